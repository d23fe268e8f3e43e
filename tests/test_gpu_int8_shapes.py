"""The int8 layers and the scored router over the sizes at which their kernels change.

Products: the sums are integers, exact in fp64 below 2^53, so a reference made
of an fp64 product of the codes and of the documented fp32 operations, one
rounding each, has the same bits.  The MoE layer and the router: against the
oracle, with the tolerances derived in test_gpu_int8.py.
"""

import numpy as np
import pytest
import torch

import oracle as O
from block_diffusion_lm_tq4_amd import inputs as I
from test_gpu_int8 import _acts, _bf16, _check_moe, _check_router, _experts, _ops, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def _randn_bf16(dev, m, k, seed, gain=1.0):
    gen = torch.Generator(device=dev).manual_seed(seed)
    return (gain * torch.randn(m, k, generator=gen, device=dev)).to(torch.bfloat16)


def _product(xg, cache, k, n):
    """float(exact sum) * sx * sw in fp32, each operation rounded once."""
    xq, sx = _ops().act_int8(xg)
    wq, sw = _ops().int8_cache_views(cache, n, k)
    acc = xq[:, :k].double() @ wq[:, :k].double().t().contiguous()
    return (acc.float() * sx[:, None]) * sw[None, :]


# one or more for every tile, with whole and part tiles, n in and out of fours,
# k of an odd number of 64-value steps and of steps that end inside one
TILES = [(33, 96, 260), (40, 2720, 96), (70, 64, 8193), (257, 352, 1100), (97, 160, 4100),
         (130, 64, 5000), (33, 1856, 8196), (300, 96, 8193), (513, 192, 4100), (1025, 32, 4101),
         (2047, 352, 2690), (1400, 64, 12004), (700, 96, 12004), (2500, 160, 2000),
         (4099, 224, 2690), (4100, 96, 2001), (1025, 352, 12004), (2500, 288, 5002),
         (4099, 64, 8193), (1, 8224, 300), (1, 16384, 77), (1, 131072, 40), (2, 8192, 1000),
         (1, 2688, 4099), (1, 8192, 2690)]


@pytest.mark.parametrize("m,k,n", TILES)
def test_linear_bits(dev, m, k, n):
    x = _randn_bf16(dev, m, k, seed=m + n)
    cache = _ops().int8_cache_bf16(_randn_bf16(dev, n, k, seed=n + k, gain=0.05))
    bias = torch.randn(n, device=dev)
    res = torch.randn(m, n, device=dev)
    p = _product(x, cache, k, n)
    assert torch.equal(_ops().linear_int8(x, cache, n), p)
    assert torch.equal(_ops().linear_int8_epilogue(x, cache, n, bias, res),
                       (p + bias[None, :]) + res)
    r16 = res.to(torch.bfloat16)
    assert torch.equal(_ops().linear_int8_epilogue_bf16(x, cache, n, bias, r16),
                       ((p + bias[None, :]) + r16.float()).to(torch.bfloat16))
    assert torch.equal(_ops().linear_int8_epilogue_bf16(x, cache, n), p.to(torch.bfloat16))


@pytest.mark.parametrize("m", [1, 9, 40, 700])
def test_linear_unaligned_tail(dev, m):
    """bias, residual and output on addresses of their type's own alignment only."""
    k, n = 160, 96
    x = _randn_bf16(dev, m, k, seed=m)
    cache = _ops().int8_cache_bf16(_randn_bf16(dev, n, k, seed=1))
    p = _product(x, cache, k, n)
    bias = torch.randn(n + 1, device=dev)[1:]
    for dt, fn in ((torch.float32, _ops().linear_int8_epilogue),
                   (torch.bfloat16, _ops().linear_int8_epilogue_bf16)):
        res = torch.randn(m * n + 1, device=dev).to(dt)[1:].view(m, n)
        out = torch.empty(m * n + 1, device=dev, dtype=dt)[1:].view(m, n)
        ref = ((p + bias[None, :]) + res.float()).to(dt)
        assert torch.equal(fn(x, cache, n, bias, res, out=out), ref)


def test_linear_past_32_bits(dev):
    """Weight codes, activation codes and outputs of more than 2^32 bytes."""
    k, n = 8192, 600000          # 4.9 GB of codes
    cache = torch.empty(_ops().int8_cache_size(n, k), dtype=torch.uint8, device=dev)
    part = 60000
    codes, scales = _ops().int8_cache_views(cache, n, k)
    for i in range(0, n, part):
        c = _ops().int8_cache_bf16(_randn_bf16(dev, part, k, seed=i))
        pc, ps = _ops().int8_cache_views(c, part, k)
        codes[i:i + part] = pc
        scales[i:i + part] = ps
    last = c
    for m in (1, 7, 40, 300):
        x = _randn_bf16(dev, m, k, seed=m)
        y = _ops().linear_int8(x, cache, n)
        assert torch.equal(y[:, n - part:], _ops().linear_int8(x, last, part))
    del cache, codes, scales, y
    m, n = 600000, 2000          # 4.9 GB of activation codes, 4.8 GB of output
    w = _ops().int8_cache_bf16(_randn_bf16(dev, n, k, seed=3))
    q = torch.empty(m, k, dtype=torch.int8, device=dev)
    s = torch.empty(m, device=dev)
    for i in range(0, m, part):
        q[i:i + part], s[i:i + part] = _ops().act_int8(_randn_bf16(dev, part, k, seed=i))
    y = _ops().linear_int8_quantized(q, s, k, w, n)
    tail = _ops().linear_int8_quantized(q[-300:].contiguous(), s[-300:].contiguous(), k, w, n)
    assert torch.equal(y[-300:], tail)
    del q, s, y


@pytest.mark.parametrize("m,k", [(4100, 96), (4097, 1856), (5000, 2080), (12300, 2112),
                                 (70000, 32), (1025, 4096), (1024, 4128)])
def test_act_codes_of_many_rows(dev, m, k):
    x = _acts(m, k, seed=m + k)
    x[m // 2] = 0
    x[m - 1, k - 1] = 0x7FC0
    codes, scales = _ops().act_int8(_bf16(x, dev))
    ref, ref_s = O.act_int8(x)
    codes = codes.cpu().numpy()
    assert np.array_equal(codes[:, :k], ref) and not codes[:, k:].any()
    assert np.array_equal(scales.cpu().numpy(), ref_s.astype(np.float32), equal_nan=True)


def test_nothing_to_do(dev):
    """No rows, and rows without elements."""
    codes, scales = _ops().act_int8(torch.zeros(0, 64, dtype=torch.bfloat16, device=dev))
    assert codes.shape == (0, 64) and scales.shape == (0,)
    for m in (1, 300):
        codes, scales = _ops().act_int8(torch.zeros(m, 0, dtype=torch.bfloat16, device=dev))
        assert codes.shape == (m, 0) and (scales == 0).all()
    c1, c2, _, _ = _experts(dev, 2, 64, 32, seed=0)
    none = torch.zeros(0, 1, device=dev)
    out = _ops().moe_grouped_int8(torch.zeros(0, 32, dtype=torch.bfloat16, device=dev),
                                  none.to(torch.int32), none, c1, c2, 2, 64)
    assert out.shape == (0, 32)


# ---- MoE ---------------------------------------------------------------------

# (tokens, experts, topk, n1, k): the single-token form's limits on pairs, topk, n1
# and k from both sides; every tile height with more than one column tile; the
# first launch with and without the quantizer; one launch and three for the buckets
MOE = [(2, 8, 6, 96, 64), (13, 5, 1, 96, 64), (12, 5, 1, 96, 64), (1, 12, 8, 64, 96),
       (1, 12, 9, 64, 96), (1, 3, 2, 2048, 64), (1, 3, 2, 2080, 64), (1, 3, 2, 64, 4096),
       (1, 3, 2, 64, 4128), (3, 4, 4, 1856, 2688), (30, 16, 2, 544, 608), (60, 4, 2, 544, 608),
       (260, 4, 2, 544, 608), (300, 2, 1, 288, 544), (700, 2, 1, 544, 608), (700, 2, 1, 608, 544),
       (20, 3, 2, 64, 4128), (4100, 5, 2, 64, 96), (4095, 3, 2, 32, 64), (4096, 3, 2, 64, 32),
       (14, 8, 1, 96, 64), (12, 16, 2, 352, 416), (20, 16, 1, 64, 4128), (13, 40, 3, 2080, 608)]


@pytest.mark.parametrize("t,e,topk,n1,k", MOE)
def test_moe_sizes(dev, t, e, topk, n1, k):
    c1, c2, w1, w2 = _experts(dev, e, n1, k, seed=t + n1)
    x = _acts(t, k, seed=t + 1)
    ids, g = I.route(np.random.default_rng(t).standard_normal((t, e)), topk)
    out = _ops().moe_grouped_int8(_bf16(x, dev), torch.from_numpy(ids).to(dev),
                                  torch.from_numpy(g).to(dev), c1, c2, e, n1)
    ref, mag = O.moe_int8(x, ids, g, w1, w2)
    _check_moe(out.cpu().numpy(), ref, mag, topk)


def _moe_fp32_range(x, ids, g, w1, w2):
    """Where the layer's documented fp32 steps leave fp32's range: (sum * sh) * sw,
    then one fma per slot.  Hidden values reach 2^127, so sh reaches 2^120 and a
    sum of up to 127^2 * 96 > 2^20 times it passes 2^128 although sw, below 2^-9,
    would bring it back: such products are infinite by the formula, and fp64
    does not show it.  Returns the outputs of that chain."""
    out = np.zeros(x.shape, np.float32)
    xq, sx = O.act_int8(x)
    for i in range(ids.shape[0]):
        for j in range(ids.shape[1]):
            u = O.linear_int8(xq[i:i + 1], sx[i:i + 1], *w1[ids[i, j]])
            h = np.where(u < 0, 0.0, u * u).astype(np.float32)
            hq, sh = O.act_int8(O.bf16_bits_from_f32(h))
            wq, sw = w2[ids[i, j]]
            acc = (hq.astype(np.int64) @ wq.astype(np.int64).T)[0].astype(np.float32)
            o = (acc * sh.astype(np.float32)) * sw.astype(np.float32)
            out[i] = (np.float64(g[i, j]) * o.astype(np.float64) + out[i]).astype(np.float32)
    return out


@pytest.mark.parametrize("t", [1, 3, 20, 200, 600])
@pytest.mark.parametrize("gain", [2.0 ** -60, 2.0 ** -30, 2.0 ** 20, 2.0 ** 62])
def test_moe_scales_far_from_one(dev, t, gain):
    """Hidden values down to fp32's subnormals and up to infinity (whose rows are
    NaN); gates of mixed signs, zero and NaN."""
    e, topk, n1, k = 3, 2, 96, 64
    c1, c2, w1, w2 = _experts(dev, e, n1, k, seed=4)
    x = _acts(t, k, seed=t, gain=gain)
    rng = np.random.default_rng(t)
    ids, _ = I.route(rng.standard_normal((t, e)), topk)
    g = rng.standard_normal((t, topk)).astype(np.float32)
    g[0, 0] = 0.0
    if t > 1:
        g[1, 1] = np.nan
    out = _ops().moe_grouped_int8(_bf16(x, dev), torch.from_numpy(ids).to(dev),
                                  torch.from_numpy(g).to(dev), c1, c2, e, n1).cpu().numpy()
    with np.errstate(all="ignore"):
        ref, mag = O.moe_int8(x, ids, g, w1, w2)
        chain = _moe_fp32_range(x, ids, g, w1, w2)
    assert np.array_equal(np.isnan(out), np.isnan(chain))
    assert np.array_equal(np.isinf(out) * np.sign(out), np.isinf(chain) * np.sign(chain),
                          equal_nan=True)
    ok = np.isfinite(chain)
    _check_moe(np.where(ok, out, 0.0), np.where(ok, ref, 0.0), np.where(ok, mag, 0.0), topk)


def test_moe_past_32_bits(dev):
    """The last experts of two stacks of more than 2^32 bytes."""
    e, n1, k, part = 512, 2048, 4352, 32
    stacks, lasts = [], []
    for rows, cols in ((n1, k), (k, n1)):
        cache = torch.empty(_ops().int8_cache_size(e * rows, cols), dtype=torch.uint8, device=dev)
        codes, scales = _ops().int8_cache_views(cache, e * rows, cols)
        for i in range(0, e, part):
            c = _ops().int8_cache_bf16(_randn_bf16(dev, part * rows, cols, seed=i, gain=0.02))
            pc, ps = _ops().int8_cache_views(c, part * rows, cols)
            codes[i * rows:(i + part) * rows] = pc
            scales[i * rows:(i + part) * rows] = ps
        stacks.append(cache)
        lasts.append(c)
    gen = torch.Generator(device=dev).manual_seed(1)
    for t in (1, 6, 700, 3000, 9000):
        x = _randn_bf16(dev, t, k, seed=t)
        ids = torch.randint(0, part, (t, 2), generator=gen, device=dev, dtype=torch.int32)
        g = torch.rand(t, 2, generator=gen, device=dev)
        big = _ops().moe_grouped_int8(x, ids + (e - part), g, *stacks, e, n1)
        assert torch.equal(big, _ops().moe_grouped_int8(x, ids, g, *lasts, part, n1))


def test_moe_single_tokens_at_the_end_of_a_stack(dev):
    """The single-token form at its largest: 512 experts of 2048 x 4096, 2^32 bytes."""
    e, n1, k = 512, 2048, 4096
    caches, lasts = [], []
    for rows, cols in ((n1, k), (k, n1)):
        cache = torch.zeros(_ops().int8_cache_size(e * rows, cols), dtype=torch.uint8, device=dev)
        c = _ops().int8_cache_bf16(_randn_bf16(dev, 2 * rows, cols, seed=rows, gain=0.02))
        codes, scales = _ops().int8_cache_views(cache, e * rows, cols)
        codes[-2 * rows:], scales[-2 * rows:] = _ops().int8_cache_views(c, 2 * rows, cols)
        caches.append(cache)
        lasts.append(c)
    x = _randn_bf16(dev, 2, k, seed=2)
    ids = torch.tensor([[511, -1], [600, 510]], dtype=torch.int32, device=dev)
    g = torch.rand(2, 2, device=dev)
    big = _ops().moe_grouped_int8(x, ids, g, *caches, e, n1)
    assert (big.abs().amax(dim=1) > 0).all()
    assert torch.equal(big, _ops().moe_grouped_int8(x, ids - 510, g, *lasts, 2, n1))


# ---- the scored router ---------------------------------------------------------

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,topk,groups,keep", [
    (48, 14, 1, 1), (48, 15, 1, 1), (96, 8, 16, 5), (102, 8, 17, 5), (256, 8, 8, 4), (512, 14, 2, 1),
    (33, 14, 1, 1), (15, 15, 1, 1), (16, 14, 8, 8), (129, 6, 3, 2), (8, 1, 8, 1)])
@pytest.mark.parametrize("t", [1, 700])
def test_router_of_bf16_logits(dev, score, e, topk, groups, keep, t):
    """Logits with 8 bits, as a bf16 gate leaves them: equal ones at every border."""
    rng = np.random.default_rng(e + topk + t)
    lg = (O.bf16_bits_from_f32(rng.standard_normal((t, e)).astype(np.float32)).astype(np.uint32)
          << 16).view(np.float32)
    bias = np.round(rng.standard_normal(e) * 4).astype(np.float32) / 8
    for b, renorm in ((None, True), (bias, False)):
        _check_router(dev, lg, topk, score=score, bias=b, n_groups=groups, topk_groups=keep,
                      renormalize=renorm, scale=1.25)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_router_wide_logits(dev, score):
    """Scores from fp32's smallest to 1, where fp32's own differences vanish: only
    the order of the fp64 scores decides."""
    rng = np.random.default_rng(3)
    lg = (40.0 * rng.standard_normal((500, 64))).astype(np.float32)
    lg[:100] = 20.0 + rng.random((100, 64)).astype(np.float32)
    lg[100:200] = -100.0 + rng.random((100, 64)).astype(np.float32)
    lg[200:300] = (1e-6 * rng.standard_normal((100, 64))).astype(np.float32)
    for bias in (None, (1e-3 * rng.standard_normal(64)).astype(np.float32)):
        for groups, keep in ((1, 1), (8, 3)):
            _check_router(dev, lg, 6, score=score, bias=bias, n_groups=groups, topk_groups=keep)


def test_router_odd_rows_and_addresses(dev):
    """Rows of an odd number of experts from an address of 4-byte alignment."""
    t, e = 333, 37
    lg = np.random.default_rng(4).standard_normal((t, e)).astype(np.float32)
    held = torch.empty(t * e + 1, device=dev)
    view = held[1:].view(t, e)
    view.copy_(torch.from_numpy(lg))
    ids, w = _ops().moe_router_scored(view, 5, renormalize=True)
    ri, rw = O.router_scored(lg, 5, renormalize=True)
    assert np.array_equal(ids.cpu().numpy(), ri)
    assert np.allclose(w.cpu().numpy(), rw, rtol=2.0 ** -23, atol=0)
