"""The int8 layers at the ends of their range, against values that do not come from
the kernels."""

import numpy as np
import pytest
import torch

import oracle as O
from block_diffusion_lm_tq4_amd import inputs as I
from test_gpu_int8 import _acts, _bf16, _experts, _ops, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def test_outputs_of_an_empty_k_past_32_bits(dev):
    """An empty sum, alone and with its tail, of 2^32 + 2^16 elements."""
    m, n = 2 ** 16 + 1, 2 ** 16
    x = torch.zeros(m, 0, dtype=torch.bfloat16, device=dev)
    cache = torch.empty(0, dtype=torch.uint8, device=dev)
    y = torch.full((m, n), 7.0, device=dev)
    assert not _ops().linear_int8(x, cache, n, out=y).any()
    bias = torch.arange(n, dtype=torch.float32, device=dev)
    row = torch.arange(m, dtype=torch.float32, device=dev)[:, None]
    y.copy_(row.expand(m, n))
    _ops().linear_int8_epilogue(x, cache, n, bias, y, out=y)   # sums below 2^18: exact
    for i in range(0, m, 8192):
        assert torch.equal(y[i:i + 8192], row[i:i + 8192] + bias)
    del y
    y = _ops().linear_int8_epilogue_bf16(x, cache, n, bias)
    for i in range(0, m, 8192):
        assert torch.equal(y[i:i + 8192], bias.to(torch.bfloat16).expand_as(y[i:i + 8192]))


def _check_small(out, ref, mag, ids, g, w2):
    """The layer's fp32 steps per slot: a = fl(sum), b = fl(a sh), o = fl(b sw), out =
    fma(g, o, out).  Each is off by 2^-24 of its value or, where that is
    subnormal, by 2^-150: (topk + 5) 2^-24 sum |g o| as for other sizes, and
    per slot 2^-150 (|g| (sw + 1) + 1)."""
    top = np.array([sw.max() for _, sw in w2], np.float64)
    steps = (np.abs(g).astype(np.float64) * (top[ids] + 1) + 1).sum(axis=1, keepdims=True)
    tol = 1.01 * ((ids.shape[1] + 5) * 2.0 ** -24 * mag + 2.0 ** -150 * steps)
    err = np.abs(out.astype(np.float64) - ref)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("t", [1, 3, 20, 200, 600])
@pytest.mark.parametrize("power", [-63, -60, -56, -52])
def test_moe_small_outputs(dev, t, power):
    """Outputs from fp32's subnormals up: hidden values about 2^(2 power + 2), so their
    rows' scales are about 2^-130 to 2^-110 and their subnormal bf16 values,
    codes and products all count."""
    e, topk, n1, k = 3, 2, 96, 64
    c1, c2, w1, w2 = _experts(dev, e, n1, k, seed=4)
    x = _acts(t, k, seed=t, gain=2.0 ** power)
    rng = np.random.default_rng(t)
    ids, _ = I.route(rng.standard_normal((t, e)), topk)
    g = rng.standard_normal((t, topk)).astype(np.float32)
    out = _ops().moe_grouped_int8(_bf16(x, dev), torch.from_numpy(ids).to(dev),
                                  torch.from_numpy(g).to(dev), c1, c2, e, n1).cpu().numpy()
    ref, mag = O.moe_int8(x, ids, g, w1, w2)
    _check_small(out, ref, mag, ids, g, w2)


def _random_cache(dev, n, k, gain, seed):
    """A cache of random codes and scales; k is a multiple of 64."""
    gen = torch.Generator(device=dev).manual_seed(seed)
    cache = torch.empty(_ops().int8_cache_size(n, k), dtype=torch.uint8, device=dev)
    codes, scales = _ops().int8_cache_views(cache, n, k)
    codes.random_(-127, 128, generator=gen)
    scales.uniform_(0.5 * gain, gain, generator=gen)
    return cache, codes, scales


def _steps(xq, sx, wq, sw):
    """The exact sums (fp64) and the documented fp32 steps, on the device."""
    acc = xq.double() @ wq.double().t().contiguous()
    return (acc.float() * sx[:, None]) * sw[None, :]


# rows at 2^31 and 2^32 bytes of codes (8192 a row), and the last ones
PLACES = [slice(262100, 262180), slice(524200, 524310), slice(-300, None)]


def test_linear_weights_past_32_bits(dev):
    n, k = 600000, 8192
    cache, wq, sw = _random_cache(dev, n, k, 0.02, seed=1)
    for m in (1, 7, 40, 300):
        x = _acts(m, k, seed=m)
        xq, sx = (torch.from_numpy(v).to(dev) for v in O.act_int8(x))
        y = _ops().linear_int8(_bf16(x, dev), cache, n)
        for at in PLACES:
            assert torch.equal(y[:, at], _steps(xq, sx, wq[at], sw[at]))


def test_linear_activations_and_outputs_past_32_bits(dev):
    m, n, k = 600000, 2000, 8192
    _, xq, sx = _random_cache(dev, m, k, 1.0, seed=2)      # laid out as codes, then scales
    cache, wq, sw = _random_cache(dev, n, k, 0.02, seed=3)
    y = _ops().linear_int8_quantized(xq, sx, k, cache, n)
    for at in PLACES + [slice(536800, 536900)]:            # 2^32 bytes of output
        assert torch.equal(y[at], _steps(xq[at], sx[at], wq, sw))


# tokens, k, tokens compared; the last case holds more than 2^32 bytes of products
# before their sum, and its last token's first slot is the last of them
@pytest.mark.parametrize("t,k,some", [(2, 4096, [0, 1]), (1, 4352, [0]), (6, 4352, [0, 3, 5]),
                                      (700, 4352, [0, 350, 699]), (9000, 4352, [0, 8999]),
                                      (125000, 4352, [0, 123400, 124999])])
def test_moe_weights_past_32_bits(dev, t, k, some):
    e, n1, topk = 512, 2048, 2
    c1, q1, s1 = _random_cache(dev, e * n1, k, 0.0005, seed=4)
    c2, q2, s2 = _random_cache(dev, e * k, n1, 0.0005, seed=5)
    # the experts on both sides of 2^31 and 2^32 bytes, and the last
    near = sorted({min(2 ** p // (n1 * k) - d, e - 1) for p in (31, 32) for d in (0, 1)} | {e - 1})
    rng = np.random.default_rng(t)
    ids = np.array(near, np.int32)[rng.integers(0, len(near), (t, topk))]
    ids[-1] = e - 1, near[0]
    g = rng.random((t, topk)).astype(np.float32)
    gen = torch.Generator(device=dev).manual_seed(6)
    x = torch.randn(t, k, generator=gen, device=dev).to(torch.bfloat16)
    out = _ops().moe_grouped_int8(x, torch.from_numpy(ids).to(dev), torch.from_numpy(g).to(dev),
                                  c1, c2, e, n1)

    def expert(q, s, rows, i):
        return q[i * rows:(i + 1) * rows].cpu().numpy(), s[i * rows:(i + 1) * rows].cpu().numpy()

    used = set(ids[some].ravel().tolist())
    w1 = [expert(q1, s1, n1, i) if i in used else None for i in range(e)]
    w2 = [expert(q2, s2, k, i) if i in used else None for i in range(e)]
    bits = x[some].view(torch.int16).cpu().numpy().view(np.uint16)
    ref, mag = O.moe_int8(bits, ids[some], g[some], w1, w2)
    assert (np.abs(ref) > 0).mean() > 0.9
    err = np.abs(out[some].cpu().numpy().astype(np.float64) - ref)
    assert (err <= (topk + 5) * 2.0 ** -24 * mag).all()


def _same_in_parts(y, xq, sx, wq, sw, part=1 << 20):
    for i in range(0, y.shape[0], part):
        at = slice(i, i + part)
        if not torch.equal(y[at], _steps(xq[at], sx[at], wq, sw)):
            return False
    return True


# rows and columns at their limit of 2^24, by every kernel family
@pytest.mark.parametrize("m,k,n", [(2 ** 24, 32, 3), (2 ** 24, 96, 17), (1, 32, 2 ** 24),
                                   (5, 64, 2 ** 24), (40, 32, 2 ** 24)])
def test_linear_of_most_rows_and_columns(dev, m, k, n):
    kp = _ops().int8_padded_k(k)
    cache, wq, sw = _random_cache(dev, n, kp, 0.02, seed=n)
    wq[:, k:] = 0
    gen = torch.Generator(device=dev).manual_seed(m)
    x = torch.randn(m, k, generator=gen, device=dev).to(torch.bfloat16)
    some = sorted({0, m // 2, m - 1})
    xq, sx = _ops().act_int8(x)
    rq, rs = O.act_int8(x[some].view(torch.int16).cpu().numpy().view(np.uint16))
    assert np.array_equal(xq[some, :k].cpu().numpy(), rq) and np.array_equal(sx[some].cpu(), rs)
    y = _ops().linear_int8(x, cache, n)
    if m > n:
        assert _same_in_parts(y, xq, sx, wq, sw)
    else:                                   # the transposed product's rows, the same steps
        for i in range(0, n, 1 << 20):
            at = slice(i, i + (1 << 20))
            assert torch.equal(y[:, at], _steps(xq, sx, wq[at], sw[at]))


def _moe_some(x, ids, g, some, caches, e, n1, k):
    """The oracle's layer for some tokens, from the caches' codes and scales."""
    used = set(ids[some].ravel().tolist())
    lists = []
    for (q, s), rows, cols in zip(caches, (n1, k), (k, n1)):
        lists.append([(q[i * rows:(i + 1) * rows, :cols].cpu().numpy(),
                       s[i * rows:(i + 1) * rows].cpu().numpy()) if i in used else None
                      for i in range(e)])
    bits = x[some].view(torch.int16).cpu().numpy().view(np.uint16)
    return O.moe_int8(bits, ids[some], g[some], *lists)


# the longest rows of both products, every expert in every slot, and the most pairs
@pytest.mark.parametrize("t,e,topk,n1,k", [(1, 2, 1, 64, 131072), (9, 2, 2, 64, 131072),
                                           (300, 2, 2, 64, 131072), (1, 2, 1, 131072, 64),
                                           (9, 2, 2, 131072, 64), (300, 2, 2, 131072, 64),
                                           (1, 512, 512, 32, 64), (7, 512, 300, 32, 64),
                                           (500, 512, 512, 32, 64), (16774911, 8, 1, 32, 32)])
def test_moe_of_the_longest_rows_and_the_most_pairs(dev, t, e, topk, n1, k):
    kp, n1p = _ops().int8_padded_k(k), _ops().int8_padded_k(n1)
    gain = 0.5 / max(k, n1) ** 0.5
    c1, q1, s1 = _random_cache(dev, e * n1, kp, gain, seed=7)
    c2, q2, s2 = _random_cache(dev, e * k, n1p, gain, seed=8)
    q1[:, k:] = 0
    q2[:, n1:] = 0
    rng = np.random.default_rng(t + topk)
    if t > 1000:
        ids = rng.integers(0, e, (t, topk)).astype(np.int32)
    else:
        ids = np.stack([rng.permutation(e)[:topk] for _ in range(t)]).astype(np.int32)
    g = rng.random((t, topk), np.float32)
    gen = torch.Generator(device=dev).manual_seed(t)
    x = torch.randn(t, k, generator=gen, device=dev).to(torch.bfloat16)
    out = _ops().moe_grouped_int8(x, torch.from_numpy(ids).to(dev), torch.from_numpy(g).to(dev),
                                  c1, c2, e, n1)
    some = sorted({0, t // 3, t - 1})
    ref, mag = _moe_some(x, ids, g, some, ((q1, s1), (q2, s2)), e, n1, k)
    assert (np.abs(ref) > 0).mean() > 0.9
    err = np.abs(out[some].cpu().numpy().astype(np.float64) - ref)
    assert (err <= (topk + 5) * 2.0 ** -24 * mag).all()


def _guarded(dev, shape, dtype, fill=7):
    """A tensor inside a longer one of a known value, and a check of its margins."""
    count, pad = int(np.prod(shape)), 256
    held = torch.full((count + 2 * pad,), fill, dtype=dtype, device=dev)
    return held[pad:pad + count].view(shape), lambda: bool(
        (held[:pad] == fill).all() and (held[pad + count:] == fill).all())


def test_memory_of_the_caller(dev):
    """Caches, codes, outputs and scratch that the caller brings: the same results, and
    nothing written outside."""
    o = _ops()
    m, k, n, e, topk, n1 = 37, 224, 96, 4, 2, 160
    gen = torch.Generator(device=dev).manual_seed(9)
    w = torch.randn(n, k, generator=gen, device=dev).to(torch.bfloat16)
    x = torch.randn(m, k, generator=gen, device=dev).to(torch.bfloat16)
    checks = []

    def own(shape, dtype):
        view, check = _guarded(dev, shape, dtype)
        checks.append(check)
        return view

    cache = o.int8_cache_bf16(w)
    assert torch.equal(o.int8_cache_bf16(w, own((o.int8_cache_size(n, k),), torch.uint8)), cache)
    packed = o.pack(w.float(), I.sign_bits())
    assert torch.equal(o.int8_cache(packed, I.sign_bits(),
                                    own((o.int8_cache_size(n, k),), torch.uint8)),
                       o.int8_cache(packed, I.sign_bits()))
    size = o.linear_int8_workspace_size(m, k, n)
    y = o.linear_int8(x, cache, n)
    assert torch.equal(o.linear_int8(x, cache, n, own((m, n), torch.float32),
                                     own((size,), torch.uint8)), y)
    assert torch.equal(o.linear_int8_quantized(*o.act_int8(x), k, cache, n,
                                               own((m, n), torch.float32)), y)
    w1, w2 = (torch.randn(e * a, b, generator=gen, device=dev).to(torch.bfloat16)
              for a, b in ((n1, k), (k, n1)))
    c1, c2 = o.int8_cache_bf16(w1), o.int8_cache_bf16(w2)
    lg = torch.randn(m, e, generator=gen, device=dev)
    ids, g = o.moe_router_scored(lg, topk, renormalize=True)
    own_ids, own_g = own((m, topk), torch.int32), own((m, topk), torch.float32)
    o.moe_router_scored(lg, topk, renormalize=True, ids=own_ids, gates=own_g)
    assert torch.equal(own_ids, ids) and torch.equal(own_g, g)
    for t in (2, m):
        size = o.moe_grouped_int8_workspace_size(t, topk, e, n1, k)
        args = (x[:t], ids[:t], g[:t], c1, c2, e, n1)
        assert torch.equal(o.moe_grouped_int8(*args, own((t, k), torch.float32),
                                              own((size,), torch.uint8)),
                           o.moe_grouped_int8(*args))
    assert all(check() for check in checks)
