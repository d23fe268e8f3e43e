"""The MXFP4 layers and the router's training step at every kernel form and at their
size limits: each dense tile with whole and odd numbers of steps, several chunks of
scales and edges in both directions; each tile height of the MoE layer and its
single-token form; operands and outputs past 2^32 bytes and 2^31 elements; two streams
at once.

Products are compared with a product of the same values in 64 bits (torch on the GPU, the
values by the oracle's rule), bit for bit: sums are exact (see test_gpu_mxfp4.py, whose
condition `_exact` holds for these inputs), a tail's adds are rounded in the same order.
"""

import numpy as np
import pytest
import torch

import oracle as O
from block_diffusion_lm_tq4_amd import inputs as I

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from block_diffusion_lm_tq4_amd import ops  # noqa: F401  (loads libtq4.so)
    return torch.device("cuda:0")


def _ops():
    from block_diffusion_lm_tq4_amd import ops
    return ops


def _bf16(bits, dev):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(dev).view(torch.bfloat16)


def _acts(m, k, seed):
    x = np.random.default_rng(seed).standard_normal((m, k))
    x[:, ::max(1, k // 3)] *= 5.0
    return O.bf16_bits_from_f32(x.astype(np.float32))


def _values(bits, dev):
    return torch.from_numpy(O.mxfp4_values(*O.act_mxfp4(bits))).to(dev)


def _product(x, w, dev):
    return torch.mm(_values(x, dev), _values(w, dev).t().contiguous()).float()


# (m, k, n): 32 x 32, 32 x 64, 64 x 64, 64 x 128, 128 x 128, 192 x 256 and 256 x 256 tiles
TILES = [(17, 2080, 130), (200, 8192, 40), (40, 160, 1000),
         (128, 128, 4096), (130, 2080, 1919), (60, 1152, 6100),
         (333, 1856, 2688), (200, 2080, 3001),
         (500, 384, 2500), (801, 2080, 4673),
         (512, 1152, 4100), (700, 2080, 4099), (4099, 256, 1030),
         (1030, 640, 8200), (1300, 2080, 8197),
         (2500, 288, 5000), (4034, 2080, 2837)]


@pytest.mark.parametrize("m,k,n", TILES)
def test_tiles(dev, m, k, n):
    o = _ops()
    rng = np.random.default_rng(m + n)
    x = _acts(m, k, seed=m)
    w = O.bf16_bits_from_f32(I.weights(n, k, seed=k))
    cache = o.mxfp4_cache_bf16(_bf16(w, dev))
    xg = _bf16(x, dev)
    want = _product(x, w, dev)
    assert torch.equal(o.linear_mxfp4(xg, cache, n), want)
    b = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(dev)
    r = torch.randn(m, n, device=dev)
    assert torch.equal(o.linear_mxfp4_epilogue(xg, cache, n, b, r), want + b + r)
    rb = r.to(torch.bfloat16)
    y = o.linear_mxfp4_epilogue_bf16(xg, cache, n, None, rb, out=rb.clone())
    assert torch.equal(y, (want + rb.float()).to(torch.bfloat16))


def _experts(dev, e, n, k, seed):
    w = O.bf16_bits_from_f32(I.weights(e * n, k, seed=seed))
    c, s = O.act_mxfp4(w)
    return (_ops().mxfp4_cache_bf16(_bf16(w, dev)),
            [(c[i * n:(i + 1) * n], s[i * n:(i + 1) * n]) for i in range(e)])


# few pairs (the single-token form, up to 24), then 64-, 128- and 256-row tiles, the last with
# one tile and with several to an expert; few workgroups have lower and narrower tiles
MOE = [(1, 4, 1, 2080, 1184), (3, 16, 8, 96, 352), (4, 8, 6, 1152, 640), (24, 30, 1, 160, 96),
       (2, 12, 9, 128, 64), (60, 12, 4, 2080, 1184), (25, 64, 1, 352, 2080),
       (100, 8, 5, 2080, 1184), (120, 8, 4, 160, 2080), (300, 6, 4, 2080, 1184),
       (513, 2, 1, 96, 1152), (700, 4, 2, 2080, 1184),
       (150, 10, 4, 2080, 1184), (600, 45, 4, 96, 1184),
       (1000, 20, 4, 2080, 1184), (1150, 45, 4, 96, 1184),
       (1250, 10, 4, 2080, 1184), (1280, 15, 6, 352, 2080)]


@pytest.mark.parametrize("t,e,topk,k,n1", MOE)
def test_moe_forms(dev, t, e, topk, k, n1):
    rng = np.random.default_rng(t)
    x = _acts(t, k, seed=t)
    ids = np.argsort(rng.random((t, e)), axis=1)[:, :topk].astype(np.int32)
    ids[rng.random((t, topk)) < 0.07] = -1
    g = rng.standard_normal((t, topk)).astype(np.float32)
    c1, r1 = _experts(dev, e, n1, k, 1)
    c2, r2 = _experts(dev, e, k, n1, 2)
    out = _ops().moe_grouped_mxfp4(_bf16(x, dev), torch.from_numpy(ids).to(dev),
                                   torch.from_numpy(g).to(dev), c1, c2, e, n1)
    want, size = O.moe_mxfp4(x, ids, g, r1, r2)
    # the down sums where hidden scales are far apart, gates and slots one rounding each
    tol = ((4 * ((n1 + 127) // 128) + 16) * 2.0 ** -23 + (topk + 2) * U) * size
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("t", [2, 4, 64])
def test_moe_with_one_expert_in_several_slots(dev, t):
    e, topk, k, n1 = 4, 3, 256, 160
    x = _acts(t, k, seed=t)
    ids = np.full((t, topk), 2, np.int32)
    ids[0] = [1, 1, 3]
    g = np.random.default_rng(0).standard_normal((t, topk)).astype(np.float32)
    c1, r1 = _experts(dev, e, n1, k, 1)
    c2, r2 = _experts(dev, e, k, n1, 2)
    out = _ops().moe_grouped_mxfp4(_bf16(x, dev), torch.from_numpy(ids).to(dev),
                                   torch.from_numpy(g).to(dev), c1, c2, e, n1)
    want, size = O.moe_mxfp4(x, ids, g, r1, r2)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= 36 * 2.0 ** -23 * size)


def test_moe_tokens_routed_nowhere_and_rows_around_the_output(dev):
    o = _ops()
    e, topk, k, n1 = 4, 2, 128, 96
    c1, _ = _experts(dev, e, n1, k, 1)
    c2, _ = _experts(dev, e, k, n1, 2)
    for t in (1, 9, 300):
        store = torch.full((t + 2, k), 5.0, device=dev)
        ids = torch.full((t, topk), -1, dtype=torch.int32, device=dev)
        out = o.moe_grouped_mxfp4(_bf16(_acts(t, k, 1), dev), ids, torch.ones(t, topk, device=dev),
                                  c1, c2, e, n1, out=store[1:t + 1])
        assert not out.any() and (store[0] == 5).all() and (store[t + 1] == 5).all()


# ---- sizes ---------------------------------------------------------------------

@pytest.mark.parametrize("m", [1, 16, 40, 300])
def test_weights_past_4_gib(dev, m):
    """Codes of 4.3 GB, zero but for rows at both ends."""
    o = _ops()
    k, n = 8192, (1 << 20) + 300
    cache = torch.zeros(o.mxfp4_cache_size(n, k), dtype=torch.uint8, device=dev)
    codes, scales = o.mxfp4_cache_views(cache, n, k)
    rows = [0, 1, 70000, n - 257, n - 2, n - 1]
    w = O.bf16_bits_from_f32(I.weights(len(rows), k, seed=3))
    wc, wsc = o.act_mxfp4(_bf16(w, dev))
    codes[rows] = wc
    scales[rows] = wsc
    x = _acts(m, k, seed=m)
    y = o.linear_mxfp4(_bf16(x, dev), cache, n)
    assert torch.equal(y[:, rows], _product(x, w, dev))
    y[:, rows] = 0
    assert not y.any()


def test_outputs_past_2_31_elements(dev):
    o = _ops()
    m, k, n = 40000, 64, 65600
    x = _acts(64, k, seed=1)
    w = O.bf16_bits_from_f32(I.weights(n, k, seed=2))
    xg = _bf16(x, dev).repeat(m // 64, 1)
    y = o.linear_mxfp4_epilogue_bf16(xg, o.mxfp4_cache_bf16(_bf16(w, dev)), n)
    assert y.shape == (m, n)
    want = _product(x, w, dev).to(torch.bfloat16)
    for i in (0, 31 * 64, m - 64):
        assert torch.equal(y[i:i + 64], want)


def test_values_past_2_32_bytes(dev):
    """Quantize and decode 2.2 G values with padded rows, and as one long row."""
    o = _ops()
    for m, k in ((1 << 19, 4128), (1 << 20, 2176)):
        x = torch.zeros(m, k, dtype=torch.bfloat16, device=dev)
        b = _bf16(_acts(70, k, seed=k), dev)
        x[m - 70:] = b
        x[m // 2:m // 2 + 70] = b
        codes, scales = o.act_mxfp4(x)
        rc, rs = o.act_mxfp4(b)
        v = o.mxfp4_values(codes, scales, k)
        want = o.mxfp4_values(rc, rs, k)
        for at in (m // 2, m - 70):
            assert torch.equal(codes[at:at + 70], rc) and torch.equal(scales[at:at + 70], rs)
            assert torch.equal(v[at:at + 70], want)
        assert not scales[:m // 2].any() and not v[m // 2 + 70:m - 70].any()
        del x, codes, scales, v


@pytest.mark.parametrize("t", [2, 90])
def test_experts_past_4_gib(dev, t):
    """Stacked experts of 4.3 GB each way, zero but for the first and the last."""
    o = _ops()
    e, topk, k, n1 = 256, 2, 4096, 8192
    rng = np.random.default_rng(t)
    r1, r2, c = {}, {}, []
    for store, n, kk in ((r1, n1, k), (r2, k, n1)):
        cache = torch.zeros(o.mxfp4_cache_size(e * n, kk), dtype=torch.uint8, device=dev)
        codes, scales = o.mxfp4_cache_views(cache, e * n, kk)
        for i in (0, e - 1):
            w = O.bf16_bits_from_f32(I.weights(n, kk, seed=i + 1))
            wc, wsc = o.act_mxfp4(_bf16(w, dev))
            codes[i * n:(i + 1) * n] = wc
            scales[i * n:(i + 1) * n] = wsc
            store[i] = _values(w, dev)
        c.append(cache)
    ids = np.stack([np.where(rng.random(t) < 0.5, 0, e - 1), rng.integers(1, e - 1, t)],
                   axis=1).astype(np.int32)
    x = _acts(t, k, seed=t)
    g = rng.standard_normal((t, topk)).astype(np.float32)
    out = o.moe_grouped_mxfp4(_bf16(x, dev), torch.from_numpy(ids).to(dev),
                              torch.from_numpy(g).to(dev), c[0], c[1], e, n1).double()
    xd = _values(x, dev)
    for i in range(t):
        u = torch.mv(r1[int(ids[i, 0])], xd[i]).float().cpu().numpy()
        u = np.maximum(u, 0)
        h = torch.from_numpy(O.mxfp4_values(*O.mxfp4_rows((u * u)[None].astype(np.float64)))[0])
        w = r2[int(ids[i, 0])]
        want = float(g[i, 0]) * torch.mv(w, h.to(dev))
        size = abs(float(g[i, 0])) * torch.mv(w.abs(), h.to(dev))
        assert torch.all((out[i] - want).abs() <= (4 * 64 + 16 + 4) * 2.0 ** -23 * size)


def test_router_step_past_2_31_logits(dev):
    o = _ops()
    t, e, topk = (1 << 22) + 77, 512, 2
    l = torch.zeros(t, e, device=dev)
    ids = torch.full((t, topk), -1, dtype=torch.int32, device=dev)
    rng = np.random.default_rng(0)
    rows = [0, 5, t // 2, t - 2, t - 1]
    ll = rng.standard_normal((len(rows), e)).astype(np.float32)
    ii = rng.integers(0, e, (len(rows), topk)).astype(np.int32)
    dg = torch.zeros(t, topk, device=dev)
    dd = rng.standard_normal((len(rows), topk)).astype(np.float32)
    for j, r in enumerate(rows):
        l[r] = torch.from_numpy(ll[j]).to(dev)
        ids[r] = torch.from_numpy(ii[j]).to(dev)
        dg[r] = torch.from_numpy(dd[j]).to(dev)
    loss, counts, tokens, mean = o.moe_balance(l, ids)
    rl, rc, rt, rm = O.moe_balance(ll, ii)
    assert int(tokens) == rt and np.array_equal(counts.cpu().numpy(), rc)
    assert np.all(np.abs(mean.double().cpu().numpy() - rm) <= 140 * U * rm)
    grad = o.moe_router_backward(l, ids, dg, counts=counts, tokens=tokens,
                                 dloss=torch.ones((), device=dev))
    want, size = O.moe_router_backward(ll, ii, dd, counts=rc, tokens=rt, dloss=1.0)
    assert np.all(np.abs(grad[rows].double().cpu().numpy() - want) <= 200 * U * size)
    grad[rows] = 0
    assert not grad.any()


# ---- calls side by side -----------------------------------------------------------

def test_two_streams_at_once(dev):
    o = _ops()
    e, topk, k, n1 = 8, 2, 512, 352
    c1, _ = _experts(dev, e, n1, k, 1)
    c2, _ = _experts(dev, e, k, n1, 2)
    rng = np.random.default_rng(0)
    work = []
    for t in (100, 300):
        l = torch.randn(t, e, device=dev)
        ids = torch.from_numpy(np.argsort(rng.random((t, e)), axis=1)[:, :topk].astype(np.int32))
        work.append((_bf16(_acts(t, k, t), dev), ids.to(dev), torch.rand(t, topk, device=dev), l))

    def step(x, ids, g, l):
        loss, counts, tokens, mean = o.moe_balance(l, ids)
        return (o.linear_mxfp4(x, c1, e * n1), o.moe_grouped_mxfp4(x, ids, g, c1, c2, e, n1), loss,
                counts, mean, o.moe_router_backward(l, ids, g, counts=counts, tokens=tokens,
                                                    dloss=loss))

    want = [step(*w) for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for s, w, out in zip(streams, work, got):
            with torch.cuda.stream(s):
                out.append(step(*w))
    torch.cuda.synchronize()
    for out, ref in zip(got, want):
        for outs in out:
            for a, b in zip(outs, ref):
                assert torch.equal(a, b)


def test_refusals_of_shapes_and_devices(dev):
    o = _ops()
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device=dev)
    cache = torch.zeros(o.mxfp4_cache_size(32, 128), dtype=torch.uint8, device=dev)
    l = torch.zeros(4, 8, device=dev)
    ids = torch.zeros(4, 2, dtype=torch.int32, device=dev)
    c = torch.zeros(8, dtype=torch.int32, device=dev)
    one = torch.zeros(1, device=dev)
    for call in (lambda: o.linear_mxfp4(x, cache, 33), lambda: o.linear_mxfp4(x[0], cache, 32),
                 lambda: o.linear_mxfp4(x[:, ::2], cache, 32),
                 lambda: o.linear_mxfp4(x, cache.cpu(), 32),
                 lambda: o.linear_mxfp4(x.float(), cache, 32),
                 lambda: o.linear_mxfp4_epilogue(x, cache, 32, torch.zeros(31, device=dev)),
                 lambda: o.linear_mxfp4_epilogue_bf16(x, cache, 32, None,
                                                      torch.zeros(4, 32, device=dev)),
                 lambda: o.linear_mxfp4(x, cache, 32, out=torch.zeros(4, 31, device=dev)),
                 lambda: o.mxfp4_values(cache.view(-1, 68), cache, 128),
                 lambda: o.moe_grouped_mxfp4(x, ids, l[:, :2].contiguous(), cache, cache, 2, 32),
                 lambda: o.moe_balance(l, ids[:3]), lambda: o.moe_balance(l, ids, score="tanh"),
                 lambda: o.moe_balance(l, ids.long()),
                 lambda: o.moe_router_backward(l, ids, l),
                 lambda: o.moe_router_backward(l, ids, counts=c),
                 lambda: o.moe_router_backward(l, ids, counts=c, tokens=c[:1], dloss=l[:, 0]),
                 lambda: o.moe_router_backward(l, ids, out=l[:3])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: o.moe_router_backward(l, ids, out=l),        # over its input
                 lambda: o.moe_balance(l, torch.zeros(4, 9, dtype=torch.int32, device=dev)),
                 lambda: o.linear_mxfp4(x[:, :100].contiguous(), cache, 32),
                 lambda: o.linear_mxfp4_epilogue_bf16(x, torch.zeros_like(cache).repeat(4), 128,
                                                      None, x, out=x)):
        with pytest.raises(RuntimeError):
            call()
    assert o.moe_router_backward(l, ids, one.expand(4, 2).contiguous()).shape == (4, 8)
