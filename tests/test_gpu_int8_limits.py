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
