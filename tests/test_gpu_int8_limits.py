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
