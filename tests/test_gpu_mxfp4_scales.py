"""MXFP4 weights from packed blocks whose half-block scales are near bf16's largest: the
decoded weights reach 2^132, past 7 * 2^127, where the scale byte stays at 254 and the codes
saturate.  The expected codes are taken here from the decoded weights by the rule, the
products from the values in fp64, where every sum is exact (one or two terms)."""

import numpy as np
import pytest
import torch

import oracle as O
from block_diffusion_lm_tq4_amd import inputs as I

pytestmark = pytest.mark.gpu
SB = I.sign_bits()
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from block_diffusion_lm_tq4_amd import ops  # noqa: F401  (loads libtq4.so)
    return torch.device("cuda:0")


def _ops():
    from block_diffusion_lm_tq4_amd import ops
    return ops


def _packed(n, k, scale, code, seed):
    """Random codes (or one code throughout) under one scale of each half block."""
    p = np.zeros((n, k // 32, 20), np.uint8)
    rng = np.random.default_rng(seed)
    p[..., :16] = rng.integers(0, 256, p[..., :16].shape) if code is None else code * 0x11
    p[..., 16:] = np.frombuffer(np.array([scale, scale], np.uint16).tobytes(), np.uint8)
    return p


def _encode(w):
    """(magnitude codes, signs, scale bytes) of decoded rows; scales near the top."""
    b = w.reshape(w.shape[0], -1, 32)
    top = np.abs(b).max(axis=-1)
    e = np.full(top.shape, 100)
    while (up := (top >= 7 * np.ldexp(1.0, e)) & (e < 127)).any():
        e = e + up
    a = np.minimum(np.abs(b) / np.ldexp(1.0, e)[..., None], 6.0)
    d = np.abs(a[..., None] - LEVELS)
    near = d.min(axis=-1, keepdims=True) == d
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(axis=-1), even.argmax(axis=-1), near.argmax(axis=-1))
    return code.reshape(w.shape), w < 0, e + 127


@pytest.mark.parametrize("scale", [0x7A00, 0x7D80, 0x7E00, 0x7E80, 0x7F00, 0x7F7F])
@pytest.mark.parametrize("code", [None, 0, 7, 15])
def test_cache_of_the_largest_weights(dev, scale, code):
    n, k = 9, 96
    p = _packed(n, k, scale, code, seed=scale)
    w = O.dequant(p, SB)
    cache = _ops().mxfp4_cache(torch.from_numpy(p).to(dev), SB)
    codes, scales = (v.cpu().numpy() for v in _ops().mxfp4_cache_views(cache, n, k))
    want, neg, byte = _encode(w)
    assert np.array_equal(scales[:, :k // 32], byte) and scales.max() <= 254
    got = O.unpack_nibbles(codes[:, :k // 2])
    assert np.array_equal(got & 7, want)
    assert np.array_equal(got >> 3, neg)
    assert not codes[:, k // 2:].any() and not scales[:, k // 32:].any()


@pytest.mark.parametrize("m", [1, 16, 40, 300])
def test_products_of_the_largest_weights(dev, m):
    """Equal codes leave one weight a block that is not zero."""
    o = _ops()
    n, k = 33, 64
    p = _packed(n, k, 0x7F7F, 15, seed=0)
    cache = o.mxfp4_cache(torch.from_numpy(p).to(dev), SB)
    x = (np.ldexp(1.0, -40) * np.ones((m, k))).astype(np.float32)
    x[::2] *= -0.5
    xb = torch.from_numpy(x).to(dev).to(torch.bfloat16)
    y = o.linear_mxfp4(xb, cache, n).double().cpu().numpy()
    w = O.dequant(p, SB)
    v = np.where(w != 0, np.sign(w) * 6 * 2.0 ** 127, 0.0)
    assert np.array_equal(y, x.astype(np.float64) @ v.T) and np.abs(y).min() > 0
