"""The oracle's scale bytes at the top of their range: decoded weights may pass 2^128, where
no byte below 255 has max|v| < 7 * 2^e.  They keep the largest scale and saturate."""

import numpy as np
import pytest

import oracle as O
from block_diffusion_lm_tq4_amd import inputs as I

SB = I.sign_bits()


@pytest.mark.parametrize("top,byte,code", [
    (6.9 * 2.0 ** 126, 253, 7), (7 * 2.0 ** 126, 254, 6), (6 * 2.0 ** 127, 254, 7),
    (7 * 2.0 ** 127, 254, 7), (2.0 ** 131.9, 254, 7), (1e60, 254, 7)])
def test_the_largest_scale_saturates(top, byte, code):
    v = np.zeros((2, 64))
    v[1, 40] = -top
    v[1, 41] = 2.0 ** 127
    codes, scales = O.mxfp4_rows(v)
    assert scales.tolist() == [[0, 0], [0, byte]]
    assert codes[1, 40] == code | 8
    unit = 2.0 ** (byte - 127)
    assert O.mxfp4_values(codes, scales)[1, 41] == 2.0 ** 127
    assert abs(O.mxfp4_values(codes, scales)[1, 40]) == O.e2m1_values()[code] * unit
    codes[1, 41] = 0
    assert (codes != 0).sum() == 1


def test_weights_decoded_past_the_largest_scale():
    """Equal codes under equal scales decode to one value, sqrt(32) times theirs."""
    p = np.zeros((3, 1, 20), np.uint8)
    p[..., :16] = 0xFF
    for i, s in enumerate((0x7E80, 0x7F00, 0x7F7F)):
        p[i, 0, 16:] = np.frombuffer(np.array([s, s], np.uint16).tobytes(), np.uint8)
    w = O.dequant(p, SB)
    assert np.abs(w[0]).max() > 7 * 2.0 ** 127
    codes, scales = O.mxfp4_cache_packed(p, SB)
    assert (scales == 254).all()
    assert np.array_equal(codes & 7, np.where(w != 0, 7, 0))
    assert np.array_equal(codes >> 3, (w < 0).astype(np.uint8))
