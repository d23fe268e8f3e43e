"""Pins of the int8 oracle: the codes against exact rational arithmetic, the
fp32 division that the device uses against the same, and the router's choices
on hand-made rows."""

from fractions import Fraction

import numpy as np
import pytest

import oracle as O


def _bf16_values(rng, n):
    """Random bf16 bit patterns of one sign and a few binades, with their values."""
    bits = (rng.integers(0x3000, 0x4200, n)).astype(np.uint16)
    return bits, O.f64_from_bf16_bits(bits)


def _exact_code(v, a):
    q = Fraction(v) * 127 / Fraction(a)
    low = q.numerator // q.denominator
    rest = q - low
    if rest > Fraction(1, 2) or (rest == Fraction(1, 2) and low % 2):
        low += 1
    return low


def test_codes_equal_exact_quotients():
    rng = np.random.default_rng(0)
    _, v = _bf16_values(rng, 400)
    rows = np.stack([v, -v])
    codes, scales = O.int8_rows(rows)
    a = np.abs(v).max()
    ref = [_exact_code(float(x), float(a)) for x in v]
    assert codes[0].tolist() == ref
    assert codes[1].tolist() == [-x for x in ref]          # rint is odd
    assert scales[0] == np.float32(a) / np.float32(127)    # one correctly rounded division


def test_every_mantissa_pair_decides_in_fp32():
    """All 128 x 128 mantissas at distances 0..9: one fp32 division rounds to the
    exact code, ties included (127 v is exact: 15 bits)."""
    man = np.arange(128, 256, dtype=np.float32)
    v, a = np.meshgrid(man, man, indexing="ij")
    ties = 0
    for d in range(10):
        vs = v * np.float32(2.0 ** -d)
        ok = vs <= a
        q32 = np.rint((vs * np.float32(127)) / a)
        num = (v.astype(np.int64) * 127) * 2
        den = a.astype(np.int64) * 2 ** d * 2
        low = num // den
        twice = 2 * (num - low * den)
        up = (twice > den) | ((twice == den) & (low % 2 == 1))
        ties += int(((twice == den) & ok).sum())
        assert np.array_equal(q32[ok], (low + up)[ok].astype(np.float32))
    assert ties > 0


def test_special_rows():
    x = np.zeros((4, 64), dtype=np.uint16)
    x[1, 3] = 0x7FC0      # NaN
    x[2, 5] = 0xFF80      # -infinity
    x[3, 7] = 0x0001      # the smallest subnormal
    codes, scales = O.act_int8(x)
    assert not codes[:3].any() and codes[3, 7] == 127
    assert scales[0] == 0 and np.isnan(scales[1]) and np.isnan(scales[2])


def test_packed_rows_are_the_decoded_weights():
    sb = 0x5A5A1234
    w = (0.05 * np.random.default_rng(3).standard_normal((6, 96))).astype(np.float32)
    p = O.pack(w, sb)
    codes, scales = O.int8_cache_packed(p, sb)
    what = O.dequant(p, sb)
    step = scales.astype(np.float64)[:, None]
    assert np.all(np.abs(codes * step - what) <= 0.5000001 * step)
    assert (np.abs(codes).max(axis=1) == 127).all()


def test_router_choices_by_hand():
    inf = np.inf
    ids, w = O.router_scored([[0.0, 1.0, 1.0, -1.0]], 3)
    assert ids.tolist() == [[1, 2, 0]]
    p = np.exp([1.0, 1.0, 0.0]) / np.exp([0.0, 1.0, 1.0, -1.0]).sum()
    assert np.allclose(w[0], p, rtol=1e-15)
    # the bias moves the choice, not the weight
    ids, w = O.router_scored([[0.0, 0.0]], 1, "sigmoid", bias=[0.0, 0.1], scale=3.0)
    assert ids.tolist() == [[1]] and w[0, 0] == 1.5
    # two groups of three: {2, 2, -9} beats {3, -9, -9}
    ids, _ = O.router_scored([[3.0, -9.0, -9.0, 2.0, 2.0, -9.0]], 2, "sigmoid", n_groups=2,
                             topk_groups=1)
    assert ids.tolist() == [[3, 4]]
    # nothing left: id -1, weight 0
    ids, w = O.router_scored([[-inf, 1.0], [-inf, -inf], [np.nan, -inf]], 2, renormalize=True)
    assert ids.tolist() == [[1, -1], [-1, -1], [-1, -1]]
    assert w.tolist() == [[1.0, 0.0], [0.0, 0.0], [0.0, 0.0]]


@pytest.mark.parametrize("topk", [1, 2])
def test_moe_of_one_expert_is_two_layers(topk):
    rng = np.random.default_rng(1)
    x = O.bf16_bits_from_f32(rng.standard_normal((3, 64)).astype(np.float32))
    w1 = [O.int8_rows(rng.standard_normal((32, 64))) for _ in range(2)]
    w2 = [O.int8_rows(rng.standard_normal((64, 32))) for _ in range(2)]
    ids = np.tile(np.arange(topk, dtype=np.int32), (3, 1))
    g = np.full((3, topk), 0.5, dtype=np.float32)
    out, _ = O.moe_int8(x, ids, g, w1, w2)
    ref = 0
    for e in range(topk):
        u = O.linear_int8(*O.act_int8(x), *w1[e])
        h = O.bf16_bits_from_f32((np.maximum(u, 0) ** 2).astype(np.float32))
        ref = ref + 0.5 * O.linear_int8(*O.act_int8(h), *w2[e])
    assert np.allclose(out, ref, rtol=1e-13)
