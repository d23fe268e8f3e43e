"""Pins of the MXFP4 and router-training oracle: each compares it with something
other than itself -- closed forms, explicit loops, differences, automatic
differentiation."""

import numpy as np
import pytest
import torch

import oracle as O
from block_diffusion_lm_tq4_amd import inputs as I

SB = I.sign_bits()


def test_e2m1_values_by_bits():
    for c in range(16):
        exp, man = (c >> 1) & 3, c & 1
        v = man * 0.5 if exp == 0 else (1 + man / 2) * 2.0 ** (exp - 1)
        assert O.e2m1_values()[c] == (-v if c & 8 else v)


def test_scale_rule_closed_forms():
    def byte(v):
        row = np.zeros((1, 32))
        row[0, 5] = v
        return int(O.mxfp4_rows(row)[1][0, 0])
    assert byte(0.0) == 0
    assert byte(6.0) == 127 and byte(-6.0) == 127 and byte(np.nextafter(7.0, 0)) == 127
    assert byte(7.0) == 128 and byte(3.5) == 127 and byte(np.nextafter(3.5, 0)) == 126
    assert byte(7 * 2.0 ** 20) == 148 and byte(6.9 * 2.0 ** -127) == 0
    assert byte(7 * 2.0 ** -127) == 1 and byte(1e-300) == 0
    assert byte(float(np.finfo(np.float32).max)) == 253
    assert byte(np.nan) == byte(np.inf) == byte(-np.inf) == 255


def test_rounding_to_the_nearest_level_by_search():
    rng = np.random.default_rng(0)
    v = rng.uniform(-6.99, 6.99, (200, 32))
    v[:, 0] = 6.99                                        # scale 2^0
    v[0, 1:15] = [.25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5]
    codes, scales = O.mxfp4_rows(v)
    assert np.all(scales == 127)
    val = O.e2m1_values()
    for i in range(200):
        for j in range(32):
            d = np.abs(val - v[i, j])
            near = [c for c in np.nonzero(d == d.min())[0] if (c >= 8) == (v[i, j] < 0)]
            pick = near[0] if len(near) == 1 else [c for c in near if c % 2 == 0][0]
            assert codes[i, j] == pick


def test_values_are_fixed_points_and_errors_stay_within_half_a_step():
    rng = np.random.default_rng(1)
    v = rng.standard_normal((50, 96)) * 2.0 ** rng.integers(-20, 20, (50, 1))
    c, s = O.mxfp4_rows(v)
    d = O.mxfp4_values(c, s)
    c2, s2 = O.mxfp4_rows(d)
    assert np.array_equal(O.mxfp4_values(c2, s2), d)
    unit = np.ldexp(1.0, s.astype(int) - 127).repeat(32, axis=1)
    assert np.all(np.abs(d - v) <= unit)                  # half of the widest step, 2
    assert np.all(np.abs(d - v)[np.abs(v) < 2 * unit] <= 0.25 * unit[np.abs(v) < 2 * unit])


def test_nibbles_round_trip():
    c = np.random.default_rng(2).integers(0, 16, (5, 64)).astype(np.uint8)
    assert np.array_equal(O.unpack_nibbles(O.pack_nibbles(c)), c)
    assert O.pack_nibbles(np.array([[1, 2]], np.uint8))[0, 0] == 0x21


def test_linear_by_explicit_loops():
    rng = np.random.default_rng(3)
    x = O.bf16_bits_from_f32(rng.standard_normal((3, 64)).astype(np.float32))
    p = O.pack(I.weights(4, 64), SB)
    xq, xs = O.act_mxfp4(x)
    wq, ws = O.mxfp4_cache_packed(p, SB)
    y = O.linear_mxfp4(xq, xs, wq, ws)
    val = O.e2m1_values()
    for m in range(3):
        for n in range(4):
            s = sum(val[xq[m, i]] * 2.0 ** (int(xs[m, i // 32]) - 127) * val[wq[n, i]]
                    * 2.0 ** (int(ws[n, i // 32]) - 127) for i in range(64))
            assert s == y[m, n]


def test_nonfinite_blocks_are_nan():
    x = O.bf16_bits_from_f32(np.ones((2, 64), np.float32))
    x[1, 40] = 0x7FC0
    c, s = O.act_mxfp4(x)
    # 7 * 2^-3 <= 1 < 7 * 2^-2
    assert s[1].tolist() == [125, 255] and not c[1, 32:].any()
    d = O.mxfp4_values(c, s)
    assert np.isnan(d[1, 32:]).all() and not np.isnan(d[1, :32]).any()


def test_moe_by_explicit_pairs():
    rng = np.random.default_rng(4)
    t, e, k, n1, topk = 4, 3, 64, 32, 2
    x = O.bf16_bits_from_f32(rng.standard_normal((t, k)).astype(np.float32))
    w1 = [O.mxfp4_rows(rng.standard_normal((n1, k))) for _ in range(e)]
    w2 = [O.mxfp4_rows(rng.standard_normal((k, n1))) for _ in range(e)]
    ids = np.array([[0, 2], [1, -1], [2, 2], [7, -5]])
    g = rng.standard_normal((t, topk))
    out, _ = O.moe_mxfp4(x, ids, g, w1, w2)
    want = np.zeros((t, k))
    xd = O.mxfp4_values(*O.act_mxfp4(x))
    for i in range(t):
        for j in range(topk):
            if 0 <= ids[i, j] < e:
                u = O.mxfp4_values(*w1[ids[i, j]]) @ xd[i]
                h = (np.maximum(u, 0).astype(np.float32) ** 2).astype(np.float64)
                want[i] += g[i, j] * (O.mxfp4_values(*w2[ids[i, j]])
                                      @ O.mxfp4_values(*O.mxfp4_rows(h[None]))[0])
    assert np.allclose(out, want, rtol=1e-13, atol=1e-13)
    assert not out[3].any()


def _case(score, seed=5):
    rng = np.random.default_rng(seed)
    t, e, topk = 6, 9, 3
    l = 2 * rng.standard_normal((t, e))
    ids = np.argsort(-l, axis=1)[:, :topk].copy()
    ids[2] = -1                                           # routed nowhere
    ids[3, 1] = 99
    ids[4, 2] = ids[4, 0]                                 # one expert twice
    l[5, 4] = -np.inf
    return l, ids, rng.standard_normal((t, topk))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_backward_against_differences(score, renorm):
    l, ids, dg = _case(score)
    loss, counts, tokens, mean = O.moe_balance(l, ids, score)

    def value(z):
        s = sum(float(dg[i] @ O.router_gates(z[i], ids[i], score, renorm, 1.7))
                for i in range(len(z)))
        return s + 0.3 * O.moe_balance(z, ids, score)[0]

    grad, _ = O.moe_router_backward(l, ids, dg, score, renorm, 1.7, counts, tokens, 0.3)
    h = 1e-5
    for i in range(l.shape[0]):
        for j in range(l.shape[1]):
            if np.isinf(l[i, j]):
                assert grad[i, j] == 0
                continue
            a, b = l.copy(), l.copy()
            a[i, j] += h
            b[i, j] -= h
            # central differences: h^2 / 6 of third derivatives of order 1, and 1e-16 / h
            assert abs((value(a) - value(b)) / (2 * h) - grad[i, j]) < 1e-9


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_backward_against_autograd(score, renorm):
    l, ids, dg = _case(score, seed=6)
    _, counts, tokens, _ = O.moe_balance(l, ids, score)
    grad, _ = O.moe_router_backward(l, ids, dg, score, renorm, 0.7, counts, tokens, 2.0)
    off = torch.from_numpy(np.isinf(l))
    z = torch.from_numpy(np.where(np.isinf(l), -50.0, l)).requires_grad_()
    i = torch.from_numpy(ids)
    ok = (i >= 0) & (i < l.shape[1])
    p = (torch.sigmoid(z) if score == "sigmoid" else
         torch.softmax(z.masked_fill(off, float("-inf")), dim=1))
    p = p.masked_fill(off, 0.0)
    q = p / p.sum(dim=1, keepdim=True)
    mean = q[ok.any(dim=1)].mean(dim=0)
    loss = l.shape[1] * (torch.from_numpy(counts / counts.sum()) * mean).sum()
    w = p.gather(1, i.where(ok, torch.zeros_like(i))) * ok
    if renorm:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    (0.7 * (w * torch.from_numpy(dg)).sum() + 2.0 * loss).backward()
    assert np.allclose(grad, z.grad.numpy(), rtol=1e-12, atol=1e-14)


def test_an_even_router_has_loss_one():
    l = np.zeros((8, 4))
    ids = np.array([[i % 4] for i in range(8)])
    loss, counts, tokens, mean = O.moe_balance(l, ids)
    assert loss == 1.0 and counts.tolist() == [2] * 4 and tokens == 8
    assert O.moe_balance(l[:0], ids[:0])[0] == 0.0
