"""MXFP4 layers and the router's training step, written out plainly in NumPy fp64.

TEST INFRASTRUCTURE ONLY -- imported by ``tests/``; never by the product path.
It shares no code with the HIP library.

Readings (Nemotron-TheHobbit-30B-A3B model card, *Running it*: the projections
every forward runs; *Help wanted*: a resident copy; *The model underneath*: 128
experts, top-6):

* 32 consecutive values of a row share a scale 2^e (byte e + 127), e the smallest
  integer from -127 to 127 with max|v| < 7 * 2^e, or 127 where there is none; a value
  is the e2m1 code nearest to v / 2^e, ties to the even code, 6 at most; a block with a
  NaN or an infinity has byte 255 and zero codes;
* weights: the decoded TQ4_1S weights or BF16 weights; activations: per call;
* y[m, n] = the exact sum of the products of the values;
* the MoE layer quantizes its hidden values fp32(fp32(relu(u))^2) the same way;
* the balance loss and the gradients by their formulas, per token.
"""

from __future__ import annotations

import numpy as np

from .tq4_oracle import dequant, f64_from_bf16_bits

__all__ = ["e2m1_values", "mxfp4_rows", "mxfp4_values", "act_mxfp4", "mxfp4_cache_packed",
           "linear_mxfp4", "moe_mxfp4", "pack_nibbles", "unpack_nibbles", "router_scores",
           "moe_balance", "router_gates", "moe_router_backward"]

_MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_values() -> np.ndarray:
    """Values of the 16 codes."""
    return np.concatenate([_MAG, -_MAG])


def mxfp4_rows(v: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """fp64 rows [rows, k] -> (codes uint8 [rows, k], scale bytes [rows, k / 32])."""
    v = np.asarray(v, dtype=np.float64)
    rows, k = v.shape
    b = v.reshape(rows, k // 32, 32)
    good = np.isfinite(b).all(axis=-1)
    top = np.max(np.abs(np.where(good[..., None], b, 0.0)), axis=-1)
    e = np.full(top.shape, -127, dtype=np.int64)
    for step in (64, 32, 16, 8, 4, 2, 1):         # raise e while 7 * 2^e does not exceed top
        while True:
            up = top >= np.ldexp(7.0, e + step - 1)
            if not up.any():
                break
            e = e + step * up
    e = np.minimum(e, 127)                        # the largest scale: what is larger saturates
    u = np.ldexp(np.where(good[..., None], b, 0.0), -e[..., None])
    a = np.minimum(np.abs(u), 6.0)
    hi = np.searchsorted(_MAG, a, side="left")                   # first level >= a
    lo = np.maximum(hi - 1, 0)
    d_hi, d_lo = np.abs(_MAG[hi] - a), np.abs(a - _MAG[lo])
    code = np.where((d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0)), hi, lo)
    code = code | np.where(np.signbit(u), 8, 0)
    code = np.where(good[..., None], code, 0)
    return (code.reshape(rows, k).astype(np.uint8),
            np.where(good, e + 127, 255).astype(np.uint8))


def mxfp4_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Values (fp64 [rows, k]) of codes and scale bytes; NaN under byte 255."""
    rows, k = codes.shape
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (e2m1_values()[codes].reshape(rows, k // 32, 32) * s[..., None]).reshape(rows, k)


def pack_nibbles(codes: np.ndarray) -> np.ndarray:
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack_nibbles(packed: np.ndarray) -> np.ndarray:
    return np.stack([packed & 15, packed >> 4], axis=-1).reshape(packed.shape[0], -1)


def act_mxfp4(x_bf16: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """bf16 rows (bit patterns) -> (codes, scale bytes)."""
    with np.errstate(invalid="ignore"):
        return mxfp4_rows(f64_from_bf16_bits(x_bf16))


def mxfp4_cache_packed(packed: np.ndarray, sign_bits: int) -> tuple[np.ndarray, np.ndarray]:
    """(codes, scale bytes) of a packed [N][K/32][20] matrix (zeros unsigned)."""
    return mxfp4_rows(dequant(packed, sign_bits) + 0.0)


def linear_mxfp4(xq, xs, wq, ws, bias=None, residual=None) -> np.ndarray:
    """fp64 [m, n]."""
    y = mxfp4_values(xq, xs) @ mxfp4_values(wq, ws).T
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)
    if residual is not None:
        y = y + np.asarray(residual, dtype=np.float64)
    return y


def moe_mxfp4(x_bf16, ids, gates, w1, w2):
    """(out fp64 [t, k], the sum of the magnitudes of its terms) with w1[e], w2[e] = (codes,
    scale bytes) of expert e; ids outside the experts contribute nothing."""
    xd = mxfp4_values(*act_mxfp4(x_bf16))
    ids = np.asarray(ids)
    g = np.asarray(gates, dtype=np.float64)
    out = np.zeros((ids.shape[0], xd.shape[1]))
    size = np.zeros_like(out)
    for e in np.unique(ids):
        if e < 0 or e >= len(w1):
            continue
        rows, js = np.nonzero(ids == e)
        u = xd[rows] @ mxfp4_values(*w1[int(e)]).T
        with np.errstate(over="ignore", invalid="ignore"):
            u = np.where(u < 0, 0.0, u).astype(np.float32)
            h = (u * u).astype(np.float64)
        hd, wd = mxfp4_values(*mxfp4_rows(h)), mxfp4_values(*w2[int(e)])
        np.add.at(out, rows, g[rows, js][:, None] * (hd @ wd.T))
        np.add.at(size, rows, np.abs(g[rows, js])[:, None] * (np.abs(hd) @ np.abs(wd).T))
    return out, size


# ---- the router's training step -----------------------------------------------

def _live_logits(row):
    l = np.asarray(row, dtype=np.float64)
    on = ~np.isnan(l) & (l != -np.inf)
    return np.where(on, np.minimum(l, float(np.finfo(np.float32).max)), -np.inf), on


def router_scores(row, score):
    """(p, q, 1 - p) of one token's logits."""
    l, on = _live_logits(row)
    zero = np.zeros_like(l)
    if not on.any():
        return zero, zero, np.ones_like(l)
    if score == "softmax":
        p = np.where(on, np.exp(l - l.max()), 0.0)
        p = p / p.sum()
        return p, p, 1.0 - p
    big = np.exp(-np.abs(np.where(on, l, 0.0)))
    p = np.where(on, np.where(l >= 0, 1.0, big) / (1.0 + big), 0.0)
    rest = np.where(on, np.where(l >= 0, big, 1.0) / (1.0 + big), 1.0)
    # relative to the largest, so that rows of very negative logits do not vanish
    m = min(l.max(), 0.0)
    rel = np.where(on, np.exp(np.minimum(l, 0.0) - m) / (1.0 + big), 0.0)
    return p, rel / rel.sum(), rest


def moe_balance(logits, ids, score="softmax"):
    """(loss, counts, tokens, mean_p)."""
    t, e = logits.shape
    ids = np.asarray(ids)
    ok = (ids >= 0) & (ids < e)
    counts = np.bincount(ids[ok], minlength=e)
    live = ok.any(axis=1)
    mean = np.zeros(e)
    for i in np.nonzero(live)[0]:
        mean += router_scores(logits[i], score)[1]
    mean = mean / max(1, live.sum())
    loss = e * float(np.sum(counts * mean)) / max(1, counts.sum())
    return loss, counts, int(live.sum()), mean


def router_gates(row, ids, score, renormalize, scale):
    """The gates of one token for its ids (0 for ids outside the experts)."""
    p, _, _ = router_scores(row, score)
    ok = (ids >= 0) & (ids < len(p))
    w = np.where(ok, p[np.where(ok, ids, 0)], 0.0)
    if renormalize:
        w = w / w.sum() if w.sum() > 0 else w * 0.0
    return scale * w


def moe_router_backward(logits, ids, dgates=None, score="softmax", renormalize=False, scale=1.0,
                        counts=None, tokens=None, dloss=None):
    """(d logits fp64 [t, E], sum of the magnitudes of the terms of each element)."""
    t, e = logits.shape
    ids = np.asarray(ids)
    out, size = np.zeros((t, e)), np.zeros((t, e))
    for i in range(t):
        p, q, rest = router_scores(logits[i], score)
        ok = (ids[i] >= 0) & (ids[i] < e)
        if counts is not None and ok.any() and tokens > 0 and counts.sum() > 0:
            c = float(dloss) * e * counts / (counts.sum() * float(tokens))
            k = rest if score == "sigmoid" else 1.0
            out[i] += k * q * (c - np.sum(q * c))
            size[i] += k * q * (np.abs(c) + np.sum(q * np.abs(c)))
        if dgates is None:
            continue
        j = np.nonzero(ok)[0]
        at = ids[i][j]
        d = scale * np.asarray(dgates[i], dtype=np.float64)[j]
        if renormalize:
            l, on = _live_logits(logits[i])
            if not on[at].any():
                continue
            # chosen scores relative to the largest chosen one
            top = l[at].max()
            if score == "softmax":
                w = np.exp(l[at] - top)
            else:
                w = np.exp(np.minimum(l[at], 0) - min(top, 0.0)) / (1 + np.exp(-np.abs(l[at])))
            w = np.where(on[at], w, 0.0)
            w = w / w.sum()
            part = w * (d - np.sum(w * d))
            mag = w * (np.abs(d) + np.sum(w * np.abs(d)))
        else:
            part = p[at] * d
            mag = np.abs(part)
        if score == "sigmoid":
            part, mag = part * rest[at], mag * rest[at]
        np.add.at(out[i], at, part)
        np.add.at(size[i], at, mag)
        if score == "softmax" and not renormalize:
            out[i] -= p * np.sum(part)
            size[i] += p * np.sum(mag)
    return out, size
