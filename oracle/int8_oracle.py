"""int8 layers and the scored router, written out plainly in NumPy fp64.

TEST INFRASTRUCTURE ONLY -- imported by ``tests/``; never by the product path.
It shares no code with the HIP library.

Readings (Nemotron-TheHobbit-30B-A3B model card, *Running it*: the projections
every forward runs; *The model underneath*: 128 experts, top-6):

* a row v with a = max|v| is held as codes rint(127 v / a), ties to even, and
  the scale fp32(a / 127); zero rows have scale 0, rows with a NaN or an
  infinity zero codes and scale NaN;
* weights: one such row per output channel, of the decoded TQ4_1S weights or of
  BF16 weights; activations: one per token;
* y[m, n] = (sum_k xq wq) * sx[m] * sw[n], the sum exact;
* the MoE layer keeps its hidden rows relu(u)^2 in bf16 (rounded from fp32) and
  quantizes them like the activations;
* the router: softmax or sigmoid scores over the experts whose logit is a number
  above -inf, a bias that only the choice sees (-inf or NaN: never chosen), groups
  valued by their two best experts, ties to the lower index, weights
  renormalized and scaled.
"""

from __future__ import annotations

import numpy as np

from .tq4_oracle import (BLOCK, RS32, bf16_bits_from_f32, dequant_rotated, f64_from_bf16_bits,
                         hadamard32, signs_from_bits)

__all__ = ["int8_rows", "act_int8", "int8_cache_packed", "linear_int8", "moe_int8",
           "router_scored"]


def int8_rows(v: np.ndarray, unit: float = 1.0) -> tuple[np.ndarray, np.ndarray]:
    """Rows unit * v (fp64) -> (codes int8 [rows, k], scales fp32 [rows])."""
    v = np.asarray(v, dtype=np.float64)
    top = np.max(np.abs(v), axis=1) if v.shape[1] else np.zeros(v.shape[0])
    good = np.isfinite(v).all(axis=1)
    live = good & (top > 0)
    codes = np.zeros(v.shape, dtype=np.int8)
    codes[live] = np.rint((v[live] * 127.0) / top[live, None]).astype(np.int8)
    scales = np.full(v.shape[0], np.nan, dtype=np.float32)
    scales[good] = ((top[good] * unit) / 127.0).astype(np.float32)
    return codes, scales


def act_int8(x_bf16: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """bf16 bit patterns [m, k] -> (codes, scales)."""
    return int8_rows(f64_from_bf16_bits(x_bf16))


def int8_cache_packed(packed: np.ndarray, sign_bits: int) -> tuple[np.ndarray, np.ndarray]:
    """Packed TQ4_1S rows [n][k/32][20] -> (codes, scales) of the decoded weights.

    The common factor 1/sqrt(32) of a row is left out of the quotients and
    enters the scale, so the codes come from exact sums."""
    z = dequant_rotated(packed)
    n = z.shape[0]
    v = (z.reshape(n, -1, BLOCK) @ hadamard32().T) * signs_from_bits(sign_bits)
    return int8_rows(v.reshape(n, -1), RS32)


def linear_int8(xq, sx, wq, sw, bias=None, residual=None) -> np.ndarray:
    """The layer in fp64 from codes and scales."""
    acc = np.asarray(xq, np.float64) @ np.asarray(wq, np.float64).T
    y = acc * np.asarray(sx, np.float64)[:, None] * np.asarray(sw, np.float64)[None, :]
    if bias is not None:
        y = y + np.asarray(bias, np.float64)[None, :]
    if residual is not None:
        y = y + np.asarray(residual, np.float64)
    return y


def moe_int8(x_bf16, ids, gates, w1, w2):
    """The MoE layer in fp64; w1, w2: per-expert lists of (codes, scales).

    Returns (out [t, k], the sum of |gate * o| per output)."""
    t, topk = ids.shape
    k = x_bf16.shape[1]
    out = np.zeros((t, k))
    mag = np.zeros((t, k))
    xq, sx = act_int8(x_bf16)
    for i in range(t):
        for j in range(topk):
            e = ids[i, j]
            if e < 0 or e >= len(w1):
                continue
            u = linear_int8(xq[i:i + 1], sx[i:i + 1], *w1[e])
            h = np.where(u < 0, 0.0, u * u).astype(np.float32)
            hq, sh = act_int8(bf16_bits_from_f32(h))
            o = float(gates[i, j]) * linear_int8(hq, sh, *w2[e])[0]
            out[i] += o
            mag[i] += np.abs(o)
    return out, mag


def router_scored(logits, topk, score="softmax", bias=None, n_groups=1, topk_groups=1,
                  renormalize=False, scale=1.0):
    """(ids int32 [t, topk], weights fp64 [t, topk]), one token after another."""
    logits = np.asarray(logits, dtype=np.float64)
    t, e = logits.shape
    per = e // n_groups
    ids = np.full((t, topk), -1, dtype=np.int32)
    w = np.zeros((t, topk))
    for i in range(t):
        on = [x for x in range(e) if logits[i, x] > -np.inf]
        l = np.minimum(logits[i], float(np.finfo(np.float32).max))
        p = np.zeros(e)
        if on and score == "softmax":
            z = np.exp(l[on] - l[on].max())
            p[on] = z / z.sum()
        elif on:
            with np.errstate(over="ignore"):
                p[on] = 1.0 / (1.0 + np.exp(-l[on]))
        c = {x: p[x] + (0.0 if bias is None else float(bias[x])) for x in on}
        c = {x: v for x, v in c.items() if v > -np.inf}
        value = []
        for g in range(n_groups):
            best = sorted((v for x, v in c.items() if x // per == g), reverse=True)[:2]
            if best:
                value.append((-sum(best), g))
        kept = {g for _, g in sorted(value)[:topk_groups]}
        order = sorted((-v, x) for x, v in c.items() if x // per in kept)[:topk]
        for j, (_, x) in enumerate(order):
            ids[i, j] = x
            w[i, j] = p[x]
        if not order or renormalize and not w[i].sum() > 0:
            continue  # zeros, whatever the factor
        if renormalize:
            w[i] /= w[i].sum()
        w[i, :len(order)] *= scale
    return ids, w
