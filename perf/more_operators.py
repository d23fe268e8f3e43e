"""Measured cases of the MXFP4 operators and of the router's training side.

Four operators, each as a user's program calls it:

* ``quant``   bf16 rows to MXFP4 codes and scale bytes, and the values these stand
              for (``ops.act_mxfp4``, ``ops.mxfp4_values``);
* ``linear``  the MXFP4 linear layer: bf16 rows quantized per 32-block, a resident
              MXFP4 copy of the weights, fp32 or bf16 output with the optional bias
              and residual (``ops.linear_mxfp4*``);
* ``moe``     the 128-expert ReLU^2 layer on MXFP4 experts (``ops.moe_grouped_mxfp4``);
* ``balance`` the router's training step: per-expert counts, mean probabilities and
              balance loss (``ops.moe_balance``), then the gradient of gates and loss
              with respect to the router logits (``ops.moe_router_backward``).

MXFP4: 32 consecutive values of a row share a scale 2^e, e the smallest integer from
-127 with max|v| < 7 * 2^e, held as the byte e + 127; a value is held as the nearest
of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (with sign) to v / 2^e, ties to the even code, 6 at
most.  Two codes a byte, the first in the low half; rows are padded with zeros to a
multiple of 128 values.

``run`` computes them in plain torch operations, or, with ``own`` set, through the
package's entry points.
"""

import math

import torch

own = False

DEV = "cuda"
BLOCK = 32
STEP = 128  # rows of codes are padded to a multiple of this


def _padded(k):
    return (k + STEP - 1) // STEP * STEP


# ---------------------------------------------------------------------------
# Cases

def listed():
    return [
        # the hidden rows of one 16-token diffusion block: launch latency
        dict(name="quant_block16", op="quant", m=16, k=2688),
        # a prompt's inner activations
        dict(name="quant_prompt", op="quant", m=4096, k=8192),
        # autoregressive decoding of one sequence: one token through a projection
        dict(name="linear_token", op="linear", m=1, k=2688, n=8192, out="fp32", bias=False,
             residual=False),
        # one diffusion block
        dict(name="linear_block16", op="linear", m=16, k=2688, n=8192, out="fp32", bias=False,
             residual=False),
        # a ragged batch of blocks through an output projection with the residual stream
        dict(name="linear_ragged", op="linear", m=333, k=1856, n=2688, out="bf16", bias=True,
             residual=True),
        # a 4096-token prefill through an output projection, bf16 residual stream
        dict(name="linear_prefill_out", op="linear", m=4096, k=8192, n=2688, out="bf16",
             bias=False, residual=True),
        # one token, one block, 64 blocks with popular experts and padding, and a prompt
        dict(name="moe_token", op="moe", t=1, e=128, topk=6, k=2688, n1=1856, routing="uniform",
             padded=0),
        dict(name="moe_block16", op="moe", t=16, e=128, topk=6, k=2688, n1=1856,
             routing="uniform", padded=0),
        dict(name="moe_step1024_zipf", op="moe", t=1024, e=128, topk=6, k=2688, n1=1856,
             routing="zipf", padded=24),
        dict(name="moe_prompt4096", op="moe", t=4096, e=128, topk=6, k=2688, n1=1856,
             routing="uniform", padded=0),
        # the router's step on 64 short sequences, some experts switched off
        dict(name="balance_step1024", op="balance", t=1024, e=128, topk=6, score="softmax",
             renorm=False, scale=1.0, masked=0.05, padded=24),
        # the same on a long packed batch with sigmoid scores
        dict(name="balance_prompt", op="balance", t=16411, e=256, topk=8, score="sigmoid",
             renorm=True, scale=2.5, masked=0.0, padded=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "moe", "balance"])
    if op == "quant":
        return dict(op=op, m=_log_int(rng, 1, 4096), k=32 * _log_int(rng, 1, 256))
    if op == "linear":
        k = 32 * _log_int(rng, 2, 256)
        return dict(op=op, m=_log_int(rng, 1, 4096), k=k,
                    n=_log_int(rng, 17, min(8192, 8192 * 2688 // k)),
                    out=rng.choice(["fp32", "bf16"]),
                    bias=rng.random() < 0.5, residual=rng.random() < 0.5)
    if op == "moe":
        e = rng.choice([8, 40, 64, 128])
        t = _log_int(rng, 1, 3000)
        return dict(op=op, t=t, e=e, topk=rng.randint(1, min(8, e)), k=32 * rng.randint(8, 84),
                    n1=32 * rng.randint(4, 58), routing=rng.choice(["uniform", "zipf"]),
                    padded=rng.randint(0, t // 4))
    e = rng.choice([5, 16, 60, 128, 160, 256, 512])
    t = _log_int(rng, 1, 16411)
    return dict(op=op, t=t if e <= 256 else min(t, 8192), e=e, topk=rng.randint(1, min(8, e)),
                score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.6,
                scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.0, 0.1, 0.5]),
                padded=rng.randint(0, t // 5))


# ---------------------------------------------------------------------------
# Inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 29)
    return g


def _rows(g, m, k):
    """Activations: N(0, 1) with a few channels several times larger, bf16."""
    gain = torch.ones(k, device=DEV)
    gain[torch.randint(0, k, (max(1, k // 128),), generator=g, device=DEV)] = 6.0
    return (torch.randn(m, k, generator=g, device=DEV) * gain).to(torch.bfloat16)


def _cache(g, n, k):
    """MXFP4 weights as the layers keep them: codes [n][kp / 2], then scale bytes
    [n][kp / 32]."""
    kp = _padded(k)
    cache = torch.zeros(n * kp // 2 + n * kp // BLOCK, dtype=torch.uint8, device=DEV)
    codes = cache[:n * kp // 2].view(n, kp // 2)
    scales = cache[n * kp // 2:].view(n, kp // BLOCK)
    part = max(1, (1 << 26) // k)
    for i in range(0, n, part):
        w = 0.02 * torch.randn(min(part, n - i), k, generator=g, device=DEV)
        c, e = _encode(w)
        codes[i:i + part, :k // 2] = c[:, 0::2] | (c[:, 1::2] << 4)
        scales[i:i + part, :k // BLOCK] = (e + 127).to(torch.uint8)
    return cache


def _logits(g, t, e, routing):
    if routing == "uniform":
        return torch.randn(t, e, generator=g, device=DEV)
    p = torch.arange(1, e + 1, device=DEV, dtype=torch.float64) ** -1.1
    u = torch.rand(t, e, generator=g, device=DEV, dtype=torch.float64).clamp_(1e-12, 1 - 1e-12)
    return (torch.log(p / p.sum()) - torch.log(-torch.log(u))).float()


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    if case["op"] == "quant":
        s["x"] = _rows(g, case["m"], case["k"])
    elif case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        s["x"] = _rows(g, m, k)
        s["cache"] = _cache(g, n, k)
        s["b"] = torch.randn(n, generator=g, device=DEV) if case["bias"] else None
        kind = torch.float32 if case["out"] == "fp32" else torch.bfloat16
        s["r"] = (torch.randn(m, n, generator=g, device=DEV).to(kind) if case["residual"]
                  else None)
    elif case["op"] == "moe":
        t, e, topk, k, n1 = (case[x] for x in ("t", "e", "topk", "k", "n1"))
        s["x"] = _rows(g, t, k)
        s["w1"] = _cache(g, e * n1, k)
        s["w2"] = _cache(g, e * k, n1)
        score, ids = torch.topk(_logits(g, t, e, case["routing"]), topk, dim=1)
        gates = torch.exp(score - score[:, :1])
        s["gates"] = (gates / gates.sum(dim=1, keepdim=True)).contiguous()
        ids = ids.to(torch.int32)
        if case["padded"]:  # the rows that fill up a batch are routed nowhere
            ids[t - case["padded"]:] = -1
        s["ids"] = ids.contiguous()
    else:
        t, e, topk = case["t"], case["e"], case["topk"]
        l = 1.5 * torch.randn(t, e, generator=g, device=DEV)
        if case["masked"]:
            off = torch.rand(t, e, generator=g, device=DEV) < case["masked"]
            l.masked_fill_(off, float("-inf"))
        # experts as a router with a balance bias chooses them
        b = 0.1 * torch.randn(e, generator=g, device=DEV)
        p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, dim=1)
        value, ids = torch.topk((p + b).masked_fill(torch.isinf(l), float("-inf")), topk, dim=1)
        ids = ids.masked_fill(torch.isinf(value), -1).to(torch.int32)
        if case["padded"]:
            ids[t - case["padded"]:] = -1
        s["logits"], s["ids"] = l, ids.contiguous()
        s["dgates"] = torch.randn(t, topk, generator=g, device=DEV)
        s["dloss"] = torch.full((), 0.01, device=DEV)
    return s


# ---------------------------------------------------------------------------
# One pass

def run(s):
    if own:
        return _own(s)
    return {"quant": _plain_quant, "linear": _plain_linear, "moe": _plain_moe,
            "balance": _plain_balance}[s["op"]](s)


def _own(s):
    from block_diffusion_lm_tq4_amd import ops

    if s["op"] == "quant":
        codes, scales = ops.act_mxfp4(s["x"])
        return ops.mxfp4_values(codes, scales, s["k"])
    if s["op"] == "linear":
        if s["out"] == "bf16":
            return ops.linear_mxfp4_epilogue_bf16(s["x"], s["cache"], s["n"], s["b"], s["r"])
        if s["b"] is not None or s["r"] is not None:
            return ops.linear_mxfp4_epilogue(s["x"], s["cache"], s["n"], s["b"], s["r"])
        return ops.linear_mxfp4(s["x"], s["cache"], s["n"])
    if s["op"] == "moe":
        return ops.moe_grouped_mxfp4(s["x"], s["ids"], s["gates"], s["w1"], s["w2"], s["e"],
                                     s["n1"])
    loss, counts, tokens, mean = ops.moe_balance(s["logits"], s["ids"], score=s["score"])
    grad = ops.moe_router_backward(s["logits"], s["ids"], s["dgates"], score=s["score"],
                                   renormalize=s["renorm"], scale=s["scale"], counts=counts,
                                   tokens=tokens, dloss=s["dloss"])
    return loss, counts, tokens, mean, grad


LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _pow2(e):
    """2^e in fp32 for int32 e from -126 to 127 (0 for -127, an all-zero block's)."""
    return ((e + 127) << 23).view(torch.float32)


def _encode(v):
    """fp32 [rows, k] -> codes (uint8 [rows, k]) and exponents (int32 [rows, k / 32])."""
    rows, k = v.shape
    b = v.reshape(rows, k // BLOCK, BLOCK)
    bits = b.abs().amax(dim=2).view(torch.int32)
    # a quarter of the exponent's step carries magnitudes from 1.75 * 2^j on into the
    # next exponent: the largest |v| / 2^e is then in [3.5, 7)
    e = (((bits + 0x200000) >> 23) - 2).clamp(min=0) - 127
    u = (b * _pow2(-e)[:, :, None]).abs()
    c = torch.zeros_like(b, dtype=torch.uint8)
    # halfway points between neighbouring levels: up where the upper code is even
    for i, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        c += u >= mid if i % 2 else u > mid
    c |= (b < 0).to(torch.uint8) << 3
    return c.reshape(rows, k), e


def _decode(codes, e, k):
    """Values (fp32 [rows, k]) of packed codes [rows, >= k / 2] and exponents."""
    rows = codes.shape[0]
    levels = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=DEV)
    c = codes[:, :k // 2]
    v = torch.stack((levels[(c & 15).int()], levels[(c >> 4).int()]), dim=2)
    return (v.view(rows, k // BLOCK, BLOCK) * _pow2(e)[:, :, None]).view(rows, k)


def _rounded(v):
    """fp32 rows at the values that their codes stand for."""
    rows, k = v.shape
    c, e = _encode(v)
    levels = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=DEV)
    return (levels[c.int()].view(rows, k // BLOCK, BLOCK) * _pow2(e)[:, :, None]).view(rows, k)


def _weights(cache, n, k):
    kp = _padded(k)
    codes = cache[:n * kp // 2].view(n, kp // 2)
    e = cache[n * kp // 2:].view(n, kp // BLOCK)[:, :k // BLOCK].int() - 127
    return _decode(codes, e, k)


def _plain_quant(s):
    return _rounded(s["x"].float()).to(torch.bfloat16)


def _plain_linear(s):
    w = _weights(s["cache"], s["n"], s["k"])
    y = _rounded(s["x"].float()) @ w.t()
    if s["b"] is not None:
        y = y + s["b"]
    if s["r"] is not None:
        y = y + s["r"].float()
    return y if s["out"] == "fp32" else y.to(torch.bfloat16)


def _plain_moe(s):
    """Pairs sorted by expert into a padded [experts, capacity] grid, one batched
    product for each projection."""
    e, topk, k, n1 = s["e"], s["topk"], s["k"], s["n1"]
    t = s["x"].shape[0]
    flat = s["ids"].reshape(-1).long()
    good = (flat >= 0) & (flat < e)
    key = torch.where(good, flat, torch.full_like(flat, e))
    expert, pair = torch.sort(key, stable=True)
    counts = torch.zeros(e + 1, dtype=torch.long, device=DEV).index_add_(
        0, key, torch.ones_like(key))
    place = torch.arange(t * topk, device=DEV) - (torch.cumsum(counts, 0) - counts)[expert]
    cap = max(1, int(counts[:e].max()))
    used = expert < e
    cell = torch.where(used, expert * cap + place, torch.full_like(expert, e * cap))
    grid = torch.full((e * cap + 1,), -1, dtype=torch.long, device=DEV)
    grid[cell] = torch.where(used, pair, torch.full_like(pair, -1))
    grid = grid[:e * cap].view(e, cap)
    x = _rounded(s["x"].float())
    live = (grid >= 0)[:, :, None]
    a = (x[grid.clamp(min=0) // topk] * live).transpose(1, 2).contiguous()
    u = torch.bmm(_weights(s["w1"], e * n1, k).view(e, n1, k), a).transpose(1, 2)
    h = torch.clamp(u, min=0).square().reshape(e * cap, n1)
    a = _rounded(h).view(e, cap, n1).transpose(1, 2).contiguous()
    o = torch.bmm(_weights(s["w2"], e * k, n1).view(e, k, n1), a).transpose(1, 2)
    o = torch.cat([o.reshape(e * cap, k), torch.zeros(1, k, device=DEV)])
    back = torch.empty_like(cell)
    back[pair] = cell
    return (o[back].view(t, topk, k) * s["gates"][:, :, None]).sum(dim=1)


def _plain_balance(s):
    """Probabilities in 32 bits, sums over tokens in 64."""
    l, ids = s["logits"], s["ids"].long()
    t, e = l.shape
    on = l > float("-inf")
    if s["score"] == "sigmoid":
        p = (1.0 / (1.0 + torch.exp(-l))).masked_fill(~on, 0.0)
        total = p.sum(dim=1, keepdim=True)
    else:
        p = torch.exp(l - l.amax(dim=1, keepdim=True)).masked_fill(~on, 0.0)
        p = p / torch.where(on.any(dim=1), p.sum(dim=1), torch.ones(t, device=DEV))[:, None]
        total = torch.ones(t, 1, device=DEV)
    q = torch.where(total > 0, p / total, torch.zeros_like(p))
    used = (ids >= 0) & (ids < e)
    live = used.any(dim=1, keepdim=True)
    tokens = live.sum()
    counts = torch.zeros(e + 1, dtype=torch.int32, device=DEV).index_add_(
        0, torch.where(used, ids, torch.full_like(ids, e)).view(-1),
        torch.ones(ids.numel(), dtype=torch.int32, device=DEV))[:e]
    mean = (q * live).sum(dim=0, dtype=torch.float64) / tokens.clamp(min=1)
    share = counts.double() / counts.sum().clamp(min=1)
    loss = e * (share * mean).sum()
    # the loss sees the probabilities only: d loss / d q_te = e * share_e / tokens
    dq = (s["dloss"] * e * share / tokens.clamp(min=1)).float() * live
    dl = q * (dq - (q * dq).sum(dim=1, keepdim=True))
    if s["score"] == "sigmoid":
        dl = dl * (1.0 - p)
    # the gates
    at = torch.where(used, ids, torch.zeros_like(ids))
    w = p.gather(1, at) * used
    dw = s["dgates"] * used * s["scale"]
    if s["renorm"]:
        sums = w.sum(dim=1, keepdim=True)
        w = torch.where(sums > 0, w / sums, torch.zeros_like(w))
        dw = dw - (w * dw).sum(dim=1, keepdim=True)
    part = w * dw
    if s["score"] == "sigmoid":
        part = part * (1.0 - p.gather(1, at))
    dl = dl.scatter_add(1, at, part)
    if s["score"] == "softmax" and not s["renorm"]:
        dl = dl - p * part.sum(dim=1, keepdim=True)
    return loss.float(), counts, tokens.to(torch.int32), mean.float(), dl


# ---------------------------------------------------------------------------
# What one pass cannot do without

def _touched(case):
    """Experts that at least one of the routed tokens is expected to visit."""
    t, e, topk = case["t"] - case["padded"], case["e"], case["topk"]
    if case["routing"] == "uniform":
        share = [topk / e] * e
    else:
        p = [(i + 1) ** -1.1 for i in range(e)]
        total = sum(p)
        share = [min(1.0, topk * x / total) for x in p]
    return sum(1.0 - (1.0 - x) ** t for x in share)


def work(case):
    if case["op"] == "quant":
        m, k = case["m"], case["k"]
        # values in, values out; codes and scales written and read between
        return {"bytes": 4 * m * k + 2 * (m * k // 2 + m * k // BLOCK), "flops": 4 * m * k}
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        each = 4 if case["out"] == "fp32" else 2
        return {"bytes": 2 * m * k + n * k // 2 + n * k // BLOCK + each * m * n +
                (each * m * n if case["residual"] else 0) + (4 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    if case["op"] == "moe":
        t, topk, k, n1 = case["t"], case["topk"], case["k"], case["n1"]
        pairs = (t - case["padded"]) * topk
        return {"bytes": 2 * t * k + _touched(case) * 2 * (n1 * k // 2 + n1 * k // BLOCK) +
                8 * t * topk + 4 * t * k, "flops": 4 * pairs * n1 * k}
    t, e, topk = case["t"], case["e"], case["topk"]
    # logits read by each half of the step, their gradient written once
    return {"bytes": 12 * t * e + 12 * t * topk + 8 * e, "flops": 20 * t * e}


# ---------------------------------------------------------------------------
# The same values in 64 bits

def _pow2_64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _value64(c):
    """The e2m1 value of a code 0 .. 15: sign, two exponent bits, one mantissa bit."""
    c = c.long()
    exp, man = (c >> 1) & 3, (c & 1).double()
    v = torch.where(exp == 0, 0.5 * man, (1 + 0.5 * man) * _pow2_64(exp - 1))
    return torch.where(c >= 8, -v, v)


def _mx64(v):
    """Rows in 64 bits at their MXFP4 values."""
    rows, k = v.shape
    b = v.double().view(rows, k // BLOCK, BLOCK)
    top = b.abs().amax(dim=2, keepdim=True)
    man, exp = torch.frexp(top)  # top = man * 2^exp, man in [0.5, 1)
    e = exp - 3 + (man >= 0.875)
    e = torch.where(top > 0, e, torch.full_like(e, -127)).clamp(min=-127)
    u = b * _pow2_64(-e)
    # spacing of the levels around u: 0.5 below 2, 1 below 4, 2 above; torch.round ties
    # to even multiples, which are the even codes
    a = u.abs()
    gap = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    r = (torch.round(a / gap) * gap).clamp(max=6.0)
    return (torch.sign(u) * r * _pow2_64(e)).view(rows, k)


def _w64(cache, n, k):
    kp = _padded(k)
    c = cache[:n * kp // 2].view(n, kp // 2)[:, :k // 2]
    e = cache[n * kp // 2:].view(n, kp // BLOCK)[:, :k // BLOCK].long() - 127
    v = torch.empty(n, k, dtype=torch.float64, device=DEV)
    v[:, 0::2] = _value64(c & 15)
    v[:, 1::2] = _value64(c >> 4)
    return (v.view(n, k // BLOCK, BLOCK) * _pow2_64(e)[:, :, None]).view(n, k)


def _exact_linear(s):
    y = torch.mm(_mx64(s["x"]), _w64(s["cache"], s["n"], s["k"]).t().contiguous())
    for extra in (s["b"], s["r"]):
        if extra is not None:
            y += extra.double()
    return y


def _exact_moe(s):
    e, topk, k, n1, t = s["e"], s["topk"], s["k"], s["n1"], s["t"]
    x = _mx64(s["x"])
    out = torch.zeros(t, k, dtype=torch.float64, device=DEV)
    kp, n1p = _padded(k), _padded(n1)

    def expert(cache, i, n, kk, kkp):
        rows = cache[:e * n * kkp // 2].view(e, -1)[i]
        scales = cache[e * n * kkp // 2:].view(e, -1)[i]
        return _w64(torch.cat([rows, scales]), n, kk)

    for i in range(e):
        tok, slot = torch.nonzero(s["ids"] == i, as_tuple=True)
        if tok.numel() == 0:
            continue
        u = torch.mm(x[tok], expert(s["w1"], i, n1, k, kp).t().contiguous())
        # the layer's hidden value is an fp32 number
        h = _mx64(torch.relu(u).pow(2).float())
        o = torch.mm(h, expert(s["w2"], i, k, n1, n1p).t().contiguous())
        out.index_add_(0, tok, o * s["gates"][tok, slot].double()[:, None])
    return out


def _exact_balance(s):
    """By automatic differentiation of the definition in 64 bits."""
    l, ids = s["logits"].double(), s["ids"].long()
    t, e = l.shape
    off = torch.isinf(l)
    z = torch.where(off, torch.full_like(l, -800.0), l).requires_grad_()
    if s["score"] == "sigmoid":
        p = torch.where(off, torch.zeros_like(z), torch.sigmoid(z))
        q = p / p.sum(dim=1, keepdim=True).clamp(min=1e-300)
    else:
        p = torch.where(off, torch.zeros_like(z), torch.softmax(z, dim=1))
        q = p
    live = ((ids >= 0) & (ids < e)).any(dim=1)
    tokens = int(live.sum())
    counts = torch.bincount(ids[ids >= 0], minlength=e)
    mean = q[live].sum(dim=0) / max(1, tokens)
    loss = e * torch.dot(counts.double() / max(1, int(counts.sum())), mean)
    w = p.gather(1, ids.clamp(min=0)) * (ids >= 0)
    if s["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    total = (s["scale"] * w * s["dgates"].double()).sum() + s["dloss"].double() * loss
    grad, = torch.autograd.grad(total, z)
    return loss.detach(), None, None, mean.detach(), grad


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        return _mx64(s["x"])
    return {"linear": _exact_linear, "moe": _exact_moe, "balance": _exact_balance}[case["op"]](s)
