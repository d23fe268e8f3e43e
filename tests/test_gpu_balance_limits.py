"""The router's training step where sums are long or differences cancel.

Bounds, in units U = 2^-24, with X the largest difference of two logits of a row.  A score is
off by at most (X + 8) of itself, a normalized one by E = 2 X + 20 (test_gpu_balance.py).
A part of the gradient is r p_e (b_e - sum_i p_i b_i) with r = 1 or 1 - p_e.  It has to be
right relative to S_e = sum_i p_i |b_e - b_i|, which is what is left of it where b_e and
the mean are all but equal.  The b are taken relative to a number m near their mean, so
|b_e - m| <= 2 S_e and sum_i p_i |b_i - m| <= 3 S_e; each difference carries 3 roundings, the
sum E and 40 roundings (a lane's 32 values and the lanes), the factors E and X + 8:
2 E + X + 8 + 2 * 3 + 3 (E + 43) <= 11 X + 250.  The mean that m comes from is off by E + 40 of
the mean magnitude A of the b where they are not integers: 3 roundings of that.
"""

import numpy as np
import pytest
import torch

import oracle as O

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


# ---- sums over tokens ----------------------------------------------------------

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t,e", [(255, 160), (4096, 160), ((1 << 24) + 5, 5), (1 << 22, 24)])
def test_equal_logits(dev, t, e, score):
    """A fresh router's: every addition over tokens rounds the same way.  All probabilities
    are 1 / E up to 8 roundings of the scores' sum (a lane's values and four joins), the
    division and the product; a lane adds at most 8 tokens in fp32 and the rest is fp64;
    the result is rounded once."""
    o = _ops()
    l = torch.zeros(t, e, device=dev)
    ids = (torch.arange(t, device=dev, dtype=torch.int32) % e)[:, None].contiguous()
    ids[5] = -1
    loss, counts, tokens, mean = o.moe_balance(l, ids, score=score)
    assert int(tokens) == t - 1
    want = torch.bincount(ids[ids >= 0].long(), minlength=e)
    assert torch.equal(counts.long(), want)
    assert torch.all((mean.double() * e - 1).abs() <= (8 + 2 + 7 + 1) * U)
    assert abs(float(loss) - 1) <= (8 + 2 + 7 + 1) * U


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_long_batch_with_rows_routed_nowhere(dev, score):
    """Whole rounds of a workgroup's tokens are left out, and the last round is part-filled."""
    o = _ops()
    t, e = 5 * 16384 + 77, 96
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    l = torch.randn(t, e, generator=g, device=dev)
    ids = l.topk(3, dim=1).indices.int()
    ids[16384:3 * 16384] = -1
    ids[::5] = e
    loss, counts, tokens, mean = o.moe_balance(l, ids, score=score)
    live = (ids[:, 0] >= 0) & (ids[:, 0] < e)
    p = torch.softmax(l[live].double(), 1) if score == "softmax" else torch.sigmoid(l[live].double())
    want = (p / p.sum(1, keepdim=True)).mean(0)
    count = torch.bincount(ids[live].flatten().long(), minlength=e)
    assert int(tokens) == int(live.sum()) and torch.equal(counts.long(), count)
    x = float(l.max() - l.min()) + 10.0
    assert torch.all((mean.double() - want).abs() <= (2 * x + 40) * U * want)
    ref = float(e * (count.double() / count.sum() * want).sum())
    assert abs(float(loss) - ref) <= (2 * x + 40) * U * ref


# ---- differences ---------------------------------------------------------------

def _parts(l, score):
    """Normalized scores and 1 - p of every row, fp64."""
    rows = [O.router_scores(r, score) for r in l]
    q = np.array([r[1] for r in rows])
    rest = np.array([r[2] for r in rows]) if score == "sigmoid" else np.ones_like(q)
    return q, rest


def _differences(p, b):
    """p_e (b_e - sum p b) and p_e sum_i p_i |b_e - b_i|, from the differences alone."""
    d = b[:, :, None] - b[:, None, :]
    return p * (d * p[:, None, :]).sum(2), p * (np.abs(d) * p[:, None, :]).sum(2)


def _loss_gradient(o, dev, l, ids, score, dloss):
    lg, ig = torch.from_numpy(l).to(dev), torch.from_numpy(ids).to(dev)
    _, counts, tokens, _ = o.moe_balance(lg, ig, score=score)
    grad = o.moe_router_backward(lg, ig, score=score, counts=counts, tokens=tokens,
                                 dloss=torch.full((), dloss, device=dev))
    n = counts.double().cpu().numpy()
    c = dloss * len(n) * n / (n.sum() * float(tokens))
    return grad.double().cpu().numpy(), np.broadcast_to(c, l.shape)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e", [1, 3, 16, 130, 512])
def test_loss_gradient_of_one_live_expert_is_zero(dev, score, e):
    o = _ops()
    rng = np.random.default_rng(e)
    t = 400
    l = np.full((t, e), -np.inf, np.float32)
    at = rng.integers(0, e, t)
    l[np.arange(t), at] = 3 * rng.standard_normal(t)
    l[::9] = rng.standard_normal((len(l[::9]), e))       # others keep the counts apart
    ids = np.argmax(l, axis=1).astype(np.int32)[:, None]
    grad, _ = _loss_gradient(o, dev, l, ids, score, 0.75)
    one = np.arange(t) % 9 != 0
    assert not grad[one].any()
    if e > 1:
        assert grad[~one].any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e", [2, 16, 130, 512])
@pytest.mark.parametrize("kind", ["dominated", "one count apart", "even", "random"])
def test_loss_gradient_relative_to_differences(dev, score, e, kind):
    o = _ops()
    rng = np.random.default_rng(e)
    t, reach = 64, 18.0
    l = rng.uniform(-0.5, 0.5, (t, e)).astype(np.float32)
    ids = rng.integers(0, e, (t, 1)).astype(np.int32)
    if kind == "dominated":                              # nearly all the weight on one expert
        l -= np.float32(4)
        l[np.arange(t), rng.integers(0, e, t)] += rng.uniform(6, 16, t).astype(np.float32)
    elif kind == "one count apart":
        t = 3 * e + 1
        l = rng.uniform(-0.5, 0.5, (t, e)).astype(np.float32)
        ids = (np.arange(t) % e).astype(np.int32)[:, None]
    elif kind == "even":
        l[:] = 0.25
    grad, c = _loss_gradient(o, dev, l, ids, score, 0.75)
    sub = slice(0, 64)
    q, rest = _parts(l[sub], score)
    want, size = _differences(q, c[sub])
    assert np.all(np.abs(grad[sub] - rest * want) <= (11 * reach + 250) * U * rest * size + 1e-36)


@pytest.mark.parametrize("e,topk", [(2, 1), (8, 1), (16, 3), (130, 8), (512, 20), (40, 40)])
@pytest.mark.parametrize("with_loss", [False, True])
def test_softmax_gates_relative_to_differences(dev, e, topk, with_loss):
    """Weights that are not renormalized: w_j = s p_j, dl_e = p_e (a_e - sum p a)."""
    o = _ops()
    rng = np.random.default_rng(e + topk)
    t, scale, reach = 60, 2.5, 18.0
    l = rng.uniform(-0.5, 0.5, (t, e)).astype(np.float32)
    top = rng.integers(0, e, t)
    # from even rows to one expert 16 above the others
    l[np.arange(t), top] += np.linspace(0, 16, t).astype(np.float32)
    ids = np.argsort(rng.random((t, e)), axis=1)[:, :topk].astype(np.int32)
    ids[::2, 0] = top[::2]                               # may be in two slots then
    dg = rng.standard_normal((t, topk)).astype(np.float32)
    lg, ig, dgg = (torch.from_numpy(v).to(dev) for v in (l, ids, dg))
    a = np.zeros((t, e))
    np.add.at(a, (np.arange(t)[:, None], ids), dg.astype(np.float64))
    b, extra = scale * a, {}
    p, _ = _parts(l, "softmax")
    want, size = _differences(p, b)
    if with_loss:
        _, counts, tokens, _ = o.moe_balance(lg, ig)
        extra = dict(counts=counts, tokens=tokens, dloss=torch.full((), 30.0, device=dev))
        n = counts.double().cpu().numpy()
        c = np.broadcast_to(30.0 * e * n / (n.sum() * float(tokens)), l.shape)
        more, size_c = _differences(p, c)
        want, size = want + more, size + size_c
    grad = o.moe_router_backward(lg, ig, dgg, scale=scale, **extra).double().cpu().numpy()
    # sums of up to topk gradients of one expert, and A's own rounding
    mean = p * (p * np.abs(b)).sum(1, keepdims=True)
    tol = (11 * reach + 250) * U * size + 3 * U * (2 * reach + 60 + topk) * U * mean
    assert np.all(np.abs(grad - want) <= tol + 1e-36), np.max(np.abs(grad - want) / (size + 1e-30))


# ---- slots of experts that are switched off -------------------------------------

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("topk", [3, 20])
def test_a_slot_whose_expert_is_off_adds_nothing(dev, score, renorm, topk):
    """Whatever stands in its gradient, an infinity or a NaN too."""
    o = _ops()
    rng = np.random.default_rng(topk)
    t, e = 30, 24
    l = rng.standard_normal((t, e)).astype(np.float32)
    l[:, 4] = -np.inf
    l[:, 5] = np.nan
    l[7] = -np.inf                                       # a row of only such experts
    ids = np.argsort(rng.random((t, e)), axis=1)[:, :topk].astype(np.int32)
    ids[:, 0], ids[:, topk - 1] = 4, 5
    ids[3, 1] = -1
    dg = rng.standard_normal((t, topk)).astype(np.float32)
    off = np.isin(ids, (4, 5)) | (ids < 0)
    off[7] = True
    args = dict(score=score, renormalize=renorm, scale=1.5)
    lg, ig = torch.from_numpy(l).to(dev), torch.from_numpy(ids).to(dev)
    clean = o.moe_router_backward(lg, ig, torch.from_numpy(np.where(off, 0, dg)).to(dev), **args)
    assert torch.isfinite(clean).all() and not clean[:, 4:6].any() and not clean[7].any()
    # three slots leave one, whose renormalized weight is 1 whatever the logits are
    assert clean.any() == (not renorm or topk > 3)
    for bad in (np.nan, np.inf, -np.inf, 3e38, 1.0):
        d = torch.from_numpy(np.where(off, bad, dg).astype(np.float32)).to(dev)
        assert torch.equal(o.moe_router_backward(lg, ig, d, **args), clean), bad
