"""GPU parity of the router's training step against the fp64 oracle.

Counts and tokens are equal.  A score is e^x of a difference x of two fp32 logits:
x carries one rounding, 2^-24 |x| of it, its exponential at most 4 ulp more
(2^-22), so with X the largest |x| of a row each score is off by at most (X + 8) 2^-24
of itself, a sum of scores by that and one rounding per addition (a lane's up to 32
values, then 4), a normalized score by twice it and 2^-23 for the division.  The
gradient multiplies one score with a difference of two weighted means of scores: within
(4 X + 160) 2^-24 of the sum of its terms' magnitudes.  Means over tokens add a
rounding per token of a lane.  Sigmoid scores have x up to |l|, so X is taken over
those too.
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


def _case(t, e, topk, seed, spread=2.0, masked=0.1):
    rng = np.random.default_rng(seed)
    l = (spread * rng.standard_normal((t, e))).astype(np.float32)
    if e > 4:
        l[rng.random((t, e)) < masked] = -np.inf
    ids = np.argsort(-l + rng.random((t, e)), axis=1)[:, :topk].astype(np.int32)
    ids[rng.random((t, topk)) < 0.1] = -1
    ids[rng.random((t, topk)) < 0.05] = e + 1
    if t > 3:
        ids[1] = -1
        l[2] = -np.inf                                   # a row without experts
        l[t - 1, 0] = np.nan
    return l, ids, rng.standard_normal((t, topk)).astype(np.float32)


def _reach(l):
    fin = np.where(np.isfinite(l), l, np.nan)
    both = np.concatenate([fin, np.zeros((l.shape[0], 1))], axis=1)
    with np.errstate(invalid="ignore"):
        return np.nanmax(both, axis=1) - np.nanmin(both, axis=1)


def _check(dev, l, ids, dg, score, renorm, scale, dloss, x=None):
    o = _ops()
    lg, ig = torch.from_numpy(l).to(dev), torch.from_numpy(ids).to(dev)
    loss, counts, tokens, mean = o.moe_balance(lg, ig, score=score)
    rl, rc, rt, rm = O.moe_balance(l, ids, score)
    x = _reach(l) if x is None else x
    worst = (2 * x.max(initial=0.0) + 120) * U
    assert np.array_equal(counts.cpu().numpy(), rc) and int(tokens) == rt
    assert np.all(np.abs(mean.double().cpu().numpy() - rm) <= worst * rm + 1e-37)
    assert abs(float(loss) - rl) <= worst * abs(rl) + 1e-37
    for gates in (True, False):
        for with_loss in (True, False):
            grad = o.moe_router_backward(
                lg, ig, torch.from_numpy(dg).to(dev) if gates else None, score=score,
                renormalize=renorm, scale=scale, counts=counts if with_loss else None,
                tokens=tokens if with_loss else None,
                dloss=torch.full((1,), dloss, device=dev) if with_loss else None)
            want, size = O.moe_router_backward(l, ids, dg if gates else None, score, renorm, scale,
                                               rc if with_loss else None, rt, np.float32(dloss))
            err = np.abs(grad.double().cpu().numpy() - want)
            # scores below fp32's normal range may vanish
            tol = ((4 * x + 160) * U)[:, None] * size + 1e-36 * (1 + np.abs(dg).max(initial=0.0))
            assert np.all(err <= tol), (gates, with_loss, np.max(err / np.maximum(size, 1e-30)))
            if not gates and not with_loss:
                assert not grad.any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("t,e,topk", [(1, 1, 1), (1, 128, 6), (2, 5, 5), (16, 128, 6), (17, 64, 8),
                                      (100, 60, 4), (63, 160, 8), (65, 256, 8), (300, 7, 2),
                                      (40, 512, 20), (9, 512, 512), (33, 130, 17), (1500, 128, 6)])
def test_against_oracle(dev, t, e, topk, score, renorm):
    l, ids, dg = _case(t, e, topk, seed=t + e)
    _check(dev, l, ids, dg, score, renorm, 2.5, 0.3)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_long_batch(dev, score):
    t, e, topk = 16411, 256, 8
    rng = np.random.default_rng(1)
    l = rng.standard_normal((t, e)).astype(np.float32)
    ids = np.argsort(-l, axis=1)[:, :topk].astype(np.int32)
    o = _ops()
    loss, counts, tokens, mean = o.moe_balance(torch.from_numpy(l).to(dev),
                                               torch.from_numpy(ids).to(dev), score=score)
    p = np.exp(l.astype(np.float64))
    if score == "sigmoid":
        p = p / (1 + p)
    q = p / p.sum(axis=1, keepdims=True)
    assert int(tokens) == t
    assert np.array_equal(counts.cpu().numpy(), np.bincount(ids.ravel(), minlength=e))
    assert np.all(np.abs(mean.double().cpu().numpy() - q.mean(axis=0)) <= 150 * U * q.mean(axis=0))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_extreme_logits(dev, score, renorm):
    e, topk = 12, 3
    big = 3.0e38
    l = np.zeros((8, e), np.float32)
    l[0] = -200.0                                        # sigmoid scores below fp32's range
    l[0, :3] = [-201, -200, -202]
    l[1] = 200.0
    l[2, 3] = np.inf                                     # counts as the largest finite value
    l[3] = -big
    l[4] = big
    l[5] = np.nan
    l[6] = -np.inf
    l[6, 5] = 1.0                                        # one expert left
    l[7, ::2] = -90.0
    ids = np.tile(np.array([[0, 1, 2]], np.int32), (8, 1))
    ids[2] = [3, 0, 1]
    ids[6] = [5, -1, -1]
    ids[7] = [0, 2, 4]                                   # chosen by their bias alone
    dg = np.random.default_rng(0).standard_normal((8, topk)).astype(np.float32)
    # differences of logits of one magnitude are exact here
    _check(dev, l, ids, dg, score, renorm, 1.0, 0.5, x=np.full(8, 210.0))


def test_one_expert_in_several_slots(dev):
    rng = np.random.default_rng(2)
    t, e, topk = 50, 20, 18
    l = rng.standard_normal((t, e)).astype(np.float32)
    ids = rng.integers(0, 4, (t, topk)).astype(np.int32)
    dg = rng.standard_normal((t, topk)).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            _check(dev, l, ids, dg, score, renorm, 1.5, 1.0)
    o = _ops()
    a = [torch.from_numpy(v).to(dev) for v in (l, ids, dg)]
    first = o.moe_router_backward(*a)
    for _ in range(5):
        assert torch.equal(o.moe_router_backward(*a), first)


def test_routed_nowhere(dev):
    o = _ops()
    l = torch.randn(40, 16, device=dev)
    ids = torch.full((40, 2), -1, dtype=torch.int32, device=dev)
    loss, counts, tokens, mean = o.moe_balance(l, ids)
    assert float(loss) == 0 and int(tokens) == 0 and not counts.any() and not mean.any()
    grad = o.moe_router_backward(l, ids, torch.randn(40, 2, device=dev), counts=counts,
                                 tokens=tokens, dloss=torch.ones((), device=dev))
    assert not grad.any()
    loss, counts, tokens, mean = o.moe_balance(l[:0], ids[:0])
    assert float(loss) == 0 and int(tokens) == 0 and not counts.any() and not mean.any()
    assert o.moe_router_backward(l[:0], ids[:0]).shape == (0, 16)


@pytest.mark.parametrize("e", [128, 30])
def test_unaligned_logits(dev, e):
    rng = np.random.default_rng(3)
    t, topk = 37, 4
    l = rng.standard_normal((t, e)).astype(np.float32)
    ids = np.argsort(-l, axis=1)[:, :topk].astype(np.int32)
    dg = rng.standard_normal((t, topk)).astype(np.float32)
    o = _ops()
    buf = torch.zeros(t * e + 1, device=dev)
    lg = buf[1:].view(t, e)
    lg.copy_(torch.from_numpy(l))
    ig, dgg = torch.from_numpy(ids).to(dev), torch.from_numpy(dg).to(dev)
    store = torch.full((t * e + 5,), 9.0, device=dev)
    out = store[3:3 + t * e].view(t, e)
    o.moe_router_backward(lg, ig, dgg, out=out)
    want, size = O.moe_router_backward(l, ids, dg)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= 200 * U * size)
    assert (store[:3] == 9).all() and (store[3 + t * e:] == 9).all()
    assert np.array_equal(o.moe_balance(lg, ig)[1].cpu().numpy(), O.moe_balance(l, ids)[1])


def test_gradient_against_differences(dev):
    """The gradient of the router's own gates and of the loss, against central differences
    of both by the kernels: the truncation is h^2 / 6 times third derivatives of order
    1, the rounding of a difference 2 * 2^-23 of the sum's magnitude over 2 h."""
    o = _ops()
    rng = np.random.default_rng(4)
    t, e, topk, h = 4, 8, 3, 2.0 ** -7
    l = torch.from_numpy(rng.standard_normal((t, e)).astype(np.float32)).to(dev)
    dg = torch.from_numpy(rng.standard_normal((t, topk)).astype(np.float32)).to(dev)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids, _ = o.moe_router_scored(l, topk, score=score, renormalize=renorm, scale=2.0)
            loss, counts, tokens, _ = o.moe_balance(l, ids, score=score)
            grad = o.moe_router_backward(l, ids, dg, score=score, renormalize=renorm, scale=2.0,
                                         counts=counts, tokens=tokens,
                                         dloss=torch.ones((), device=dev)).double().cpu()

            def value(z):
                n, g = o.moe_router_scored(z, topk, score=score, renormalize=renorm, scale=2.0)
                order = (n[:, None, :] == ids[:, :, None]).int().argmax(dim=2)
                assert torch.equal(n.sort(dim=1).values, ids.sort(dim=1).values)
                return (float((g.gather(1, order).double() * dg.double()).sum())
                        + float(o.moe_balance(z, ids, score=score)[0]))

            for i in range(t):
                for j in range(e):
                    a, b = l.clone(), l.clone()
                    a[i, j] += h
                    b[i, j] -= h
                    # 6 * 2^-14 / 6 of truncation, 40 * 2^-23 / 2^-6 of rounding
                    assert abs((value(a) - value(b)) / (2 * h) - grad[i, j]) < 3e-4 + 3e-4


def test_a_training_step_from_logits_to_gradient(dev):
    """Router, MXFP4 experts, statistics and gradient as a program runs them: the
    gradient of sum(out) + 0.01 loss with respect to the logits."""
    o = _ops()
    from block_diffusion_lm_tq4_amd import inputs as I
    rng = np.random.default_rng(5)
    t, e, topk, k, n1 = 48, 8, 2, 128, 96
    x = O.bf16_bits_from_f32(rng.standard_normal((t, k)).astype(np.float32))
    l = rng.standard_normal((t, e)).astype(np.float32)
    w1 = O.bf16_bits_from_f32(I.weights(e * n1, k, seed=1))
    w2 = O.bf16_bits_from_f32(I.weights(e * k, n1, seed=2))
    as_bf16 = lambda b: torch.from_numpy(b.view(np.int16)).to(dev).view(torch.bfloat16)
    c1, c2 = o.mxfp4_cache_bf16(as_bf16(w1)), o.mxfp4_cache_bf16(as_bf16(w2))
    lg = torch.from_numpy(l).to(dev)
    ids, gates = o.moe_router_scored(lg, topk, renormalize=True)
    out = o.moe_grouped_mxfp4(as_bf16(x), ids, gates, c1, c2, e, n1)
    loss, counts, tokens, _ = o.moe_balance(lg, ids)
    # d sum(out) / d gates: each slot's output alone, summed
    dgates = torch.stack([o.moe_grouped_mxfp4(as_bf16(x), ids[:, j:j + 1].contiguous(),
                                              torch.ones(t, 1, device=dev), c1, c2, e, n1)
                          .sum(dim=1) for j in range(topk)], dim=1).contiguous()
    grad = o.moe_router_backward(lg, ids, dgates, renormalize=True, counts=counts, tokens=tokens,
                                 dloss=torch.full((), 0.01, device=dev))
    rid, rg = O.router_scored(l, topk, renormalize=True)
    assert np.array_equal(ids.cpu().numpy(), rid)
    split = lambda w, n: [tuple(v[i * n:(i + 1) * n] for v in O.act_mxfp4(w)) for i in range(e)]
    r1, r2 = split(w1, n1), split(w2, k)
    want, size = O.moe_mxfp4(x, rid, rg, r1, r2)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= 32 * 2.0 ** -23 * size)
    rdg = np.stack([O.moe_mxfp4(x, rid[:, j:j + 1], np.ones((t, 1)), r1, r2)[0].sum(axis=1)
                    for j in range(topk)], axis=1)
    _, rc, rt, _ = O.moe_balance(l, rid)
    rgrad, rsize = O.moe_router_backward(l, rid, rdg, renormalize=True, counts=rc, tokens=rt,
                                         dloss=0.01)
    # dgates are sums of k terms whose magnitudes the layer's bound covers
    slack = 256 * U * np.abs(size).sum(axis=1, keepdims=True)
    assert np.all(np.abs(grad.double().cpu().numpy() - rgrad) <= 200 * U * rsize + slack)


def test_captured_step_replays(dev):
    o = _ops()
    t, e, topk = 70, 32, 4
    l = torch.randn(t, e, device=dev)
    dg = torch.randn(t, topk, device=dev)
    dl = torch.full((), 0.1, device=dev)

    def step():
        ids, gates = o.moe_router_scored(l, topk)
        loss, counts, tokens, mean = o.moe_balance(l, ids)
        return ids, loss, counts, tokens, mean, o.moe_router_backward(
            l, ids, dg, counts=counts, tokens=tokens, dloss=dl)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(4):
        l.copy_(torch.randn(t, e, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)
