"""The scored router at the ends of its range: scores below fp64's normal range,
slots without an expert, biases that bar an expert, and more tokens than one
launch holds.  Ids are equal to the fp64 oracle's and weights one rounding
(2^-24 relative, and fp32's last bit where they are subnormal) of its own.
"""

import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_int8 import _check_router, _ops, dev  # noqa: F401

pytestmark = pytest.mark.gpu


# four tokens a wave; that and its fp64 pass (equal biases: the border is not
# clear); a wave a token, by its slots and by its groups
FORMS = [(64, 4, 1, 1, False), (64, 4, 1, 1, True), (256, 8, 8, 4, False), (64, 15, 1, 1, False),
         (102, 6, 17, 4, False)]


@pytest.mark.parametrize("e,topk,groups,keep,equal", FORMS)
@pytest.mark.parametrize("scale", [1.0, 2.5])
def test_router_renormalizes_scores_below_the_normal_range(dev, e, topk, groups, keep, equal,
                                                           scale):
    """A bias brings in experts whose softmax scores are fp64 subnormals: the sum's
    reciprocal is infinite, its quotients are not.  Scores are above e^-716 > 2^-1034
    and so have 40 bits, of which two exponentials may differ in the last."""
    rng = np.random.default_rng(e + topk)
    lg = (-714.0 - 1.9 * rng.random((40, e))).astype(np.float32)
    lg[:, ::3] = -np.abs(rng.standard_normal((40, lg[:, ::3].shape[1])))
    lg[:, 0] = 0
    bias = np.full(e, 3.0, np.float32) if equal else rng.permutation(e).astype(np.float32) + 3
    bias[::3] = -3
    ids, w = _check_router(dev, lg, topk, score="softmax", bias=bias, n_groups=groups,
                           topk_groups=keep, renormalize=True, scale=scale)
    assert (ids.cpu().numpy() % 3 != 0).all()
    total = w.cpu().numpy().astype(np.float64).sum(axis=1)
    assert (np.abs(total - scale) <= scale * topk * 2.0 ** -24).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,topk,groups,keep", [(6, 5, 1, 1), (64, 15, 1, 1), (34, 4, 17, 2)])
@pytest.mark.parametrize("scale", [np.inf, -np.inf, np.nan])
def test_router_slots_without_an_expert_weigh_nothing(dev, score, e, topk, groups, keep, scale):
    """Rows with 0, 1, ... experts on, under a factor that is no number."""
    lg = np.full((topk + 2, e), -np.inf, np.float32)
    for i in range(topk + 2):
        lg[i, :i] = np.arange(i) / 8
    lg[topk + 1, :topk] = np.nan
    for renorm in (False, True):
        ids, w = _ops().moe_router_scored(torch.from_numpy(lg).to(dev), topk, score=score,
                                          n_groups=groups, topk_groups=keep, renormalize=renorm,
                                          scale=scale)
        ri, rw = O.router_scored(lg, topk, score, None, groups, keep, renorm, scale)
        assert np.array_equal(ids.cpu().numpy(), ri) and (ri < 0).any()
        assert np.array_equal(w.cpu().numpy(), rw.astype(np.float32), equal_nan=True)
        assert (rw[ri < 0] == 0).all()
    low = torch.full((3, e), -800.0, device=dev)     # sigmoid scores of 0: nothing to divide by
    ids, w = _ops().moe_router_scored(low, topk, score="sigmoid", n_groups=groups,
                                      topk_groups=keep, renormalize=True, scale=scale)
    assert (ids >= 0).all() and (w == 0).all()


def _repeat(rows, t):
    """The given rows over and over, t in all."""
    return rows.repeat((t + len(rows) - 1) // len(rows), 1)[:t]


# past 2^32 threads at 16 and at 64 threads a token
@pytest.mark.parametrize("t,e,topk,groups,keep", [(2 ** 28 + 21, 2, 1, 1, 1),
                                                  (2 ** 26 + 13, 17, 2, 17, 2)])
def test_router_of_more_tokens_than_a_launch_holds(dev, t, e, topk, groups, keep):
    lg = np.random.default_rng(e).standard_normal((997, e)).astype(np.float32)
    base, base_w = _check_router(dev, lg, topk, score="sigmoid", n_groups=groups,
                                 topk_groups=keep)
    ids, w = _ops().moe_router_scored(_repeat(torch.from_numpy(lg).to(dev), t), topk,
                                      score="sigmoid", n_groups=groups, topk_groups=keep)
    assert torch.equal(ids, _repeat(base, t)) and torch.equal(w, _repeat(base_w, t))


def test_softmax_router_of_more_tokens_than_a_launch_holds(dev):
    t, e, topk = 2 ** 26 + 13, 3, 2
    lg = torch.from_numpy(np.random.default_rng(1).standard_normal((997, e)).astype(np.float32))
    base, base_w = _ops().moe_router(lg.to(dev), topk)
    ri, rw = O.router_scored(lg.numpy(), topk)
    assert np.array_equal(base.cpu().numpy(), ri) and np.allclose(base_w.cpu().numpy(), rw, 1e-5)
    ids, w = _ops().moe_router(_repeat(lg.to(dev), t), topk)
    assert torch.equal(ids, _repeat(base, t)) and torch.equal(w, _repeat(base_w, t))


# by the fp32 choice, by its fp64 pass (a bias of +inf), by the wave a token
@pytest.mark.parametrize("case", ["fast", "again", "wave"])
@pytest.mark.parametrize("barred", [-np.inf, np.nan])
def test_router_bias_that_bars_leaves_the_softmax_alone(dev, barred, case):
    """exp(l) = 1, 2, 4, 1 over and over, 64 in all over 32 experts.  The fours are
    barred but keep their share, so that weights are 2 / 64 and 1 / 64."""
    e, topk = 32, 16 if case == "wave" else 10
    lg = torch.log(torch.tensor([1.0, 2.0, 4.0, 1.0], dtype=torch.float64)).float().to(dev)
    bias = torch.zeros(e)
    bias[2::4] = barred
    if case == "again":
        bias[5] = np.inf
    ids, w = _ops().moe_router_scored(lg.repeat(5, e // 4), topk, bias=bias.to(dev))
    two, one = list(range(1, 32, 4)), sorted([*range(0, 32, 4), *range(3, 32, 4)])
    order = [5] + [x for x in two if x != 5] if case == "again" else two
    assert ids.cpu().tolist() == [(order + one)[:topk]] * 5
    ref = torch.tensor([2 / 64] * 8 + [1 / 64] * (topk - 8), dtype=torch.float64)
    # log 2 and log 4 are off by 2^-25 and 2^-24, their shares of the sum make 0.63 *
    # 2^-24 of that, and the weight is rounded: 2.2 * 2^-24
    assert ((w.cpu().double() - ref).abs() <= 3 * 2.0 ** -24 * ref).all()
