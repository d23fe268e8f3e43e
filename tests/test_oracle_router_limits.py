"""Hand-written values of the scored router's oracle at the ends of its range."""

import numpy as np
import pytest

import oracle as O


@pytest.mark.parametrize("scale", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_slots_without_an_expert_weigh_nothing_whatever_the_factor(score, scale):
    lg = [[0.0, -np.inf, -np.inf], [-np.inf, np.nan, -np.inf]]
    for renorm in (False, True):
        ids, w = O.router_scored(lg, 2, score, renormalize=renorm, scale=scale)
        assert ids.tolist() == [[0, -1], [-1, -1]]
        assert np.array_equal(w, [[scale, 0.0], [0.0, 0.0]], equal_nan=True)


def test_a_sum_of_zero_gives_weights_of_zero_whatever_the_factor():
    """exp(800) is infinite in fp64: both scores are 0."""
    with np.errstate(over="ignore"):
        ids, w = O.router_scored([[-800.0, -900.0, -850.0]], 2, "sigmoid", renormalize=True,
                                 scale=np.inf)
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]


@pytest.mark.parametrize("barred", [-np.inf, np.nan])
def test_a_barring_bias_leaves_the_softmax_alone(barred):
    """exp(l) = 1, 2, 4, 1: the barred expert keeps its share of 8; one whose logit is
    off has none."""
    lg = np.log([[1.0, 2.0, 4.0, 1.0]])
    ids, w = O.router_scored(lg, 4, bias=[0.0, 0.0, barred, 0.0])
    assert ids.tolist() == [[1, 0, 3, -1]]
    assert np.allclose(w, [[2 / 8, 1 / 8, 1 / 8, 0]], rtol=1e-15)
    lg[0, 2] = barred
    ids, w = O.router_scored(lg, 4)
    assert ids.tolist() == [[1, 0, 3, -1]]
    assert np.allclose(w, [[2 / 4, 1 / 4, 1 / 4, 0]], rtol=1e-15)
