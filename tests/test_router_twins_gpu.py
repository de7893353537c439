"""Routing by scores where some experts of a token are the same, logit and bias
(twins), and others come closer to them than fp32 can tell: the choice and the
groups that stay are those of 64 bits, exactly."""
import numpy as np
import pytest

from oracle import training_oracle as O

from test_router_gpu import _check, _many, _run

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -31       # fp32 numbers next to 1/2 lie 2^-25 apart, the pairs' error is below 2^-38


def _rows(rng, T, E, score, twins, near):
    """(logits, bias): every token's experts `twins` have logit and bias 0, those
    of `near` values u that lie whole STEPs, at most 64 and each another number, above
    or below the twins', and all others lie far below."""
    l = np.full((T, E), -4.0, np.float32)
    l[:, twins] = 0
    l[:, near] = rng.integers(1, 64, len(near)) * 2.0 ** -13
    bias = np.zeros(E, np.float32)
    s = O.scores(l[:1], score)[0]
    level = s[twins[0]]
    bias[near] = level - s[near]
    steps = np.argsort(rng.random((T, 128)), 1)[:, :len(near)] - 64.0
    want = level - bias[near].astype(np.float64) + np.where(steps < 0, steps, steps + 1) * STEP
    l[:, near] = np.log(want / (1 - want)) if score == "sigmoid" else np.log(want / level)
    return l, bias


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,twins,near,how", [
    (34, 32, 33, 1, {}), (34, 31, 30, 4, {}), (64, 32, 60, 2, {}), (1024, 32, 400, 3, {}), (1024, 31, 200, 2, {}),
    (1024, 6, 100, 5, {}), (1024, 1, 40, 1, {}), (256, 8, 90, 2, {}), (128, 32, 50, 2, dict(groups=2, top_groups=1, group_top=1)),
    (256, 31, 70, 3, dict(groups=2, top_groups=1, group_top=2))])
@pytest.mark.parametrize("many", [False, True])
def test_twins_past_the_candidates(score, E, k, twins, near, how, many):
    """More twins than candidates have places, close ones of lower and of higher value in front of
    them, between them and behind."""
    rng = np.random.default_rng(E + k)
    for front in (True, False):
        # all of one group; a close one of lower index comes first among equal fp32 values
        at = np.arange(near + twins)
        close = at[:near] if front else np.sort(rng.permutation(at)[:near])
        l, bias = _rows(rng, 64, E, score, np.setdiff1d(at, close), close)
        x, r, dg, dl = _run(_many(l, many), bias, k, score=score, **how)
        _check(x, bias, k, r, dg, dl, score=score, **how)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,top_groups", [(64, 8, 3), (256, 8, 4), (60, 6, 2), (96, 3, 1), (320, 32, 9), (256, 4, 1)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("many", [False, True])
def test_groups_whose_best_are_twins(score, E, groups, top_groups, group_top, many):
    """A group's best by its fp32 values are twins, or one of them and a close one: which of them
    count, and so which groups stay, only 64 bits tell."""
    rng = np.random.default_rng(E + groups + group_top)
    size = E // groups
    for each in (2, 3):
        at = np.stack([g * size + rng.permutation(min(size, 7))[:each + 1] for g in range(groups)])
        l, bias = _rows(rng, 600, E, score, at[:, 1:].reshape(-1), at[:, 0])
        how = dict(score=score, groups=groups, top_groups=top_groups, group_top=group_top)
        x, r, dg, dl = _run(_many(l, many), bias, 4, **how)
        _check(x, bias, 4, r, dg, dl, **how)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,top_groups", [(64, 8, 3), (256, 8, 4), (60, 6, 2), (96, 3, 1), (320, 32, 9)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("many", [False, True])
def test_two_groups_with_a_close_one_next_to_twins(score, E, groups, top_groups, group_top, many):
    """The same where the other groups have twins alone, whose best are certain."""
    rng = np.random.default_rng(2 * E + groups + group_top)
    size = E // groups
    for each in (2, 3):
        at = np.stack([g * size + rng.permutation(min(size, 7))[:each + 1] for g in range(groups)])
        l, bias = _rows(rng, 600, E, score, at[:, 1:].reshape(-1), at[:2, 0])
        how = dict(score=score, groups=groups, top_groups=top_groups, group_top=group_top)
        x, r, dg, dl = _run(_many(l, many), bias, 4, **how)
        _check(x, bias, 4, r, dg, dl, **how)
