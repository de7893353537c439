"""Gates of sigmoid scores that leave the range of fp32, relative to others that do not:
within the tolerance of all gates (test_router_gpu)."""
import numpy as np
import pytest

from test_router_gpu import _check, _many, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("low,high", [(-100, -40), (-130, -55), (-100, 5), (-92, -80), (-300, -200)])
@pytest.mark.parametrize("E,k,how", [(2, 2, {}), (8, 8, dict(groups=2, top_groups=2, group_top=1)), (40, 32, {}), (40, 5, {})])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("many", [False, True])
def test_renormalised_gates_of_small_scores(low, high, E, k, how, biased, many):
    rng = np.random.default_rng(E + k - low)
    l = rng.uniform(low, high, (300, E)).astype(np.float32)
    l[::5, 1:] = low                                             # one score, and others that vanish next to it
    l[1::7, 0] = -np.inf
    bias = rng.standard_normal(E).astype(np.float32) if biased else None
    how = dict(score="sigmoid", scale=2.5, **how)
    x, r, dg, dl = _run(_many(l, many), bias, k, **how)
    _check(x, bias, k, r, dg, dl, **how)
    assert r.device_status() == 0
