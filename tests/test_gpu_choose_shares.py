"""Weights of experts far below a row's largest logit."""
import numpy as np
import pytest

from tests import choose_ref as R
from tests.gpu_harness import ensure_built, need_gpu
from tests.test_gpu_choose import _close, _run_experts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    need_gpu()
    ensure_built()


@pytest.mark.parametrize("run", ["eager", "executor"])
@pytest.mark.parametrize("E,K", [(64, 8), (256, 8), (512, 10), (256, 20)])
def test_shares_of_far_experts(E, K, run):
    """A bias chooses experts 33 to 79 below the largest, whose distance from it no float holds: as exact as all others."""
    rng = np.random.default_rng(E)
    x = (-rng.uniform(33, 78, (400, 1)) + 35 + rng.uniform(0, 1, (400, E))).astype(np.float32)
    x[:, 7] = np.float32(35.123457)
    bias = (2 + rng.random(E)).astype(np.float32)
    bias[7] = -3.0
    for normalise in (True, False):
        ids, w = _run_experts(run, x, True, 0, K, bias, sigmoid=False, groups=1, keep=1, top2=False, normalise=normalise, scale=1.0)
        wids, ww = R.experts(x, K, False, bias, 1, 1, False, normalise, 1.0)
        assert (ids == wids).all()
        # a score: ex2 2^-22, four roundings of 2^-24 (the exponential's correction, 1 / the row's sum, a product, the
        # distance's rest): 2^-21. A sum of scores is off by as much and by five roundings (2^-24 each, 32 lanes), a quotient by two
        # in its last place, 2^-22: 2^-20 + 5 x 2^-24 + 2^-22 < 1.6 x 2^-20
        _close(w, ww, 1.6 * 2.0 ** -20 * ww)


@pytest.mark.parametrize("run", ["eager", "executor"])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("E,K", [(64, 4), (256, 8), (512, 10), (600, 5)])
def test_infinite_logits_share_the_weight(E, K, biased, run):
    rng = np.random.default_rng(E)
    x = rng.standard_normal((6, E)).astype(np.float32)
    x[0, 9] = x[1, 3] = x[1, 60] = x[2, 5] = np.inf
    x[2, 7] = 3.3e38
    x[3] = np.inf
    x[4, ::2] = np.inf
    bias = np.full(E, 0.5, np.float32) if biased else None
    ids, w = _run_experts(run, x, True, 0, K, bias, sigmoid=False, groups=1, keep=1, top2=False, normalise=False, scale=1.0)
    for r in range(5):
        at = np.flatnonzero(np.isposinf(x[r]))
        n = min(len(at), K)
        assert ids[r, :n].tolist() == at[:n].tolist()
        _close(w[r, :n], np.full(n, 1.0 / len(at)), 2.0 ** -18 / len(at))
        assert (w[r, n:] == 0).all()
    _close(w[5], R.experts(x[5:], K, False, bias, 1, 1, False, False, 1.0)[1][0], R.EXPERTS_TOL)
