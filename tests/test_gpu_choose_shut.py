"""Experts shut by a bias of -infinity, chosen beside others that are near."""
import numpy as np
import pytest

from tests.gpu_harness import ensure_built, need_gpu
from tests.test_gpu_choose import _run_experts
from tests.test_gpu_choose_alike import SHAPES
from tests.test_gpu_choose_order import _choice

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    need_gpu()
    ensure_built()


@pytest.mark.parametrize("run", ["eager", "executor"])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("E,K,groups,keep", SHAPES + [(16, 10, 16, 16), (32, 12, 8, 8)])
def test_shut_experts_beside_near_ones(E, K, groups, keep, sigmoid, run):
    """Fewer live experts than are chosen, two of them near: the others come after them, the lowest first."""
    rng = np.random.default_rng(E * K)
    x = rng.standard_normal((20, E)).astype(np.float32)
    live = rng.permutation(E)[:max(2, K // 2)]
    x[:, live[1]] = x[:, live[0]] + np.float32(2e-7)
    for shut in (-np.inf, np.nan):
        bias = np.full(E, shut, np.float32)
        bias[live] = 0.01 * rng.standard_normal(len(live))
        bias[live[1]] = bias[live[0]]
        clean = np.where(np.isnan(bias), np.float32(-np.inf), bias)
        ids, _ = _run_experts(run, x, True, 0, K, bias, sigmoid=sigmoid, groups=groups, keep=keep, top2=False)
        want = np.array([_choice(r, K, sigmoid, clean, groups, keep, False) for r in x])
        assert (ids == want).all(), (ids[(ids != want).any(1)][:2], want[(ids != want).any(1)][:2])
