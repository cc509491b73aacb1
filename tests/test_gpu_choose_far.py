"""Experts' groups whose sums of two no float holds."""
import numpy as np
import pytest

from tests.gpu_harness import ensure_built, need_gpu
from tests.test_gpu_choose import _run_experts
from tests.test_gpu_choose_order import _choice

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    need_gpu()
    ensure_built()


@pytest.mark.parametrize("run", ["eager", "executor"])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("E,K,groups,keep", [(64, 6, 8, 3), (96, 4, 3, 1), (256, 8, 8, 4), (512, 10, 16, 7), (1024, 20, 32, 9)])
def test_groups_by_sums_beyond_fp32(E, K, groups, keep, sigmoid, run):
    rng = np.random.default_rng(E)
    x = rng.standard_normal((7, E)).astype(np.float32)
    size = E // groups
    at = np.arange(groups) * size
    up, down = np.zeros(E, np.float32), np.zeros(E, np.float32)
    worth = rng.permutation(groups)
    # each finite and none near another, their sums beyond 3.4e38
    up[at + 1], up[at + size - 1] = 1.8e38 + worth * 4e36, 1.75e38 + worth * 4.3e36
    down[:] = np.repeat(-1.8e38 - worth * 4e36, size) - np.tile(np.arange(size) * 2e34, groups)
    some = np.where(np.arange(E) // size % 2 == 0, 0.1 * rng.standard_normal(E), -3.4028235e38).astype(np.float32)  # masked by the lowest value
    shut = some.copy()
    shut[:size] = -np.inf
    for bias in (up, down, some, shut):
        ids, _ = _run_experts(run, x, True, 0, K, bias, sigmoid=sigmoid, groups=groups, keep=keep, top2=True)
        with np.errstate(invalid="ignore"):
            want = np.array([_choice(r, K, sigmoid, bias, groups, keep, True) for r in x])
        assert (ids == want).all(), (np.argwhere((ids != want).any(1)).ravel(), ids[(ids != want).any(1)][:2], want[(ids != want).any(1)][:2])
