"""How many digits a log-probability next to 0 keeps."""
import numpy as np
import pytest

from tests.gpu_harness import ensure_built, need_gpu
from tests.test_gpu_choose import _close, _run_top

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    need_gpu()
    ensure_built()


@pytest.mark.parametrize("run", ["eager", "executor"])
def test_log_probability_of_a_likely_token(run):
    """Two tokens, logits 0 and -gap: log-probability -log(1 + e^-gap), e^-gap at most 0.136.

    In units of 2^-24: the sum's one rounding, next to 1, is 1 at most. The other exponential is off by its argument's
    roundings, a product's and those of log2 e in 24 bits, 1.25 of gap, times gap e^-gap (0.28 at most), and by ex2's four of
    itself: 0.35 + 0.55. The logarithm, below 2^-3, is off by one in its last place, 0.13, and both differences are exact: 2.03."""
    rng = np.random.default_rng(17)
    gap = rng.uniform(2.0, 20.0, 4096).astype(np.float32)
    x = np.zeros((4096, 2), np.float32)
    at = rng.integers(0, 2, 4096)
    x[np.arange(4096), 1 - at] = -gap
    ids, lp, lse = _run_top(run, x, True, 0, 1)
    assert (ids[:, 0] == at).all()
    want = np.log1p(np.exp(-gap.astype(np.float64)))
    _close(lp[:, 0], -want, 2.03 * 2.0 ** -24, "logprobs")
    _close(lse, want, 2.03 * 2.0 ** -24, "lse")
