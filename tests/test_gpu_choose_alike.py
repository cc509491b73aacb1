"""Experts that are alike, equal logits and biases, between others that only
64-bit arithmetic tells apart."""
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


SHAPES = [(8, 1, 1, 1), (16, 5, 1, 1), (64, 8, 1, 1), (64, 6, 4, 2), (96, 8, 1, 1), (256, 8, 8, 4), (256, 12, 1, 1), (512, 10, 4, 3), (600, 7, 1, 1), (128, 20, 2, 2)]


def _check(run, x, K, bias, f32=True, **kw):
    ids, _ = _run_experts(run, x, f32, 0, K, bias, **kw)
    with np.errstate(all="ignore"):
        want = np.array([_choice(r, K, kw["sigmoid"], bias, kw["groups"], kw["keep"], kw["top2"]) for r in x])
    bad = np.argwhere((ids != want).any(1)).ravel()
    assert bad.size == 0, (bad, ids[bad][:2], want[bad][:2])


@pytest.mark.parametrize("run", ["eager", "executor"])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("E,K,groups,keep", SHAPES)
def test_alike_where_the_choice_ends(E, K, groups, keep, sigmoid, run):
    """Whole logits, so that many are equal, whose scores beside their biases differ by less than fp32 tells."""
    rng = np.random.default_rng(E + K)
    x = np.concatenate([rng.integers(lo, hi, (12, E)) for lo, hi in ((24, 33), (-31, -27), (12, 15), (-20, -16))]).astype(np.float32)
    if not sigmoid:
        x[:, rng.integers(0, E)] = 40 + x.max()  # the others' shares are far below it
    zeros = np.zeros(E, np.float32)
    quarters = (np.round(rng.standard_normal(E) * 2) / 4).astype(np.float32)
    for bias in (zeros, zeros + np.float32(1.25), quarters):
        for top2 in ((False, True) if groups > 1 else (False,)):
            for f32 in (True, False):
                _check(run, x, K, bias, f32, sigmoid=sigmoid, groups=groups, keep=keep, top2=top2)


@pytest.mark.parametrize("run", ["eager", "executor"])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("E,K,groups,keep", SHAPES)
def test_only_the_last_chosen_has_its_like(E, K, groups, keep, sigmoid, run):
    """K - 1 experts far apart, then some that are alike, and behind them by number one that is better by 1e-13."""
    rng = np.random.default_rng(E - K)
    open_ = E // groups * keep
    for alike in (2, 3, min(7, open_ - K)):
        if open_ < K + alike:
            continue
        x = np.zeros((16, E), np.float32)
        bias = (-5.0 - rng.random(E)).astype(np.float32)
        at = rng.permutation(open_)[:K + alike]
        bias[at[:K - 1]] = 3 + 0.1 * np.arange(K - 1)
        last = np.sort(at[K - 1:])
        bias[last] = 1.25
        base = 30.0 if sigmoid else -29.0
        x[:, last] = base
        x[:, last[-1]] = base + rng.integers(1, 3, 16)
        x[::4, last[-1]] = base  # (none is better: the lowest)
        x[1::4, last[-2]] = base - 1
        for top2 in ((False, True) if groups > 1 else (False,)):
            _check(run, x, K, bias, sigmoid=sigmoid, groups=groups, keep=keep, top2=top2)
            _check(run, x, K, bias, False, sigmoid=sigmoid, groups=groups, keep=keep, top2=top2)
