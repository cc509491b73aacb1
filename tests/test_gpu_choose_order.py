"""Which experts are chosen where 64-bit scores are equal and logits are not:
without a bias the order is the logits', with one it is that of 64-bit sums."""
import numpy as np
import pytest

from tests.gpu_harness import ensure_built, need_gpu
from tests.test_gpu_choose import _run_experts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    need_gpu()
    ensure_built()


def _scores(x, sigmoid):
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    with np.errstate(all="ignore"):
        if sigmoid:
            return x, 1 / (1 + np.exp(-x))
        e = np.exp(x - x.max()) if np.isfinite(x.max()) else np.zeros_like(x)
        return x, e / max(e.sum(), 1e-300)


def _choice(x, K, sigmoid, bias, groups, keep, top2):
    """One token's experts, from the definition in include/gpuos.h, by Python's own sort."""
    x, s = _scores(x, sigmoid)
    value = x if bias is None else s + bias.astype(np.float64)
    size = len(x) // groups
    kept = range(len(x))
    if groups > 1:
        def worth(g):
            part = sorted((s if bias is None else value)[g * size:(g + 1) * size] if top2 else value[g * size:(g + 1) * size], reverse=True)
            return part[0] + part[1] if top2 else part[0]
        best = sorted(range(groups), key=lambda g: (-worth(g), g))[:keep]
        kept = [e for e in kept if e // size in best]
    return sorted(kept, key=lambda e: (-value[e], e))[:K]


def _rows(E, seed):
    rng = np.random.default_rng(seed)
    x = np.zeros((14, E), np.float32)
    x[0, 5] = 1e-20                                          # 0.5 in 64 bits, like the others
    x[1] = rng.permutation(E) * np.float32(1e-20)            # so near 0 that no 64-bit score tells
    x[2] = -x[1]
    x[3] = 95 + rng.standard_normal(E)                       # 1 in 64 bits
    x[4] = 20 + 25 * rng.random(E)                           # from where scores still differ to where they do not
    x[5] = -800 - 100 * rng.random(E)                        # 0 in 64 bits
    x[6] = np.where(rng.random(E) < 0.5, 95, 96)             # two values
    x[7] = -95 + rng.standard_normal(E)                      # far below, but told apart
    x[8] = 3e38 * rng.random(E)
    x[9] = -3e38 * rng.random(E)
    x[10] = rng.standard_normal(E) * 300                     # some of everything
    x[11] = np.where(rng.random(E) < 0.5, 40 + rng.random(E), -np.inf)
    x[12, ::2] = np.float32(1e-30)
    x[13] = np.where(rng.random(E) < 0.3, 50 + rng.random(E), rng.standard_normal(E))
    return x


@pytest.mark.parametrize("run", ["eager", "executor"])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("E,K,groups,keep", [(8, 2, 1, 1), (64, 6, 1, 1), (64, 8, 4, 2), (256, 8, 1, 1), (256, 8, 8, 4), (512, 10, 4, 2), (96, 20, 3, 2)])
def test_order_where_scores_are_equal(E, K, groups, keep, sigmoid, run):
    x = _rows(E, E + K)
    zeros = np.zeros(E, np.float32)
    some = np.where(np.arange(E) % 5 == 0, 0.25, 0.0).astype(np.float32)
    for bias in (None, zeros, some):
        for top2 in ((False, True) if groups > 1 else (False,)):
            ids, _ = _run_experts(run, x, True, 0, K, bias, sigmoid=sigmoid, groups=groups, keep=keep, top2=top2)
            want = np.array([_choice(r, K, sigmoid, bias, groups, keep, top2) for r in x])
            assert (ids == want).all(), (bias is None, top2, np.argwhere((ids != want).any(1)).ravel(), ids[(ids != want).any(1)][:2], want[(ids != want).any(1)][:2])


def test_a_bias_of_zeros_is_not_the_same_as_none():
    """Eight experts, all logits 0 but one of 1e-20: its score is 0.5 like the others' in 64 bits."""
    x = np.zeros((1, 8), np.float32)
    x[0, 5] = 1e-20
    kw = dict(sigmoid=True, groups=1, keep=1, top2=False)
    assert _run_experts("eager", x, True, 0, 2, None, **kw)[0].tolist() == [[5, 0]]
    assert _run_experts("eager", x, True, 0, 2, np.zeros(8, np.float32), **kw)[0].tolist() == [[0, 1]]
