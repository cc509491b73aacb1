"""What a decode step chooses, on the GPU against the definitions in 64 bits
(tests/choose_ref.py): as launches and through the persistent executor, with
staging buffers and without."""
import numpy as np
import pytest

from tests import choose_ref as R
from tests.gpu_harness import ensure_built, need_gpu
from tests.test_gpu_kv4 import RUNNERS, _dev, _f64

pytestmark = pytest.mark.gpu

# a staging buffer smaller than a tile's counters: windows
RUNS = dict(RUNNERS, executor_small=lambda *d, **k: RUNNERS["executor"](*d, stage_bytes=1024, **k))


@pytest.fixture(scope="module", autouse=True)
def _setup():
    need_gpu()
    ensure_built()


def _rows(x, f32, pad, junk=777.0):
    """x on the device in rows that are `pad` longer (filled with junk), and the whole buffer."""
    import torch
    B, V = x.shape
    whole = torch.full((B, V + pad), junk, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    whole[:, :V] = torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()
    return whole[:, :V], whole


def _close(got, want, tol, what=""):
    assert got.shape == want.shape
    same = (np.isnan(got) & np.isnan(want)) | (got == want)
    with np.errstate(invalid="ignore"):
        ok = same | (np.abs(got - want) <= tol)
    bad = np.argwhere(~ok)
    assert bad.size == 0, (what, len(bad), bad[:3], got[tuple(bad[0])], want[tuple(bad[0])], np.broadcast_to(tol, want.shape)[tuple(bad[0])])


# ---- adjust


def _adjust_case(seed, B, V, L, nb, M, f32, odd=False):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((B, V)).astype(np.float32) * 3
    if odd:  # what masks and overflows leave
        x[rng.random((B, V)) < 0.02] = -np.inf
        x[rng.random((B, V)) < 0.01] = np.inf
        x[rng.random((B, V)) < 0.01] = np.nan
        x[rng.random((B, V)) < 0.01] = -3.3e38
        x[rng.random((B, V)) < 0.01] = -0.0
    if not f32:
        x = R.bf16(x)
    s = np.zeros(B, R.SETTING)
    s["repetition"] = rng.choice([1.0, 1.2, 0.8, 1.07], B)
    s["presence"] = rng.choice([0.0, 0.4, -0.3], B)
    s["frequency"] = rng.choice([0.0, 0.25, -0.1], B)
    s["temperature"] = rng.choice([1.0, 0.7, 1.3, 0.0, -1.0], B)
    tokens = bias = mask = None
    if L:
        tokens = (V * rng.random((B, L)) ** 3).astype(np.int32)
        tokens[rng.random((B, L)) < 0.05] = -1  # images, padding
        tokens[rng.random((B, L)) < 0.05] = V
        tokens[rng.random((B, L)) < 0.02] = 2 ** 31 - 1
        s["length"] = rng.integers(0, L + 1, B)
        s["length"][:3] = [L, 0, 1][:B]
        s["prompt"] = rng.integers(0, s["length"] + 1)
        s["prompt"][0] = 0
    if nb:
        bias = np.zeros((B, nb), R.BIAS)
        bias["token"] = rng.integers(-1, V + 2, (B, nb))
        bias["token"][:, nb // 2:] = bias["token"][:, :nb - nb // 2]  # listed twice: the later one counts
        if L:
            bias["token"][:, ::3] = tokens[:, :1]  # of a token that the request has had
        bias["value"] = rng.standard_normal((B, nb)) * 5
        s["biases"] = rng.integers(0, nb + 1, B)
        s["biases"][0] = nb
    if M:
        mask = rng.integers(0, 1 << 32, (M, -(-V // 32)), dtype=np.uint32)
        mask[-1] = 0  # leaves nothing
        s["mask"] = rng.integers(-1, M, B)
        s["mask"][-1] = M - 1
    else:
        s["mask"] = -1
    return x, s, tokens, bias, mask


def _adjust_args(s, tokens, bias, mask):
    import torch
    t = torch.from_numpy(s.view(np.int32).reshape(-1, 8)).cuda()
    w = lambda x, shape: None if x is None else torch.from_numpy(np.ascontiguousarray(x).view(np.int32).reshape(shape)).cuda()  # noqa: E731
    return t, dict(tokens=None if tokens is None else _dev(tokens), bias=w(bias, (len(s), -1, 2)),
                   mask=None if mask is None else w(mask, mask.shape))


ADJUST = [
    # B, V, pad in, pad out, L, biases, masks
    (1, 1, 0, 0, 1, 1, 1), (1, 7, 0, 0, 0, 0, 0), (3, 9, 1, 3, 5, 3, 2), (4, 33, 0, 0, 300, 8, 2), (5, 256, 8, 8, 64, 0, 3),
    (2, 4096, 0, 0, 1000, 40, 1), (3, 4089, 0, 7, 257, 5, 2), (3, 5001, 47, 0, 700, 70, 3), (2, 33003, 1, 1, 3000, 3, 2),
    (2, 32000, 0, 0, 5000, 0, 0), (3, 33003, 1, 0, 9000, 40, 2), (2, 70000, 8, 8, 20000, 600, 1), (2, 3000, 0, 0, 40, 1024, 1), (1, 2001, 0, 0, 300000, 3, 1), (6, 8200, 56, 56, 31, 33, 4), (33, 1000, 0, 1, 17, 2, 1),
]


@pytest.mark.parametrize("run", sorted(RUNS))
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("case", ADJUST, ids=str)
def test_adjust(case, f32, run):
    from persistent_micro_dispatch_gb300 import choose
    B, V, pi, po, L, nb, M = case
    x, s, tokens, bias, mask = _adjust_case(hash(case) & 0xFFFF, B, V, L, nb, M, f32, odd=V % 2 == 1)
    want, tol = R.adjust(x, s, tokens, bias, mask, f32)
    t, kw = _adjust_args(s, tokens, bias, mask)
    logits, before = _rows(x, f32, pi)
    out, whole = _rows(np.zeros((B, V)), f32, po)
    RUNS[run](choose.adjust(logits, out, t, **kw))
    _close(_f64(out), want, tol)
    assert (whole[:, V:] == 777.0).all() and (before[:, V:] == 777.0).all()
    _close(_f64(logits), x.astype(np.float64), 0.0)
    # in place
    RUNS[run](choose.adjust(logits, logits, t, **kw))
    _close(_f64(logits), want, tol)
    assert (before[:, V:] == 777.0).all()


@pytest.mark.parametrize("run", ["eager", "executor"])
def test_adjust_without_anything_is_a_copy(run):
    import torch
    from persistent_micro_dispatch_gb300 import choose
    x = torch.randn(3, 5000, device="cuda")
    out, settings = torch.zeros_like(x), choose.new_settings(3)
    RUNS[run](choose.adjust(x, out, settings))
    assert torch.equal(x, out)


@pytest.mark.parametrize("run", sorted(RUNS))
def test_adjust_records_that_do_not_fit(run):
    """Each such request keeps its row; the others are done; the executor says so."""
    from persistent_micro_dispatch_gb300 import choose
    x, s, tokens, bias, mask = _adjust_case(5, 8, 5000, 40, 3, 2, True)
    s["length"], s["prompt"] = 20, 10
    s["length"][1], s["length"][2], s["prompt"][3], s["prompt"][4], s["mask"][5], s["biases"][6] = 41, -1, 21, -1, 2, 4
    bad = [1, 2, 3, 4, 5, 6]
    fit = s.copy()
    fit[bad] = s[0]
    want, tol = R.adjust(x, fit, tokens, bias, mask, True)
    t, kw = _adjust_args(s, tokens, bias, mask)
    logits, _ = _rows(x, True, 0)
    out, _ = _rows(np.full((8, 5000), 5.0), True, 0)
    d = choose.adjust(logits, out, t, **kw)
    RUNS[run](d, **(dict(expect=[2]) if "executor" in run else {}))
    want[bad], tol[bad] = 5.0, 0.0
    _close(_f64(out), want, tol)


@pytest.mark.parametrize("run", ["eager", "executor"])
def test_adjust_long_history(run):
    """More tokens than the vocabulary has, and one token most of the time."""
    from persistent_micro_dispatch_gb300 import choose
    x, s, tokens, bias, mask = _adjust_case(9, 3, 1501, 70001, 0, 0, False)
    tokens[1] = 3  # (one token 69,901 times)
    s["length"], s["prompt"] = 70001, [0, 100, 70001]
    s["repetition"], s["presence"], s["frequency"] = 1.1, 0.2, 1e-4
    want, tol = R.adjust(x, s, tokens, bias, mask, False)
    t, kw = _adjust_args(s, tokens, bias, mask)
    logits, _ = _rows(x, False, 0)
    out, _ = _rows(np.zeros((3, 1501)), False, 0)
    RUNS[run](choose.adjust(logits, out, t, **kw))
    _close(_f64(out), want, tol)


# ---- top


def _top_rows(seed, B, V, f32, kind):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((B, V)).astype(np.float32) * 4
    if kind == "ties":
        x = np.round(x)
    if kind == "masked":  # a grammar's mask: few are left, in some rows one, in some none
        x[rng.random((B, V)) < 0.99] = -np.inf
        x[0] = -np.inf
        x[-1, :] = -np.inf
        x[-1, V // 2] = 1.5
    if kind == "lowest":  # masked by the type's lowest value
        x[rng.random((B, V)) < 0.95] = -3.3895314e38
        x[0] = -3.3895314e38
    if kind == "nan":
        x[rng.random((B, V)) < 0.3] = np.nan
        x[0] = np.nan
    if kind == "up":  # every element is better than all before it
        x = np.sort(x, axis=1)
    if kind == "down":
        x = -np.sort(x, axis=1)
    if kind == "zeros":
        x = np.where(rng.random((B, V)) < 0.5, np.float32(0.0), np.float32(-0.0))
    return x if f32 else R.bf16(x)


TOP = [(1, 1, 0, 1), (2, 5, 1, 5), (3, 64, 0, 64), (1, 1000, 0, 1), (7, 1023, 3, 20), (2, 1025, 0, 33), (3, 4099, 1, 8),
       (1, 33001, 0, 20), (2, 32000, 0, 64), (5, 9000, 8, 32), (2049, 70, 0, 3), (700, 3001, 2, 5)]


def _run_top(run, x, f32, pad, K):
    import torch
    from persistent_micro_dispatch_gb300 import choose
    B = len(x)
    logits, _ = _rows(x, f32, pad, junk=1e30)
    ids = torch.full((B, K), -7, dtype=torch.int32, device="cuda")
    lp, lse = torch.zeros(B, K, device="cuda"), torch.zeros(B, device="cuda")
    ws = choose.new_workspace()
    d = choose.top(logits, ids, lp, lse, ws)
    RUNS[run](d)
    assert not ws[:choose.COUNTER_BYTES].any()
    return ids.cpu().numpy(), _f64(lp), _f64(lse)


def _check_top(run, x, f32, pad, K):
    ids, lp, lse = _run_top(run, x, f32, pad, K)
    wids, wlp, wlse, tlp, tlse = R.top(x, K)
    assert (ids == wids).all(), np.argwhere(ids != wids)[:4]
    _close(lse, wlse, tlse, "lse")
    _close(lp, wlp, tlp, "logprobs")


@pytest.mark.parametrize("run", sorted(RUNNERS))
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("case", TOP, ids=str)
def test_top(case, f32, run):
    B, V, pad, K = case
    _check_top(run, _top_rows(B + V, B, V, f32, "plain"), f32, pad, K)


@pytest.mark.parametrize("run", ["eager", "executor"])
@pytest.mark.parametrize("kind", ["ties", "masked", "lowest", "nan", "up", "down", "zeros"])
@pytest.mark.parametrize("case", [(3, 5003, 1, 20), (2, 20000, 0, 64), (300, 2000, 0, 1)], ids=str)
def test_top_of_odd_rows(case, kind, run):
    B, V, pad, K = case
    for f32 in (True, False):
        _check_top(run, _top_rows(B + V, B, V, f32, kind), f32, pad, K)


@pytest.mark.parametrize("kind", ["plain", "up", "masked"])
def test_top_of_many_rows(kind):
    """More rows than a launch has blocks: runs of several rows, and pieces of rows."""
    _check_top("eager", _top_rows(2, 460, 9000, False, kind), False, 1, 7)
    _check_top("eager", _top_rows(1, 1300, 20001, True, kind), True, 0, 64)
    _check_top("executor", _top_rows(1, 1300, 20001, False, kind), False, 3, 33)


@pytest.mark.parametrize("run", ["eager", "executor"])
def test_top_of_an_infinite_logit(run):
    """+infinity is the best; the row's lse is infinite, the others' log-probabilities -infinity."""
    x = _top_rows(3, 2, 3000, True, "plain")
    x[1, 77] = np.inf
    ids, lp, lse = _run_top(run, x, True, 0, 4)
    wids, wlp, wlse, tlp, tlse = R.top(x[:1], 4)
    assert (ids[0] == wids[0]).all() and ids[1, 0] == 77 and lse[1] == np.inf
    _close(lp[:1], wlp, tlp)
    assert np.isnan(lp[1, 0]) and (lp[1, 1:] == -np.inf).all()


def test_top_without_lse_and_twice_with_one_workspace():
    import torch
    from persistent_micro_dispatch_gb300 import choose
    x = _top_rows(4, 3, 20000, False, "plain")
    logits, _ = _rows(x, False, 0)
    ws = choose.new_workspace()
    for K in (5, 40):
        ids, lp = torch.zeros(3, K, dtype=torch.int32, device="cuda"), torch.zeros(3, K, device="cuda")
        RUNS["eager"](choose.top(logits, ids, lp, None, ws))
        wids, wlp, _, tlp, _ = R.top(x, K)
        assert (ids.cpu().numpy() == wids).all()
        _close(_f64(lp), wlp, tlp)


# ---- experts


EXPERTS = [
    # N, E, pad, K, sigmoid, bias, groups, keep, top2
    (1, 1, 0, 1, False, False, 1, 1, False), (1, 8, 0, 2, False, False, 1, 1, False), (7, 60, 4, 4, False, False, 1, 1, False),
    (9, 64, 0, 6, False, True, 1, 1, False), (33, 256, 0, 8, True, True, 8, 4, True), (17, 256, 1, 8, True, False, 8, 3, True),
    (20, 160, 0, 6, False, False, 8, 3, False), (12, 384, 0, 8, True, True, 1, 1, False), (5, 1024, 0, 32, True, True, 32, 7, True),
    (6, 512, 3, 10, False, True, 4, 2, True), (40, 12, 0, 3, True, True, 3, 2, True), (11, 96, 0, 1, False, False, 32, 1, False),
    (3, 32, 0, 32, True, True, 1, 1, False), (300, 128, 0, 8, False, False, 1, 1, False), (13, 66, 0, 5, True, False, 3, 2, True),
]


def _run_experts(run, x, f32, pad, K, bias, rows=None, **kw):
    import torch
    from persistent_micro_dispatch_gb300 import choose
    N = len(x)
    logits, _ = _rows(x, f32, pad, junk=1e30)
    ids, w = torch.full((N, K), -7, dtype=torch.int32, device="cuda"), torch.full((N, K), -7.0, device="cuda")
    b = None if bias is None else _dev(bias.astype(np.float32))
    r = None if rows is None else torch.tensor([rows], dtype=torch.int32, device="cuda")
    RUNS[run](choose.experts(logits, ids, w, bias=b, rows=r, **kw))
    return ids.cpu().numpy(), _f64(w)


def _check_experts(run, x, f32, pad, K, bias, normalise=True, scale=1.0, **kw):
    ids, w = _run_experts(run, x, f32, pad, K, bias, normalise=normalise, scale=scale, **kw)
    wids, ww = R.experts(x, K, kw["sigmoid"], bias, kw["groups"], kw["keep"], kw["top2"], normalise, scale)
    assert (ids == wids).all(), (np.argwhere(ids != wids)[:4], ids[ids != wids][:4], wids[ids != wids][:4])
    _close(w, ww, R.EXPERTS_TOL * np.abs(ww) + 2.0 ** -149)


@pytest.mark.parametrize("run", ["eager", "executor"])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("case", EXPERTS, ids=str)
def test_experts(case, f32, run):
    N, E, pad, K, sigmoid, biased, groups, keep, top2 = case
    rng = np.random.default_rng(N * E)
    x = rng.standard_normal((N, E)).astype(np.float32) * 1.5
    x = x if f32 else R.bf16(x)
    bias = rng.standard_normal(E).astype(np.float32) * 0.1 if biased else None
    for normalise, scale in ((True, 2.5), (False, 1.0)):
        _check_experts(run, x, f32, pad, K, bias, normalise, scale, sigmoid=sigmoid, groups=groups, keep=keep, top2=top2)


@pytest.mark.parametrize("run", ["eager", "executor"])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_experts_choose_as_in_64_bits(sigmoid, run):
    """Values that fp32 cannot tell apart: scores and biases that make up for each other but for a little."""
    rng = np.random.default_rng(3)
    N, E, K = 200, 64, 6
    x = rng.standard_normal((N, E)).astype(np.float32)
    x[:] = x[0]
    s = 1 / (1 + np.exp(-x[0].astype(np.float64))) if sigmoid else np.exp(x[0].astype(np.float64)) / np.exp(x[0].astype(np.float64)).sum()
    bias = (1.0 - s).astype(np.float32)  # all values near 1
    x += (rng.standard_normal((N, E)) * 1e-6).astype(np.float32)
    _check_experts(run, x, True, 0, K, bias, sigmoid=sigmoid, groups=1, keep=1, top2=False)
    _check_experts(run, x, True, 0, K, bias, sigmoid=sigmoid, groups=8, keep=3, top2=True)
    _check_experts(run, x, True, 0, K, None, sigmoid=sigmoid, groups=8, keep=3, top2=True)


@pytest.mark.parametrize("run", ["eager", "executor"])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("groups,keep", [(1, 1), (4, 2)])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_experts_ties_and_masked(sigmoid, groups, keep, biased, run):
    """Equal scores go to the lower expert; experts shut by -infinity; NaN; rows of nothing else; far logits."""
    rng = np.random.default_rng(8)
    E = 64
    x = np.zeros((12, E), np.float32)
    x[1] = rng.integers(0, 3, E)
    x[2] = -np.inf
    x[3] = np.nan
    x[4, :60] = -np.inf
    x[5] = np.where(rng.random(E) < 0.5, np.nan, rng.standard_normal(E))
    x[6] = rng.standard_normal(E) * 40
    x[7] = -70 + rng.standard_normal(E)
    x[8] = -95 + rng.standard_normal(E)
    x[9] = 95 + rng.standard_normal(E)
    x[10] = -3.3e38
    x[11] = rng.permutation(E) / 8
    bias = np.where(np.arange(E) % 5 == 0, 0.25, 0.0).astype(np.float32) if biased else None
    for top2 in ((False, True) if groups > 1 else (False,)):
        # (far logits: 64-bit scores of several are equal where the logits are not)
        keepers = [i for i in range(12) if i not in ((9,) if sigmoid and top2 else ())]
        _check_experts(run, x[keepers], True, 0, 8, bias, sigmoid=sigmoid, groups=groups, keep=keep, top2=top2)


@pytest.mark.parametrize("run", ["eager", "executor"])
@pytest.mark.parametrize("E,K", [(64, 6), (256, 8), (256, 20)])
@pytest.mark.parametrize("f32", [True, False])
def test_experts_whose_scores_no_float_holds(f32, E, K, run):
    """A softmax whose bias chooses experts far below the largest: their weights are shares of one another."""
    rng = np.random.default_rng(12)
    x = (rng.standard_normal((9, E)) * 2 - np.array([60, 79, 81, 85, 90, 100, 150, 300, 600])[:, None]).astype(np.float32)
    x[:, 3] = 0.0
    x[4, 10:] = -np.inf
    x = x if f32 else R.bf16(x)
    bias = (8 + rng.random(E)).astype(np.float32)
    bias[3] = -4.0
    _check_experts(run, x, f32, 0, K, bias, sigmoid=False, groups=1, keep=1, top2=False)
    _check_experts(run, x, f32, 0, K, bias, sigmoid=False, groups=4, keep=2, top2=True)


@pytest.mark.parametrize("run", ["eager", "executor"])
def test_experts_of_a_padded_batch(run):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 32)).astype(np.float32)
    for rows in (0, 1, 37, 50, 99, -3):
        n = min(max(rows, 0), 50)
        ids, w = _run_experts(run, x, True, 0, 4, None, rows=rows)
        wids, ww = R.experts(x, 4, False, None, 1, 1, False, True, 1.0)
        assert (ids[:n] == wids[:n]).all() and (ids[n:] == -1).all() and (w[n:] == 0).all()
        _close(w[:n], ww[:n], R.EXPERTS_TOL * ww[:n])


# ---- plan


@pytest.mark.parametrize("run", sorted(RUNNERS))
@pytest.mark.parametrize("case", [(1, 1, 1), (0, 2, 8), (5, 2, 8), (64, 8, 256), (511, 8, 60), (512, 8, 1024), (1025, 4, 8), (9000, 6, 1000), (33000, 8, 256)], ids=str)
def test_plan(case, run):
    import torch
    from persistent_micro_dispatch_gb300 import choose
    N, K, E = case
    rng = np.random.default_rng(N + E)
    ids = rng.integers(0, E, (N, K)).astype(np.int32)
    ids[rng.random((N, K)) < 0.2] = -1
    ids[rng.random((N, K)) < 0.02] = E
    ids[rng.random((N, K)) < 0.2] = E // 2
    ws = choose.new_workspace()
    P = N * K
    order, place = torch.full((P + 8,), -9, dtype=torch.int32, device="cuda"), torch.full((N, K), -9, dtype=torch.int32, device="cuda")
    offsets = torch.full((E + 1,), -9, dtype=torch.int32, device="cuda")
    pairs = _dev(ids)
    d = choose.plan(pairs, order[:P], place, offsets, ws)
    assert len(d) == (1 if P <= choose.PLAN_ONE else 2)
    RUNS[run](d)
    worder, wplace, woffsets = R.plan(ids, E)
    assert (offsets.cpu().numpy() == woffsets).all()
    assert (order[:P].cpu().numpy() == worder).all() and (order[P:] == -9).all()
    assert (place.cpu().numpy() == wplace).all()
    assert not ws[:choose.COUNTER_BYTES].any()
