"""What a decode step chooses, at the sizes where launches and tiles take
their other ways: more places a thread, better bars, many pieces of a row,
several turns of a block and several tokens of a tile."""
import numpy as np
import pytest

from tests import choose_ref as R
from tests.gpu_harness import ensure_built, need_gpu
from tests.test_gpu_choose import RUNS, _adjust_args, _adjust_case, _close, _rows
from tests.test_gpu_kv4 import RUNNERS, _dev, _f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    need_gpu()
    ensure_built()


# More than 4,000,000 logits: three (f32) or four (bf16) eights a thread. Rows
# alike and lying otherwise than the output's; ends inside a thread's places.
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("case", [(32, 128000, 0, 0, 3000, 40, 3), (63, 65537, 7, 7, 900, 5, 2), (33, 125003, 1, 0, 2500, 40, 2),
                                  (500, 8201, 0, 3, 60, 1024, 4), (40, 100352, 0, 0, 0, 0, 1)], ids=str)
def test_adjust_of_a_large_batch(case, f32):
    from persistent_micro_dispatch_gb300 import choose
    B, V, pi, po, L, nb, M = case
    assert B * V > 4_000_000
    x, s, tokens, bias, mask = _adjust_case(B, B, V, L, nb, M, f32, odd=V % 2 == 1)
    want, tol = R.adjust(x, s, tokens, bias, mask, f32)
    t, kw = _adjust_args(s, tokens, bias, mask)
    logits, before = _rows(x, f32, pi)
    out, whole = _rows(np.zeros((B, V)), f32, po)
    RUNS["eager"](choose.adjust(logits, out, t, **kw))
    _close(_f64(out), want, tol)
    assert (whole[:, V:] == 777.0).all() and (before[:, V:] == 777.0).all()
    RUNS["eager"](choose.adjust(logits, logits, t, **kw))  # in place
    _close(_f64(logits), want, tol)
    assert (before[:, V:] == 777.0).all()


def _long_rows(seed, V, f32):
    """Twelve rows in which a bar is found late, early, or not at all."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((12, V)).astype(np.float32) * 4
    x[1] = np.round(x[1])                                   # ties
    x[2, :V // 2] = -np.inf                                 # masked, but for its end
    x[3] = np.sort(x[3])                                    # each better than all before it
    x[4] = -np.sort(x[4])
    x[5, rng.random(V) < 0.99] = -np.inf
    x[6, rng.random(V) < 0.5] = np.nan
    x[7] = np.where(rng.random(V) < 0.95, np.float32(-3.3895314e38), x[7])
    x[8] = 2.5                                              # all alike
    x[9] = -np.inf
    x[9, V - 1] = 1.0
    x[10] = np.floor(np.arange(V) / 4096) + rng.random(V) * np.float32(0.5)  # each unit better than the one before
    x[11] = rng.integers(-2, 3, V)
    return x if f32 else R.bf16(x)


# One row of 32 pieces; 16 pieces of 28; rows in runs across rows (two or three
# pieces a block); rows whole, of 32 units; and vocabularies beyond all tables.
@pytest.mark.parametrize("K", [1, 7, 33, 64])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("V,copies", [(128000, 0), (262147, 0), (128000, 1), (40001, 25), (40001, 38)], ids=str)
def test_top_of_long_rows(V, copies, f32, K):
    import torch
    from persistent_micro_dispatch_gb300 import choose
    x = _long_rows(V + K, V, f32)
    wids, wlp, wlse, tlp, tlse = R.top(x, K)
    ws = choose.new_workspace()
    logits, _ = _rows(x, f32, 1 if V % 2 else 0, junk=1e30)
    # (0: a row a call)
    for at in ([slice(0, 12)] if copies else [slice(r, r + 1) for r in range(12)]):
        n = max(copies, 1)
        many = logits[at] if n == 1 else logits[at].repeat(n, 1)
        B = many.shape[0]
        ids, lp, lse = torch.full((B, K), -7, dtype=torch.int32, device="cuda"), torch.zeros(B, K, device="cuda"), torch.zeros(B, device="cuda")
        RUNNERS["eager"](choose.top(many, ids, lp, lse, ws))
        ids, lp, lse = ids.cpu().numpy().reshape(n, -1, K), _f64(lp).reshape(n, -1, K), _f64(lse).reshape(n, -1)
        for c in range(n):
            assert (ids[c] == wids[at]).all(), np.argwhere(ids[c] != wids[at])[:4]
            _close(lp[c], wlp[at], tlp[at], "logprobs")
            _close(lse[c], wlse[at], tlse[at], "lse")
    assert not ws[:choose.COUNTER_BYTES].any()


def test_top_of_long_rows_in_the_executor():
    import torch
    from persistent_micro_dispatch_gb300 import choose
    x = _long_rows(5, 128000, False)
    logits, _ = _rows(x, False, 0)
    ids, lp, lse = torch.zeros(12, 40, dtype=torch.int32, device="cuda"), torch.zeros(12, 40, device="cuda"), torch.zeros(12, device="cuda")
    ws = choose.new_workspace()
    RUNNERS["executor"](choose.top(logits, ids, lp, lse, ws))
    wids, wlp, wlse, tlp, tlse = R.top(x, 40)
    assert (ids.cpu().numpy() == wids).all()
    _close(_f64(lp), wlp, tlp, "logprobs")
    _close(_f64(lse), wlse, tlse, "lse")


# Launches take a second turn of their blocks from 9,728 tokens (sixteen lanes a
# token) or 19,456 (eight); the executor's tiles have several tokens from 1,537.
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("run,N,E,K,sigmoid,biased,groups,keep,top2", [
    ("eager", 20011, 256, 8, True, True, 8, 4, True), ("eager", 20011, 256, 8, False, False, 1, 1, False), ("eager", 40003, 64, 6, False, True, 1, 1, False),
    ("eager", 30001, 60, 4, True, True, 1, 1, False), ("eager", 10007, 384, 10, True, True, 4, 2, True), ("eager", 6007, 640, 9, False, True, 1, 1, False),
    ("executor", 2003, 256, 8, True, True, 8, 4, True), ("executor", 20011, 64, 8, False, False, 8, 3, False)])
def test_experts_of_many_tokens(run, N, E, K, sigmoid, biased, groups, keep, top2, f32):
    import torch
    from persistent_micro_dispatch_gb300 import choose
    rng = np.random.default_rng(N)
    x = rng.standard_normal((N, E)).astype(np.float32) * 1.5
    x[::97] = np.round(x[::97])            # ties, more than a token has room for among them
    x[5::101, E // 8:] = -np.inf
    x[7::103] = np.nan
    x[11::89] = 0.0
    x = x if f32 else R.bf16(x)
    bias = (rng.standard_normal(E) * 0.05).astype(np.float32) if biased else None
    logits, _ = _rows(x, f32, E % 8, junk=1e30)
    ids, w = torch.full((N, K), -7, dtype=torch.int32, device="cuda"), torch.full((N, K), -7.0, device="cuda")
    b, rows = None if bias is None else _dev(bias), torch.tensor([N - 5], dtype=torch.int32, device="cuda")
    RUNS[run](choose.experts(logits, ids, w, sigmoid=sigmoid, bias=b, groups=groups, keep=keep, top2=top2, scale=2.5, rows=rows))
    wids, ww = R.experts(x, K, sigmoid, bias, groups, keep, top2, True, 2.5)
    wids[N - 5:], ww[N - 5:] = -1, 0.0
    ids = ids.cpu().numpy()
    assert (ids == wids).all(), (np.argwhere(ids != wids)[:4], ids[ids != wids][:4], wids[ids != wids][:4])
    _close(_f64(w), ww, R.EXPERTS_TOL * np.abs(ww) + 2.0 ** -149)


# From 393,217 pairs on a run is more than a block's turn.
@pytest.mark.parametrize("run", ["eager", "executor"])
@pytest.mark.parametrize("N,K,E", [(65537, 8, 256), (200003, 4, 1000), (49153, 8, 7)], ids=str)
def test_plan_of_a_long_prompt(N, K, E, run):
    import torch
    from persistent_micro_dispatch_gb300 import choose
    rng = np.random.default_rng(N)
    ids = rng.integers(0, E, (N, K)).astype(np.int32)
    ids[rng.random((N, K)) < 0.1] = -1
    ids[rng.random((N, K)) < 0.01] = E
    ids[rng.random((N, K)) < 0.3] = E // 2
    ids[-N // 9:] = -1
    P = N * K
    assert P > 96 * 4096
    ws = choose.new_workspace()
    order, place = torch.full((P + 8,), -9, dtype=torch.int32, device="cuda"), torch.full((N, K), -9, dtype=torch.int32, device="cuda")
    offsets = torch.full((E + 1,), -9, dtype=torch.int32, device="cuda")
    pairs = _dev(ids)
    RUNS[run](choose.plan(pairs, order[:P], place, offsets, ws))
    worder, wplace, woffsets = R.plan(ids, E)
    assert (offsets.cpu().numpy() == woffsets).all()
    assert (order[:P].cpu().numpy() == worder).all() and (order[P:] == -9).all()
    assert (place.cpu().numpy() == wplace).all()
