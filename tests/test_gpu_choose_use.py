"""What a decode step chooses, as it is used: one step's ops one after another,
in captured graphs, on other streams, beside a resident executor, through
aliases; and what is refused."""
import time

import numpy as np
import pytest

from tests import choose_ref as R
from tests.gpu_harness import ensure_built, need_gpu
from tests.test_gpu_choose import RUNS, _adjust_args, _adjust_case, _check_experts, _close, _rows, _top_rows
from tests.test_gpu_kv4 import RUNNERS, _dev, _f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    need_gpu()
    ensure_built()


class Step:
    """One decode step's choices: adjusted logits, their best tokens, a router's experts and their plan."""

    def __init__(self, seed=0, B=5, V=9001, N=40, E=64, K=6):
        import torch
        from persistent_micro_dispatch_gb300 import choose
        self.x, self.s, self.tokens, self.bias, self.mask = _adjust_case(seed, B, V, 200, 5, 3, False)
        self.t, self.kw = _adjust_args(self.s, self.tokens, self.bias, self.mask)
        self.logits, _ = _rows(self.x, False, 7)
        self.out = torch.zeros(B, V, dtype=torch.bfloat16, device="cuda")
        self.ids, self.lp = torch.zeros(B, 9, dtype=torch.int32, device="cuda"), torch.zeros(B, 9, device="cuda")
        self.lse, self.ws = torch.zeros(B, device="cuda"), choose.new_workspace()
        self.E, self.K = E, K
        rng = np.random.default_rng(seed)
        self.r = rng.standard_normal((N, E)).astype(np.float32)
        self.rbias = (rng.standard_normal(E) * 0.1).astype(np.float32)
        self.router, self.balance = _dev(self.r), _dev(self.rbias)
        self.eids, self.w = torch.zeros(N, K, dtype=torch.int32, device="cuda"), torch.zeros(N, K, device="cuda")
        self.order, self.place = torch.zeros(N * K, dtype=torch.int32, device="cuda"), torch.zeros(N, K, dtype=torch.int32, device="cuda")
        self.offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")

    def descs(self):
        from persistent_micro_dispatch_gb300 import choose
        return np.concatenate([
            choose.experts(self.router, self.eids, self.w, sigmoid=True, bias=self.balance, groups=4, keep=2, top2=True, scale=2.0),
            choose.plan(self.eids, self.order, self.place, self.offsets, self.ws),
            choose.adjust(self.logits, self.out, self.t, **self.kw),
            choose.top(self.out, self.ids, self.lp, self.lse, self.ws)])

    def check(self):
        want, tol = R.adjust(self.x, self.s, self.tokens, self.bias, self.mask, False)
        _close(_f64(self.out), want, tol)
        ids, lp, lse, tlp, tlse = R.top(self.out.float().cpu().numpy(), 9)
        assert (self.ids.cpu().numpy() == ids).all()
        _close(_f64(self.lp), lp, tlp)
        _close(_f64(self.lse), lse, tlse)
        ids, w = R.experts(self.r, self.K, True, self.rbias, 4, 2, True, True, 2.0)
        assert (self.eids.cpu().numpy() == ids).all()
        _close(_f64(self.w), w, R.EXPERTS_TOL * w)
        order, place, offsets = R.plan(ids, self.E)
        assert (self.order.cpu().numpy() == order).all() and (self.place.cpu().numpy() == place).all()
        assert (self.offsets.cpu().numpy() == offsets).all()


@pytest.mark.parametrize("run", sorted(RUNS))
@pytest.mark.parametrize("N", [40, 900])  # one record for the plan, and two
def test_a_step(N, run):
    s = Step(N, N=N)
    RUNS[run](s.descs())
    s.check()


def test_a_step_in_a_graph():
    """Captured once, replayed on inputs that change; another graph shares the workspace."""
    import torch
    from persistent_micro_dispatch_gb300 import gpuos as G
    s, o = Step(1, N=900), Step(2, N=700)
    o.ws = s.ws
    stream = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(stream):
        for x in (s, o):
            G.eager_run(x.descs(), stream.cuda_stream)
            stream.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                G.eager_run(x.descs(), stream.cuda_stream)
            graphs.append(g)
    for seed in (3, 4):
        for x, n in ((s, 900), (o, 700)):
            y = Step(seed, N=n)
            for a in ("x", "s", "tokens", "bias", "mask", "r", "rbias"):
                setattr(x, a, getattr(y, a))
            x.logits.copy_(y.logits)
            x.t.copy_(y.t)
            for k in x.kw:
                x.kw[k].copy_(y.kw[k])
            x.router.copy_(y.router)
            x.balance.copy_(y.balance)
        torch.cuda.synchronize()
        for g in graphs + graphs:
            g.replay()
        torch.cuda.synchronize()
        s.check()
        o.check()


def test_two_steps_at_once():
    """On two streams, each with a workspace of its own."""
    import torch
    from persistent_micro_dispatch_gb300 import gpuos as G
    steps = [Step(k, B=33, N=900) for k in (5, 6)]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, st in zip(steps, streams):
            G.eager_run(x.descs(), st.cuda_stream)
    torch.cuda.synchronize()
    for x in steps:
        x.check()


def test_a_step_beside_a_resident_executor():
    import torch
    from persistent_micro_dispatch_gb300 import gpuos as G
    from workloads.device import warm_torch
    s, o = Step(7, N=900), Step(8, N=900)
    st, done = torch.cuda.Stream(), torch.cuda.Event()
    warm_torch()
    torch.cuda.synchronize()
    ex = G.Executor(blocks=8, idle_exit_ms=10_000)
    try:
        G.eager_run(s.descs(), st.cuda_stream)
        done.record(st)
        d = o.descs()
        d["flags"], d["dep"][1:, 0] = G.FLAG_DEP_REL, 1
        ex.submit_batch(d)
        t0 = time.monotonic()
        while not done.query() and time.monotonic() - t0 < 5:
            time.sleep(0.01)
        late, running = not done.query(), ex.stats()["running"]
        ex.sync(timeout_ms=30_000)
    finally:
        assert ex.shutdown() == G.OK
    assert not late and running == 1
    s.check()
    o.check()


def test_rows_far_apart():
    """Offsets that pass 2^31 elements and 2^32 bytes."""
    import torch
    from persistent_micro_dispatch_gb300 import choose, gpuos as G
    ld, V, B = (1 << 30) + 8, 3000, 3
    buf = torch.empty(2 * ld + V, dtype=torch.bfloat16, device="cuda")
    x, s, tokens, bias, mask = _adjust_case(11, B, V, 50, 3, 2, False)
    logits = torch.as_strided(buf, (B, V), (ld, 1))
    logits.copy_(_dev(x).to(torch.bfloat16))
    t, kw = _adjust_args(s, tokens, bias, mask)
    wide = torch.empty(B, 1 << 28, dtype=torch.int32, device="cuda")  # rows of tokens a gigabyte apart
    wide[:, :50] = kw["tokens"]
    out = torch.zeros(B, V, dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    G.eager_run(choose.adjust(logits, out, t, tokens=wide, bias=kw["bias"], mask=kw["mask"]), stream)
    want, tol = R.adjust(x, s, tokens, bias, mask, False)
    _close(_f64(out), want, tol)
    RUNNERS["executor"](choose.adjust(logits, logits, t, tokens=wide, bias=kw["bias"], mask=kw["mask"]))
    _close(_f64(logits), want, tol)
    y = logits.float().cpu().numpy()
    ids, lp, ws = torch.zeros(B, 4, dtype=torch.int32, device="cuda"), torch.zeros(B, 4, device="cuda"), choose.new_workspace()
    eids, w = torch.zeros(B, 4, dtype=torch.int32, device="cuda"), torch.zeros(B, 4, device="cuda")
    router = torch.as_strided(buf, (B, 64), (ld, 1))
    for run in ("eager", "executor"):
        RUNNERS[run](choose.top(logits, ids, lp, None, ws), choose.experts(router, eids, w, sigmoid=True))
        assert (ids.cpu().numpy() == R.top(y, 4)[0]).all()
        assert (eids.cpu().numpy() == R.experts(y[:, :64], 4, True, None, 1, 1, False, True, 1.0)[0]).all()


@pytest.mark.parametrize("run", ["eager", "executor"])
@pytest.mark.parametrize("f32", [True, False])
def test_rows_that_begin_anywhere(f32, run):
    """Columns of a wider tensor: rows begin between the vectors' boundaries."""
    import torch
    from persistent_micro_dispatch_gb300 import choose
    for off in (1, 2, 5, 7):
        V, B = 4500 + off, 3
        x, s, tokens, bias, mask = _adjust_case(20 + off, B, V, 60, 4, 2, f32)
        t, kw = _adjust_args(s, tokens, bias, mask)
        big = torch.full((B, V + 24), 5.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        logits = big[:, off:off + V]
        logits.copy_(_dev(x).to(big.dtype))
        other = torch.full_like(big, 5.0)
        out = other[:, 8 - off:8 - off + V]
        ids, lp, lse, ws = (torch.zeros(B, 7, dtype=torch.int32, device="cuda"), torch.zeros(B, 7, device="cuda"), torch.zeros(B, device="cuda"),
                            choose.new_workspace())
        RUNNERS[run](choose.adjust(logits, out, t, **kw), choose.top(logits, ids, lp, lse, ws))
        want, tol = R.adjust(x, s, tokens, bias, mask, f32)
        _close(_f64(out), want, tol)
        wids, wlp, wlse, tlp, tlse = R.top(x, 7)
        assert (ids.cpu().numpy() == wids).all()
        _close(_f64(lp), wlp, tlp)
        _close(_f64(lse), wlse, tlse)
        for b, at in ((big, off), (other, 8 - off)):
            assert (b[:, :at] == 5.0).all() and (b[:, at + V:] == 5.0).all()
    rng = np.random.default_rng(4)
    wide = np.full((6, 80), 1e30, np.float32)
    wide[:, 3:67] = R.bf16(rng.standard_normal((6, 64)))
    src = _dev(wide).to(torch.float32 if f32 else torch.bfloat16)
    ids, w = torch.zeros(6, 5, dtype=torch.int32, device="cuda"), torch.zeros(6, 5, device="cuda")
    RUNNERS[run](choose.experts(src[:, 3:67], ids, w))
    assert (ids.cpu().numpy() == R.experts(wide[:, 3:67], 5, False, None, 1, 1, False, True, 1.0)[0]).all()


@pytest.mark.parametrize("run", ["eager", "executor"])
def test_experts_whose_bias_shuts_them(run):
    """A bias of -infinity or NaN: chosen last, the lower number first."""
    rng = np.random.default_rng(9)
    x = rng.standard_normal((20, 64)).astype(np.float32)
    b = (rng.standard_normal(64) * 0.1).astype(np.float32)
    b[::2] = -np.inf
    shut = b.copy()
    shut[10::8] = np.nan
    for sigmoid in (True, False):
        for groups, keep, K in ((1, 1, 8), (8, 2, 8), (8, 5, 15), (1, 1, 32)):
            for bias in (b, shut):
                import torch
                from persistent_micro_dispatch_gb300 import choose
                ids, w = torch.zeros(20, K, dtype=torch.int32, device="cuda"), torch.zeros(20, K, device="cuda")
                t, tb = _dev(x), _dev(bias)
                RUNNERS[run](choose.experts(t, ids, w, sigmoid=sigmoid, bias=tb, groups=groups, keep=keep))
                wids, ww = R.experts(x, K, sigmoid, b, groups, keep, False, True, 1.0)
                assert (ids.cpu().numpy() == wids).all(), (sigmoid, groups, K)
                _close(_f64(w), ww, R.EXPERTS_TOL * ww)


@pytest.mark.parametrize("run", ["eager", "executor"])
def test_experts_of_every_layout(run):
    """Numbers of experts, groups and choices around what lanes hold."""
    rng = np.random.default_rng(2)
    for E, groups, keep, K in ((16, 16, 9, 3), (48, 16, 2, 6), (64, 2, 1, 16), (72, 8, 3, 8), (128, 8, 2, 8), (136, 8, 8, 8), (160, 4, 1, 12),
                               (200, 1, 1, 15), (256, 16, 3, 15), (257, 1, 1, 8), (480, 2, 2, 10), (512, 32, 4, 9), (520, 8, 3, 8), (1000, 1, 1, 7)):
        x = rng.standard_normal((37, E)).astype(np.float32) * 2
        bias = (rng.standard_normal(E) * 0.05).astype(np.float32)
        for b in (None, bias):
            for top2 in ((False, True) if E // groups > 1 and groups > 1 else (False,)):
                _check_experts(run, x, True, 0, K, b, sigmoid=True, groups=groups, keep=keep, top2=top2)
                _check_experts(run, R.bf16(x), False, 3, K, b, normalise=False, sigmoid=False, groups=groups, keep=keep, top2=top2)


@pytest.mark.parametrize("run", ["eager", "executor"])
def test_groups_choose_as_in_64_bits(run):
    """Groups whose two best differ, but whose sums fp32 cannot tell apart."""
    rng = np.random.default_rng(12)
    N, E = 300, 64
    x = rng.standard_normal((N, E)).astype(np.float32) - 1.0
    s = 1 / (1 + np.exp(-x[0].astype(np.float64)))
    bias = np.zeros(E, np.float32)
    for g in range(8):  # each group's two best values add up to nearly the same
        at = slice(8 * g, 8 * g + 8)
        best = np.argsort(-s[at])[:2] + 8 * g
        bias[at] = -1.0
        bias[best[0]] = 1.0 - s[best[0]] + 0.01 * g
        bias[best[1]] = 1.0 - s[best[1]] - 0.01 * g
    x[:] = x[0]
    x += (rng.standard_normal((N, E)) * 3e-7).astype(np.float32)
    for keep in (1, 3, 7):
        _check_experts(run, x, True, 0, 2, bias, sigmoid=True, groups=8, keep=keep, top2=True)
        _check_experts(run, x, True, 0, 2, bias, sigmoid=True, groups=8, keep=keep, top2=False)


@pytest.mark.parametrize("run", ["eager", "executor"])
def test_top_of_a_language_model_like_row(run):
    """One token far ahead: its log-probability is next to 0 and keeps its digits."""
    x = _top_rows(6, 4, 32000, True, "plain")
    x[:, 777] = [14.0, 25.0, 40.0, 60.0]
    from tests.test_gpu_choose import _check_top
    _check_top(run, x, True, 0, 5)


@pytest.mark.parametrize("run", ["eager", "executor"])
def test_nothing_to_do(run):
    import torch
    from persistent_micro_dispatch_gb300 import choose
    ws, dev = choose.new_workspace(), "cuda"
    x, i, w = torch.zeros(0, 64, device=dev), torch.zeros(0, 4, dtype=torch.int32, device=dev), torch.zeros(0, 4, device=dev)
    offsets = torch.full((9,), 5, dtype=torch.int32, device=dev)
    s = choose.new_settings(0)
    RUNNERS[run](choose.adjust(x, x, s), choose.top(x, i, w, None, ws), choose.experts(x, i, w), choose.plan(i, i.view(-1), i, offsets, ws))
    assert not offsets.any()


@pytest.mark.parametrize("run", ["eager", "executor"])
def test_reset_after_an_abandoned_call(run):
    """Counters that a call left raised: reset, the next one is right."""
    import torch
    from persistent_micro_dispatch_gb300 import choose
    ws = choose.new_workspace()
    ws.copy_(torch.randint(0, 256, (choose.WORKSPACE_BYTES,), dtype=torch.uint8, device="cuda"))
    choose.reset_workspace(ws)
    x = _top_rows(2, 3, 33001, False, "plain")
    logits, _ = _rows(x, False, 0)
    ids, lp = torch.zeros(3, 20, dtype=torch.int32, device="cuda"), torch.zeros(3, 20, device="cuda")
    for _ in range(2):
        RUNNERS[run](choose.top(logits, ids, lp, None, ws))
        assert (ids.cpu().numpy() == R.top(x, 20)[0]).all()


@pytest.mark.parametrize("run", ["eager", "executor"])
def test_a_placement_without_its_count(run):
    """Counts that are not of these pairs give a wrong order, and nothing outside it."""
    import torch
    from persistent_micro_dispatch_gb300 import choose
    rng = np.random.default_rng(3)
    ids = _dev(rng.integers(0, 16, 9000).astype(np.int32))
    for fill in (0, 1000, 2 ** 31 - 1, -1):
        ws = choose.new_workspace()
        ws.view(torch.int32)[choose.COUNTER_BYTES // 4:] = fill
        guard = torch.full((9000 + 20000,), -9, dtype=torch.int32, device="cuda")
        place, offsets = torch.zeros_like(ids), torch.zeros(17, dtype=torch.int32, device="cuda")
        d = choose.plan(ids, guard[10000:19000], place, offsets, ws)[1:].copy()
        d["flags"], d["dep"] = 0, 0
        RUNNERS[run](d)
        assert (guard[:10000] == -9).all() and (guard[19000:] == -9).all()


def test_adjust_of_more_rows_than_a_grid_holds():
    import torch
    from persistent_micro_dispatch_gb300 import choose
    B, V = 65537 + 60, 40
    x, s, tokens, bias, mask = _adjust_case(1, B, V, 6, 2, 3, True)
    t, kw = _adjust_args(s, tokens, bias, mask)
    logits, out = _dev(x), torch.zeros(B, V, device="cuda")
    RUNNERS["eager"](choose.adjust(logits, out, t, **kw))
    at = np.r_[0:40, 65500:B]
    want, tol = R.adjust(x[at], s[at], tokens[at], bias[at], mask, True)
    _close(_f64(out)[at], want, tol)


def test_aliased_ops_check_their_sizes():
    """An alias is a user op: the host passes its sizes and tile count on, and
    the op itself refuses what it cannot do."""
    import torch
    from persistent_micro_dispatch_gb300 import gpuos as G
    from workloads.device import warm_torch
    s = Step(9, N=900)
    good = s.descs()
    names = ["expert_route", "expert_count", "expert_place", "logits_adjust", "logits_top"]
    assert [int(i) for i in good["op_id"]] == [G.OP[n] for n in names]
    tiles = [G.op_ntiles(good[i:i + 1]) for i in range(5)]
    good["ntiles"] = tiles
    bad = []

    def refused(i, dim=None, value=0, field=None, shift=0, ntiles=None):
        d = good[i:i + 1].copy()
        if dim is not None:
            d["dims"][0, dim] = value
        if field:
            d[field] = d[field] + shift if shift else 0
        if ntiles is not None:
            d["ntiles"] = ntiles
        bad.append(d)

    for dim, value in ((1, 0), (1, 63), (2, 60), (3, 0), (3, 33), (4, 5 | 2 << 16), (4, 4), (5, 8)):
        refused(0, dim, value)
    for i, dim, value in ((1, 1, 0), (1, 1, 1025), (2, 1, 1025), (3, 2, 9000), (3, 3, 9000), (3, 4, (1 << 28) + 1), (4, 2, 9000), (4, 3, 65),
                          (4, 3, 0)):
        refused(i, dim, value)
    for i, field, shift in ((0, "a", 1), (0, "out", 0), (0, "aux1", 2), (1, "aux2", 8), (2, "b", 0), (2, "aux0", 2), (3, "aux0", 8), (3, "b", 0),
                            (3, "aux1", 2), (3, "aux2", 4), (4, "aux2", 0), (4, "aux0", 1), (4, "a", 1)):
        refused(i, field=field, shift=shift)
    for i in range(5):
        refused(i, ntiles=tiles[i] + 1)
        refused(i, ntiles=1)
    d = np.concatenate([good] + bad)
    for i, n in enumerate(names):
        d["op_id"][d["op_id"] == G.OP[n]] = 90 + i
    d["flags"] = G.FLAG_DEP_REL
    d["dep"][1:, 0] = 1
    warm_torch()
    torch.cuda.synchronize()
    ex = G.Executor()
    try:
        for i, n in enumerate(names):
            ex.alias_op(90 + i, G.OP[n])
        with pytest.raises(G.GpuosError):
            ex.alias_op(95, 20)
        with pytest.raises(G.GpuosError):
            ex.alias_op(20, G.OP["add"])
        hist = ex.set_history(0, len(d))
        ex.submit_batch(d)
        rc = ex.sync(raise_on_error=False, timeout_ms=60_000)
    finally:
        assert ex.shutdown() == G.OK
    assert rc == G.EDEVICE and hist["status"].tolist() == [0] * 5 + [2] * len(bad)
    s.check()
    assert not s.ws[:8192].any().item()


def test_binding_refusals():
    import torch
    from persistent_micro_dispatch_gb300 import choose
    dev, B, V = "cuda", 3, 100
    x, i32 = torch.zeros(B, V, device=dev), lambda *n: torch.zeros(*n, dtype=torch.int32, device=dev)  # noqa: E731
    good = dict(logits=x, out=torch.zeros_like(x), settings=choose.new_settings(B), tokens=i32(B, 4), bias=i32(B, 2, 2), mask=i32(1, 4))
    choose.adjust(**good)
    flat = i32(1 + 8 * B)
    for name, bad, err in [
            ("logits", x.half(), TypeError), ("logits", x[0], ValueError), ("logits", x.cpu(), ValueError), ("logits", x.t().contiguous().t(), ValueError),
            ("logits", x[:, :0], ValueError), ("logits", x[:1].expand(B, V), ValueError), ("out", x.bfloat16(), ValueError), ("out", x[:2], ValueError),
            ("out", x[:, 1:], ValueError), ("out", x.cpu(), ValueError), ("settings", choose.new_settings(2), ValueError),
            ("settings", choose.new_settings(B).float(), TypeError), ("settings", flat[1:].view(B, 8), ValueError), ("tokens", i32(2, 4), ValueError),
            ("tokens", i32(B, 4).long(), TypeError), ("tokens", i32(4, B).t(), ValueError), ("tokens", i32(B), ValueError), ("bias", i32(B, 2), ValueError),
            ("bias", i32(B, 2, 3), ValueError), ("bias", flat[1:13].view(B, 2, 2), ValueError), ("bias", i32(B, 1025, 2), ValueError),
            ("mask", i32(1, 3), ValueError), ("mask", i32(4), ValueError), ("mask", i32(1 << 16, 4), ValueError), ("mask", i32(1, 4).cpu(), ValueError)]:
        with pytest.raises(err):
            choose.adjust(**{**good, name: bad})
    with pytest.raises(ValueError):  # its own memory, rows elsewhere
        choose.adjust(torch.as_strided(x, (2, 10), (20, 1)), torch.as_strided(x, (2, 10), (30, 1)), choose.new_settings(2))
    f = lambda *n: torch.zeros(*n, device=dev)  # noqa: E731
    ws = choose.new_workspace()
    good = dict(logits=x, ids=i32(B, 4), logprobs=f(B, 4), lse=f(B), workspace=ws)
    choose.top(**good)
    for name, bad in [("ids", i32(B, 0)), ("ids", i32(B, 65)), ("ids", i32(2, 4)), ("ids", i32(B, 4).long()), ("ids", i32(4, B).t()), ("logprobs", f(B, 5)),
                      ("logprobs", f(B, 4).half()), ("lse", f(2)), ("lse", i32(B)), ("workspace", ws[16:]), ("workspace", ws[1:]),
                      ("workspace", ws.view(2, -1)), ("workspace", ws.cpu()), ("workspace", ws.view(torch.int32))]:
        with pytest.raises((TypeError, ValueError)):
            choose.top(**{**good, name: bad})
    with pytest.raises(ValueError):
        choose.top(x[:, :3], i32(B, 4), f(B, 4), None, ws)
    r = f(B, 64)
    good = dict(logits=r, ids=i32(B, 4), weights=f(B, 4), bias=f(64), groups=8, keep=2, rows=i32(1))
    choose.experts(**good)
    for name, bad in [("groups", 0), ("groups", 7), ("groups", 64), ("keep", 0), ("keep", 9), ("ids", i32(B, 0)), ("ids", i32(B, 17)), ("ids", i32(2, 4)),
                      ("ids", f(B, 4)), ("weights", f(B, 5)), ("weights", i32(B, 4)), ("bias", f(63)), ("bias", f(64).half()), ("rows", i32(2)),
                      ("rows", i32(1).cpu()), ("logits", f(B, 1032))]:
        with pytest.raises((TypeError, ValueError)):
            choose.experts(**{**good, name: bad})
    with pytest.raises(ValueError):
        choose.experts(f(B, 8), i32(B, 2), f(B, 2), groups=8, keep=8, top2=True)
    good = dict(ids=i32(B, 4), order=i32(12), place=i32(B, 4), offsets=i32(9), workspace=ws)
    choose.plan(**good)
    for name, bad in [("ids", f(B, 4)), ("ids", i32(4, B).t()), ("order", i32(11)), ("order", i32(B, 4)), ("place", i32(12)), ("offsets", i32(1)),
                      ("offsets", i32(1026)), ("offsets", i32(3, 3)), ("workspace", ws[16:]), ("workspace", ws.view(torch.int32))]:
        with pytest.raises((TypeError, ValueError)):
            choose.plan(**{**good, name: bad})
