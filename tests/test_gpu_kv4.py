"""The 4-bit paged cache's ops on the GPU against their definitions in 64 bits
(tests/kv4_ref.py), eagerly and through the persistent executor."""
import numpy as np
import pytest

from tests import kv4_ref as R
from tests.gpu_harness import ensure_built, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    need_gpu()
    ensure_built()


def _dev(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def _f64(t):
    return t.double().cpu().numpy()


def _eager(*descs, stage=16384):
    import torch
    from persistent_micro_dispatch_gb300 import gpuos as G
    G.eager_run(np.concatenate(descs), torch.cuda.current_stream().cuda_stream, stage)
    torch.cuda.synchronize()


def _executor(*descs, expect=None, **cfg):
    """Each descriptor after the one before it; the statuses."""
    import torch
    from persistent_micro_dispatch_gb300 import gpuos as G
    from workloads.device import warm_torch
    d = np.concatenate(descs)
    d["flags"] = G.FLAG_DEP_REL
    d["dep"][1:, 0] = 1
    warm_torch()
    torch.cuda.synchronize()
    ex = G.Executor(**cfg)
    try:
        hist = ex.set_history(0, len(d))
        ex.submit_batch(d)
        rc = ex.sync(raise_on_error=False, timeout_ms=60_000)
    finally:
        assert ex.shutdown() == G.OK
    assert rc == (G.EDEVICE if expect and any(expect) else G.OK), G.strerror(rc)
    assert hist["status"].tolist() == (expect or [0] * len(d))


RUNNERS = {"eager": _eager, "eager_nostage": lambda *d, **k: _eager(*d, stage=0), "executor": _executor,
           "executor_nostage": lambda *d, **k: _executor(*d, stage_bytes=0, **k)}


def _attend_case(seed, B, H, heads, D, T, lens, spare=0, qsize=1.0, pool=None):
    rng = np.random.default_rng(seed)
    need = [-(-max(n, 0) // 32) for n in lens]
    P = max(max(need) + spare, 1)
    npages = sum(need) + 2
    if pool is None:
        pool = R.random_pool(rng, npages, heads, D)
    order = rng.permutation(npages)
    table = np.full((B, P), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    q = R.bf16(rng.standard_normal((B, T, H, D)) * qsize)
    return q, pool, table, np.array(lens, np.int32)


def _attend(run, q, pool, table, lens, scale, ws=None, out=None, **kw):
    import torch
    from persistent_micro_dispatch_gb300 import kv4
    qt = _dev(q, torch.bfloat16)
    o = torch.full_like(qt, 7.0) if out is None else out
    ws = kv4.new_workspace() if ws is None else ws
    held = _dev(pool), _dev(table), _dev(lens)  # alive until the descriptor has completed
    run(kv4.sdpa(qt, *held, o, ws, scale), **kw)
    assert not ws[:8192].any().item(), "counters left nonzero"
    return _f64(o)


def _close(got, want, tol):
    """bf16 output: half a step of rounding on top of the bound."""
    lim = tol + 2.0 ** -8 * np.abs(want) + 1e-30
    bad = ~(np.abs(got - want) <= lim)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], lim[bad][:5])


CASES = [
    # B, H, heads, D, T, lens
    (1, 1, 1, 128, 1, [1]),
    (1, 8, 1, 128, 1, [33]),
    (2, 8, 2, 64, 1, [31, 64]),
    (3, 4, 4, 128, 1, [1, 257, 32]),
    (5, 14, 2, 64, 1, [5, 0, 100, 31, 33]),
    (2, 16, 1, 128, 1, [700, 3]),         # sixteen rows a head
    (2, 20, 1, 64, 1, [129, 40]),         # twenty: an uneven last row tile
    (2, 6, 2, 128, 3, [2, 90]),           # the first token of request 0 sees nothing
    (2, 5, 1, 64, 32, [40, 17]),          # 160 rows
    (4, 8, 2, 128, 4, [0, 4, 65, 3]),
    (40, 2, 1, 64, 1, list(range(40))),   # more than a warp's lanes of requests
    (201, 3, 3, 64, 1, [7 * i % 90 for i in range(201)]),
    (1, 4, 1, 128, 1, [20011]),           # long: many partial states
    (3, 24, 1, 128, 5, [1500, 97, 3]),    # 120 rows
    (3, 32, 4, 128, 2, [3000, 7, 1023]),
]


@pytest.mark.parametrize("runner", sorted(RUNNERS))
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:5]) + f"-{max(c[5])}")
def test_attention(case, runner):
    B, H, heads, D, T, lens = case
    x = _attend_case(hash(case[:5]) & 0xFFFF, B, H, heads, D, T, lens, spare=B % 3)
    want, tol = R.attend(*x, D ** -0.5)
    _close(_attend(RUNNERS[runner], *x, D ** -0.5), want, tol)


@pytest.mark.parametrize("D,H,T,lens", [(128, 16, 1, [9000, 31, 0, 4097]), (64, 11, 3, [2, 700, 5000, 33]), (128, 64, 7, [1200, 5, 33])])
def test_attention_wide_tables(D, H, T, lens):
    """Tables wide enough for the launch to take sixteen rows at a time,
    whatever the lengths."""
    q, pool, table, lens = _attend_case(91, len(lens), H, 1, D, T, lens)
    wide = np.full((len(lens), 16384), -1, np.int32)
    wide[:, :table.shape[1]] = table
    want, tol = R.attend(q, pool, table, lens, D ** -0.5)
    for t in (table, wide):
        _close(_attend(_eager, q, pool, t, lens, D ** -0.5), want, tol)
    first = _attend(_eager, q, pool, wide, lens, 0.1)
    assert np.array_equal(_attend(_eager, q, pool, wide, lens, 0.1), first)


@pytest.mark.parametrize("runner", ["eager", "executor"])
def test_attention_most_heads(runner):
    """65,535 query heads over one cache head, two tokens: 131,070 rows."""
    q, pool, table, lens = _attend_case(101, 1, 65535, 1, 64, 2, [40])
    K, V, S = R.unpack(pool)
    at = np.arange(40)
    k, v, sc = (x[table[0, at // 32], 0, at % 32] for x in (K, V, S))
    want, tol = np.zeros(q.shape), np.zeros(q.shape)
    for t in range(2):
        n = 39 + t
        s = q[0, t] @ k[:n].T * 0.1
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        want[0, t] = p @ v[:n]
        reach = (np.abs(q[0, t]) @ np.abs(k[:n]).T * 0.1).max()
        tol[0, t] = R.bound(p, np.abs(v[:n]), sc[:n].max(0), reach, 64)
    _close(_attend(RUNNERS[runner], q, pool, table, lens, 0.1), want, tol)


def test_first_call_captured():
    """The first call of a process may be inside a capture."""
    import os
    import subprocess
    import sys
    code = """
import torch
from persistent_micro_dispatch_gb300 import gpuos as G, kv4
q = torch.randn(2, 1, 4, 128, device="cuda").bfloat16()
pool, ws, out = kv4.new_pool(8, 2, 128), kv4.new_workspace(), torch.zeros_like(q)
k = torch.randn(70, 2, 128, device="cuda").bfloat16()
slots = torch.arange(70, device="cuda", dtype=torch.int32)
table = torch.tensor([[0, 1, 2], [0, -1, -1]], device="cuda", dtype=torch.int32)
lens = torch.tensor([70, 1], device="cuda", dtype=torch.int32)
pairs = torch.tensor([[0, 5]], device="cuda", dtype=torch.int32)
st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g, stream=st):
    for d in (kv4.write(k, k, slots, pool), kv4.page_copy(pool.view(1, 8, -1), pairs),
              kv4.sdpa(q, pool, table, lens, out, ws, 0.1), kv4.read(pool, slots, k, k)):
        G.eager_run(d, st.cuda_stream)
g.replay()
torch.cuda.synchronize()
assert torch.equal(out[1, 0, 0], k[0, 0]) and torch.equal(out[1, 0, 3], k[0, 1]) and torch.equal(pool[5], pool[0])
print("captured ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert "captured ok" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("runner", ["eager", "executor"])
def test_attention_is_the_same_each_time(runner):
    """Partial states merge in the order of the keys, whoever arrives last."""
    x = _attend_case(5, 3, 8, 2, 128, 1, [4000, 999, 2500])
    first = _attend(RUNNERS[runner], *x, 0.09)
    for _ in range(3):
        assert np.array_equal(_attend(RUNNERS[runner], *x, 0.09), first)


@pytest.mark.parametrize("qsize,scale", [(1e-30, 1e30), (1e30, 1e-31), (300.0, 0.01), (1.0, -0.1), (1.0, 0.0)])
def test_attention_query_sizes(qsize, scale):
    """Queries far from one: their rows are scaled by powers of two."""
    x = _attend_case(11, 2, 4, 2, 64, 1, [70, 300], qsize=qsize)
    want, tol = R.attend(*x, scale)
    _close(_attend(_eager, *x, scale), want, tol)


@pytest.mark.parametrize("runner", ["eager", "executor"])
def test_attention_value_scales_far_apart(runner):
    """Value scales 2^-60 to 2^60 in one group: what a key adds is kept to
    2^-20 of the largest value, whichever order they come in."""
    rng = np.random.default_rng(3)
    lens = [97, 64, 200]
    q, pool, table, lens = _attend_case(3, 3, 4, 2, 64, 1, lens)
    D = 64
    key, c = np.meshgrid(np.arange(32), np.arange(D), indexing="ij")
    vs = R.offsets(D, key, c)[3][:, ::32]
    pool[:, :, vs] = rng.integers(127 - 60, 127 + 60, (pool.shape[0], 2, 32, 2)).astype(np.uint8)
    want, tol = R.attend(q, pool, table, lens, 0.125)
    _close(_attend(RUNNERS[runner], q, pool, table, lens, 0.125), want, tol)


@pytest.mark.parametrize("runner", ["eager", "executor"])
def test_attention_sink(runner):
    """One key takes nearly all the weight and its value is nothing: the
    output is what thousands of keys with weights near 2^-20 add up to."""
    q, pool, table, lens = _attend_case(61, 1, 4, 1, 128, 1, [12001])
    k0, v0, ks, vs = R.offsets(128, 0, np.arange(128))
    pool[:, :, 32 * 128:33 * 128] = 121  # the other keys are small
    pool[table[0, 0], 0, v0] = 0
    pool[table[0, 0], 0, k0] = 0x22  # every channel 1.0
    pool[table[0, 0], 0, ks] = 127
    q[:] = R.bf16(0.5 + np.random.default_rng(1).standard_normal(q.shape) * 0.03)
    scale = 14.0 / 64  # the sink's score 14, 20 octaves; the others' near 0
    want, tol = R.attend(q, pool, table, lens, scale)
    K, V, _ = R.unpack(pool)
    s = (K[table[0, 0], 0, 0] * q[0, 0, 0]).sum() * scale
    assert 13 < s < 15 and 1e-5 < np.abs(want).max() < 1e-2
    _close(_attend(RUNNERS[runner], q, pool, table, lens, scale), want, tol)


def test_attention_graphs_share_a_workspace():
    """Two captured calls with one workspace, replayed one after another."""
    import torch
    from persistent_micro_dispatch_gb300 import gpuos as G, kv4
    ws, st = kv4.new_workspace(), torch.cuda.Stream()
    graphs, held = [], []
    for seed, (B, H, heads, D, T, ls) in ((71, (2, 8, 2, 128, 1, [700, 2100])), (72, (1, 24, 1, 64, 1, [5000]))):
        q, pool, table, lens = _attend_case(seed, B, H, heads, D, T, ls)
        t = [_dev(q, torch.bfloat16), _dev(pool), _dev(table), _dev(lens)]
        out = torch.zeros(B, T, H, D, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            G.eager_run(kv4.sdpa(*t, out, ws, 0.1), st.cuda_stream)
        graphs.append(g)
        held.append((t, out, R.attend(q, pool, table, lens, 0.1)))
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for _, out, (want, tol) in held:
        _close(_f64(out), want, tol)
    assert not ws[:8192].any().item()


@pytest.mark.parametrize("runner", ["eager", "executor"])
def test_attention_stale_rows_and_nan_groups(runner):
    """Scale bytes of 255: behind the last key they are ignored; a visible
    value group gives NaN there and only there; a visible key gives NaN rows."""
    D, heads, H, T = 128, 2, 4, 2
    q, pool, table, lens = _attend_case(9, 4, H, heads, D, T, [37, 64, 50, 41])
    key = np.arange(32)
    for b, n in enumerate(lens):
        last = table[b, (n - 1) // 32]
        for k in key[n % 32 or 32:]:  # stale rows
            for cc in range(0, D, 32):
                _, _, ks, vs = R.offsets(D, k, cc)
                pool[last, :, [ks, vs]] = 255
    # request 2: value group 1 of head 0, key 10; request 3: key 40 of head 1 (seen by the last token only)
    _, _, _, vs = R.offsets(D, 10, 32)
    pool[table[2, 0], 0, vs] = 255
    k0, _, ks, _ = R.offsets(D, 8, np.arange(64, 96))
    pool[table[3, 1], 1, ks] = 255
    pool[table[3, 1], 1, k0] = 0
    want, tol = R.attend(q, pool, table, lens, 0.1)
    want[2, :, 0:2, 32:64] = np.nan
    want[3, 1, 2:4] = np.nan
    got = _attend(RUNNERS[runner], q, pool, table, lens, 0.1)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = ~np.isnan(want)
    _close(got[fine], want[fine], np.where(fine, tol, 0)[fine])


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_attention_bad_queries(bad):
    """A NaN or infinity in a query row makes that row NaN and no other."""
    q, pool, table, lens = _attend_case(21, 2, 4, 1, 64, 2, [1, 80])
    q[1, 0, 2, 17] = bad
    q[0, 0, 1, 3] = bad  # a row that sees no key: zeros all the same
    clean = np.where(np.isfinite(q), q, 0)
    want, tol = R.attend(clean, pool, table, lens, 0.2)
    got = _attend(_eager, q, pool, table, lens, 0.2)
    assert np.isnan(got[1, 0, 2]).all()
    keep = np.ones(q.shape[:3], bool)
    keep[1, 0, 2] = False
    _close(got[keep], want[keep], tol[keep])


@pytest.mark.parametrize("runner", ["eager", "executor"])
def test_attention_bad_pages_and_lengths(runner):
    """Pages that are not in the pool count as no keys; a length that the
    table cannot hold leaves its request's rows alone. Status 2 for both."""
    q, pool, table, lens = _attend_case(31, 5, 4, 2, 64, 1, [100, 96, 64, 33, 64])
    table[0, 1] = pool.shape[0]
    table[1, 0] = -5
    table[2, :] = 1 << 30
    lens[3] = 32 * table.shape[1] + 1
    lens[4] = -1
    sane = lens.copy()
    sane[3:] = 0
    want, tol = R.attend(q, pool, table, sane, 0.1)
    want[2] = np.nan  # sees positions, but none holds a key
    want[3:] = 7.0
    kw = {"expect": [2]} if runner == "executor" else {}
    got = _attend(RUNNERS[runner], q, pool, table, lens, 0.1, **kw)
    assert np.isnan(got[2]).all()
    keep = [0, 1, 3, 4]
    _close(got[keep], want[keep], tol[keep])


def test_attention_replayed_and_two_streams():
    """A captured call replayed on changed inputs; two calls at once on two
    streams with a workspace each."""
    import torch
    from persistent_micro_dispatch_gb300 import gpuos as G, kv4
    D, scale = 128, 0.08
    q, pool, table, lens = _attend_case(41, 3, 8, 2, D, 1, [900, 40, 333])
    t = [_dev(q, torch.bfloat16), _dev(pool), _dev(table), _dev(lens)]
    ws, out = kv4.new_workspace(), torch.zeros(3, 1, 8, D, dtype=torch.bfloat16, device="cuda")
    d = kv4.sdpa(*t, out, ws, scale)
    _eager(d)
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        G.eager_run(d, st.cuda_stream)
    for n in ([900, 40, 333], [1, 0, 12], [512, 65, 31]):
        lens[:] = n
        t[3].copy_(_dev(lens))
        want, tol = R.attend(q, pool, table, lens, scale)
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        _close(_f64(out), want, tol)
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [(kv4.new_workspace(), torch.zeros_like(out)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (w, o) in zip(streams, sets):
            G.eager_run(kv4.sdpa(*t, o, w, scale), s.cuda_stream)
    torch.cuda.synchronize()
    for _, o in sets:
        _close(_f64(o), want, tol)


def test_attention_far_pages():
    """A pool of more than 4 GB: page offsets pass 32 bits."""
    import torch
    from persistent_micro_dispatch_gb300 import kv4
    D, heads, npages = 128, 8, 150_000  # 5.2 GB
    q, small, table, lens = _attend_case(51, 1, 16, heads, D, 1, [3 * 32 + 5])
    pool = torch.zeros(npages, heads, 34 * D, dtype=torch.uint8, device="cuda")
    far = np.array([npages - 1, 123_457, 0, 149_000], np.int32)
    for i, pg in enumerate(far):
        pool[int(pg)] = _dev(small[table[0, i]])
    out = torch.zeros(1, 1, 16, D, dtype=torch.bfloat16, device="cuda")
    held = _dev(q, torch.bfloat16), _dev(far[None]), _dev(lens), kv4.new_workspace()
    _eager(kv4.sdpa(held[0], pool, held[1], held[2], out, held[3], 0.1))
    want, tol = R.attend(q, small, table, lens, 0.1)
    _close(_f64(out), want, tol)
    # the row ops at the far end
    slots = _dev(np.array([(npages - 1) * 32 + 31, 123_457 * 32 + 1], np.int32))
    k = torch.randn(2, heads, D, device="cuda")
    v = torch.randn(2, heads, D, device="cuda")
    kb, vb = torch.empty_like(k), torch.empty_like(v)
    _eager(kv4.write(k, v, slots, pool), kv4.read(pool, slots, kb, vb))
    for x, y in ((k, kb), (v, vb)):
        assert np.array_equal(_f64(y), R.values(*R.quantise(_f64(x))))


def test_launches_wait_for_their_predecessors():
    """A chain of short and long launches on one stream, ordinary kernels
    among them: each op sees what every earlier one wrote, also past a launch
    between them that has nothing to do."""
    import torch
    from persistent_micro_dispatch_gb300 import gpuos as G, kv4
    rng = np.random.default_rng(5)
    heads, D, n = 8, 128, 40_000
    pool = kv4.new_pool(n // 32, heads, D)
    k = _dev(R.bf16(rng.standard_normal((n, heads, D))), torch.bfloat16)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    hole = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    one = torch.empty(1, heads, D, dtype=torch.bfloat16, device="cuda")
    src, a, b = torch.empty_like(k), torch.empty_like(k), torch.empty_like(k)
    pairs = _dev(np.array([[i, n // 32 - 1 - i] for i in range(n // 64)], np.int32))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for r in range(8):
            torch.mul(k, float(2 ** r), out=src)  # an ordinary kernel, then ours
            G.eager_run(kv4.write(src, src, slots, pool), st.cuda_stream)
            G.eager_run(kv4.read(pool, hole, one, one), st.cuda_stream)
            G.eager_run(kv4.page_copy(pool.view(1, n // 32, -1), pairs), st.cuda_stream)
            G.eager_run(kv4.read(pool, hole, one, one), st.cuda_stream)
            G.eager_run(kv4.read(pool, slots, a, b), st.cuda_stream)
            got = a.clone()  # ours, then an ordinary kernel
            want = R.values(*R.quantise(_f64(k[:32 * 4]) * 2.0 ** r))
            st.synchronize()
            assert np.array_equal(_f64(got[:128]), want)
            m = torch.arange(n, device="cuda").view(-1, 32)
            m[n // 32 - n // 64:] = m[:n // 64].flip(0)
            assert torch.equal(got, got[m.flatten()])


def _rows(rng, n, heads, D, f32):
    x = rng.standard_normal((n, heads, D)) * np.exp(2 * rng.standard_normal((n, heads, D // 32))).repeat(32, -1)
    return x.astype(np.float32).astype(np.float64) if f32 else R.bf16(x)


@pytest.mark.parametrize("runner", ["eager", "executor"])
@pytest.mark.parametrize("n,heads,D,f32", [(1, 1, 128, False), (1, 1, 64, True), (37, 3, 64, False), (5, 8, 128, True),
                                           (700, 2, 128, False), (2100, 1, 64, True), (600, 40, 64, False)])
def test_write_and_read(runner, n, heads, D, f32):
    """Codes and scales byte for byte, everything else of the pool untouched;
    the rows read back exactly."""
    import torch
    from persistent_micro_dispatch_gb300 import kv4
    rng = np.random.default_rng(n)
    npages = n // 20 + 2
    pool = rng.integers(0, 256, (npages, heads, 34 * D)).astype(np.uint8)
    if n >= 600:  # runs of neighbouring slots, as prompts have them
        slots = (rng.permutation(npages)[:, None] * 32 + np.arange(32)).ravel()[3:n + 3].astype(np.int32)
    else:
        slots = rng.permutation(npages * 32)[:n].astype(np.int32)
    slots[n // 2:n // 2 + n // 10] = -1
    k, v = _rows(rng, n, heads, D, f32), _rows(rng, n, heads, D, f32)
    dt = torch.float32 if f32 else torch.bfloat16
    kt, vt, st, pt = _dev(k, dt), _dev(v, dt), _dev(slots), _dev(pool)
    kb, vb = torch.full_like(kt, 9), torch.full_like(vt, 9)
    RUNNERS[runner](kv4.write(kt, vt, st, pt), kv4.read(pt, st, kb, vb))
    (kc, ks), (vc, vs) = R.quantise(k), R.quantise(v)
    want = pool.copy()
    for i in range(n):
        for h in range(heads if slots[i] >= 0 else 0):
            R.put(want, slots[i], h, kc[i, h], ks[i, h], vc[i, h], vs[i, h])
    assert np.array_equal(pt.cpu().numpy(), want)
    hole = (slots < 0)[:, None, None]
    assert np.array_equal(_f64(kb), np.where(hole, 0, R.values(kc, ks)))
    assert np.array_equal(_f64(vb), np.where(hole, 0, R.values(vc, vs)))


def test_write_edges():
    """Every border between codes, signed zeros, subnormal and largest
    numbers, NaN and infinities, each in a group of its own."""
    import torch
    from persistent_micro_dispatch_gb300 import kv4
    f = np.float32
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], f)
    near = np.concatenate([borders, np.nextafter(borders, f(0)), np.nextafter(borders[:7], f(9)), np.zeros(8, f)])
    groups = [np.concatenate([[f(6)], near * s]) for s in (1, -1)]
    groups += [g * f(2.0) ** e for g in groups[:1] for e in (-126, -100, 60, 124)]
    for top in (1e-45, 2e-45, 3e-39, 1.1754944e-38, 3.4028235e38, 3.0e38, 2.5521178e38, 2.6e38, 0.0, -0.0):
        groups.append(np.full(32, top, f) * np.array([1, -1] * 16, f))
    for bad in (np.nan, np.inf, -np.inf):
        g = np.ones(32, f)
        g[7] = bad
        groups.append(g)
    x = np.concatenate(groups).reshape(-1, 1, 32).astype(f)
    x = np.concatenate([x, x], -1)  # D = 64
    n = len(x)
    slots = np.arange(n, dtype=np.int32)
    pool = torch.zeros(n // 32 + 1, 1, 34 * 64, dtype=torch.uint8, device="cuda")
    kt, st = _dev(x), _dev(slots)
    vt = _dev(x[::-1].copy())
    kb, vb = torch.empty_like(kt), torch.empty_like(vt)
    kh, vh = torch.empty_like(kt, dtype=torch.bfloat16), torch.empty_like(vt, dtype=torch.bfloat16)
    _eager(kv4.write(kt, vt, st, pool), kv4.read(pool, st, kb, vb), kv4.read(pool, st, kh, vh))
    want = np.zeros(tuple(pool.shape), np.uint8)
    (kc, ks), (vc, vs) = R.quantise(x), R.quantise(x[::-1])
    for i in range(n):
        R.put(want, i, 0, kc[i, 0], ks[i, 0], vc[i, 0], vs[i, 0])
    assert np.array_equal(pool.cpu().numpy(), want)
    for got, c, s in ((kb, kc, ks), (vb, vc, vs), (kh, kc, ks), (vh, vc, vs)):
        assert np.array_equal(_f64(got), R.values(c, s), equal_nan=True)


def test_slots_outside_the_pool():
    import torch
    from persistent_micro_dispatch_gb300 import kv4
    pool = torch.full((2, 1, 34 * 64), 0x5A, dtype=torch.uint8, device="cuda")
    k = torch.ones(3, 1, 64, device="cuda")
    slots = _dev(np.array([64, 2, (1 << 31) - 1], np.int32))
    kb, vb = torch.full_like(k, 9), torch.full_like(k, 9)
    _executor(kv4.write(k, k, slots, pool), kv4.read(pool, slots, kb, vb), expect=[2, 2])
    got = _f64(kb)
    assert (got[0] == 0).all() and (got[2] == 0).all() and (got[1] == 1).all()
    R_pool = np.full((2, 1, 34 * 64), 0x5A, np.uint8)
    c, s = R.quantise(np.ones((1, 64)))
    R.put(R_pool, 2, 0, c[0], s[0], c[0], s[0])
    assert np.array_equal(pool.cpu().numpy(), R_pool)


@pytest.mark.parametrize("runner", ["eager", "executor"])
@pytest.mark.parametrize("layers,npages,nbytes,n", [(1, 2, 16, 1), (3, 40, 2176, 15), (2, 9, 34816, 4), (5, 70, 16400, 33),
                                                    (1, 600, 272, 299)])
def test_page_copy(runner, layers, npages, nbytes, n):
    from persistent_micro_dispatch_gb300 import kv4
    rng = np.random.default_rng(n)
    pool = rng.integers(0, 256, (layers, npages, nbytes)).astype(np.uint8)
    order = rng.permutation(npages)
    src, dst = order[:n].copy(), order[n:2 * n]
    n = len(dst)
    src = np.where(np.arange(n) % 4 == 3, src[0], src[:n])  # one page forks often
    pairs = np.stack([src, dst], 1).astype(np.int32)
    if n > 3:
        pairs[1] = -1, pairs[1, 1]
        pairs[2] = pairs[2, 0], -7
    want = pool.copy()
    for s, d in pairs:
        if s >= 0 and d >= 0:
            want[:, d] = pool[:, s]
    pt, pr = _dev(pool), _dev(pairs)
    RUNNERS[runner](kv4.page_copy(pt, pr))
    assert np.array_equal(pt.cpu().numpy(), want)


def test_page_copy_far_and_outside():
    import torch
    from persistent_micro_dispatch_gb300 import kv4
    pool = torch.zeros(3, 100_000, 16384, dtype=torch.uint8, device="cuda")  # 4.9 GB
    pool[:, 3] = torch.arange(16384, device="cuda").to(torch.uint8)
    pairs = _dev(np.array([[3, 99_999], [3, 50_000]], np.int32))
    _eager(kv4.page_copy(pool, pairs))
    assert (pool[:, 99_999] == pool[:, 3]).all() and (pool[:, 50_000] == pool[:, 3]).all()
    assert not pool[:, 99_998].any() and not pool[:, 49_999].any() and not pool[:, 50_001].any()
    small = torch.zeros(2, 4, 64, dtype=torch.uint8, device="cuda")
    small[:, 1] = 5
    pairs = _dev(np.array([[4, 0], [1, 9], [1, 2]], np.int32))
    _executor(kv4.page_copy(small, pairs), expect=[2])
    assert small[:, 2].eq(5).all() and not small[:, 0].any() and not small[:, 3].any()


@pytest.mark.parametrize("runner", ["eager", "executor"])
def test_serving_steps(runner):
    """A prompt is written, forked, and both branches take decode steps of
    their own: write, then attend, over a cache that the copies made."""
    import torch
    from persistent_micro_dispatch_gb300 import kv4
    rng = np.random.default_rng(77)
    heads, H, D, npages, steps = 2, 8, 128, 12, 5
    pool = kv4.new_pool(npages, heads, D)
    ws = kv4.new_workspace()
    n = 75
    table = np.full((2, 4), -1, np.int32)
    table[0, :3] = [7, 2, 9]
    k, v = _rows(rng, n, heads, D, False), _rows(rng, n, heads, D, False)
    at = np.arange(n)
    keep, descs, outs, qs = [], [], [], []

    def dev(x, dt=None):
        keep.append(_dev(x, dt))
        return keep[-1]

    slots = table[0, at // 32] * 32 + at % 32
    descs.append(kv4.write(dev(k, torch.bfloat16), dev(v, torch.bfloat16), dev(slots.astype(np.int32)), pool))
    # the fork shares the full pages and copies the last one
    table[1, :3] = [7, 2, 4]
    descs.append(kv4.page_copy(pool.view(1, npages, -1), dev(np.array([[9, 4]], np.int32))))
    ref = np.zeros((npages, heads, 34 * D), np.uint8)

    def put(slot, kr, vr):
        for h in range(heads):
            (kc, ks), (vc, vs) = R.quantise(kr[h]), R.quantise(vr[h])
            R.put(ref, slot, h, kc, ks, vc, vs)

    for i in range(n):
        put(slots[i], k[i], v[i])
    ref[4] = ref[9]
    table[0, 3], table[1, 3] = 11, 0
    tb = dev(table)
    want = []
    for s in range(steps):
        pos = n + s
        kn, vn = _rows(rng, 2, heads, D, False), _rows(rng, 2, heads, D, False)
        sl = table[:, pos // 32] * 32 + pos % 32
        q = R.bf16(rng.standard_normal((2, 1, H, D)))
        lens = np.array([pos + 1] * 2, np.int32)
        outs.append(torch.zeros(2, 1, H, D, dtype=torch.bfloat16, device="cuda"))
        descs.append(kv4.write(dev(kn, torch.bfloat16), dev(vn, torch.bfloat16), dev(sl.astype(np.int32)), pool))
        descs.append(kv4.sdpa(dev(q, torch.bfloat16), pool, tb, dev(lens), outs[-1], ws, D ** -0.5))
        for b in range(2):
            put(sl[b], kn[b], vn[b])
        want.append(R.attend(q, ref, table, lens, D ** -0.5))
    RUNNERS[runner](*descs)
    for o, (w, tol) in zip(outs, want):
        _close(_f64(o), w, tol)
    assert np.array_equal(pool.cpu().numpy(), ref)


def test_aliased_ops_check_their_sizes():
    """An alias is a user op: the host passes its sizes and tile count on, and
    the op itself refuses what it cannot do."""
    import torch
    from persistent_micro_dispatch_gb300 import gpuos as G, kv4
    from workloads.device import warm_torch
    q, pool, table, lens = _attend_case(81, 2, 4, 2, 64, 1, [700, 33])
    t = [_dev(q, torch.bfloat16), _dev(pool), _dev(table), _dev(lens)]
    out, ws = torch.zeros_like(t[0]), kv4.new_workspace()
    k = torch.ones(3, 2, 64, device="cuda")
    s = _dev(np.array([0, 1, 2], np.int32))
    pairs = _dev(np.array([[0, 1], [0, 1]], np.int32))
    good = kv4.sdpa(*t, out, ws, 0.1)
    reads, copies = kv4.read(t[1], s, k, k), kv4.page_copy(t[1][None], pairs)
    bad = []

    def refused(alias, desc, dim=None, value=0, field=None, shift=0):
        d = desc.copy()
        d["op_id"] = alias
        if dim is not None:
            d["dims"][0, dim] = value
        if field:
            d[field] = d[field] + shift if shift else 0
        bad.append(d)

    for dim, value in ((1, 4), (1, 4 | 3 << 16), (2, 96 | 1 << 16), (2, 64), (3, 0), (4, 0)):
        refused(90, good, dim, value)
    for field, shift in (("a", 8), ("b", 2), ("out", 1), ("aux0", 2), ("aux1", 1), ("aux2", 8), ("b", 0)):
        refused(90, good, field=field, shift=shift)
    for dim, value in ((1, 0), (2, 96), (3, 0)):
        refused(91, reads, dim, value)
    refused(91, reads, field="aux1", shift=4)
    for dim, field, shift in ((1, None, 0), (3, None, 0), (None, "a", 0), (None, "aux0", 4)):
        refused(92, copies, dim, 0, field, shift)
    good["op_id"], good["ntiles"] = 90, 5000  # more tiles than the workspace holds states for
    d = np.concatenate([good] + bad)
    d["ntiles"][1:] = 4
    d["flags"] = G.FLAG_DEP_REL
    d["dep"][1:, 0] = 1
    warm_torch()
    torch.cuda.synchronize()
    ex = G.Executor()
    try:
        ex.alias_op(90, G.OP["kv4_sdpa"])
        ex.alias_op(91, G.OP["kv4_read"])
        ex.alias_op(92, G.OP["page_copy"])
        hist = ex.set_history(0, len(d))
        ex.submit_batch(d)
        rc = ex.sync(raise_on_error=False, timeout_ms=60_000)
    finally:
        assert ex.shutdown() == G.OK
    assert rc == G.EDEVICE and hist["status"].tolist() == [0] + [2] * len(bad)
    want, tol = R.attend(q, pool, table, lens, 0.1)
    _close(_f64(out), want, tol)
    assert not ws[:8192].any().item()


def test_binding_refusals():
    import torch
    from persistent_micro_dispatch_gb300 import kv4
    pool = kv4.new_pool(4, 2, 64)
    ws = kv4.new_workspace()
    q = torch.zeros(3, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    ok = dict(q=q, pool=pool, table=table, lens=lens, out=torch.empty_like(q), workspace=ws, scale=1.0)
    kv4.sdpa(**ok)
    flat = torch.zeros(4096, dtype=torch.bfloat16, device="cuda")
    for name, bad, err in [("q", q.float(), TypeError), ("q", q.cpu(), ValueError), ("q", q[:, :, :3], ValueError),
                           ("q", flat[1:769].view(3, 1, 4, 64), ValueError), ("table", table[:2], ValueError),
                           ("table", table.long(), TypeError), ("lens", lens[:2], ValueError), ("pool", pool[:, :, 1:], ValueError),
                           ("out", q[:2].clone(), ValueError), ("workspace", ws[:-16], ValueError),
                           ("q", torch.zeros(3, 33, 4, 64, dtype=torch.bfloat16, device="cuda"), ValueError),
                           ("q", q.transpose(0, 2), ValueError), ("table", table[:, :0], ValueError)]:
        with pytest.raises(err):
            kv4.sdpa(**{**ok, name: bad})
    k = torch.zeros(3, 2, 64, device="cuda")
    s = torch.zeros(3, dtype=torch.int32, device="cuda")
    for args in [(k, k.bfloat16(), s, pool), (k.half(), k.half(), s, pool), (k, k, s[:2], pool), (k, k, s.long(), pool),
                 (k[:, :1], k[:, :1], s, pool), (k, k, s, pool.view(-1))]:
        with pytest.raises((TypeError, ValueError)):
            kv4.write(*args)
        with pytest.raises((TypeError, ValueError)):
            kv4.read(args[3], args[2], args[0], args[1])
    p = torch.zeros(2, 4, 24, dtype=torch.uint8, device="cuda")
    pr = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    for args in [(p, pr), (p[:, :, :16], pr), (p[0], pr), (torch.zeros(2, 4, 16, device="cuda"), pr.view(2, 1))]:
        with pytest.raises(ValueError):
            kv4.page_copy(*args)
    kv4.write(k[:0], k[:0], s[:0], pool)
    _eager(kv4.write(k[:0], k[:0], s[:0], pool), kv4.sdpa(q[:0], pool, table[:0], lens[:0], q[:0], ws, 1.0))
