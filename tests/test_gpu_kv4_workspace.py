"""A workspace after an attention that did not run to its end."""
import re

import pytest

from tests import kv4_ref as R
from tests.gpu_harness import ensure_built, need_gpu
from tests.test_gpu_kv4 import RUNNERS, _attend, _attend_case, _close


def test_counter_bytes_are_the_headers():
    from persistent_micro_dispatch_gb300 import build, kv4
    text = open(f"{build.INCLUDE}/gpuos.h").read()
    assert int(re.search(r"#define GPUOS_KV4_COUNTERS (\d+)u", text).group(1)) == kv4.COUNTER_BYTES


def test_reset_refuses_what_is_no_workspace():
    import torch
    from persistent_micro_dispatch_gb300 import kv4
    ws = kv4.new_workspace(device="cpu").fill_(7)
    for bad in (ws[:-1], ws.view(torch.int32), ws.view(2, -1), torch.zeros(8192, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            kv4.reset_workspace(bad)
    kv4.reset_workspace(ws)
    assert not ws[:kv4.COUNTER_BYTES].any() and (ws[kv4.COUNTER_BYTES:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("runner", ["eager", "executor"])
def test_reset_after_an_abandoned_attention(runner):
    """Counters raised as tiles that ran before the others were given up leave
    them, and any states behind them: reset, the next attention is right."""
    import torch
    from persistent_micro_dispatch_gb300 import kv4
    need_gpu()
    ensure_built()
    x = _attend_case(5, 3, 8, 2, 128, 1, [4000, 999, 2500])
    want, tol = R.attend(*x, 0.09)
    ws = kv4.new_workspace()
    ws.copy_(torch.randint(0, 256, (kv4.WORKSPACE_BYTES,), dtype=torch.uint8, device="cuda"))
    ws.view(torch.int32)[:kv4.COUNTER_BYTES // 4] = (torch.arange(kv4.COUNTER_BYTES // 4, device="cuda") % 3 == 1).int()
    kv4.reset_workspace(ws)
    torch.cuda.synchronize()
    for _ in range(2):
        _close(_attend(RUNNERS[runner], *x, 0.09, ws=ws), want, tol)


@pytest.mark.gpu
def test_a_wait_that_runs_out_and_the_workspace():
    """An attention behind a fence whose wait runs out completes with status
    3; after a reset its workspace serves again."""
    import torch
    from persistent_micro_dispatch_gb300 import gpuos as G, kv4
    from tests.test_gpu_kv4 import _dev
    from tests.test_gpu_protocol import _big_add
    need_gpu()
    ensure_built()
    q, pool, table, lens = _attend_case(6, 2, 8, 2, 64, 1, [3000, 999])
    t = [_dev(q, torch.bfloat16), _dev(pool), _dev(table), _dev(lens)]
    out, ws = torch.zeros_like(t[0]), kv4.new_workspace()
    attend = kv4.sdpa(*t, out, ws, 0.1)
    attend["flags"] = G.FLAG_FENCE
    big, keep = _big_add(1 << 26)
    ex = G.Executor(blocks=1, warps_per_block=2, dep_timeout_ms=20)
    try:
        ex.submit(big)
        ticket = ex.submit(attend)
        assert ex.sync(timeout_ms=60_000, raise_on_error=False) == G.EDEVICE
        assert ex.query(ticket).status == G.ST_DEP_TIMEOUT
    finally:
        assert ex.shutdown() == G.OK
    kv4.reset_workspace(ws)
    want, tol = R.attend(q, pool, table, lens, 0.1)
    for runner in ("executor", "eager"):
        _close(_attend(RUNNERS[runner], q, pool, table, lens, 0.1, ws=ws), want, tol)
    del keep
