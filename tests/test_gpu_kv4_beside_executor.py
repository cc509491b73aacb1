"""The cache's ops launched beside a resident executor of a few SMs."""
import time

import numpy as np
import pytest

from tests import kv4_ref as R
from tests.gpu_harness import ensure_built, need_gpu
from tests.test_gpu_kv4 import _attend_case, _close, _dev, _f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("spread", [0, 60])
def test_launches_beside_a_resident_executor(spread):
    """Attention (its slow path's stack included), copies and row ops complete
    while the executor stays, and the executor runs the same op meanwhile.
    (The executor leaves after ten idle seconds, so that a launch that waited
    for its end would show as late, not hang.)"""
    import torch
    from persistent_micro_dispatch_gb300 import gpuos as G, kv4
    from workloads.device import warm_torch
    need_gpu()
    ensure_built()
    rng = np.random.default_rng(spread)
    q, pool, table, lens = _attend_case(71, 3, 24, 1, 128, 2, [700, 33, 2000])
    if spread:
        pool[:, :, 33 * 128:] = rng.integers(127 - spread, 127 + spread, pool[:, :, 33 * 128:].shape)
    wide = np.full((3, 8192), -1, np.int32)
    wide[:, :table.shape[1]] = table
    t = [_dev(q, torch.bfloat16), _dev(pool)]
    tables, ln = [_dev(table), _dev(wide)], _dev(lens)
    outs = [torch.zeros_like(t[0]) for _ in range(3)]
    ws = [kv4.new_workspace() for _ in range(2)]
    k = torch.zeros(40, 1, 128, device="cuda")
    s = torch.arange(40, dtype=torch.int32, device="cuda")
    other = kv4.new_pool(4, 1, 128)
    pairs = _dev(np.array([[0, 3]], np.int32))
    st, done = torch.cuda.Stream(), torch.cuda.Event()
    warm_torch()
    torch.cuda.synchronize()
    ex = G.Executor(blocks=8, idle_exit_ms=10_000)
    try:
        for tb, out in zip(tables, outs):
            G.eager_run(kv4.sdpa(*t, tb, ln, out, ws[0], 0.1), st.cuda_stream)
        G.eager_run(np.concatenate([kv4.write(k, k, s, other), kv4.page_copy(other.view(1, 4, -1), pairs),
                                    kv4.read(other, s, k, k)]), st.cuda_stream)
        done.record(st)
        ex.submit(kv4.sdpa(*t, tables[0], ln, outs[2], ws[1], 0.1))
        t0 = time.monotonic()
        while not done.query() and time.monotonic() - t0 < 5:
            time.sleep(0.01)
        late, running = not done.query(), ex.stats()["running"]
        ex.sync(timeout_ms=30_000)
    finally:
        assert ex.shutdown() == G.OK
    assert not late and running == 1
    if spread:
        from tests.test_gpu_kv4_scales import _want
        want, tol = _want(q, pool, table, lens, 0.1)
    else:
        want, tol = R.attend(q, pool, table, lens, 0.1)
    for out in outs:
        _close(_f64(out), want, tol)
