"""The executor's tile profile across a hand-off: every bucket, also those of
the 4-bit cache's ops and of user ops, counts from the executor's last launch."""
import numpy as np
import pytest

from tests.gpu_harness import ensure_built, need_gpu
from tests.test_gpu_kv4 import _attend_case, _dev
from tests.test_gpu_protocol import _NEG_SRC

pytestmark = pytest.mark.gpu


def test_profile_restarts_with_the_executor():
    import torch
    from persistent_micro_dispatch_gb300 import gpuos as G, kv4
    from workloads.device import warm_torch
    need_gpu()
    ensure_built()
    q, pool, table, lens = _attend_case(5, 3, 8, 2, 64, 1, [700, 33, 90])
    t = [_dev(q, torch.bfloat16), _dev(pool), _dev(table), _dev(lens)]
    out, ws = torch.zeros_like(t[0]), kv4.new_workspace()
    k = torch.ones(40, 2, 64, device="cuda")
    s = _dev(np.arange(40, dtype=np.int32))
    spare = torch.zeros(3, 2, 2, 34 * 64, dtype=torch.uint8, device="cuda")
    pairs = _dev(np.array([[0, 1]], np.int32))
    n = 5000
    x = torch.randn(n, device="cuda")
    y, z = torch.zeros_like(x), torch.zeros_like(x)
    add, user = G.make_descs(1), G.make_descs(1)
    add["op_id"], add["dtype"] = G.OP["add"], G.F32
    add["a"], add["b"], add["out"], add["dims"][0, 0] = x.data_ptr(), x.data_ptr(), y.data_ptr(), n
    user["op_id"], user["dtype"], user["ntiles"] = 80, G.F32, 5
    user["a"], user["b"], user["out"], user["dims"][0, 0] = x.data_ptr(), x.data_ptr(), z.data_ptr(), n
    cache = {"kv4_write": kv4.write(k, k, s, spare[0]), "kv4_read": kv4.read(spare[0], s, k, k),
             "kv4_sdpa": kv4.sdpa(*t, out, ws, 0.1), "page_copy": kv4.page_copy(spare, pairs)}
    tiles = {**{name: G.op_ntiles(d) for name, d in cache.items()}, "add": G.op_ntiles(add), "user": 5}

    def chain(*descs):
        d = np.concatenate(descs)
        d["flags"], d["dep"] = G.FLAG_DEP_REL, 0
        d["dep"][1:, 0] = 1
        return d

    def got(ex):
        ex.sync(timeout_ms=30_000)
        return {name: p["tiles"] for name, p in ex.tile_profile().items()}

    warm_torch()
    torch.cuda.synchronize()
    ex = G.Executor()
    try:
        ex.alias_op(80, G.OP["add"])
        ex.submit_batch(chain(*cache.values(), add, user, *cache.values(), user))
        ex.sync(timeout_ms=30_000)
        first = None
        for _ in range(200):  # the profile follows the completion records by a moment
            first = got(ex)
            if first == {**{name: 2 * tiles[name] for name in cache}, "add": tiles["add"], "user": 10}:
                break
        assert first == {**{name: 2 * tiles[name] for name in cache}, "add": tiles["add"], "user": 10}
        ex.register_op(90, G.compile_op(_NEG_SRC, "neg.cu"), "op_neg_ptr")  # hand-off
        assert ex.stats()["handoffs"] == 1
        ex.submit_batch(chain(*cache.values(), user))
        want = {**{name: tiles[name] for name in cache}, "user": 5}  # (no add since)
        ex.sync(timeout_ms=30_000)
        for _ in range(200):
            last = got(ex)
            if last == want:
                break
        assert last == want
        assert ex.stop() == G.OK
        prof = ex.tile_profile()
    finally:
        assert ex.shutdown() == G.OK
    assert {name: p["tiles"] for name, p in prof.items()} == want
    assert all(0 < p["body_us"] < 1e5 and p["finish_us"] < 1e5 and p["dep_us"] < 1e6 for p in prof.values())
    assert torch.equal(z, x + x)
