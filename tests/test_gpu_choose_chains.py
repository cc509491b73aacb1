"""What a decode step chooses, as the documents say to submit it: chains of
dependencies in the executor, and a process's first call inside a capture."""
import numpy as np
import pytest

from tests.gpu_harness import ensure_built, need_gpu
from tests.test_gpu_choose_use import Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    need_gpu()
    ensure_built()


def test_two_chains_side_by_side():
    """Tokens and experts, each chain with a workspace of its own, many times in one batch."""
    import torch
    from persistent_micro_dispatch_gb300 import choose, gpuos as G
    from workloads.device import warm_torch
    steps = [Step(k, N=n, B=7) for k, n in ((1, 900), (2, 40), (3, 2000))]
    batch = []
    for s in steps:
        s.ws2 = choose.new_workspace()
        tokens = np.concatenate([choose.adjust(s.logits, s.out, s.t, **s.kw), choose.top(s.out, s.ids, s.lp, s.lse, s.ws)])
        experts = np.concatenate([choose.experts(s.router, s.eids, s.w, sigmoid=True, bias=s.balance, groups=4, keep=2, top2=True, scale=2.0),
                                  choose.plan(s.eids, s.order, s.place, s.offsets, s.ws2)])
        for d in (tokens, experts):
            d["flags"], d["dep"][1:, 0] = G.FLAG_DEP_REL, 1
            batch.append(d)
    d = np.concatenate(batch)
    warm_torch()
    torch.cuda.synchronize()
    ex = G.Executor()
    try:
        for _ in range(20):
            ex.submit_batch(d)
            ex.sync(timeout_ms=60_000)
    finally:
        assert ex.shutdown() == G.OK
    for s in steps:
        s.check()
        assert not s.ws[:choose.COUNTER_BYTES].any() and not s.ws2[:choose.COUNTER_BYTES].any()


def test_first_call_captured():
    """The first call of a process may be inside a capture: kernels that need their shared memory raised, and clusters, too."""
    import os
    import subprocess
    import sys
    code = """
import torch
from persistent_micro_dispatch_gb300 import choose, gpuos as G
dev, i32 = "cuda", torch.int32
x, ws = torch.randn(2, 9000, device=dev), choose.new_workspace()
out, ids, lp = torch.empty_like(x), torch.zeros(2, 3, dtype=i32, device=dev), torch.zeros(2, 3, device=dev)
settings = choose.new_settings(2)
tokens = torch.randint(0, 9000, (2, 20000), device=dev).int()
f = choose.fields(settings)
f["length"][:], f["presence"][:] = 20000, 0.5
r, eids, w = torch.randn(700, 1024, device=dev), torch.zeros(700, 8, dtype=i32, device=dev), torch.zeros(700, 8, device=dev)
order, place, offsets = torch.zeros(5600, dtype=i32, device=dev), torch.zeros(700, 8, dtype=i32, device=dev), torch.zeros(1025, dtype=i32, device=dev)
st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g, stream=st):
    for d in (choose.adjust(x, out, settings, tokens=tokens), choose.top(out, ids, lp, None, ws), choose.experts(r, eids, w),
              choose.plan(eids, order, place, offsets, ws)):
        G.eager_run(d, st.cuda_stream)
g.replay()
torch.cuda.synchronize()
had = torch.zeros(2, 9000, device=dev).scatter_(1, tokens.long(), 1.0)
assert torch.allclose(out, x - 0.5 * had, atol=1e-6) and torch.equal(ids, out.topk(3).indices.int())
assert torch.equal(eids, r.topk(8).indices.int()) and int(offsets[-1]) == 5600
assert torch.equal(order.long(), eids.flatten().sort(stable=True).indices)
print("captured ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert "captured ok" in r.stdout, r.stderr[-2000:]
