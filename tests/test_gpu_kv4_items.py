"""Launched attention where every warp has many short items in turn: an item's
pages take the place of the one before it in shared memory."""
import numpy as np
import pytest

from tests import kv4_ref as R
from tests.gpu_harness import ensure_built, need_gpu
from tests.test_gpu_kv4 import _attend_case, _close, _dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,H,heads,longest", [(64, 8, 8, 70), (128, 8, 8, 40), (128, 20, 1, 33)])
def test_many_short_items_a_warp(D, H, heads, longest):
    """Thousands of items of one to three pages, replayed: the same bits each
    time, and right (a sample of the requests against the reference)."""
    import torch
    from persistent_micro_dispatch_gb300 import gpuos as G, kv4
    need_gpu()
    ensure_built()
    B = 2500
    rng = np.random.default_rng(longest)
    lens = rng.integers(0, longest + 1, B)
    q, pool, table, lens = _attend_case(longest, B, H, heads, D, 1, list(lens), pool=R.random_pool(rng, 64, heads, D))
    table = np.where(table >= 0, table % 64, table).astype(np.int32)  # (the requests share 64 pages)
    t = [_dev(q, torch.bfloat16), _dev(pool), _dev(table), _dev(lens)]
    ws, out = kv4.new_workspace(), torch.zeros(B, 1, H, D, dtype=torch.bfloat16, device="cuda")
    d = kv4.sdpa(*t, out, ws, 0.1)
    st = torch.cuda.current_stream().cuda_stream
    G.eager_run(d, st)
    first = out.clone()
    for _ in range(20):
        out.zero_()
        G.eager_run(d, st)
        assert torch.equal(out, first)
    pick = rng.permutation(B)[:60]
    want, tol = R.attend(q[pick], pool, table[pick], lens[pick], 0.1)
    _close(first.double().cpu().numpy()[pick], want, tol)
