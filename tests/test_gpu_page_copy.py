"""Pairs of a page copy that name one page twice."""
import numpy as np
import pytest

from tests.gpu_harness import ensure_built, need_gpu
from tests.test_gpu_kv4 import _dev, _executor

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pair,status", [((2, 2), 0), ((4, 4), 2), ((1 << 30, 1 << 30), 2), ((-3, -3), 0), ((-1, 9), 0)])
def test_a_page_onto_itself(pair, status):
    """Nothing to do inside the pool, bad arguments outside it as for any
    other pair; a negative page is a hole."""
    import torch
    from persistent_micro_dispatch_gb300 import kv4
    need_gpu()
    ensure_built()
    was = np.arange(2 * 4 * 64, dtype=np.uint8).reshape(2, 4, 64)
    pool = _dev(was)
    pairs = _dev(np.array([pair, (1, 3)], np.int32))
    _executor(kv4.page_copy(pool, pairs), expect=[status])
    was[:, 3] = was[:, 1]
    assert torch.equal(pool.cpu(), torch.from_numpy(was))
