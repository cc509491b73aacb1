"""Attention over the 4-bit cache when value sizes lie far apart: a key adds
what its weight and its value make together, whatever the other keys, the
other rows and the keys that a row may not see hold."""
import numpy as np
import pytest

from tests import kv4_ref as R
from tests.gpu_harness import ensure_built, need_gpu
from tests.test_gpu_kv4 import RUNNERS, _attend, _attend_case, _close

pytestmark = pytest.mark.gpu
WAYS = ["eager", "executor", "executor_nostage"]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    need_gpu()
    ensure_built()


def _want(q, pool, table, lens, scale):
    """Output and bound of (float64 [B, T, H, D] each). The bound: weights and
    scores as in R.bound (2^-11, 2 (D + 8) 2^-24 reach, 2^-18), relative to
    p @ |v|; 6 * 2^-27 for each key of the largest weight times value scale
    that the row meets in the group (a weight times a scale is held in f16
    steps of 2^-25, where that largest is 2^2 at least: 2^14 over the window's
    2^12; a code is 6 at most); weights below 2^-140 count as zero."""
    B, T, H, D = q.shape
    g = H // pool.shape[1]
    K, V, S = R.unpack(pool)
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        at = np.arange(int(lens[b]))
        page = table[b][at // 32]
        kb, vb, sb = (x[page, :, at % 32] for x in (K, V, S))
        for t in range(T):
            n = int(lens[b]) - T + t + 1
            if n <= 0:
                continue
            for h in range(H):
                k, v, s = (x[:n, h // g] for x in (kb, vb, sb))
                x = k @ q[b, t, h] * scale
                p = np.exp(x - x.max())
                p /= p.sum()
                out[b, t, h] = p @ v
                reach = (np.abs(k) @ np.abs(q[b, t, h])).max() * abs(scale)
                rel = 2.0 ** -11 + 2 * (D + 8) * 2.0 ** -24 * reach + 2.0 ** -18
                tol[b, t, h] = (rel * (p @ np.abs(v)) + n * 6 * 2.0 ** -27 * (p[:, None] * s).max(0)
                                + 2.0 ** -140 * np.abs(v).sum(0))
    return out, tol


def _check(run, q, pool, table, lens, scale):
    want, tol = _want(q, pool, table, lens, scale)
    got = _attend(RUNNERS[run], q, pool, table, lens, scale)
    _close(got, want, tol)
    return got


def _plain_pool(seed, B, H, heads, D, T, lens, scale_byte=127, lo=126):
    """A case whose value scales are lo .. scale_byte, and whose scores stay within a few nats."""
    q, pool, table, lens = _attend_case(seed, B, H, heads, D, T, lens)
    rng = np.random.default_rng(seed + 1)
    pool[:, :, 33 * D:] = rng.integers(lo, scale_byte + 1, pool[:, :, 33 * D:].shape)
    pool[:, :, 32 * D:33 * D] = 123
    q[:] = R.bf16(0.5 + 0.1 * rng.standard_normal(q.shape))
    return q, pool, table, lens


def _key(pool, page, head, key, code=None, scale=None, value=None, value_scale=None):
    """Set all of a key's codes and scale bytes, or its value's."""
    D = pool.shape[2] // 34
    k, v, ks, vs = R.offsets(D, key, np.arange(D))
    for at, x in ((k, code), (v, value)):
        if x is not None:
            pool[page, head, at] = x | x << 4
    for at, x in ((ks, scale), (vs, value_scale)):
        if x is not None:
            pool[page, head, at] = x


@pytest.mark.parametrize("run", WAYS)
@pytest.mark.parametrize("D,H,heads", [(64, 4, 2), (128, 12, 1)])
@pytest.mark.parametrize("up", [10, 14, 23, 60, 100])
def test_light_outlier_at_every_position(run, D, H, heads, up):
    """One key of a hundred has a value 2^up times the others' and a score
    about 70 octaves below them: nothing but for the largest, then all."""
    where = [0, 1, 15, 31, 32, 63, 64, 95, 96, 99]
    q, pool, table, lens = _plain_pool(7, len(where), H, heads, D, 1, [100] * len(where))
    for b, n in enumerate(where):
        for h in range(heads):
            _key(pool, table[b, n // 32], h, n % 32, code=15, scale=128 if D == 64 else 127, value_scale=127 + up)
    _check(run, q, pool, table, lens, 0.125)


@pytest.mark.parametrize("run", WAYS)
@pytest.mark.parametrize("octaves", [20, 36, 60, 110])
def test_outlier_as_heavy_as_it_is_light(run, octaves):
    """A weight 2^-octaves, a value 2^octaves: it adds as much as the rest. A
    page of such keys, first, in the middle and last."""
    D, scale = 64, 0.125
    q, pool, table, lens = _plain_pool(11, 3, 4, 2, D, 1, [130] * 3)
    q[:] = 0.5
    # the other keys' channels cancel: score 0. These: -64 x 0.5 x scale = -4 for each unit of size
    pool[:, :, :16 * D] = 0xA2  # +1, -1
    size = octaves * np.log(2) / 4
    e = int(np.ceil(np.log2(size / 6)))
    code = int(np.abs(R.MAG - size / 2.0 ** e).argmin())
    for b, pg in enumerate((0, 1, 3)):
        for h in range(2):
            for key in range(32):
                _key(pool, table[b, pg], h, key, code=8 + code, scale=127 + e, value_scale=127 + octaves)
    _check(run, q, pool, table, lens, scale)


@pytest.mark.parametrize("run", WAYS)
@pytest.mark.parametrize("T,H,lens", [(2, 2, [4, 33, 64]), (4, 8, [4, 40, 99]), (8, 12, [70, 9, 8]), (32, 2, [32, 64, 100])])
@pytest.mark.parametrize("up", [10, 23, 100])
def test_hidden_outliers(run, T, H, lens, up):
    """The last T - 1 keys, which the first token does not see, hold ever
    larger values: each token weighs what it sees."""
    q, pool, table, lens = _plain_pool(13, len(lens), H, 1, 64, T, lens)
    for b, n in enumerate(lens):
        for k in range(T - 1):
            at = n - T + 1 + k
            _key(pool, table[b, at // 32], 0, at % 32, value_scale=127 + up * (k + 1) // (T - 1))
    got = _check(run, q, pool, table, lens, 0.125)
    assert np.abs(got[0, 0]).max() < 16


@pytest.mark.parametrize("run", WAYS)
def test_hidden_outliers_leave_the_bits(run):
    """The first token's output, bit for bit, with and without a later token's
    value of 2^23 in place of one: neither page takes another path for it."""
    q, pool, table, lens = _plain_pool(17, 1, 2, 1, 64, 2, [3], lo=127)
    first = _check(run, q, pool, table, lens, 0.125)
    _key(pool, table[0, 0], 0, 2, value_scale=150)
    second = _check(run, q, pool, table, lens, 0.125)
    lim = 2.0 ** -8 * np.abs(first[0, 0])  # (another order of roundings: within a step)
    assert (np.abs(first[0, 0] - second[0, 0]) <= lim).all()


@pytest.mark.parametrize("run", WAYS)
@pytest.mark.parametrize("T,H", [(1, 4), (3, 6), (1, 24)])
@pytest.mark.parametrize("spread", [14, 60, 120])
def test_random_scales(run, T, H, spread):
    rng = np.random.default_rng(spread)
    q, pool, table, lens = _attend_case(3, 4, H, 1, 64, T, [97, 64, 200, 9])
    pool[:, :, 33 * 64:] = rng.integers(127 - spread, 127 + spread + 1, pool[:, :, 33 * 64:].shape).clip(0, 252)
    _check(run, q, pool, table, lens, 0.125)


@pytest.mark.parametrize("run", WAYS)
@pytest.mark.parametrize("step", [2, -2, 0.5, -0.5])
def test_scales_that_climb_and_fall(run, step):
    """Every key's value scale is a little above, or below, the one before."""
    q, pool, table, lens = _plain_pool(19, 2, 6, 2, 128, 1, [120, 61])
    for b, n in enumerate(lens):
        for at in range(n):
            byte = int(127 + step * (at - 60))
            for h in range(2):
                _key(pool, table[b, at // 32], h, at % 32, value_scale=byte)
    _check(run, q, pool, table, lens, 0.125)


@pytest.mark.parametrize("run", WAYS)
@pytest.mark.parametrize("up", [14, 40, 100])
def test_one_row_heeds_what_the_next_does_not(run, up):
    """Two query heads of one cache head: the large values' keys take all of
    the first's weight and none of the second's."""
    D = 64
    q, pool, table, lens = _plain_pool(23, 2, 2, 1, D, 1, [100, 400], lo=120)
    for b, n in enumerate(lens):
        for at in range(3, n, 37):
            _key(pool, table[b, at // 32], 0, at % 32, code=7, scale=128, value_scale=127 + up)
    q[:, :, 1] *= -1  # 64 x 12 x 0.5 x 0.125 = 48 nats, up and down
    got = _check(run, q, pool, table, lens, 0.125)
    assert np.abs(got[:, :, 0]).max() > 2.0 ** (up - 4) and (up == 100 or np.abs(got[:, :, 1]).max() < 16)


@pytest.mark.parametrize("run", WAYS)
@pytest.mark.parametrize("n,first", [(100, 1), (100, 32), (100, 40), (5000, 3)])
def test_sink_of_no_value(run, n, first):
    """The first keys take all the weight but 2^-30 or so, and hold zeros
    under a scale byte of zero: the output is what the others add."""
    D = 64
    q, pool, table, lens = _plain_pool(29, 1, 4, 1, D, 1, [n])
    for at in range(first):
        _key(pool, table[0, at // 32], 0, at % 32, code=7, scale=127, value=0, value_scale=0)
    got = _check(run, q, pool, table, lens, 0.125)
    assert 0 < np.abs(got).max() < 1e-3


@pytest.mark.parametrize("run", WAYS)
def test_alone_and_in_a_batch(run):
    """A request's runs are cut elsewhere when others stand beside it: the
    same output to within the bound, with outliers all along."""
    lens = [700, 5, 2100, 33, 0, 900]
    q, pool, table, lens = _plain_pool(31, len(lens), 8, 2, 64, 1, lens)
    for at in range(11, 2100, 97):
        for h in range(2):
            _key(pool, table[2, at // 32], h, at % 32, code=15, scale=128, value_scale=150)
    got = _check(run, q, pool, table, lens, 0.125)
    one = _check(run, q[2:3], pool, table[2:3], lens[2:3], 0.125)
    want, tol = _want(q[2:3], pool, table[2:3], lens[2:3], 0.125)
    assert (np.abs(one - got[2:3]) <= 2 * tol + 2.0 ** -7 * np.abs(want)).all()


@pytest.mark.parametrize("run", WAYS)
def test_nan_groups_among_far_scales(run):
    """A value scale of 255 is NaN for the rows that see it, in its group
    alone, in a page whose other scales lie far apart too."""
    D, T = 64, 3
    q, pool, table, lens = _plain_pool(37, 2, 4, 1, D, T, [60, 90], lo=80)
    clean = pool.copy()
    # request 0: group 1 of key 20; request 1: group 0 of the last key, which the last token alone sees
    for page, key, c in ((table[0, 0], 20, 32), (table[1, 2], 89 - 64, 0)):
        vs = R.offsets(D, key, c)[3]
        pool[page, 0, vs], clean[page, 0, vs] = 255, 127
    want, tol = _want(q, clean, table, lens, 0.125)
    nan = np.zeros(q.shape, bool)
    nan[0, :, :, 32:] = True
    nan[1, 2, :, :32] = True
    got = _attend(RUNNERS[run], q, pool, table, lens, 0.125)
    assert np.array_equal(np.isnan(got), nan)
    _close(got[~nan], want[~nan], tol[~nan])


@pytest.mark.parametrize("run", WAYS)
@pytest.mark.parametrize("T,H", [(1, 4), (2, 24)])
@pytest.mark.parametrize("up", [60, 66, 100, 112, 118])
@pytest.mark.parametrize("scale", [1.0, 0.125, 0.001])
def test_large_keys_under_small_queries(run, T, H, up, scale):
    """Keys 2^up times their common size, queries 2^-up times theirs: scores
    of order one, as they are without."""
    D = 64
    q, pool, table, lens = _attend_case(41, 3, H, 1, D, T, [70, 33, 1 + T])
    was = pool[:, :, 32 * D:33 * D].astype(int)
    pool[:, :, 32 * D:33 * D] = (was + up).clip(0, 252)
    q = R.bf16(q * 2.0 ** -up / scale * 0.125)
    want, tol = _want(q, pool, table, lens, scale)
    assert 0.01 < np.abs(want).max() < 100
    _check(run, q, pool, table, lens, scale)


@pytest.mark.parametrize("run", WAYS)
@pytest.mark.parametrize("byte", [0, 1, 9])
def test_small_keys_under_large_queries(run, byte):
    """Key scales from 2^-127 on: a code of them is not zero."""
    D = 64
    q, pool, table, lens = _attend_case(43, 2, 4, 2, D, 1, [70, 33])
    pool[:, :, 32 * D:33 * D] = byte
    q = R.bf16(q * 2.0 ** 120)
    K, _, _ = R.unpack(pool)
    scale = 2.0 ** (7 - byte)
    x = K[table[0, 0], 0] @ q[0, 0, 0] * scale
    assert 2 < np.abs(x).max() < 60
    _check(run, q, pool, table, lens, scale)


@pytest.mark.parametrize("run", WAYS)
def test_key_sizes_apart(run):
    """One group of every key is 2^90 times the others, under query channels
    that are small there; some keys in pages of common ones."""
    D = 64
    q, pool, table, lens = _attend_case(47, 2, 4, 1, D, 1, [100, 300])
    q[..., 32:] *= 2.0 ** -90
    q = R.bf16(q)
    for b, n in enumerate(lens):
        for at in range(5, n, 7):
            ks = R.offsets(D, at % 32, 32)[2]
            pool[table[b, at // 32], 0, ks] += 90
    _check(run, q, pool, table, lens, 0.125)


@pytest.mark.parametrize("run", WAYS)
@pytest.mark.parametrize("code", [0, 1, 7, 9, 15])
def test_key_scale_of_nan_beside_any_code(run, code):
    """A key scale of 255 is NaN whatever the codes are, for the rows that see
    the key; behind the last key it is nothing."""
    D, T = 64, 2
    q, pool, table, lens = _attend_case(53, 3, 4, 2, D, T, [40, 50, 70])
    clean = pool.copy()
    for page, key, h in ((table[0, 1], 39 - 32, 0), (table[1, 0], 4, 1), (table[2, 2], 70 - 64, 0)):
        k, _, ks, _ = R.offsets(D, key, np.arange(32))
        pool[page, h, k] = code | code << 4
        pool[page, h, ks] = 255
        clean[page, h, k], clean[page, h, ks] = 0, 127
    want, tol = _want(q, clean, table, lens, 0.125)
    nan = np.zeros(q.shape, bool)
    nan[0, 1, :2] = True  # the last key: the last token alone sees it
    nan[1, :, 2:] = True
    got = _attend(RUNNERS[run], q, pool, table, lens, 0.125)
    assert np.array_equal(np.isnan(got), nan)
    _close(got[~nan], want[~nan], tol[~nan])


def test_far_scales_after_a_handoff():
    """The slow way of a page in an executor that was linked anew with a
    module of user ops."""
    import torch
    from persistent_micro_dispatch_gb300 import gpuos as G, kv4
    from tests.test_gpu_kv4 import _dev, _f64
    from tests.test_gpu_protocol import _NEG_SRC
    from workloads.device import warm_torch
    rng = np.random.default_rng(61)
    q, pool, table, lens = _attend_case(3, 4, 12, 1, 128, 2, [97, 64, 2000, 9])
    pool[:, :, 33 * 128:] = rng.integers(67, 188, pool[:, :, 33 * 128:].shape)
    t = [_dev(q, torch.bfloat16), _dev(pool), _dev(table), _dev(lens)]
    out, ws = torch.zeros_like(t[0]), kv4.new_workspace()
    img = G.compile_op(_NEG_SRC, "neg.cu")
    warm_torch()
    torch.cuda.synchronize()
    ex = G.Executor()
    try:
        ex.register_op(90, img, "op_neg_ptr")
        assert ex.stats()["handoffs"] == 1
        ex.submit(kv4.sdpa(*t, out, ws, 0.1))
        ex.sync(timeout_ms=30_000)
    finally:
        assert ex.shutdown() == G.OK
    want, tol = _want(q, pool, table, lens, 0.1)
    _close(_f64(out), want, tol)


@pytest.mark.parametrize("run", WAYS)
def test_pages_outside_among_far_scales(run):
    """A page that is not in the pool is left out, between pages that go the
    slow way; one request has none in the pool."""
    q, pool, table, lens = _plain_pool(67, 2, 4, 1, 64, 1, [200, 64], lo=60)
    table[0, 2], table[0, 4], table[1, :2] = -7, pool.shape[0], 1 << 20
    got = _attend(RUNNERS[run], q, pool, table, lens, 0.125, **({"expect": [2]} if run != "eager" else {}))
    inside = table.copy()
    inside[0, :5] = table[0, [0, 1, 3, 5, 6]]  # the last page has 8 keys, and stays last
    want, tol = _want(q[:1], pool, inside[:1], np.array([200 - 64]), 0.125)
    _close(got[:1], want, tol)
    assert np.isnan(got[1]).all()
