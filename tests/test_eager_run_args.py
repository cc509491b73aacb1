"""What eager_run passes to the library, with the library call replaced: the
address of as many 128-byte records as it says there are (CPU)."""
import ctypes

import numpy as np
import pytest

from persistent_micro_dispatch_gb300 import gpuos as G


@pytest.fixture
def seen(monkeypatch):
    calls = []

    class Stub:
        @staticmethod
        def gpuos_eager_run(ptr, count, stage, stream):
            if isinstance(ptr, bytes):
                assert len(ptr) == 128 * count, "fewer bytes than records"
                raw = ptr
            else:
                raw = ctypes.string_at(ptr, 128 * count)
            calls.append((np.frombuffer(raw, dtype=G.DESC_DTYPE), stream))
            return G.OK

    monkeypatch.setattr(G, "lib", lambda: Stub)
    return calls


def _descs(n):
    d = G.make_descs(n)
    d["op_id"] = np.arange(n) % 8
    d["a"] = 4096 * (1 + np.arange(n))
    return d


FORMS = {
    "array": lambda d: (d, len(d)),
    "record": lambda d: (d[0], 1),
    "0-d array": lambda d: (d[:1].reshape(()), 1),
    "list of records": lambda d: (list(d), len(d)),
    "2-d array": lambda d: (d.reshape(1, -1), len(d)),
    "every other": lambda d: (d[::2], -(-len(d) // 2)),
    "recarray": lambda d: (d.view(np.recarray), len(d)),
    "equal dtype": lambda d: (d.view(np.dtype(G.DESC_DTYPE.descr)), len(d)),
}


@pytest.mark.parametrize("n", [1, 3, 16, 17, 40])
@pytest.mark.parametrize("form", sorted(FORMS))
def test_every_record_and_no_more(seen, form, n):
    d = _descs(n)
    arg, count = FORMS[form](d)
    want = d[::2] if form == "every other" else d[:count]
    G.eager_run(arg, 0x77)
    (got, stream), = seen
    assert stream == 0x77 and len(got) == count
    assert got.tobytes() == np.ascontiguousarray(want).tobytes()


def test_no_records(seen):
    G.eager_run(G.make_descs(0))
    G.eager_run([])
    assert [len(got) for got, _ in seen] == [0, 0]


@pytest.mark.parametrize("bad", [None, "descs", (1, 2, 3), [object()]])
def test_what_is_no_record_is_refused(seen, bad):
    with pytest.raises((TypeError, ValueError)):
        G.eager_run(bad)
    assert not seen
