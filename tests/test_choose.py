"""What a decode step chooses, without a GPU: the tiling rules and refusals of
its ops, the binding's checks, and the reference's own pins."""
import numpy as np
import pytest
import torch

from tests import choose_ref as R


@pytest.fixture(scope="module")
def G():
    from persistent_micro_dispatch_gb300 import build
    build.build()
    from persistent_micro_dispatch_gb300 import gpuos
    gpuos.lib()
    return gpuos


def _desc(G, op, dims, dtype=1, **kw):
    d = G.make_descs(1)
    d["op_id"], d["dtype"] = G.OP[op], dtype
    d["dims"] = list(dims) + [0] * (6 - len(dims))
    for f in ("a", "b", "out", "aux0", "aux1", "aux2"):
        d[f] = kw.get(f, 0x1000)
    return d


GOOD = {
    "logits_adjust": (2, 1000, 1000, 1000, 50, 1 | 3 << 16),
    "logits_top": (2, 1000, 1000, 20),
    "expert_route": (9, 64, 64, 8, 8 | 4 << 16, 7),
    "expert_count": (9000, 64),
    "expert_place": (9000, 64),
}


def test_tiles(G):
    n = lambda *a, **k: G.op_ntiles(_desc(G, *a, **k))  # noqa: E731
    # 4,096 tokens a tile, of a row that may begin seven elements behind its first vector
    assert n("logits_adjust", (2, 4089, 4089, 4089, 0, 0)) == 2
    assert n("logits_adjust", (2, 4090, 4090, 4090, 0, 0)) == 4
    assert n("logits_adjust", (3, 128000, 128000, 128000, 0, 0), dtype=0) == 3 * 32
    assert n("logits_adjust", (0, 5, 5, 5)) == n("logits_adjust", (5, 0, 0, 0)) == 1
    # 1,024 tokens a tile, and 1,536 tiles at most while rows are cut
    assert n("logits_top", (1, 1000, 1000, 1)) == 1
    assert n("logits_top", (1, 1018, 1018, 1)) == 2
    assert n("logits_top", (1, 128000, 128000, 20)) == 126
    assert n("logits_top", (64, 128000, 128000, 20)) == 64 * 24
    assert n("logits_top", (65, 128000, 128000, 20)) == 65 * 23
    assert n("logits_top", (769, 128000, 128000, 20)) == 769
    assert n("logits_top", (5000, 128000, 128000, 20)) == 5000
    assert n("logits_top", (0, 0, 0, 0)) == 1
    route = lambda N: n("expert_route", (N, 64, 64, 8, 1 | 1 << 16, 0))  # noqa: E731
    assert [route(N) for N in (1, 17, 1536, 1537, 4608, 12288, 12289, 32768)] == [1, 17, 1536, 769, 1536, 1536, 1537, 4096]
    assert n("expert_route", (0, 0, 0, 0)) == 1
    for op in ("expert_count", "expert_place"):
        assert n(op, (4096, 64)) == 1 and n(op, (4097, 64)) == 3 and n(op, (1 << 20, 64)) == 96 and n(op, (0, 64)) == 1


@pytest.mark.parametrize("op,at,value", [
    *[("logits_adjust", i, v) for i, v in ((1, 0x7FFFFF00), (2, 999), (3, 999), (4, (1 << 28) + 1), (0, 1 << 31), (5, 1 | 1025 << 16))],
    *[("logits_top", i, v) for i, v in ((1, 0), (1, 19), (1, 0x7FFFFF00), (2, 999), (3, 0), (3, 65))],
    *[("expert_route", i, v) for i, v in (
        (0, 0x7FFFFF01), (1, 0), (1, 63), (1, 1032), (2, 63), (3, 0), (3, 33), (4, 8), (4, 4 << 16), (4, 7 | 4 << 16), (4, 8 | 9 << 16),
        (4, 64 | 64 << 16), (4, 16 | 1 << 16), (5, 8))],
    *[(op, i, v) for op in ("expert_count", "expert_place") for i, v in ((0, 0x7FFFFF01), (1, 0), (1, 1025))],
])
def test_size_refusals(G, op, at, value):
    dims = list(GOOD[op]) + [0] * (6 - len(GOOD[op]))
    G.op_ntiles(_desc(G, op, dims))
    dims[at] = value
    with pytest.raises(G.GpuosError) as e:
        G.op_ntiles(_desc(G, op, dims))
    assert e.value.code == G.EINVAL


@pytest.mark.parametrize("op,field,value", [
    *[("logits_adjust", f, v) for f, v in (("a", 0), ("a", 0x1001), ("out", 0), ("out", 0x1003), ("b", 0), ("b", 0x1002), ("aux0", 0),
                                           ("aux0", 0x1008), ("aux1", 0), ("aux1", 0x1002), ("aux2", 0), ("aux2", 0x1004))],
    *[("logits_top", f, v) for f, v in (("a", 0), ("a", 0x1001), ("out", 0), ("out", 0x1002), ("aux0", 0), ("aux0", 0x1001), ("aux1", 0x1002),
                                        ("aux2", 0), ("aux2", 0x1008))],
    *[("expert_route", f, v) for f, v in (("a", 0), ("b", 0x1002), ("out", 0), ("out", 0x1001), ("aux0", 0), ("aux0", 0x1002), ("aux1", 0x1001))],
    *[("expert_place", f, v) for f, v in (("a", 0), ("a", 0x1002), ("b", 0), ("b", 0x1002), ("out", 0), ("out", 0x1001), ("aux0", 0),
                                          ("aux0", 0x1002), ("aux2", 0), ("aux2", 0x1008))],
    *[("expert_count", f, v) for f, v in (("a", 0), ("a", 0x1002), ("aux2", 0), ("aux2", 0x1008))],
    *[(op, "dtype", 2) for op in ("logits_adjust", "logits_top", "expert_route")],
])
def test_pointer_and_type_refusals(G, op, field, value):
    kw = {field: value} if field != "dtype" else {}
    with pytest.raises(G.GpuosError) as e:
        G.op_ntiles(_desc(G, op, GOOD[op], **kw, **({"dtype": value} if field == "dtype" else {})))
    assert e.value.code == G.EINVAL


def test_the_reserved_id_is_no_op(G):
    assert 20 not in G.OP.values()
    d = G.make_descs(1)
    d["op_id"] = 20
    with pytest.raises(G.GpuosError) as e:
        G.op_ntiles(d)
    assert e.value.code == G.EINVAL
    assert G.lib().gpuos_eager_run(d.ctypes.data, 1, 0, None) == G.EINVAL


def test_in_place_needs_rows_alike(G):
    G.op_ntiles(_desc(G, "logits_adjust", (2, 10, 12, 12, 0, 0)))
    with pytest.raises(G.GpuosError):
        G.op_ntiles(_desc(G, "logits_adjust", (2, 10, 12, 13, 0, 0)))
    G.op_ntiles(_desc(G, "logits_adjust", (2, 10, 12, 13, 0, 0), out=0x2000))


def test_constants_of_the_header(G):
    import os
    import re
    from persistent_micro_dispatch_gb300 import choose
    text = open(os.path.join(os.path.dirname(G.HERE), "include", "gpuos.h")).read()
    value = lambda n: eval(re.search(rf"#define {n} (.*?)(?:/\*|\n)", text).group(1).replace("u", ""))  # noqa: E731
    assert choose.WORKSPACE_BYTES == value("GPUOS_CHOOSE_WORKSPACE") and choose.COUNTER_BYTES == value("GPUOS_CHOOSE_COUNTERS")
    assert choose.PLAN_ONE == value("GPUOS_PLAN_ONE")
    assert [value(f"GPUOS_ROUTE_{n}") for n in ("SIGMOID", "TOP2", "NORM")] == [1, 2, 4]
    body = re.search(r"typedef struct gpuos_logits_request \{(.*?)\}", text, re.S).group(1)
    assert re.findall(r"(\w+)(?=[,;])", re.sub(r"/\*.*?\*/", "", body)) == list(choose._FIELDS)


def test_settings_by_name():
    from persistent_micro_dispatch_gb300 import choose
    s = choose.new_settings(3, device="cpu")
    f = choose.fields(s)
    f["temperature"][1] = 0.5
    f["length"][2] = 7
    r = s.numpy().view(R.SETTING)[:, 0]
    assert r["temperature"].tolist() == [1.0, 0.5, 1.0] and r["length"].tolist() == [0, 0, 7] and r["mask"].tolist() == [-1] * 3
    assert r["repetition"].tolist() == [1.0] * 3 and not r["presence"].any() and not r["biases"].any()
    with pytest.raises(ValueError):
        choose.fields(s[:, :7])


def test_binding_refuses_before_any_launch(G):
    """Host tensors (the rest is in the GPU tests)."""
    from persistent_micro_dispatch_gb300 import choose
    x, i, w = torch.zeros(3, 64), torch.zeros(3, 8, dtype=torch.int32), torch.zeros(3, 8)
    ws = choose.new_workspace("cpu")
    with pytest.raises(ValueError, match="CUDA"):
        choose.adjust(x, x, choose.new_settings(3, "cpu"))
    with pytest.raises(ValueError, match="CUDA"):
        choose.top(x, i, w, None, ws)
    with pytest.raises(ValueError, match="CUDA"):
        choose.experts(x, i, w)
    with pytest.raises(ValueError, match="CUDA"):
        choose.plan(i, i.view(-1), i, torch.zeros(65, dtype=torch.int32), ws)
    with pytest.raises(ValueError):
        choose.reset_workspace(ws[1:])


# ---- the reference's own pins


def test_reference_adjusts_by_the_definition():
    s = np.zeros(1, R.SETTING)
    s[0] = (2.0, 0.5, 0.25, 0.5, 1, 4, 0, 2)
    tokens = np.array([[3, 1, 1, 2, 0]], np.int32)  # 3 in the prompt, 1 twice and 2 once after it; 0 is not there yet
    bias = np.zeros((1, 2), R.BIAS)
    bias[0] = [(4, 9.0), (4, 1.0)]
    mask = np.array([[0b011111]], np.uint32)
    want, _ = R.adjust(np.array([[1.0, 4.0, -1.0, 6.0, 2.0, 5.0]]), s, tokens, bias, mask, True)
    assert want.tolist() == [[2.0, (4 / 2 - 1.0) * 2, (-2 - 0.75) * 2, 6.0, 6.0, -np.inf]]


def test_reference_ranks_ties_by_number():
    ids, lp, lse, _, _ = R.top(np.array([[1.0, 3.0, np.nan, 3.0, -np.inf]]), 5)
    assert ids.tolist() == [[1, 3, 0, 2, 4]] and lp[0, 3] == lp[0, 4] == -np.inf
    assert np.isclose(lse[0], np.log(2 * np.exp(3) + np.e)) and np.isclose(np.exp(lp[0]).sum(), 1)
    # the groups' sums of exp(x): 1 + e, e + e^0.5, e^2
    ids, w = R.experts(np.array([[0.0, 1.0, 1.0, 0.5, -np.inf, 2.0]]), 2, False, None, 3, 2, True, True, 2.0)
    assert ids.tolist() == [[5, 2]] and np.allclose(w, [[2 * np.e / (np.e + 1), 2 / (np.e + 1)]])
    ids, w = R.experts(np.array([[0.0, 1.0, 1.0, 0.5, -np.inf, 2.0]]), 2, False, None, 3, 1, False, False, 1.0)
    assert ids.tolist() == [[5, 4]] and w[0, 1] == 0


def test_reference_plans_in_order():
    order, place, offsets = R.plan(np.array([[2, 0], [-1, 2], [0, 3]], np.int32), 3)
    assert order.tolist() == [1, 4, 0, 3, -1, -1] and place.tolist() == [[2, 0], [-1, 3], [1, -1]] and offsets.tolist() == [0, 2, 2, 4]
