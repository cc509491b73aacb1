"""The 4-bit paged cache without a GPU: the tiling rules and refusals of its
ops, the binding's checks, and the reference's own pins."""
import numpy as np
import pytest
import torch

from tests import kv4_ref as R


@pytest.fixture(scope="module")
def G():
    from persistent_micro_dispatch_gb300 import build
    build.build()
    from persistent_micro_dispatch_gb300 import gpuos
    gpuos.lib()
    return gpuos


def _desc(G, op, dims, dtype=1, fparam=1.0, **kw):
    d = G.make_descs(1)
    d["op_id"], d["dtype"] = G.OP[op], dtype
    d["dims"] = list(dims) + [0] * (6 - len(dims))
    d["fparam"][0, 0] = fparam
    for f in ("a", "b", "out", "aux0", "aux1", "aux2"):
        d[f] = kw.get(f, 0x1000)
    return d


def _sdpa(G, B=2, H=8, Hkv=2, D=128, T=1, P=4, npages=9, **kw):
    return _desc(G, "kv4_sdpa", (B, H | Hkv << 16, D | T << 16, P, npages), **kw)


def test_tiles(G):
    n = lambda d: G.op_ntiles(d)  # noqa: E731
    # rows: eight tokens of a head, up to 64 once that makes more than 8192 tiles
    assert n(_desc(G, "kv4_write", (1, 1, 128, 1))) == 1
    assert n(_desc(G, "kv4_write", (65, 8, 128, 99))) == 9 * 8
    assert n(_desc(G, "kv4_read", (8192, 8, 64, 999), dtype=0)) == 8192
    assert n(_desc(G, "kv4_read", (8193, 8, 64, 999), dtype=0)) == -(-8193 // 16) * 8
    assert n(_desc(G, "kv4_read", (1 << 20, 8, 64, 1 << 20))) == (1 << 20) // 64 * 8
    assert n(_desc(G, "kv4_write", (0, 0, 0, 0), a=0, b=0, out=0, aux0=0)) == 1
    # attention: the table's pages and six by (request, head, row tile), until 1536
    assert n(_sdpa(G)) == 2 * 2 * (4 + 6)
    assert n(_sdpa(G, H=16, T=2)) == 2 * 2 * (4 + 6) * 2  # 16 rows a head: two row tiles
    assert n(_sdpa(G, B=64, Hkv=8, P=512)) == 1536
    assert n(_sdpa(G, B=0)) == 1
    # pages: 16 KB a tile
    assert n(_desc(G, "page_copy", (3, 1024, 9, 2))) == 6
    assert n(_desc(G, "page_copy", (3, 1025, 9, 2))) == 12
    assert n(_desc(G, "page_copy", (0, 0, 0, 0), a=0, aux0=0)) == 1


@pytest.mark.parametrize("bad", [
    dict(D=96), dict(D=0), dict(D=256), dict(T=0), dict(T=33), dict(H=7), dict(H=0), dict(Hkv=0), dict(P=0),
    dict(P=(1 << 26) + 1), dict(npages=0), dict(npages=(1 << 26) + 1), dict(dtype=0), dict(a=0), dict(b=0), dict(out=0),
    dict(aux0=0), dict(aux1=0), dict(aux2=0), dict(a=0x1008), dict(b=0x1004), dict(out=0x1002), dict(aux2=0x1008),
    dict(aux0=0x1002), dict(aux1=0x1001), dict(B=0xFFFFFFFF, P=1 << 26), dict(B=1 << 16, Hkv=16, H=16, P=4096)])
def test_sdpa_refusals(G, bad):
    with pytest.raises(G.GpuosError) as e:
        G.op_ntiles(_sdpa(G, **bad))
    assert e.value.code == G.EINVAL


@pytest.mark.parametrize("op", ["kv4_write", "kv4_read"])
@pytest.mark.parametrize("bad", [
    dict(dims=(1, 0, 128, 1)), dict(dims=(1, 65536, 128, 1)), dict(dims=(1, 1, 100, 1)), dict(dims=(1, 1, 128, 0)),
    dict(dims=(1, 1, 128, (1 << 26) + 1)), dict(dims=(1 << 31, 1, 128, 1)), dict(dtype=2), dict(a=0), dict(out=0), dict(aux0=0), dict(aux0=0x1002),
    dict(a=0x1004), dict(out=0x1008), dict(second=0), dict(second=0x1008)])
def test_row_refusals(G, op, bad):
    bad = dict(bad)
    if "second" in bad:
        bad["b" if op == "kv4_write" else "aux1"] = bad.pop("second")
    with pytest.raises(G.GpuosError) as e:
        G.op_ntiles(_desc(G, op, bad.pop("dims", (1, 1, 128, 1)), **bad))
    assert e.value.code == G.EINVAL


@pytest.mark.parametrize("bad", [
    dict(dims=(1, 0, 4, 1)), dict(dims=(1, 4, 0, 1)), dict(dims=(1, 4, 1 << 31, 1)), dict(dims=(1, 4, 4, 0)), dict(a=0),
    dict(aux0=0), dict(a=0x1008), dict(aux0=0x1004), dict(dims=(1 << 20, 4, 4, 1 << 12)),
    dict(dims=(0xFFFFFFFF, 0xFFFFFFFF, 4, 0xFFFFFFFF))])
def test_page_copy_refusals(G, bad):
    bad = dict(bad)
    with pytest.raises(G.GpuosError) as e:
        G.op_ntiles(_desc(G, "page_copy", bad.pop("dims", (1, 4, 4, 1)), **bad))
    assert e.value.code == G.EINVAL


def test_pool_bytes(G):
    L = G.lib()
    assert L.gpuos_kv4_pool_bytes(3, 8, 128) == 3 * 8 * 4352
    assert L.gpuos_kv4_pool_bytes(1 << 26, 65535, 128) == (1 << 26) * 65535 * 4352
    for bad in ((0, 1, 64), (1, 0, 64), (1, 1, 32), ((1 << 26) + 1, 1, 64), (1, 65536, 64)):
        assert L.gpuos_kv4_pool_bytes(*bad) == 0


def test_binding_refuses_before_any_launch(G):
    """Host tensors and sizes that no pool has (the rest is in the GPU tests)."""
    from persistent_micro_dispatch_gb300 import kv4
    pool = torch.zeros(4, 2, 34 * 64, dtype=torch.uint8)
    k = torch.zeros(3, 2, 64)
    s = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kv4.write(k, k, s, pool)
    with pytest.raises(ValueError, match="CUDA"):
        kv4.page_copy(pool, s.view(1, 3))
    with pytest.raises(ValueError):
        kv4.new_pool(4, 2, 96, device="cpu")
    assert kv4.new_pool(4, 2, 64, device="cpu").shape == (4, 2, 34 * 64)
    assert kv4.WORKSPACE_BYTES == 32 << 20 and kv4.PAGE == 32


@pytest.mark.parametrize("D", [64, 128])
def test_page_layout_is_a_bijection(D):
    key, c = np.meshgrid(np.arange(32), np.arange(D), indexing="ij")
    k, v, ks, vs = R.offsets(D, key, c)
    seen = np.zeros(34 * D, int)
    for at in (k[:, ::2], v[:, ::2], ks[:, ::32], vs[:, ::32]):
        np.add.at(seen, at.ravel(), 1)
    assert (seen == 1).all()
    assert (k[:, ::2] == k[:, 1::2]).all() and (v[:, ::2] == v[:, 1::2]).all()


def test_reference_quantises_by_the_definition():
    x = np.zeros((1, 32))
    x[0, :8] = [6.0, 5.0, 2.5, 0.25, 0.75, -0.0, -3.5, 1.25]
    code, byte = R.quantise(x)
    assert byte[0, 0] == 127
    assert code[0, :8].tolist() == [7, 6, 4, 0, 2, 8, 14, 2]  # ties to the even code
    for top, want in ((6.0, 127), (6.5, 128), (3.0, 126), (1e-45, 0), (0.0, 0), (3e38, 252), (np.inf, 255), (np.nan, 255)):
        assert R.quantise(np.full((1, 32), top))[1][0, 0] == want, top
    assert np.isnan(R.values(*R.quantise(np.full((1, 32), np.nan)))).all()
