"""Descriptors of the 4-bit paged key/value cache's ops from PyTorch tensors.

Argument checks and marshalling only, as in the ctypes binding: each function
returns one ``gpuos_desc`` record (an array of one) for ``Executor.submit``,
``Executor.submit_batch`` (joined with ``numpy.concatenate``) or
``gpuos.eager_run``; the ops run in the library's CUDA kernels
(include/gpuos.h, GPUOS_OP_KV4_WRITE and the ops after it, has the pool's
format). The tensors must stay alive until the descriptor has completed, and a
descriptor may be submitted again while they do. GPUOS page, §3 Q2, operator
library, has the dense cache update and attention that these stand beside.

    pool = kv4.new_pool(npages, Hkv, D)
    ws = kv4.new_workspace()
    stream = torch.cuda.current_stream().cuda_stream
    gpuos.eager_run(kv4.write(k, v, slots, pool), stream)
    gpuos.eager_run(kv4.sdpa(q, pool, table, lens, out, ws, D ** -0.5), stream)

Nothing here reads device memory. Slots, page tables, lengths and pairs that
point outside the pool are found by the kernels: such an entry is skipped
(attention: the page counts as no keys; a request whose length does not fit
its table row keeps its output rows as they were), and the executor reports
status 2 (bad arguments) for the descriptor.
"""
from __future__ import annotations

import struct

import numpy as np
import torch

from . import gpuos as G

PAGE = 32
WORKSPACE_BYTES = 32 << 20
MAX_QUERY_TOKENS = 32

_DESC = struct.Struct("<HBBI2Q6Q6I2f3Q")
assert _DESC.size == 128
_DTYPE = {torch.float32: G.F32, torch.bfloat16: G.BF16}


def new_pool(npages: int, heads: int, head_dim: int, device="cuda") -> torch.Tensor:
    """A zeroed pool uint8 [npages, heads, 34 * head_dim]."""
    if G.lib().gpuos_kv4_pool_bytes(npages, heads, head_dim) == 0:
        raise ValueError(f"no such pool: {npages} pages, {heads} heads of {head_dim} (64 or 128)")
    return torch.zeros(npages, heads, 34 * head_dim, dtype=torch.uint8, device=device)


def new_workspace(device="cuda") -> torch.Tensor:
    """The attention's workspace, for one descriptor at a time."""
    return torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device=device)


def _check(what: str, ok: bool) -> None:
    if not ok:
        raise ValueError(what)


def _tensor(name: str, t: torch.Tensor, dtypes, ndim: int, like: torch.Tensor) -> int:
    """Device pointer of a contiguous tensor on `like`'s device."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, wanted {' or '.join(str(d) for d in dtypes)}")
    if t.ndim != ndim:
        raise ValueError(f"{name}: {t.ndim} dimensions, wanted {ndim}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    if t.device != like.device or t.device.type != "cuda":
        raise ValueError(f"{name}: on {t.device}, wanted the pool's CUDA device")
    return t.data_ptr()


def _pool(pool: torch.Tensor):
    p = _tensor("pool", pool, (torch.uint8,), 3, pool)
    npages, heads, nbytes = pool.shape
    _check(f"pool: {nbytes} bytes a head and page, wanted 34 * 64 or 34 * 128", nbytes in (34 * 64, 34 * 128))
    _check("pool: 1 to 2^26 pages and 1 to 65535 heads", 1 <= npages <= 1 << 26 and 1 <= heads <= 65535)
    _check("pool: not 16-byte aligned", p % 16 == 0)
    return p, npages, heads, nbytes // 34


def _desc(op: str, dtype: int, a=0, b=0, out=0, aux0=0, aux1=0, aux2=0, dims=(), fparam=0.0) -> np.ndarray:
    dims = tuple(dims) + (0,) * (6 - len(dims))
    raw = bytearray(_DESC.pack(G.OP[op], dtype, 0, 0, 0, 0, a, b, out, aux0, aux1, aux2, *dims, fparam, 0.0, 0, 0, 0))
    return np.frombuffer(raw, dtype=G.DESC_DTYPE)


def _rows(op: str, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, pool: torch.Tensor) -> np.ndarray:
    pp, npages, heads, D = _pool(pool)
    kp = _tensor("k", k, _DTYPE, 3, pool)
    vp = _tensor("v", v, (k.dtype,), 3, pool)
    sp = _tensor("slots", slots, (torch.int32,), 1, pool)
    n = slots.shape[0]
    _check(f"k, v: {tuple(k.shape)} and {tuple(v.shape)}, wanted {(n, heads, D)}", k.shape == v.shape == (n, heads, D))
    _check("k, v: not 16-byte aligned", kp % 16 == 0 and vp % 16 == 0)
    if op == "kv4_write":
        return _desc(op, _DTYPE[k.dtype], a=kp, b=vp, out=pp, aux0=sp, dims=(n, heads, D, npages))
    return _desc(op, _DTYPE[k.dtype], a=pp, out=kp, aux0=sp, aux1=vp, dims=(n, heads, D, npages))


def write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, pool: torch.Tensor) -> np.ndarray:
    """Quantise rows k, v [N, heads, D] (float32 or bfloat16) into the slots
    int32 [N] (page * 32 + key; negative: skipped; distinct) of the pool."""
    return _rows("kv4_write", k, v, slots, pool)


def read(pool: torch.Tensor, slots: torch.Tensor, k: torch.Tensor, v: torch.Tensor) -> np.ndarray:
    """The rows held in the slots into k, v [N, heads, D] (float32 or
    bfloat16, both exact); zeros for a negative slot."""
    return _rows("kv4_read", k, v, slots, pool)


def sdpa(q: torch.Tensor, pool: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, out: torch.Tensor,
         workspace: torch.Tensor, scale: float) -> np.ndarray:
    """Attention of q [B, T, H, D] (bfloat16, T <= 32 tokens a request, the
    last T of its lens[b]) over the pages table[b] (int32 [B, P]) into out:
    token t sees keys 0 .. lens[b] - T + t; zeros where that is none. Query
    head h reads cache head h // (H / heads). Descriptors that share a
    workspace must run one after another."""
    pp, npages, heads, D = _pool(pool)
    qp = _tensor("q", q, (torch.bfloat16,), 4, pool)
    op = _tensor("out", out, (torch.bfloat16,), 4, pool)
    tp = _tensor("table", table, (torch.int32,), 2, pool)
    lp = _tensor("lens", lens, (torch.int32,), 1, pool)
    wp = _tensor("workspace", workspace, (torch.uint8,), 1, pool)
    B, T, H, d = q.shape
    P = table.shape[1]
    _check(f"q: {d} channels a head, the pool has {D}", d == D)
    _check(f"q: {H} heads over the pool's {heads}", 1 <= H <= 65535 and H % heads == 0)
    _check(f"q: {T} tokens, wanted 1 to {MAX_QUERY_TOKENS}", 1 <= T <= MAX_QUERY_TOKENS)
    _check("out: not q's shape", out.shape == q.shape)
    _check("table, lens: not one row and one length a request", table.shape[0] == B and lens.shape[0] == B)
    _check("table: 1 to 2^26 pages a request", 1 <= P <= 1 << 26)
    _check("q, out, workspace: not 16-byte aligned", (qp | op | wp) % 16 == 0)
    _check(f"workspace: {workspace.numel()} bytes, wanted {WORKSPACE_BYTES}", workspace.numel() >= WORKSPACE_BYTES)
    return _desc("kv4_sdpa", G.BF16, a=qp, b=pp, out=op, aux0=lp, aux1=tp, aux2=wp,
                 dims=(B, H | heads << 16, D | T << 16, P, npages), fparam=scale)


def page_copy(pool: torch.Tensor, pairs: torch.Tensor) -> np.ndarray:
    """pool[l, dst] = pool[l, src] for the pairs int32 [n, 2] of (src, dst)
    and every layer l. pool: [layers, npages, ...] of any dtype, a multiple of
    16 bytes a page. Pairs with a negative page are skipped; a source may be
    in several pairs, a destination is in one and is no pair's source."""
    _check(f"pool: {pool.ndim} dimensions, wanted layers, pages and the page's own", pool.ndim >= 3)
    pp = _tensor("pool", pool, (pool.dtype,), pool.ndim, pool)
    ap = _tensor("pairs", pairs, (torch.int32,), 2, pool)
    layers, npages = pool.shape[:2]
    nbytes = pool[0, 0].numel() * pool.element_size() if layers and npages else 0
    _check("pool: no layers, no pages, or pages that are not a multiple of 16 bytes", nbytes > 0 and nbytes % 16 == 0)
    _check("pool: more than 2^31 - 1 pages or 2^36 bytes a page", npages < 1 << 31 and nbytes < 1 << 36)
    _check("pairs: wanted [n, 2]", pairs.shape[1] == 2)
    _check("pool, pairs: not 16- and 8-byte aligned", pp % 16 == 0 and ap % 8 == 0)
    return _desc("page_copy", G.BF16, a=pp, aux0=ap, dims=(pairs.shape[0], nbytes // 16, npages, layers))
