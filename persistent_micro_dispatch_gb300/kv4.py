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

Nothing here reads device memory or computes gradients. Launch with the
tensors' device current, on one of its streams. Slots, page tables, lengths and
pairs that point outside the pool are found by the kernels, and the executor
reports status 2 (bad arguments) for the descriptor; a launch reports nothing.
Of such an entry, a written row is skipped, a row read back is zeros, a pair is
skipped, a page's keys are left out of the attention (a query that has
positions to see, but none of whose pages is in the pool, is NaN), and a
request whose length does not fit its table row keeps its output rows as they
were.
"""
from __future__ import annotations

import struct

import numpy as np
import torch

from . import gpuos as G

PAGE = 32
WORKSPACE_BYTES = 32 << 20
COUNTER_BYTES = 8192  # of the workspace: zero before each attention
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


def reset_workspace(workspace: torch.Tensor) -> None:
    """Make a workspace fit for use again after an attention that did not run
    to its end (status 3, a dependency's wait ran out, or 4, the executor was
    leaving): what it left would be joined to the next one's states. Runs on
    the current stream."""
    if workspace.dtype is not torch.uint8 or workspace.ndim != 1 or workspace.numel() < WORKSPACE_BYTES:
        raise ValueError(f"workspace: {workspace.dtype} {tuple(workspace.shape)}, wanted uint8 ({WORKSPACE_BYTES},)")
    workspace[:COUNTER_BYTES].zero_()


def _refuse(pool: torch.Tensor, *named) -> None:
    """Raise what is wrong with a call's arguments, each (name, tensor,
    dtypes, shape; None in the shape: any size)."""
    for name, t, dtypes, shape in named:
        if t.dtype not in dtypes:
            raise TypeError(f"{name}: dtype {t.dtype}, wanted {' or '.join(str(d) for d in dtypes)}")
        if t.ndim != len(shape) or any(w is not None and n != w for n, w in zip(t.shape, shape)):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, wanted {tuple('any' if w is None else w for w in shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: not contiguous")
        if t.get_device() < 0 or t.device != pool.device:
            raise ValueError(f"{name}: on {t.device}, wanted the pool's CUDA device")
        if t.data_ptr() % 16 and name not in ("slots", "table", "lens"):
            raise ValueError(f"{name}: not 16-byte aligned")
    raise ValueError(f"pool {tuple(pool.shape)}: 1 to 2^26 pages of 1 to 65535 heads of 34 * 64 or 34 * 128 bytes, wanted")


def _desc(op: int, dtype: int, a: int, b: int, out: int, aux0: int, aux1: int, aux2: int, d0: int, d1: int, d2: int,
          d3: int, d4: int, fparam: float) -> np.ndarray:
    raw = bytearray(_DESC.pack(op, dtype, 0, 0, 0, 0, a, b, out, aux0, aux1, aux2, d0, d1, d2, d3, d4, 0, fparam, 0.0,
                               0, 0, 0))
    return np.frombuffer(raw, dtype=G.DESC_DTYPE)


_WRITE, _READ, _SDPA, _COPY = (G.OP[n] for n in ("kv4_write", "kv4_read", "kv4_sdpa", "page_copy"))
_U8, _I32, _BF16 = torch.uint8, torch.int32, torch.bfloat16
_HEAD_DIM = {34 * 64: 64, 34 * 128: 128}


def _rows(op: int, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, pool: torch.Tensor) -> np.ndarray:
    dt, dev, ks, ps = _DTYPE.get(k.dtype), pool.get_device(), k.shape, pool.shape
    if len(ks) == 3 and len(ps) == 3 and slots.ndim == 1:
        (n, heads, D), (npages, _, nbytes) = ks, ps
        kp, vp, pp = k.data_ptr(), v.data_ptr(), pool.data_ptr()
        if (dt is not None and v.dtype is k.dtype and v.shape == ks and slots.dtype is _I32 and pool.dtype is _U8
                and slots.shape[0] == n and _HEAD_DIM.get(nbytes) == D and ps[1] == heads and 1 <= npages <= 1 << 26
                and 1 <= heads <= 65535 and dev >= 0 and k.get_device() == dev and v.get_device() == dev
                and slots.get_device() == dev and k.is_contiguous() and v.is_contiguous() and slots.is_contiguous()
                and pool.is_contiguous() and not (kp | vp | pp) & 15):
            if op == _WRITE:
                return _desc(op, dt, kp, vp, pp, slots.data_ptr(), 0, 0, n, heads, D, npages, 0, 0.0)
            return _desc(op, dt, pp, 0, kp, slots.data_ptr(), vp, 0, n, heads, D, npages, 0, 0.0)
    n, heads = slots.numel(), ps[1] if len(ps) == 3 else None
    D = _HEAD_DIM.get(ps[2]) if len(ps) == 3 else None
    _refuse(pool, ("pool", pool, (_U8,), (None, None, None)), ("k", k, tuple(_DTYPE), (n, heads, D)),
            ("v", v, (k.dtype,), (n, heads, D)), ("slots", slots, (_I32,), (n,)))


def write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, pool: torch.Tensor) -> np.ndarray:
    """Quantise rows k, v [N, heads, D] (float32 or bfloat16) into the slots
    int32 [N] (page * 32 + key; negative: skipped; distinct) of the pool."""
    return _rows(_WRITE, k, v, slots, pool)


def read(pool: torch.Tensor, slots: torch.Tensor, k: torch.Tensor, v: torch.Tensor) -> np.ndarray:
    """The rows held in the slots into k, v [N, heads, D] (float32 or
    bfloat16, both exact); zeros for a negative slot."""
    return _rows(_READ, k, v, slots, pool)


def sdpa(q: torch.Tensor, pool: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, out: torch.Tensor,
         workspace: torch.Tensor, scale: float) -> np.ndarray:
    """Attention of q [B, T, H, D] (bfloat16, T <= 32 tokens a request, the
    last T of its lens[b]) over the pages table[b] (int32 [B, P]) into out:
    token t sees keys 0 .. lens[b] - T + t; zeros where that is none. Query
    head h reads cache head h // (H / heads). Descriptors that share a
    workspace must run one after another."""
    dev, qs, ps, ts = pool.get_device(), q.shape, pool.shape, table.shape
    if len(qs) == 4 and len(ps) == 3 and len(ts) == 2 and lens.ndim == 1:
        (B, T, H, D), (npages, heads, nbytes), P = qs, ps, ts[1]
        qp, pp, op, wp = q.data_ptr(), pool.data_ptr(), out.data_ptr(), workspace.data_ptr()
        if (q.dtype is _BF16 and out.dtype is _BF16 and pool.dtype is _U8 and table.dtype is _I32 and lens.dtype is _I32
                and workspace.dtype is _U8 and out.shape == qs and _HEAD_DIM.get(nbytes) == D and ts[0] == B
                and lens.shape[0] == B and 1 <= npages <= 1 << 26 and 1 <= heads and 1 <= H <= 65535 and H % heads == 0
                and 1 <= T <= MAX_QUERY_TOKENS and 1 <= P <= 1 << 26 and workspace.numel() >= WORKSPACE_BYTES
                and dev >= 0 and q.get_device() == dev and out.get_device() == dev and table.get_device() == dev
                and lens.get_device() == dev and workspace.get_device() == dev and q.is_contiguous()
                and out.is_contiguous() and pool.is_contiguous() and table.is_contiguous() and lens.is_contiguous()
                and workspace.is_contiguous() and not (qp | pp | op | wp) & 15):
            return _desc(_SDPA, G.BF16, qp, pp, op, lens.data_ptr(), table.data_ptr(), wp, B, H | heads << 16, D | T << 16,
                         P, npages, scale)
        if len(qs) == 4 and not 1 <= T <= MAX_QUERY_TOKENS:
            raise ValueError(f"q: {T} tokens a request, wanted 1 to {MAX_QUERY_TOKENS}")
        if heads and H % heads or not 1 <= H <= 65535:
            raise ValueError(f"q: {H} heads over the pool's {heads}")
        if not 1 <= P <= 1 << 26:
            raise ValueError(f"table: {P} pages a request, wanted 1 to 2^26")
        if workspace.numel() < WORKSPACE_BYTES:
            raise ValueError(f"workspace: {workspace.numel()} bytes, wanted {WORKSPACE_BYTES}")
    B, D = qs[0] if qs else None, _HEAD_DIM.get(ps[2]) if len(ps) == 3 else None
    _refuse(pool, ("pool", pool, (_U8,), (None, None, None)), ("q", q, (_BF16,), (None, None, None, D)),
            ("out", out, (_BF16,), tuple(qs)), ("table", table, (_I32,), (B, None)), ("lens", lens, (_I32,), (B,)),
            ("workspace", workspace, (_U8,), (None,)))


def page_copy(pool: torch.Tensor, pairs: torch.Tensor) -> np.ndarray:
    """pool[l, dst] = pool[l, src] for the pairs int32 [n, 2] of (src, dst)
    and every layer l. pool: [layers, npages, ...] of any dtype, a multiple of
    16 bytes a page. Pairs with a negative page are skipped; a source may be
    in several pairs, a destination is in one and is no pair's source."""
    ps, dev = pool.shape, pool.get_device()
    nbytes = pool.element_size()
    for n in ps[2:]:
        nbytes *= n
    pp, ap = pool.data_ptr(), pairs.data_ptr()
    if (len(ps) >= 3 and ps[0] >= 1 and 1 <= ps[1] < 1 << 31 and 0 < nbytes < 1 << 36 and not nbytes & 15
            and pairs.dtype is _I32 and pairs.ndim == 2 and pairs.shape[1] == 2 and dev >= 0 and pairs.get_device() == dev
            and pool.is_contiguous() and pairs.is_contiguous() and not pp & 15 and not ap & 7):
        return _desc(_COPY, G.BF16, pp, 0, 0, ap, 0, 0, pairs.shape[0], nbytes >> 4, ps[1], ps[0], 0, 0.0)
    if len(ps) < 3 or not pool.numel() or nbytes & 15 or nbytes >= 1 << 36 or ps[1] >= 1 << 31:
        raise ValueError(f"pool {tuple(ps)}: wanted [layers, pages, ...], a multiple of 16 bytes a page")
    if pairs.dtype is _I32 and ap & 7:
        raise ValueError("pairs: not 8-byte aligned")
    _refuse(pool, ("pool", pool, (pool.dtype,), tuple(ps)), ("pairs", pairs, (_I32,), (None, 2)))
