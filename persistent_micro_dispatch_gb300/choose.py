"""Descriptors of the ops with which a decode step makes its choices, from
PyTorch tensors: logits adjusted for the next token (``adjust``), the best
tokens of a row with their log-probabilities (``top``), the experts of a token
(``experts``) and the experts' order (``plan``).

Argument checks and marshalling only, as in the ctypes binding: each function
returns ``gpuos_desc`` records (an array of one; ``plan`` of one or two, to be
run in that order) for ``Executor.submit_batch`` (joined with
``numpy.concatenate``) or ``gpuos.eager_run``; the ops run in the library's
CUDA kernels (include/gpuos.h, GPUOS_OP_LOGITS_ADJUST and the ops after it, has
their definitions). The tensors must stay alive until the descriptor has
completed, and a descriptor may be submitted again while they do. GPUOS page,
§3 Q2, operator library, has the softmax and row reductions that these stand
beside.

    settings = choose.new_settings(B)                    # one record for each request
    choose.fields(settings)["temperature"][:] = 0.7
    ws = choose.new_workspace()
    stream = torch.cuda.current_stream().cuda_stream
    gpuos.eager_run(choose.adjust(logits, logits, settings, tokens=tokens, mask=mask), stream)
    gpuos.eager_run(choose.top(logits, ids, logprobs, lse, ws), stream)

    gpuos.eager_run(choose.experts(router_logits, ids, weights, sigmoid=True, bias=bias, groups=8, keep=4, top2=True), stream)
    gpuos.eager_run(choose.plan(ids, order, place, offsets, ws), stream)

In the executor a descriptor starts when a worker is free, whatever came before
it in the batch: each must depend on those whose results it reads, and on the
last one that used its workspace. ``plan``'s second record depends on its first;
nothing else is set here. A step as a chain, each record after the one before:

    d = numpy.concatenate([choose.adjust(...), choose.top(...), choose.experts(...), choose.plan(...)])
    d["flags"], d["dep"][1:, 0] = gpuos.FLAG_DEP_REL, 1
    ex.submit_batch(d)

(Two chains side by side, tokens and experts, take a workspace each. Launches on
one stream run in order by themselves.)

Logits are [rows, columns], float32 or bfloat16, with neighbouring columns next
to each other and rows any distance apart; everything else is contiguous.
Nothing here reads device memory or computes gradients. Launch with the
tensors' device current, on one of its streams. What the device finds wrong (a
request's record that does not fit) gives status 2 (bad arguments) in the
executor; a launch reports nothing, and keeps such a request's row as it was.
"""
from __future__ import annotations

from typing import Optional

import numpy as np
import torch

from . import gpuos as G
from .kv4 import _DESC

WORKSPACE_BYTES = 2 << 20
COUNTER_BYTES = 8192  # of the workspace: zero before each use
MAX_BIASES = 1024
MAX_TOP = 64
MAX_EXPERTS = 1024
MAX_EXPERTS_PER_TOKEN = 32
PLAN_ONE = 4096  # pairs of a plan that one descriptor places

_FLAGS_SIGMOID, _FLAGS_TOP2, _FLAGS_NORM = 1, 2, 4
_DTYPE = {torch.float32: G.F32, torch.bfloat16: G.BF16}
_U8, _I32, _F32 = torch.uint8, torch.int32, torch.float32
_ADJUST, _TOP, _ROUTE, _COUNT, _PLACE = (G.OP[n] for n in ("logits_adjust", "logits_top", "expert_route", "expert_count", "expert_place"))
_FIELDS = ("repetition", "presence", "frequency", "temperature", "prompt", "length", "mask", "biases")


def new_settings(requests: int, device="cuda") -> torch.Tensor:
    """Records int32 [requests, 8] (``gpuos_logits_request``) that change
    nothing: no penalties, temperature 1, no tokens, no mask, no biases."""
    s = torch.zeros(requests, 8, dtype=_I32, device=device)
    s[:, :4] = torch.tensor([1.0, 0.0, 0.0, 1.0]).view(_I32).to(device)
    s[:, 6] = -1
    return s


def fields(settings: torch.Tensor) -> dict:
    """The records' columns by name, as views to write to: ``repetition``,
    ``presence``, ``frequency``, ``temperature`` (float32), ``prompt``,
    ``length`` (tokens so far, the first ``prompt`` of them the prompt),
    ``mask`` (its row; negative: none) and ``biases`` (entries; int32)."""
    if settings.dtype is not _I32 or settings.ndim != 2 or settings.shape[1] != 8 or not settings.is_contiguous():
        raise ValueError(f"settings: {settings.dtype} {tuple(settings.shape)}, wanted int32 (any, 8), contiguous")
    f = settings.view(_F32)
    return {n: (f if i < 4 else settings)[:, i] for i, n in enumerate(_FIELDS)}


def new_workspace(device="cuda") -> torch.Tensor:
    """The workspace of ``top`` and ``plan``, for one of them at a time."""
    return torch.zeros(WORKSPACE_BYTES, dtype=_U8, device=device)


def reset_workspace(workspace: torch.Tensor) -> None:
    """Make a workspace fit for use again after a ``top`` that did not run to
    its end (status 3, a dependency's wait ran out, or 4, the executor was
    leaving). Runs on the current stream."""
    if workspace.dtype is not _U8 or workspace.ndim != 1 or workspace.numel() < WORKSPACE_BYTES or not workspace.is_contiguous():
        raise ValueError(f"workspace: {workspace.dtype} {tuple(workspace.shape)}, wanted uint8 ({WORKSPACE_BYTES},)")
    workspace[:COUNTER_BYTES].zero_()


def _refuse(like: torch.Tensor, *named) -> None:
    """Raise what is wrong with a call's arguments, each (name, tensor,
    dtypes, shape (None in it: any size), alignment)."""
    for name, t, dtypes, shape, align in named:
        if t is None:
            continue
        if t.dtype not in dtypes:
            raise TypeError(f"{name}: dtype {t.dtype}, wanted {' or '.join(str(d) for d in dtypes)}")
        if t.ndim != len(shape) or any(w is not None and n != w for n, w in zip(t.shape, shape)):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, wanted {tuple('any' if w is None else w for w in shape)}")
        if t.get_device() < 0 or t.device != like.device:
            raise ValueError(f"{name}: on {t.device}, wanted the logits' or ids' CUDA device")
        if not t.is_contiguous():
            raise ValueError(f"{name}: not contiguous")
        if t.data_ptr() % align:
            raise ValueError(f"{name}: not {align}-byte aligned")


def _rows(name: str, x: torch.Tensor):
    """Type, rows, columns, row distance and address of logits."""
    dt, shape = _DTYPE.get(x.dtype), x.shape
    if dt is not None and len(shape) == 2 and x.get_device() >= 0:
        n, cols = shape
        ld, step = (cols, 1) if x.is_contiguous() or n < 2 else x.stride()
        if n < 2:
            step = x.stride(1)
        if (step == 1 or cols == 1) and 1 <= cols <= ld < 1 << 32 and cols < 0x7FFFFF00 and n < 1 << 31:
            return dt, n, cols, ld, x.data_ptr()
    if dt is None:
        raise TypeError(f"{name}: dtype {x.dtype}, wanted torch.float32 or torch.bfloat16")
    if x.ndim != 2 or not x.shape[1]:
        raise ValueError(f"{name}: shape {tuple(x.shape)}, wanted (rows, columns)")
    if x.get_device() < 0:
        raise ValueError(f"{name}: on {x.device}, wanted a CUDA device")
    raise ValueError(f"{name}: shape {tuple(x.shape)}, strides {x.stride()}, wanted rows that lie one behind the other")


def _desc(*records) -> np.ndarray:
    """Descriptors of (op, dtype, flags, dep, a, b, out, aux0, aux1, aux2, dims..., fparam)."""
    raw = bytearray()
    for op, dt, flags, dep, a, b, out, x0, x1, x2, d0, d1, d2, d3, d4, d5, f in records:
        raw += _DESC.pack(op, dt, flags, 0, dep, 0, a, b, out, x0, x1, x2, d0, d1, d2, d3, d4, d5, f, 0.0, 0, 0, 0)
    return np.frombuffer(raw, G.DESC_DTYPE)


def adjust(logits: torch.Tensor, out: torch.Tensor, settings: torch.Tensor, tokens: Optional[torch.Tensor] = None,
           bias: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None) -> np.ndarray:
    """Logits [B, V] under each request's settings into out [B, V] (of the same
    type; it may be the logits themselves, but not overlap them otherwise):
    penalties for the tokens int32 [B, L] that it has had (its first ``length``
    of them), biases for listed tokens (int32 [B, n <= 1024, 2]: a token, and the
    bits of a float32; its first ``biases``), the temperature, and -infinity for the
    tokens whose bit in its row of the mask (int32 [M, ceil(V / 32)], token v at
    bit v % 32 of word v // 32) is 0."""
    dt, B, V, ld, a = _rows("logits", logits)
    dt2, B2, V2, ldo, o = _rows("out", out)
    dev, sp = logits.get_device(), settings.data_ptr()
    L = M = n = tp = mp = bp = 0
    ok = (dt2 == dt and B2 == B and V2 == V and out.get_device() == dev and settings.dtype is _I32 and settings.shape == (B, 8)
          and settings.get_device() == dev and settings.is_contiguous() and not sp & 15)
    if tokens is not None:
        ts, tp = tokens.shape, tokens.data_ptr()
        L = ts[-1] if ts else 0
        ok = (ok and len(ts) == 2 and ts[0] == B and L <= 1 << 28 and tokens.dtype is _I32 and tokens.get_device() == dev
              and tokens.is_contiguous())
    if mask is not None:
        ms, mp = mask.shape, mask.data_ptr()
        M = ms[0] if ms else 0
        ok = (ok and len(ms) == 2 and ms[1] == V + 31 >> 5 and M < 1 << 16 and mask.dtype is _I32 and mask.get_device() == dev
              and mask.is_contiguous())
    if bias is not None:
        bs, bp = bias.shape, bias.data_ptr()
        n = bs[1] if len(bs) == 3 else 0
        ok = (ok and len(bs) == 3 and bs[0] == B and bs[2] == 2 and n <= MAX_BIASES and bias.dtype is _I32 and bias.get_device() == dev
              and bias.is_contiguous() and not bp & 7)
    if not ok or (a == o and ld != ldo):
        if dt2 != dt or (B2, V2) != (B, V) or out.get_device() != dev:
            raise ValueError(f"out: {out.dtype} {tuple(out.shape)} on {out.device}, wanted {logits.dtype} {(B, V)} on {logits.device}")
        if a == o and ld != ldo:
            raise ValueError(f"out: the logits' own memory with rows {ldo} apart, wanted {ld}")
        _refuse(logits, ("settings", settings, (_I32,), (B, 8), 16), ("tokens", tokens, (_I32,), (B, None), 4),
                ("mask", mask, (_I32,), (None, (V + 31) // 32), 4), ("bias", bias, (_I32,), (B, None, 2), 8))
        raise ValueError(f"{L} tokens, {M} masks and {n} biases: at most 2^28, 65535 and {MAX_BIASES}")
    return _desc((_ADJUST, dt, 0, 0, a, tp, o, sp, mp, bp, B, V, ld, ldo, L, M | n << 16, 0.0))


def top(logits: torch.Tensor, ids: torch.Tensor, logprobs: torch.Tensor, lse: Optional[torch.Tensor],
        workspace: torch.Tensor) -> np.ndarray:
    """The K <= 64 best tokens of each row of logits [B, V] into ids int32
    [B, K] (by value, then by id), their log-probabilities into logprobs
    float32 [B, K] and the rows' log-sum-exp into lse float32 [B] (None: not
    wanted). Descriptors that share a workspace must run one after another."""
    dt, B, V, ld, a = _rows("logits", logits)
    dev, K = logits.get_device(), ids.shape[-1] if ids.ndim else 0
    shape, wp = (B, K), workspace.data_ptr()
    if not (1 <= K <= MAX_TOP and K <= V and ids.dtype is _I32 and ids.shape == shape and logprobs.dtype is _F32
            and logprobs.shape == shape and ids.get_device() == dev and logprobs.get_device() == dev and ids.is_contiguous()
            and logprobs.is_contiguous()
            and (lse is None or (lse.dtype is _F32 and lse.shape == (B,) and lse.get_device() == dev and lse.is_contiguous()))
            and workspace.dtype is _U8 and workspace.ndim == 1 and workspace.numel() >= WORKSPACE_BYTES
            and workspace.get_device() == dev and workspace.is_contiguous() and not wp & 15):
        if not 1 <= K <= min(MAX_TOP, V):
            raise ValueError(f"ids: {K} of {V} tokens a row, wanted 1 to {min(MAX_TOP, V)}")
        _refuse(logits, ("ids", ids, (_I32,), (B, None), 4), ("logprobs", logprobs, (_F32,), (B, K), 4), ("lse", lse, (_F32,), (B,), 4),
                ("workspace", workspace, (_U8,), (None,), 16))
        raise ValueError(f"workspace: {workspace.numel()} bytes, wanted {WORKSPACE_BYTES}")
    return _desc((_TOP, dt, 0, 0, a, 0, ids.data_ptr(), logprobs.data_ptr(), 0 if lse is None else lse.data_ptr(), wp, B, V, ld, K, 0, 0,
                  0.0))


def experts(logits: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, *, sigmoid: bool = False,
            bias: Optional[torch.Tensor] = None, groups: int = 1, keep: int = 1, top2: bool = False, normalise: bool = True,
            scale: float = 1.0, rows: Optional[torch.Tensor] = None) -> np.ndarray:
    """The K experts of each token of the router's logits [N, E] into ids int32
    [N, K], best first, and their weights into weights float32 [N, K]. Scores
    are the row's softmax, or sigmoids; the choice goes by score + bias
    (float32 [E]) as in 64-bit arithmetic, or without a bias by the logits, whose
    order is the scores' (also where 64-bit scores run out of digits: a bias of
    zeros may choose otherwise there), among the ``keep`` best of ``groups`` groups of neighbouring
    experts (by their best, or with top2 by the sum of their two best scores plus biases), ties to
    the lower number. Weights are the scores, divided by their sum
    with normalise, times scale. rows (int32 [1]): the tokens from there on are
    padding, with ids -1 and weights 0."""
    dt, N, E, ld, a = _rows("logits", logits)
    dev, K = logits.get_device(), ids.shape[-1] if ids.ndim else 0
    shape = (N, K)
    if not (E <= MAX_EXPERTS and 1 <= K <= MAX_EXPERTS_PER_TOKEN and 1 <= groups <= 32 and E % groups == 0 and 1 <= keep <= groups
            and K <= keep * (E // groups) and not (top2 and E // groups < 2) and ids.dtype is _I32 and ids.shape == shape
            and weights.dtype is _F32 and weights.shape == shape and ids.get_device() == dev and weights.get_device() == dev
            and ids.is_contiguous() and weights.is_contiguous()
            and (bias is None or (bias.dtype is _F32 and bias.shape == (E,) and bias.get_device() == dev and bias.is_contiguous()))
            and (rows is None or (rows.dtype is _I32 and rows.shape == (1,) and rows.get_device() == dev))):
        if not 1 <= E <= MAX_EXPERTS or not 1 <= groups <= 32 or E % groups or not 1 <= keep <= groups or (top2 and E // groups < 2):
            raise ValueError(f"{E} experts in {groups} groups of which {keep}: wanted at most {MAX_EXPERTS} in 1 to 32 equal groups"
                             + (" of two or more" if top2 else ""))
        if not 1 <= K <= min(MAX_EXPERTS_PER_TOKEN, keep * (E // groups)):
            raise ValueError(f"ids: {K} experts a token, wanted 1 to {min(MAX_EXPERTS_PER_TOKEN, keep * (E // groups))}")
        _refuse(logits, ("ids", ids, (_I32,), (N, None), 4), ("weights", weights, (_F32,), (N, K), 4), ("bias", bias, (_F32,), (E,), 4),
                ("rows", rows, (_I32,), (1,), 4))
    return _desc((_ROUTE, dt, 0, 0, a, 0 if bias is None else bias.data_ptr(), ids.data_ptr(), weights.data_ptr(),
                  0 if rows is None else rows.data_ptr(), 0, N, E, ld, K, groups | keep << 16,
                  (_FLAGS_SIGMOID if sigmoid else 0) | (_FLAGS_TOP2 if top2 else 0) | (_FLAGS_NORM if normalise else 0), scale))


def plan(ids: torch.Tensor, order: torch.Tensor, place: torch.Tensor, offsets: torch.Tensor, workspace: torch.Tensor) -> np.ndarray:
    """The pairs of ids int32 [N, K] (token, expert) in the experts' order:
    order int32 [N * K] lists pair numbers (token * K + k) by expert, and -1
    behind the last; place int32 [N, K] says where each pair went (-1: its id
    is no expert's); offsets int32 [E + 1] says where each expert's pairs begin. One
    record, or two (a count and a placement that depends on the record before
    it) for more than 4,096 pairs. Descriptors that share a workspace must run
    one after another, these two with nothing between that shares it."""
    dev, P, E, ws = ids.get_device(), ids.numel(), offsets.numel() - 1, workspace.data_ptr()
    if not (dev >= 0 and ids.dtype is _I32 and order.dtype is _I32 and place.dtype is _I32 and offsets.dtype is _I32
            and P < 0x7FFFFF00 and 1 <= E <= MAX_EXPERTS and order.numel() == P and order.ndim == offsets.ndim == 1
            and place.shape == ids.shape and order.get_device() == dev and place.get_device() == dev and offsets.get_device() == dev
            and ids.is_contiguous() and order.is_contiguous() and place.is_contiguous() and offsets.is_contiguous()
            and workspace.dtype is _U8 and workspace.ndim == 1 and workspace.numel() >= WORKSPACE_BYTES
            and workspace.get_device() == dev and workspace.is_contiguous() and not ws & 15):
        if dev < 0:
            raise ValueError(f"ids: on {ids.device}, wanted a CUDA device")
        _refuse(ids, ("ids", ids, (_I32,), tuple(ids.shape), 4), ("order", order, (_I32,), (P,), 4),
                ("place", place, (_I32,), tuple(ids.shape), 4), ("offsets", offsets, (_I32,), (None,), 4),
                ("workspace", workspace, (_U8,), (None,), 16))
        if not 1 <= E <= MAX_EXPERTS or P >= 0x7FFFFF00:
            raise ValueError(f"{P} pairs of {E} experts: wanted below 2^31 of 1 to {MAX_EXPERTS}")
        raise ValueError(f"workspace: {workspace.numel()} bytes, wanted {WORKSPACE_BYTES}")
    a = ids.data_ptr()
    place_it = (_PLACE, 0, 0, 0, a, place.data_ptr(), order.data_ptr(), offsets.data_ptr(), 0, ws, P, E, 0, 0, 0, 0, 0.0)
    if P <= PLAN_ONE:
        return _desc(place_it)
    return _desc((_COUNT, 0, 0, 0, a, 0, 0, 0, 0, ws, P, E, 0, 0, 0, 0, 0.0), (_PLACE, 0, G.FLAG_DEP_REL, 1) + place_it[4:])
