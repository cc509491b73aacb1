"""What a decode step chooses, by its definitions in 64 bits (numpy), with how
far results in fp32 may be off."""
import numpy as np

SETTING = np.dtype([("repetition", "<f4"), ("presence", "<f4"), ("frequency", "<f4"), ("temperature", "<f4"),
                    ("prompt", "<i4"), ("length", "<i4"), ("mask", "<i4"), ("biases", "<i4")])
BIAS = np.dtype([("token", "<i4"), ("value", "<f4")])
HALF_STEP = {True: 2.0 ** -24, False: 2.0 ** -8}  # of f32, of bf16, relative


def bf16(x):
    """x rounded to bfloat16 (nearest, ties to even), as float32; NaN stays NaN."""
    x = np.ascontiguousarray(x, np.float32)
    b = x.view(np.uint32)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), x, r)


def _held(x, f32):
    """x with what the type cannot hold infinite (beyond its largest and half a step)."""
    return np.where(np.abs(x) >= (3.4028235677973366e38 if f32 else 3.3961775292304e38), np.copysign(np.inf, x), x)


def adjust(logits, settings, tokens, bias, mask, f32):
    """(adjusted logits f64 [B, V], how far an fp32 result rounded to the type may be off)."""
    B, V = logits.shape
    want, tol = np.empty((B, V)), np.empty((B, V))
    for b in range(B):
        s = settings[b]
        rep, pres, freq, temp = (float(s[n]) for n in ("repetition", "presence", "frequency", "temperature"))
        had = [t for t in tokens[b, :s["length"]] if 0 <= t < V] if tokens is not None else []
        own = [t for t in tokens[b, s["prompt"]:s["length"]] if 0 <= t < V] if tokens is not None else []
        seen = np.bincount(had, minlength=V) > 0
        c = np.bincount(own, minlength=V).astype(np.float64)
        x = logits[b].astype(np.float64)
        with np.errstate(all="ignore"):
            y = np.where(seen, np.where(x > 0, x / rep, x * rep), x)
            off = np.where(c > 0, freq * c + pres, 0.0)
            add = np.zeros(V)
            for e in (bias[b, :s["biases"]] if bias is not None else []):
                if 0 <= e["token"] < V:
                    add[e["token"]] = e["value"]
            t = temp if temp > 0 else 1.0
            # roundings, each 2^-24 of a part: 1 / temperature, that over (or times) rep, frequency, presence; the penalty's;
            # the multiply-adds'
            part = np.abs(y) + np.abs(off) + np.abs(add)
            y = _held((y - off + add) / t, f32)
            near = 8 * 2.0 ** -24 * part / t
            tol[b] = np.where(np.isfinite(y), near + HALF_STEP[f32] * (np.abs(y) + near) + 2.0 ** -133, 0.0)
        if s["mask"] >= 0:
            bits = np.unpackbits(np.ascontiguousarray(mask[s["mask"]]).view(np.uint8), bitorder="little")[:V]
            y[bits == 0] = -np.inf
            tol[b][bits == 0] = 0
        want[b] = y
    return want, tol


def top(logits, K):
    """(ids, log-probabilities, lse, their tolerances)."""
    B, V = logits.shape
    x = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    ids = np.empty((B, K), np.int32)
    lp, lse = np.empty((B, K)), np.empty(B)
    tlp, tlse = np.empty((B, K)), np.empty(B)
    for b in range(B):
        ids[b] = np.argsort(-x[b], kind="stable")[:K]
        m = x[b].max()
        with np.errstate(all="ignore"):
            ls = np.log(np.exp(x[b] - m).sum()) if np.isfinite(m) else 0.0
            lse[b] = m + ls
            v = x[b][ids[b]]
            lp[b] = np.where(v == -np.inf, -np.inf, v - m - ls)
        # The sum, relative: an exponential is off by 2^-22 (ex2) and by the argument's roundings, 2^-23 of it, whose
        # mean under the softmax is ln V at most; one rounding for each unit of 1,024, for the 37 sums within it and over the
        # lanes, and three for each of up to 128 runs that meet. The logarithm: 2^-23 of itself. Then three differences.
        r = 2.0 ** -22 + np.log(V) * 2.0 ** -23 + (V / 1024 + 40 + 3 * 128) * 2.0 ** -24
        tlse[b] = r + 2.0 ** -22 * abs(ls) + (2.0 ** -24 * abs(lse[b]) if np.isfinite(lse[b]) else 0)
        with np.errstate(all="ignore"):
            tlp[b] = np.where(np.isfinite(lp[b]), r + 2.0 ** -22 * (np.abs(v - m) + abs(ls)), 0.0)
    return ids, lp, lse, tlp, tlse


def experts(logits, K, sigmoid, bias, groups, keep, top2, normalise, scale):
    """(ids, weights f64); the weights' tolerance is `experts_tol` of themselves."""
    x = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    N, E = x.shape
    with np.errstate(all="ignore"):
        if sigmoid:
            s = np.where(x > 0, 1 / (1 + np.exp(-x)), np.exp(x) / (1 + np.exp(x)))
        else:
            m = np.where(np.isfinite(x.max(1)), x.max(1), 0.0)[:, None]
            e = np.exp(x - m)
            s = e / np.where(e.sum(1) > 0, e.sum(1), 1.0)[:, None]
    c = s + bias.astype(np.float64) if bias is not None else s
    # without a bias the scores' order is the logits', also where scores run out of digits
    order = c if bias is not None else x
    if groups > 1:
        g = (c if top2 else order).reshape(N, groups, E // groups)
        best = -np.sort(-g, axis=2)
        value = best[:, :, 0] + best[:, :, 1] if top2 else best[:, :, 0]
        kept = np.argsort(-value, axis=1, kind="stable")[:, :keep]
        shut = np.ones((N, groups), bool)
        np.put_along_axis(shut, kept, False, 1)
        # (shut ones behind all others, those of -infinity among them)
        rank = np.lexsort((np.arange(E) + np.zeros((N, 1)), -order, np.repeat(shut, E // groups, 1)), axis=1)
    else:
        rank = np.argsort(-order, axis=1, kind="stable")
    ids = rank[:, :K]
    w = np.take_along_axis(s, ids, 1)
    if normalise:
        t = w.sum(1, keepdims=True)
        w = np.divide(w, t, out=np.zeros_like(w), where=t > 0)
    return ids.astype(np.int32), w * scale


# A score is off by less than 2^-19 of itself (ex2 2^-22 twice, the sum's roundings), and so is a sum of them; a quotient
# by twice that, then two roundings.
EXPERTS_TOL = 2.0 ** -18 + 2.0 ** -23


def plan(ids, E):
    """(order, place, offsets)."""
    flat = ids.reshape(-1).astype(np.int64)
    here = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(here, flat, E), kind="stable")
    n = int(here.sum())
    place = np.full(flat.size, -1, np.int32)
    place[order[:n]] = np.arange(n)
    offsets = np.concatenate(([0], np.cumsum(np.bincount(flat[here], minlength=E)))).astype(np.int32)
    return np.where(np.arange(flat.size) < n, order, -1).astype(np.int32), place.reshape(ids.shape), offsets
