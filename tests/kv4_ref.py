"""The 4-bit paged cache in 64 bits, from its definition (numpy): the reference
of the KV4 ops' tests. It shares no code with the library."""
import numpy as np

PAGE = 32
MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16(x):
    """Nearest bfloat16 (ties to even) of finite float64 values, as float64."""
    f = np.asarray(x, np.float64).astype(np.float32)
    u = f.view(np.uint32)
    return (((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)).view(np.float32).astype(np.float64)


def offsets(D, key, c):
    """Byte offsets in a head's page of channel c of a key: key code, value
    code, key scale, value scale. The even channel of a pair is the low half."""
    G, g, x = D // 32, c // 32, c % 32
    t, quad, r = key // 16, key // 4 % 4, key % 4
    k = t * 8 * D + ((quad * 2 + r % 2) * 4 + x // 8) * 8 * G + (r // 2) * 4 * G + 4 * g + x % 8 // 2
    v = 16 * D + t * 8 * D + (x // 4 * 4 + quad) * 8 * G + r * 2 * G + 2 * g + x % 4 // 2
    return k, v, 32 * D + key * G + g, 33 * D + t * 16 * G + quad * 4 * G + g * 4 + r


def quantise(x):
    """Codes and scale bytes of rows x [..., D]."""
    x = np.asarray(x, np.float64)
    y = x.reshape(x.shape[:-1] + (-1, 32))
    fine = np.isfinite(y).all(-1)
    top = np.where(fine, np.abs(np.where(np.isfinite(y), y, 0)).max(-1), 0.0)
    # the least e >= -127 with top <= 6 2^e (frexp: top in [2^(n-1), 2^n)), at most 125
    n = np.frexp(top)[1]
    e = np.clip(np.where(top <= 6 * 2.0 ** (n - 3.0), n - 3, n - 2), -127, 125)
    e = np.where(top == 0, -127, e)
    with np.errstate(invalid="ignore"):
        a = np.abs(np.where(fine[..., None], y, 0)) / 2.0 ** e[..., None].astype(float)
    d = np.abs(a[..., None] - MAG)
    best = d.min(-1, keepdims=True)
    near = d == best
    idx = np.arange(8)
    # the nearest; of two nearest the even code
    code = np.where(near & (idx % 2 == 0), idx, -1).max(-1)
    code = np.where(near.sum(-1) == 1, near.argmax(-1), code)
    code = np.where(fine[..., None], code + 8 * np.signbit(y), 0)
    return code.reshape(x.shape).astype(np.uint8), np.where(fine, e + 127, 255).astype(np.uint8)


def values(code, byte):
    """Values [..., D] of codes and scale bytes."""
    c = code.reshape(code.shape[:-1] + (-1, 32))
    v = np.where(c > 7, -1.0, 1.0) * MAG[c & 7] * 2.0 ** (byte.astype(float) - 127)[..., None]
    v = np.where((byte == 255)[..., None], np.nan, v)
    return v.reshape(code.shape)


def put(pool, slot, head, kc, kb, vc, vb):
    """Write one row's codes and scale bytes into pool uint8 [pages, heads, 34 D]."""
    D = len(kc)
    blob, key = pool[slot // PAGE, head], slot % PAGE
    for c in range(0, D, 2):
        k, v, ks, vs = offsets(D, key, c)
        blob[k] = kc[c] | kc[c + 1] << 4
        blob[v] = vc[c] | vc[c + 1] << 4
        blob[ks], blob[vs] = kb[c // 32], vb[c // 32]


_maps = {}


def unpack(pool):
    """Keys, values and the values' scales float64 [pages, heads, 32, D] of a pool."""
    D = pool.shape[2] // 34
    if D not in _maps:
        key, c = np.meshgrid(np.arange(PAGE), np.arange(D), indexing="ij")
        _maps[D] = offsets(D, key, c), c
    (k, v, ks, vs), c = _maps[D]
    out = []
    for at, sc in ((k, ks), (v, vs)):
        code = pool[:, :, at] >> (4 * (c % 2)).astype(np.uint8) & 15
        out.append(values(code, pool[:, :, sc][..., ::32]))
    out.append(2.0 ** (np.repeat(pool[:, :, vs][..., ::32], 32, -1).astype(float) - 127))
    return out


def attend(q, pool, table, lens, scale):
    """Output float64 [B, T, H, D] of q (float64) and a bound on what a kernel
    may be off by, apart from the rounding of its output (see bound())."""
    B, T, H, D = q.shape
    heads = pool.shape[1]
    g = H // heads
    K, V, S = unpack(pool)
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        n = int(lens[b])
        at = np.arange(n)
        page = table[b][at // PAGE]
        inside = (page >= 0) & (page < pool.shape[0])
        kb, vb, sb = (x[np.where(inside, page, 0), :, at % PAGE] for x in (K, V, S))  # [n, heads, D]
        for t in range(T):
            see = inside & (at <= n - T + t)
            if not see.any():
                continue
            for h in range(H):
                k, v = kb[see, h // g], vb[see, h // g]
                s = k @ q[b, t, h] * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                out[b, t, h] = p @ v
                reach = np.abs(k) @ np.abs(q[b, t, h]) * abs(scale)
                tol[b, t, h] = bound(p, np.abs(v), sb[see, h // g].max(0), reach.max(), D)
    return out, tol


def bound(p, v, scale, reach, D):
    """|error| before the output's rounding, from the kernel's arithmetic:
    weights rounded to f16 (2^-11 each, or 2^-31 of the largest where they are
    subnormal); scores summed in fp32 over D products and D / 32 scale groups,
    scaled and shifted (each a rounding of at most 2^-24 of `reach`, the
    largest sum of |q k| scale), so a weight is off by twice that many nats
    against the sum; exp2 and the rescaling of the accumulators good to 2^-18.
    Values: a weight is multiplied by 2^(b - E + 7) in f16, b the exponent of
    the value's scale and E the largest of the group's, which is zero for b
    <= E - 22: such a value is at most 6 * 2^-22 of the largest scale; a
    product below 2^-14 is off by 2^-25, when the largest weight times the
    largest scale is 2^13 or more: 6 * 2^-38 of that scale for each key."""
    rel = 2.0 ** -11 + 2 * (D + 8) * 2.0 ** -24 * reach + 2.0 ** -18
    return rel * (p @ v) + 2.0 ** -31 * v.sum(0) + (6 * 2.0 ** -22 + len(v) * 6 * 2.0 ** -38) * scale


def random_pool(rng, pages, heads, D, spread=3.0):
    """A pool whose every slot holds a quantised random row, and those rows."""
    pool = np.zeros((pages, heads, 34 * D), np.uint8)
    key, c = np.meshgrid(np.arange(PAGE), np.arange(0, D, 2), indexing="ij")
    k, v, ks, vs = offsets(D, key, c)
    for at, sc, size in ((k, ks, 1.0), (v, vs, 1.0)):
        x = rng.standard_normal((pages, heads, PAGE, D)) * np.exp(rng.standard_normal((pages, heads, PAGE, 1)) * spread / 3) * size
        code, byte = quantise(x)
        pool[:, :, at] = code[..., 0::2] | code[..., 1::2] << 4
        pool[:, :, sc[:, ::16]] = byte
    return pool
