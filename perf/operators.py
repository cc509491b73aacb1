"""The 4-bit paged key/value cache: its operators in plain form, and the calls a user makes of them.

A cache page holds 32 tokens of every key/value head. For one head a page is 34 D bytes (D = head dimension, G = D / 32
scale groups): the keys' codes (16 D bytes), the values' codes (16 D), the keys' scales (D), the values' scales (D).
A code is a sign and a magnitude of {0, 0.5, 1, 1.5, 2, 3, 4, 6}; 32 neighbouring channels of a token share one scale, a
power of two held as its exponent + 127 (255: the group held a NaN or an infinity). Codes lie in the order in which a
warp's matrix fragments take them, two neighbouring channels to a byte, the even one in the low half:

  keys          [key>>4][key>>2 & 3][key & 1][channel>>3 & 3][key>>1 & 1][group][channel>>1 & 3]
  values        [key>>4][channel>>2 & 7][key>>2 & 3][key & 3][group][channel>>1 & 1]
  key scales    [key][group]
  value scales  [key>>4][key>>2 & 3][group][key & 3]

with `channel` counted within its group of 32. A slot is page * 32 + key.

Four kinds of case: "attend" (attention of one or a few query tokens over the cache), "append" (new rows quantised into
their slots, then the whole context read back), "gather" (rows read back) and "pages" (page copies for a fork or a
compaction).
"""
import random

import torch

own = False

PAGE = 32
WORKSPACE = 32 << 20  # bytes of scratch that the attention takes, whatever the sizes
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one user's chat turn: latency is all
        dict(name="attend_one", kind="attend", B=1, H=32, Hkv=8, D=128, T=1, lo=1000, hi=1000, empty=0, spare=0),
        # the 32-head decode step with a cache head for each query head, ragged lengths up to 4096
        dict(name="attend_mha", kind="attend", B=8, H=32, Hkv=32, D=128, T=1, lo=17, hi=4096, empty=0, spare=3),
        # a full server with long contexts, two of its places free: the largest
        dict(name="attend_batch", kind="attend", B=64, H=32, Hkv=8, D=128, T=1, lo=2000, hi=16383, empty=2, spare=0),
        # one long document
        dict(name="attend_long", kind="attend", B=1, H=64, Hkv=8, D=128, T=1, lo=131071, hi=131071, empty=0, spare=1),
        # four drafted tokens of each request are checked at once
        dict(name="attend_draft", kind="attend", B=16, H=32, Hkv=4, D=128, T=4, lo=2, hi=4099, empty=0, spare=0),
        # a small model with 64 channels a head, an odd batch
        dict(name="attend_small", kind="attend", B=33, H=14, Hkv=2, D=64, T=1, lo=1, hi=3001, empty=1, spare=5),
        # a decode step's new tokens go into the cache
        dict(name="append_step", kind="append", B=64, Hkv=8, D=128, T=1, lo=1, hi=129, f32=False),
        # a chunk of four prompts, and the context read back for the chunk's own attention
        dict(name="append_chunk", kind="append", B=4, Hkv=8, D=128, T=2048, lo=2048, hi=6001, f32=False),
        # a long prefix read back
        dict(name="gather_long", kind="gather", B=2, Hkv=8, D=128, lo=65537, hi=98304, f32=False),
        # one short prefix read back in 32 bits, odd sizes
        dict(name="gather_short", kind="gather", B=1, Hkv=3, D=64, lo=911, hi=911, f32=True),
        # a beam forks: each part-filled last page is copied, in every layer
        dict(name="pages_fork", kind="pages", layers=32, npages=257, page=34816, n=15),
        # a pool of bf16 pages is compacted
        dict(name="pages_compact", kind="pages", layers=4, npages=1500, page=131072, n=611),
    ]


def draw(rng):
    def spread(lo, hi):
        return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))

    kind = rng.choice(["attend", "attend", "attend", "append", "gather", "pages"])
    if kind == "pages":
        page = 16 * spread(136, 8192)
        layers, n = spread(1, 32), spread(1, 1024)
        while layers * n * page > 400 << 20:
            layers, n = max(1, layers // 2), max(1, n * 2 // 3)
        return dict(kind=kind, layers=layers, npages=2 * n + spread(1, 200), page=page, n=n)
    D, Hkv = rng.choice([64, 128, 128]), rng.choice([1, 2, 3, 4, 8, 8, 32])
    if kind == "attend":
        B, H, T = spread(1, 64), Hkv * rng.choice([1, 2, 4, 5, 7, 8, 16]), rng.choice([1, 1, 1, 2, 3, 5, 8])
        hi = spread(1, 131072)
        while B * hi * Hkv * D > 25 * 16384 * 8 * 128 or B * hi * T * H * D > 25 * 16384 * 32 * 128:
            B, hi = max(1, B * 2 // 3), max(1, hi * 3 // 4)
        return dict(kind=kind, B=B, H=H, Hkv=Hkv, D=D, T=T, lo=spread(1, hi), hi=hi, empty=rng.choice([0, 0, 1]) if B > 1 else 0, spare=rng.randrange(9))
    B, f32 = spread(1, 64), rng.random() < 0.3
    hi = spread(1, 98304)
    while B * hi * Hkv * D * (2 if f32 else 1) > (150000 if kind == "gather" else 100000) * 8 * 128:
        B, hi = max(1, B * 2 // 3), max(1, hi * 3 // 4)
    if kind == "gather":
        return dict(kind=kind, B=B, Hkv=Hkv, D=D, lo=spread(1, hi), hi=hi, f32=f32)
    T = spread(1, min(hi, 4096))
    return dict(kind=kind, B=B, Hkv=Hkv, D=D, T=T, lo=spread(T, hi), hi=hi, f32=f32)


def _lengths(case):
    """The requests' lengths: they belong to the case, whatever the seed. The longest is the first."""
    rng = random.Random(case["B"] * 1000003 + case["hi"])
    lens = [case["hi"]] + [round(case["lo"] * (case["hi"] / case["lo"]) ** rng.random()) for _ in range(case["B"] - 1)]
    for i in range(case.get("empty", 0)):
        lens[-1 - 7 * i] = 0
    return lens


def _quantised(x):
    """Codes 0..15 and scale bytes of rows x[..., D], in 32 bits. The scale is the least power of two (at least 2^-127, at
    most 2^125) under which the group's largest magnitude is at most 6; codes go to the nearest value, ties to the even
    code. A group with a NaN or an infinity in it has scale 255 and codes 0."""
    x = x.float().unflatten(-1, (-1, 32))
    top = x.abs().amax(-1)
    fine = torch.isfinite(top)
    m, e = torch.frexp(torch.where(fine, top, 0.0))
    e = torch.where(m == 0, -127, e - 3 + (m > 0.75).int()).clamp(-127, 125)
    y = torch.ldexp(x, -e.unsqueeze(-1))
    a = y.abs()
    code = (a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5).byte()
    code = torch.where(fine.unsqueeze(-1), code + 8 * torch.signbit(y).byte(), 0)
    return code.flatten(-2).byte(), torch.where(fine, e + 127, 255).byte()


def _keys_first(slots):
    """Page and key of each slot; negative slots (holes) go to page 0."""
    s = slots.long().clamp(min=0)
    return s // PAGE, s % PAGE


def _plan(D, device):
    """Where a head's page holds what: byte offsets [32 keys, D / 2 pairs] of the keys' and the values' codes and
    [32 keys, G] of their scales; and the values of the sixteen codes."""
    G = D // 32
    key, pair, g = torch.arange(PAGE, device=device)[:, None], torch.arange(D // 2, device=device)[None], torch.arange(G, device=device)[None]
    grp, c = pair // 16, 2 * (pair % 16)
    kc = ((((((key >> 4) * 4 + (key >> 2 & 3)) * 2 + (key & 1)) * 4 + (c >> 3)) * 2 + (key >> 1 & 1)) * G + grp) * 4 + (c >> 1 & 3)
    vc = ((((key >> 4) * 8 + (c >> 2)) * 4 + (key >> 2 & 3)) * 4 + (key & 3)) * G * 2 + grp * 2 + (c >> 1 & 1)
    ks = key * G + g
    vs = (((key >> 4) * 4 + (key >> 2 & 3)) * G + g) * 4 + (key & 3)
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=device)
    return kc, 16 * D + vc, 32 * D + ks, 33 * D + vs, table


def _values(codes, scales, table):
    """Values in 32 bits of code bytes [..., D / 2] and scale bytes [..., G]."""
    b = codes.int()
    v = table[torch.stack((b & 15, b >> 4), -1)].flatten(-2).unflatten(-1, (-1, 32))
    e = scales.int()
    s = torch.where(e == 255, float("nan"), torch.ldexp(torch.ones_like(e, dtype=torch.float32), e - 127))
    return (v * s.unsqueeze(-1)).flatten(-2)


def _unpacked(pages, plan):
    """Keys and values [..., head, 32, D] of page bytes [..., head, 34 D]."""
    kc, vc, ks, vs, table = plan
    return _values(pages[..., kc], pages[..., ks], table), _values(pages[..., vc], pages[..., vs], table)


def _attend(s):
    q, pool, table, lens, scale = s["q"], s["pool"], s["table"], s["lens"], s["scale"]
    B, T, H, D = q.shape
    Hkv = pool.shape[1]
    K, V = _unpacked(pool[table.clamp(min=0).long()], s["plan"])  # [B, P, Hkv, 32, D]
    K, V = (x.transpose(1, 2).flatten(2, 3) for x in (K, V))  # [B, Hkv, n, D]
    n = K.shape[2]
    rows = q.float().view(B, T, Hkv, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    dots = (rows @ K.transpose(-1, -2)).view(B, Hkv, T, H // Hkv, n) * scale
    at, last = torch.arange(n, device=q.device), lens[:, None] - T + torch.arange(T, device=q.device)[None]
    seen = (at[None, None] <= last[:, :, None])[:, None, :, None]  # query t sees the keys up to its own position
    dots = torch.where(seen, dots, float("-inf"))
    most = dots.amax(-1, keepdim=True)
    p = torch.exp(dots - torch.where(most == float("-inf"), 0.0, most)).flatten(2, 3)
    V = torch.where((at[None] < lens[:, None])[:, None, :, None], V, 0.0)
    out = (p @ V) / p.sum(-1, keepdim=True).clamp(min=1e-38)  # a row that sees nothing is zero
    return out.view(B, Hkv, T, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, T, H, D).to(q.dtype)


def _write(pool, slots, k, v, plan):
    kc, vc, ks, vs, _ = plan
    page, key = _keys_first(slots)
    flat, base = pool.view(-1), (page[:, None] * pool.shape[1] + torch.arange(pool.shape[1], device=pool.device)) * pool.shape[2]
    for x, codes_at, scales_at in ((k, kc, ks), (v, vc, vs)):
        code, scale = _quantised(x)
        flat[base[..., None] + codes_at[key][:, None]] = code[..., ::2] | code[..., 1::2] << 4
        flat[base[..., None] + scales_at[key][:, None]] = scale


def _read(pool, slots, dtype, plan):
    kc, vc, ks, vs, table = plan
    page, key = _keys_first(slots)
    base = ((page[:, None] * pool.shape[1] + torch.arange(pool.shape[1], device=pool.device)) * pool.shape[2])[..., None]
    flat = pool.view(-1)
    k = _values(flat[base + kc[key][:, None]], flat[base + ks[key][:, None]], table)
    v = _values(flat[base + vc[key][:, None]], flat[base + vs[key][:, None]], table)
    hole = (slots < 0)[:, None, None]
    return torch.where(hole, 0.0, k).to(dtype), torch.where(hole, 0.0, v).to(dtype)


def _rows(gen, n, heads, D, dtype):
    """Key and value rows as a model gives them: a few key channels stand out, tokens differ in size."""
    dev = gen.device
    out = 1 + 7 * (torch.rand(heads, D, device=dev, generator=gen) > 0.96)
    size = torch.exp(0.4 * torch.randn(n, heads, 1, device=dev, generator=gen))
    k = torch.randn(n, heads, D, device=dev, generator=gen) * out
    v = torch.randn(n, heads, D, device=dev, generator=gen) * size * 0.5
    return k.to(dtype), v.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = gen.device
    if case["kind"] == "pages":
        pool = torch.randint(0, 256, (case["layers"], case["npages"], case["page"]), device=dev, generator=gen, dtype=torch.uint8)
        order = torch.randperm(case["npages"], device=dev, generator=gen)
        n = case["n"]
        source = order[:n]
        source = torch.where(torch.arange(n, device=dev) % 5 == 4, source.roll(1), source)  # some pages fork twice
        return dict(case, pool=pool, pairs=torch.stack((source, order[n:2 * n]), 1).int().contiguous())
    Hkv, D, B = case["Hkv"], case["D"], case["B"]
    lens = _lengths(case)
    used = [-(-n // PAGE) for n in lens]
    npages = sum(used) + 3
    order = torch.randperm(npages, device=dev, generator=gen).int()
    # the pool as earlier steps left it: every page filled, so stale rows lie behind each last token
    pool = torch.empty(npages, Hkv, 34 * D, device=dev, dtype=torch.uint8)
    k, v = _rows(gen, npages * PAGE, Hkv, D, torch.bfloat16)
    plan, step = _plan(D, dev), 1 << 17
    for i in range(0, npages * PAGE, step):
        at = torch.arange(i, min(i + step, npages * PAGE), device=dev, dtype=torch.int32)
        _write(pool, at, k[i:i + step], v[i:i + step], plan)
    del k, v
    width = max(used) + case.get("spare", 0)
    counts, cols = torch.tensor(used, device=dev)[:, None], torch.arange(width, device=dev)[None]
    first = counts.cumsum(0) - counts
    table = torch.where(cols < counts, order[(first + cols).clamp(max=npages - 1)], -1).int().contiguous()
    lens_t = torch.tensor(lens, device=dev, dtype=torch.int32)
    if case["kind"] == "attend":
        q = torch.randn(B, case["T"], case["H"], D, device=dev, generator=gen).to(torch.bfloat16)
        return dict(case, plan=plan, q=q, pool=pool, table=table, lens=lens_t, scale=D ** -0.5, out=torch.empty_like(q),
                    workspace=torch.zeros(WORKSPACE, device=dev, dtype=torch.uint8))
    dtype = torch.float32 if case["f32"] else torch.bfloat16
    at = torch.arange(max(lens), device=dev)[None]
    slots = table.gather(1, (at // PAGE).expand(B, -1)) * PAGE + at % PAGE
    here = at < lens_t[:, None]
    rows = slots[here].int().contiguous()  # every row of every request
    s = dict(case, plan=plan, pool=pool, rows=rows, back_k=torch.empty(len(rows), Hkv, D, device=dev, dtype=dtype),
             back_v=torch.empty(len(rows), Hkv, D, device=dev, dtype=dtype))
    if case["kind"] == "gather":
        s["rows"][6::7] = -1  # holes: rows that the caller keeps elsewhere
        return s
    new = here & (at >= lens_t[:, None] - case["T"])  # the last T rows of each request are the new ones
    s["slots"] = slots[new].int().contiguous()
    s["k"], s["v"] = _rows(gen, len(s["slots"]), Hkv, D, dtype)
    return s


def run(s):
    if own:
        from persistent_micro_dispatch_gb300 import gpuos, kv4

        stream = torch.cuda.current_stream().cuda_stream
        if s["kind"] == "attend":
            gpuos.eager_run(kv4.sdpa(s["q"], s["pool"], s["table"], s["lens"], s["out"], s["workspace"], s["scale"]), stream)
            return s["out"]
        if s["kind"] == "pages":
            gpuos.eager_run(kv4.page_copy(s["pool"], s["pairs"]), stream)
            return s["pool"]
        if s["kind"] == "append":
            gpuos.eager_run(kv4.write(s["k"], s["v"], s["slots"], s["pool"]), stream)
        gpuos.eager_run(kv4.read(s["pool"], s["rows"], s["back_k"], s["back_v"]), stream)
        return s["back_k"], s["back_v"]
    if s["kind"] == "attend":
        return _attend(s)
    if s["kind"] == "pages":
        pairs = s["pairs"].long()
        s["pool"][:, pairs[:, 1]] = s["pool"][:, pairs[:, 0]]
        return s["pool"]
    if s["kind"] == "append":
        _write(s["pool"], s["slots"], s["k"], s["v"], s["plan"])
    return _read(s["pool"], s["rows"], s["back_k"].dtype, s["plan"])


def work(case):
    if case["kind"] == "pages":
        sources = len(set(i - 1 if i % 5 == 4 else i for i in range(case["n"])))
        return {"bytes": case["layers"] * (sources + case["n"]) * case["page"], "flops": 0}
    lens, Hkv, D = _lengths(case), case["Hkv"], case["D"]
    row = Hkv * (D + D // 16)  # a token's codes and scales, keys and values
    if case["kind"] == "attend":
        B, T, H = case["B"], case["T"], case["H"]
        pages = sum(-(-n // PAGE) for n in lens)
        return {"bytes": sum(lens) * row + 4 * B * T * H * D + 4 * pages + 4 * B, "flops": 4 * sum(lens) * T * H * D}
    size = 4 if case["f32"] else 2
    back = sum(lens) * (4 + 2 * Hkv * D * size)
    if case["kind"] == "gather":
        return {"bytes": sum(lens) * row * 6 // 7 + back, "flops": 0}
    new = sum(min(n, case["T"]) for n in lens)
    # new rows are read, their codes written; old codes are read, every row is written in full
    return {"bytes": new * (4 + 2 * Hkv * D * size) + sum(lens) * row + back, "flops": 0}


def exact(case, seed):
    """From the definitions, in 64 bits: each request by itself, code by code."""
    s = prepare(case, seed)
    if case["kind"] == "pages":
        pool = s["pool"]
        was = pool.clone()
        for src, dst in s["pairs"].tolist():
            pool[:, dst] = was[:, src]
        return pool
    D, Hkv, pool = case["D"], case["Hkv"], s["pool"]
    G, dev = D // 32, pool.device
    ch = torch.arange(D, device=dev)

    def held(slots, head):
        """The keys and values of one head at these slots, decoded nibble by nibble."""
        blob, key = pool[(slots // PAGE).long(), head], (slots % PAGE).long()[:, None]
        grp, c = ch // 32, ch % 32
        tile, quad, r = key // 16, key % 16 // 4, key % 4
        lane_k = (quad * 2 + r % 2) * 4 + c // 8
        lane_v = c // 4 * 4 + quad
        at_k = tile * 8 * D + lane_k * 8 * G + r // 2 * 4 * G + grp * 4 + c % 8 // 2
        at_v = 16 * D + tile * 8 * D + lane_v * 8 * G + r * 2 * G + grp * 2 + c % 4 // 2
        at_ks = 32 * D + key * G + grp
        at_vs = 33 * D + tile * 16 * G + quad * 4 * G + grp * 4 + r
        got = []
        for at, sc in ((at_k, at_ks), (at_v, at_vs)):
            code = blob.gather(1, at).long() >> 4 * (c % 2) & 15
            two, one = (code >> 1 & 3).double(), (code & 1).double()
            size = torch.where(two == 0, one / 2, (1 + one / 2) * torch.exp2(two - 1))
            e = blob.gather(1, sc).double()
            got.append(torch.where(e == 255, float("nan"), torch.where(code > 7, -size, size) * torch.exp2(e - 127)))
        return got

    if case["kind"] == "attend":
        B, T, H = case["B"], case["T"], case["H"]
        if sum(_lengths(case)) * Hkv > 6_000_000:
            return None
        g, out = H // Hkv, torch.zeros(B, T, H, D, device=dev, dtype=torch.float64)
        for b, n in enumerate(_lengths(case)):
            at = torch.arange(n, device=dev)
            slots = s["table"][b].long()[at // PAGE] * PAGE + at % PAGE
            for h in range(Hkv if n else 0):
                k, v = held(slots, h)
                for t in range(max(0, T - n), T):
                    m = n - T + t + 1
                    x = s["q"][b, t, h * g:h * g + g].double() @ k[:m].T * s["scale"]
                    out[b, t, h * g:h * g + g] = torch.softmax(x, -1) @ v[:m]
        return out

    def rounded(x):
        """The values that the cache holds of rows x: nearest of sixteen, ties to the even code."""
        x = x.double().unflatten(-1, (G, 32))
        top = x.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(top / 6))
        e = torch.where(top > 6 * torch.exp2(e), e + 1, torch.where(top <= 6 * torch.exp2(e - 1), e - 1, e)).clamp(-127, 125)
        y, values = x.abs() / torch.exp2(e), torch.tensor(MAGNITUDES, device=dev, dtype=torch.float64)
        hi = torch.searchsorted(values, y.contiguous()).clamp(max=7)
        lo = (hi - 1).clamp(min=0)
        up, down = values[hi] - y, y - values[lo]
        code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        return (torch.sign(x) * values[code] * torch.exp2(e)).flatten(-2)

    back = [torch.zeros(len(s["rows"]), Hkv, D, device=dev, dtype=torch.float64) for _ in range(2)]
    here = (s["rows"] >= 0).nonzero()[:, 0]
    for i in here.split(1 << 15):
        for h in range(Hkv):
            for x, y in zip(back, held(s["rows"][i], h)):
                x[i, h] = y
    if case["kind"] == "append":
        order = torch.argsort(s["rows"])
        at = order[torch.searchsorted(s["rows"][order], s["slots"])]
        for x, new in zip(back, (s["k"], s["v"])):
            for i in range(0, len(at), 1 << 15):
                x[at[i:i + (1 << 15)]] = rounded(new[i:i + (1 << 15)])
    return tuple(back)
