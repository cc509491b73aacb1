"""What a decode step chooses: its operators in plain form, and the calls a user makes of them.

Four kinds of case:

  "adjust"   logits [B, V] before a token is chosen: penalties for the tokens that a request has had, biases for listed
             tokens, a temperature, a grammar's mask
  "top"      the K best tokens of each row with their log-probabilities, and the row's log-sum-exp
  "experts"  router logits [N, E] -> the K experts of each token and their weights
  "plan"     the pairs (token, expert) in the experts' order, as the experts' products take them: a stable counting sort

Settings of a request are eight words of 32 bits (int32 [B, 8]): repetition, presence and frequency penalty and
temperature as float32, then the prompt's tokens, all tokens, the row of the mask (-1: none) and the listed biases.
Biases are pairs of words (int32 [B, n, 2]): a token and a float32. A mask is a bit for each token (int32 [M, V / 32]),
token v at bit v % 32 of word v / 32; 1 allows it.
"""
import random

import torch

own = False


def listed():
    return [
        # one user's chat turn with a grammar: latency is all
        dict(name="adjust_one", kind="adjust", B=1, V=128000, pad=0, f32=False, lo=900, hi=900, biases=4, masks=1),
        # a full server's batch, logits in 32 bits: the largest
        dict(name="adjust_batch", kind="adjust", B=256, V=128000, pad=0, f32=True, lo=100, hi=4000, biases=16, masks=16),
        # a vocabulary of odd size, whose rows the last product has padded
        dict(name="adjust_odd", kind="adjust", B=33, V=50001, pad=47, f32=False, lo=1, hi=2000, biases=3, masks=3),
        # long documents: the tokens so far outnumber the vocabulary
        dict(name="adjust_long", kind="adjust", B=8, V=32000, pad=0, f32=False, lo=20000, hi=131071, biases=0, masks=0),
        # greedy choice for one request
        dict(name="top_greedy", kind="top", B=1, V=32000, pad=0, f32=True, K=1),
        # twenty log-probabilities for each request of a batch
        dict(name="top_batch", kind="top", B=64, V=128000, pad=0, f32=False, K=20),
        # a prompt is scored: a row for each of its tokens
        dict(name="top_score", kind="top", B=509, V=128000, pad=0, f32=True, K=5),
        # the router of one decode step of 64 requests: sigmoid scores, balance bias, eight groups of which four
        dict(name="experts_step", kind="experts", N=64, E=256, pad=0, K=8, sigmoid=True, bias=True, groups=8, keep=4, two=True, f32=True),
        # a small router over a ragged batch
        dict(name="experts_odd", kind="experts", N=5001, E=60, pad=4, K=4, sigmoid=False, bias=False, groups=1, keep=1, two=False, f32=False),
        # the router of a long prompt
        dict(name="experts_prompt", kind="experts", N=32768, E=256, pad=0, K=8, sigmoid=True, bias=True, groups=8, keep=4, two=True, f32=True),
        # the pairs of that prompt
        dict(name="plan_prompt", kind="plan", N=32768, E=256, K=8, absent=7),
        # the pairs of that step
        dict(name="plan_step", kind="plan", N=64, E=256, K=8, absent=0),
    ]


def draw(rng):
    def spread(lo, hi):
        return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))

    kind = rng.choice(["adjust", "adjust", "top", "top", "experts", "experts", "plan"])
    f32 = rng.random() < 0.5
    if kind in ("adjust", "top"):
        V = rng.choice([32000, 50001, 65536, 100003, 128000, spread(1000, 262144)])
        B, pad = spread(1, 512), rng.choice([0, 0, 1, 24, 64])
        while B * V * (2 if f32 else 1) > 500 * 128000:
            B = max(1, B * 2 // 3)
        if kind == "top":
            return dict(kind=kind, B=B, V=V, pad=pad, f32=f32, K=rng.choice([1, 1, 5, 8, 20, spread(1, 64)]))
        hi = spread(1, 131072)
        while B * hi > 1 << 20:
            hi = max(1, hi // 2)
        return dict(kind=kind, B=B, V=V, pad=pad, f32=f32, lo=spread(1, hi), hi=hi, biases=rng.choice([0, 3, spread(1, 100)]), masks=rng.choice([0, 1, 5]))
    E = rng.choice([8, 16, 60, 64, 128, 160, 256, 256, 384, 512])
    K = rng.choice([k for k in (1, 2, 4, 6, 8, 8, 10) if k <= E // 2])
    N = spread(1, 32768 * 256 // max(E, 256))
    if kind == "plan":
        return dict(kind=kind, N=N, E=E, K=K, absent=rng.choice([0, 0, 5]))
    groups = rng.choice([1, 1] + [g for g in (2, 4, 8) if E % g == 0 and E // g >= 2])
    keep = rng.randint(1, groups)
    while keep * (E // groups) < K:
        keep += 1
    return dict(kind=kind, N=N, E=E, pad=rng.choice([0, 0, 4, 1]), K=K, sigmoid=rng.random() < 0.5, bias=rng.random() < 0.5, groups=groups, keep=keep,
                two=groups > 1 and rng.random() < 0.5, f32=f32)


# ---- the inputs


def _lengths(case):
    """The requests' tokens so far: they belong to the case, whatever the seed. The most are the first's."""
    rng = random.Random(case["B"] * 1000003 + case["hi"])
    return [case["hi"]] + [round(case["lo"] * (case["hi"] / case["lo"]) ** rng.random()) for _ in range(case["B"] - 1)]


def _mask_rows(case):
    """The mask row of each request: one in four has none where there are several requests."""
    return [-1 if not case["masks"] or b % 4 == 3 else b % case["masks"] for b in range(case["B"])]


def _padded(rows, n, pad, gen, f32, size):
    """Logits [rows, n] in rows of n + pad, as the product before leaves them."""
    x = torch.randn(rows, n + pad, device=gen.device, generator=gen) * size
    return (x if f32 else x.to(torch.bfloat16))[:, :n]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = gen.device
    if case["kind"] == "plan":
        N, E, K = case["N"], case["E"], case["K"]
        # a few experts are asked for more often, as routers do
        ids = (torch.rand(N, E, device=dev, generator=gen) + 0.3 * torch.rand(E, device=dev, generator=gen)).topk(K).indices.int()
        if case["absent"]:
            ids[N - N // case["absent"]:] = -1  # a padded batch: its last tokens have no experts
        P = N * K
        return dict(case, ids=ids, order=torch.empty(P, device=dev, dtype=torch.int32), place=torch.empty(N, K, device=dev, dtype=torch.int32),
                    offsets=torch.empty(E + 1, device=dev, dtype=torch.int32), workspace=torch.zeros(4 << 20, device=dev, dtype=torch.uint8))
    if case["kind"] == "experts":
        N, E, K = case["N"], case["E"], case["K"]
        x = _padded(N, E, case["pad"], gen, case["f32"], 1.5)
        bias = 0.05 * torch.randn(E, device=dev, generator=gen) if case["bias"] else None
        return dict(case, logits=x, balance=bias, ids=torch.empty(N, K, device=dev, dtype=torch.int32), weights=torch.empty(N, K, device=dev))
    B, V = case["B"], case["V"]
    x = _padded(B, V, case["pad"], gen, case["f32"], 3.0)
    if case["kind"] == "top":
        K = case["K"]
        return dict(case, logits=x, ids=torch.empty(B, K, device=dev, dtype=torch.int32), logprobs=torch.empty(B, K, device=dev),
                    lse=torch.empty(B, device=dev), workspace=torch.zeros(4 << 20, device=dev, dtype=torch.uint8))
    lens = torch.tensor(_lengths(case), device=dev)
    settings = torch.zeros(B, 8, device=dev, dtype=torch.int32)
    some = torch.rand(B, 4, device=dev, generator=gen)
    # repetition 1 to 1.3, presence and frequency 0 to 0.5, temperature 0.5 to 1.5
    settings[:, :4] = torch.stack((1 + 0.3 * some[:, 0], 0.5 * some[:, 1], 0.5 * some[:, 2], 0.5 + some[:, 3]), 1).view(torch.int32)
    settings[:, 4] = lens // 2
    settings[:, 5] = lens
    settings[:, 6] = torch.tensor(_mask_rows(case), device=dev)
    settings[:, 7] = case["biases"]
    # tokens come back as in text: a few often, most never
    tokens = (V * torch.rand(B, case["hi"], device=dev, generator=gen) ** 4).int().clamp(max=V - 1)
    bias = mask = None
    if case["biases"]:
        n = case["biases"]
        first = torch.randint(0, V, (B, 1), device=dev, generator=gen)
        value = 4 * torch.randn(B, n, device=dev, generator=gen)
        bias = torch.stack((((first + torch.arange(n, device=dev) * 7) % V).int(), value.view(torch.int32)), -1).contiguous()
    if case["masks"]:
        words = (case["masks"], -(-V // 32))
        mask = torch.randint(-1 << 31, 1 << 31, words, device=dev, generator=gen).int()
        # every second grammar allows little, as within a name or a number
        tight = torch.randint(-1 << 31, 1 << 31, words, device=dev, generator=gen).int() & (torch.rand(words, device=dev, generator=gen) < 0.02)
        mask[1::2] = tight[1::2]
    out = torch.empty(B, V, device=dev, dtype=x.dtype)
    return dict(case, logits=x, out=out, settings=settings, tokens=tokens, bias_pairs=bias, mask=mask)


# ---- the plain forms


def _adjust(s):
    x, V = s["logits"].float(), s["V"]
    p = s["settings"]
    rep, presence, frequency, temperature = p[:, :4].contiguous().view(torch.float32)[:, :, None].unbind(1)
    at = torch.arange(s["tokens"].shape[1], device=x.device)
    here = at < p[:, 5:6]
    tokens = s["tokens"].long()
    nowhere = torch.zeros(x.shape[0], V + 1, device=x.device)
    had = nowhere.scatter(1, torch.where(here, tokens, V), 1.0)[:, :V] > 0
    count = nowhere.scatter_add(1, torch.where(here & (at >= p[:, 4:5]), tokens, V), torch.ones_like(tokens, dtype=torch.float32))[:, :V]
    y = torch.where(had, torch.where(x > 0, x / rep, x * rep), x)
    y = y - torch.where(count > 0, frequency * count + presence, 0.0)
    if s["bias_pairs"] is not None:
        pairs = s["bias_pairs"]
        listed_here = torch.arange(pairs.shape[1], device=x.device) < p[:, 7:8]
        y = y + nowhere.scatter(1, torch.where(listed_here, pairs[:, :, 0].long(), V), pairs[:, :, 1].contiguous().view(torch.float32))[:, :V]
    y = y / temperature
    if s["mask"] is not None:
        v = torch.arange(V, device=x.device)
        row = p[:, 6]
        allowed = (s["mask"][row.clamp(min=0).long()][:, v // 32] >> (v % 32).int()) & 1
        y = torch.where((allowed == 1) | (row < 0)[:, None], y, float("-inf"))
    return y.to(s["logits"].dtype)


def _top(s):
    x = s["logits"].float()
    value, at = torch.sort(x, dim=1, descending=True, stable=True)  # of equal values the lowest token first
    most = value[:, :1]
    total = torch.exp(x - most).sum(1, keepdim=True)
    return at[:, :s["K"]].int(), value[:, :s["K"]] - most - torch.log(total), (most + torch.log(total))[:, 0]


def _experts(s):
    x = s["logits"].double()  # which experts are chosen hangs on differences of neighbouring scores
    if s["sigmoid"]:
        score = 1 / (1 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    choice = score if s["balance"] is None else score + s["balance"]
    if s["groups"] > 1:
        g = choice.unflatten(1, (s["groups"], -1))
        best = torch.sort(g, dim=2, descending=True).values
        value = best[:, :, 0] + best[:, :, 1] if s["two"] else best[:, :, 0]
        kept = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :s["keep"]]
        shut = torch.ones_like(value).scatter(1, kept, 0.0)
        choice = torch.where(shut.unsqueeze(2) > 0, float("-inf"), g).flatten(1)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :s["K"]]
    w = score.gather(1, ids)
    return ids.int(), (w / w.sum(1, keepdim=True) * 2.5).float()


def _plan(s):
    ids, E = s["ids"].flatten().long(), s["E"]
    here = (ids >= 0) & (ids < E)
    key = torch.where(here, ids, E)
    order = torch.sort(key, stable=True).indices
    count = torch.zeros(E + 1, device=ids.device, dtype=torch.int64).scatter_add(0, key, torch.ones_like(key))
    offsets = torch.cat((count.new_zeros(1), count[:E].cumsum(0)))
    at = torch.arange(len(ids), device=ids.device)
    place = torch.empty_like(order).scatter(0, order, at)
    return torch.where(at < offsets[E], order, -1).int(), torch.where(here, place, -1).int().view_as(s["ids"]), offsets.int()


def run(s):
    if own:
        from persistent_micro_dispatch_gb300 import choose, gpuos

        stream = torch.cuda.current_stream().cuda_stream
        if s["kind"] == "adjust":
            gpuos.eager_run(choose.adjust(s["logits"], s["out"], s["settings"], tokens=s["tokens"], bias=s["bias_pairs"], mask=s["mask"]), stream)
            return s["out"]
        if s["kind"] == "top":
            gpuos.eager_run(choose.top(s["logits"], s["ids"], s["logprobs"], s["lse"], s["workspace"]), stream)
            return s["ids"], s["logprobs"], s["lse"]
        if s["kind"] == "experts":
            gpuos.eager_run(choose.experts(s["logits"], s["ids"], s["weights"], sigmoid=s["sigmoid"], bias=s["balance"], groups=s["groups"],
                                           keep=s["keep"], top2=s["two"], scale=2.5), stream)
            return s["ids"], s["weights"]
        gpuos.eager_run(choose.plan(s["ids"], s["order"], s["place"], s["offsets"], s["workspace"]), stream)
        return s["order"], s["place"], s["offsets"]
    return {"adjust": _adjust, "top": _top, "experts": _experts, "plan": _plan}[s["kind"]](s)


def work(case):
    if case["kind"] == "plan":
        P = case["N"] * case["K"]
        return {"bytes": 12 * P + 4 * case["E"] + 4, "flops": 0}
    size = 4 if case["f32"] else 2
    if case["kind"] == "experts":
        N, E, K = case["N"], case["E"], case["K"]
        return {"bytes": N * E * size + 8 * N * K + (4 * E if case["bias"] else 0), "flops": 4 * N * E}
    B, V = case["B"], case["V"]
    if case["kind"] == "top":
        return {"bytes": B * V * size + 8 * B * case["K"] + 4 * B, "flops": 4 * B * V}
    masks = len(set(r for r in _mask_rows(case) if r >= 0)) * -(-V // 32) * 4
    return {"bytes": 2 * B * V * size + 4 * sum(_lengths(case)) + 8 * B * case["biases"] + 32 * B + masks, "flops": 6 * B * V}


def exact(case, seed):
    """From the definitions, in 64 bits. What is a whole number has no such value."""
    s = prepare(case, seed)
    if case["kind"] == "plan":
        return None
    x = s["logits"].double()
    if case["kind"] == "top":
        lse = torch.logsumexp(x, 1)
        return None, x.topk(case["K"]).values - lse[:, None], lse
    if case["kind"] == "experts":
        score = torch.sigmoid(x) if case["sigmoid"] else torch.softmax(x, 1)
        c = score.clone() if s["balance"] is None else score + s["balance"].double()
        N, E, G = case["N"], case["E"], case["groups"]
        parts = c.view(N, G, E // G)
        value = parts.topk(2, dim=2).values.sum(2) if case["two"] else parts.amax(2)
        floor = value.topk(case["keep"], dim=1).values[:, -1:]
        parts[value < floor] = -float("inf")
        w = score.gather(1, c.topk(case["K"]).indices)
        return None, 2.5 * w / w.sum(1, keepdim=True)
    V, out = case["V"], []
    words = s["settings"].cpu()
    numbers = words.view(torch.float32).double()
    word, bit = torch.arange(V, device=x.device) // 32, 1 << torch.arange(V, device=x.device) % 32
    for b in range(case["B"]):
        rep, presence, frequency, temperature = numbers[b, :4].tolist()
        prompt, length, row, biases = words[b, 4:].tolist()
        had = torch.bincount(s["tokens"][b, :length], minlength=V)
        count = torch.bincount(s["tokens"][b, prompt:length], minlength=V).double()
        y = x[b]
        y = torch.where(had > 0, torch.where(y > 0, y / rep, y * rep), y) - frequency * count - presence * (count > 0)
        if biases:
            pairs = s["bias_pairs"][b]
            y[pairs[:, 0].long()] += pairs[:, 1].contiguous().view(torch.float32).double()
        y = y / temperature
        if row >= 0:
            y[(s["mask"][row].long()[word] & bit) == 0] = -float("inf")
        out.append(y)
    return torch.stack(out)
