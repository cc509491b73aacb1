/*
 * What a decode step chooses (included by gpuos_device.cu, whose memory, bf16
 * and staging helpers it uses): logits adjusted for the next token, the best
 * tokens of a row, the experts of a token, and the experts' order.
 *
 * Each op has a body for one warp (a tile of the executor), first, and kernels
 * of its own for launches, behind them. Everything is bound by memory or by
 * latency; there are no products of matrices. The bodies need no shared memory,
 * and use the warp's staging buffer for counters where there is one.
 *
 * Times are of one GB300 (measured copy bandwidth 6.8 TB/s), device time of
 * launches one after another in a CUDA graph, unless they say executor (there:
 * first tile to done).
 */
#ifndef GPUOS_CHOOSE_CUH
#define GPUOS_CHOOSE_CUH

#define GPUOS_FULL 0xFFFFFFFFu

/* A row of f32 or bf16 elements, seen from the last 16-byte boundary at or
 * before it: element i of the row has place i + lo, places that are multiples
 * of eight begin 16-byte vectors, and only places in [lo, hi) are read. */
template <bool F32>
struct ChooseRow {
    uint64_t base;
    uint32_t lo, hi;
    DEV ChooseRow(uint64_t a, uint32_t row, uint32_t ld, uint32_t n)
    {
        const uint64_t p = a + (uint64_t)row * ld * (F32 ? 4u : 2u);
        lo = (uint32_t)(p & 15u) / (F32 ? 4u : 2u);
        hi = lo + n;
        base = p & ~15ull;
    }
    DEV const uint4 *vec(uint32_t at) const { return reinterpret_cast<const uint4 *>(base + (uint64_t)at * (F32 ? 4u : 2u)); }
    DEV float one(uint32_t at) const
    {
        if (F32) return __ldcg(reinterpret_cast<const float *>(base) + at);
        return bf1(__ldcg(reinterpret_cast<const uint16_t *>(base) + at));
    }
    DEV void put(uint32_t at, float x) const
    {
        if (F32) __stcg(reinterpret_cast<float *>(base) + at, x);
        else __stcg(reinterpret_cast<uint16_t *>(base) + at, to_bf(x));
    }
};
/* Eight elements from place `at` (a multiple of eight); `none` outside [lo, hi). */
template <bool F32>
DEV void choose_load8(const ChooseRow<F32> &r, uint32_t at, uint32_t lo, uint32_t hi, float none, float (&x)[8])
{
    if (at >= lo && at + 8u <= hi) {
        if (F32) {
            const uint4 a = __ldcg(r.vec(at)), b = __ldcg(r.vec(at) + 1);
            x[0] = __uint_as_float(a.x), x[1] = __uint_as_float(a.y), x[2] = __uint_as_float(a.z), x[3] = __uint_as_float(a.w);
            x[4] = __uint_as_float(b.x), x[5] = __uint_as_float(b.y), x[6] = __uint_as_float(b.z), x[7] = __uint_as_float(b.w);
        } else {
            unpack8(__ldcg(r.vec(at)), x);
        }
    } else {
#pragma unroll
        for (uint32_t j = 0; j < 8; j++) x[j] = at + j >= lo && at + j < hi ? r.one(at + j) : none;
    }
}

/* A float's place in the order of the floats, as a whole number (-0 as +0;
 * not for NaN): 0 is below every float's. */
DEV uint32_t choose_key(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
/* e^x for x <= 80 (-infinity included; exp_ex2 takes no larger arguments either way). */
DEV float choose_exp(float x) { return exp_ex2(fmaxf(x, -200.0f)); }
/* The largest of three in one instruction; a NaN is passed over. */
DEV float choose_max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
DEV float choose_unkey(uint32_t k) { return __uint_as_float(k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u)); }

/* ---------------------------------------------------------------------------
 * Logits adjusted. One pass: each logit is read once and written once, so it
 * is bound by memory; what a token's penalty needs, its count among the
 * request's tokens, comes from counters of the tile's window of the
 * vocabulary in shared memory, filled by one look at the request's tokens.
 * A counter holds the count after the prompt and two flags. Executor: one
 * request over 128,000 tokens 21 us, 256 of them (f32) 131; a request's 100,000
 * tokens are one warp's work in each tile, 200 us.
 * ------------------------------------------------------------------------- */
#define GPUOS_ADJUST_HAD 0x80000000u    /* in the prompt */
#define GPUOS_ADJUST_LISTED 0x40000000u /* has a bias: written after the others */
#define GPUOS_ADJUST_COUNT 0x3FFFFFFFu

struct AdjustArgs {
    gpuos_logits_request q;
    const int32_t *tokens;
    const uint32_t *mask; /* its row; null: none */
    const int2 *bias;
    /* divided by the temperature: 1, 1 / repetition, repetition, frequency, presence */
    float plain, above, below, frequency, presence;
    bool penal;
};
/* The settings of request b; false if its record does not fit. */
DEV bool adjust_args(const gpuos_devdesc *d, uint32_t b, AdjustArgs &a)
{
    const uint32_t V = d->dims[1], Lcap = d->dims[4], M = d->dims[5] & 0xFFFFu, Nb = d->dims[5] >> 16;
    const uint4 *rq = reinterpret_cast<const uint4 *>(d->aux0) + (uint64_t)b * 2u;
    const uint4 r0 = __ldcg(rq), r1 = __ldcg(rq + 1);
    a.q.repetition = __uint_as_float(r0.x);
    a.q.presence = __uint_as_float(r0.y);
    a.q.frequency = __uint_as_float(r0.z);
    a.q.temperature = __uint_as_float(r0.w);
    a.q.prompt = (int32_t)r1.x;
    a.q.length = (int32_t)r1.y;
    a.q.mask = (int32_t)r1.z;
    a.q.biases = (int32_t)r1.w;
    a.tokens = reinterpret_cast<const int32_t *>(d->b) + (uint64_t)b * Lcap;
    a.bias = reinterpret_cast<const int2 *>(d->aux2) + (uint64_t)b * Nb;
    a.mask = a.q.mask < 0 ? nullptr : reinterpret_cast<const uint32_t *>(d->aux1) + (uint64_t)(uint32_t)a.q.mask * ((V + 31u) / 32u);
    a.plain = a.q.temperature > 0.0f ? rcp_approx(a.q.temperature) : 1.0f;
    a.above = a.plain * rcp_approx(a.q.repetition);
    a.below = a.plain * a.q.repetition;
    a.frequency = a.plain * a.q.frequency;
    a.presence = a.plain * a.q.presence;
    a.penal = a.q.length > 0 && !(a.q.repetition == 1.0f && a.q.presence == 0.0f && a.q.frequency == 0.0f);
    return (uint32_t)a.q.length <= Lcap && (uint32_t)a.q.prompt <= (uint32_t)a.q.length && (a.q.mask < 0 || (uint32_t)a.q.mask < M) &&
           (uint32_t)a.q.biases <= Nb;
}
/* x under a token's counter, divided by the temperature: a factor for each
 * request and side, and one multiply-add. (The factors are off by 5 x 2^-24 at
 * most, two hardware reciprocals of 2^-23 and a product; divisions would be ten
 * times the code, for each thread.) */
DEV float adjust_penalty(const AdjustArgs &a, float x, uint32_t w)
{
    const uint32_t c = w & GPUOS_ADJUST_COUNT;
    const float f = w & (GPUOS_ADJUST_COUNT | GPUOS_ADJUST_HAD) ? (x > 0.0f ? a.above : a.below) : a.plain;
    return fmaf(x, f, c ? -fmaf(a.frequency, (float)c, a.presence) : 0.0f);
}
/* The mask's bits of eight tokens from v (some of which may lie outside the
 * vocabulary); all ones without a mask. */
DEV uint32_t adjust_bits(const AdjustArgs &a, int32_t v, uint32_t V)
{
    if (!a.mask) return 0xFFu;
    const int32_t w = v >> 5; /* -1 for v < 0 */
    const uint32_t words = (V + 31u) / 32u;
    const uint32_t lo = w >= 0 ? __ldcg(a.mask + w) : 0u;
    const uint32_t hi = (v & 31) > 24 && (uint32_t)(w + 1) < words ? __ldcg(a.mask + w + 1) : 0u;
    return __funnelshift_r(lo, hi, (uint32_t)v & 31u);
}
DEV bool adjust_allowed(const AdjustArgs &a, uint32_t v) { return !a.mask || (__ldcg(a.mask + (v >> 5)) >> (v & 31u) & 1u); }
/* Each lane's entry i, of this token, is listed again behind it: the later
 * entry counts. Every lane of the warp. */
DEV bool adjust_again(const AdjustArgs &a, uint32_t i, int32_t token)
{
    const uint32_t n = (uint32_t)a.q.biases;
    bool again = false;
#pragma unroll 1
    for (uint32_t k0 = i & ~31u; k0 < n; k0 += 32) {
        const int32_t t = k0 + lane_id() < n ? __ldcg(&a.bias[k0 + lane_id()].x) : -1;
#pragma unroll 1
        for (uint32_t k = 0; k < 32 && k0 + k < n; k++) again |= __shfl_sync(GPUOS_FULL, t, (int)k) == token && k0 + k > i;
    }
    return again;
}

/* One warp's tile: GPUOS_ADJUST_CHUNK places of one row. */
template <bool F32>
DEV int adjust_tile(const gpuos_devdesc *d, uint32_t tile)
{
    const uint32_t V = d->dims[1], chunks = gpuos_adjust_chunks(V), lane = lane_id();
    const uint32_t b = tile / chunks;
    if (b >= d->dims[0]) return GPUOS_ST_OK;
    AdjustArgs a;
    if (!adjust_args(d, b, a)) return GPUOS_ST_BAD_ARGS;
    /* places go by the output's alignment: its stores are whole vectors */
    const ChooseRow<F32> in(d->a, b, d->dims[2], V), out(d->out, b, d->dims[3], V);
    const int32_t shift = (int32_t)in.lo - (int32_t)out.lo;
    const uint32_t from = (tile - b * chunks) * GPUOS_ADJUST_CHUNK;
    const uint32_t lo = max(from, out.lo), hi = min(from + GPUOS_ADJUST_CHUNK, out.hi);
    if (lo >= hi) return GPUOS_ST_OK;
    const uint32_t room = min(stage_hdr()->stage_bytes / 4u, (uint32_t)GPUOS_ADJUST_CHUNK);
    const bool counted = a.penal || a.q.biases > 0;
    /* without staging, counters of 256 places in registers, eight a lane */
    const uint32_t window = !counted ? GPUOS_ADJUST_CHUNK : (room ? room : 256u);
    uint32_t *ctr = reinterpret_cast<uint32_t *>(warp_stage_buf());
#pragma unroll 1
    for (uint32_t w0 = from; w0 < hi; w0 += window) {
        const uint32_t w1 = min(w0 + window, hi);
        uint32_t mine[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        auto mark = [&](int32_t token, bool here, uint32_t prompt) { /* every lane */
            const uint32_t at = (uint32_t)token + out.lo - w0;
            const bool in_window = here && (uint32_t)token < V && at < w1 - w0;
            if (room) {
                if (in_window) {
                    if (prompt) atomicOr(ctr + at, prompt);
                    else atomicAdd(ctr + at, 1u);
                }
            } else {
                uint32_t left = __ballot_sync(GPUOS_FULL, in_window);
                while (left) {
                    const int src = __ffs((int)left) - 1;
                    left &= left - 1u;
                    const uint32_t k = __shfl_sync(GPUOS_FULL, at, src), f = __shfl_sync(GPUOS_FULL, prompt, src);
#pragma unroll
                    for (uint32_t j = 0; j < 8; j++)
                        if (k == lane * 8u + j) mine[j] = f ? mine[j] | f : mine[j] + 1u;
                }
            }
        };
        if (counted) {
            if (room) {
                for (uint32_t i = lane; i < window; i += 32) ctr[i] = 0u;
                __syncwarp();
            }
            if (a.penal) {
                const uint32_t n = (uint32_t)a.q.length;
#pragma unroll 1
                for (uint32_t i0 = 0; i0 < n; i0 += 32 * 24) { /* (a warp alone: what it waits for is the time) */
                    int32_t t[24];
#pragma unroll
                    for (uint32_t k = 0; k < 24; k++) {
                        const uint32_t i = i0 + k * 32u + lane;
                        t[k] = i < n ? __ldcg(a.tokens + i) : -1;
                    }
#pragma unroll
                    for (uint32_t k = 0; k < 24; k++)
                        mark(t[k], true, i0 + k * 32u + lane < (uint32_t)a.q.prompt ? GPUOS_ADJUST_HAD : 0u);
                }
            }
            for (uint32_t i0 = 0; i0 < (uint32_t)a.q.biases; i0 += 32)
                mark(i0 + lane < (uint32_t)a.q.biases ? __ldcg(&a.bias[i0 + lane].x) : -1, true, GPUOS_ADJUST_LISTED);
            __syncwarp();
        }
        const uint32_t v0 = max(w0, lo);
#pragma unroll 1
        for (uint32_t at = w0 + lane * 8u; at < w1; at += 256u) {
            float x[8];
            if (shift == 0) {
                choose_load8(in, at, v0, w1, 0.0f, x);
            } else {
#pragma unroll
                for (uint32_t j = 0; j < 8; j++) x[j] = at + j >= v0 && at + j < w1 ? in.one(at + j + shift) : 0.0f;
            }
            const uint32_t bits = adjust_bits(a, (int32_t)at - (int32_t)out.lo, V);
            uint32_t skip = 0;
#pragma unroll
            for (uint32_t j = 0; j < 8; j++) {
                uint32_t w = counted ? (room ? ctr[at - w0 + j] : mine[j]) : 0u;
                if (w & GPUOS_ADJUST_LISTED || at + j < v0 || at + j >= w1) skip |= 1u << j;
                x[j] = bits >> j & 1u ? adjust_penalty(a, x[j], w) : -INFINITY;
            }
            if (skip == 0) {
                uint4 *o = const_cast<uint4 *>(out.vec(at));
                if (F32) {
                    __stcg(o, make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])));
                    __stcg(o + 1, make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7])));
                } else {
                    __stcg(o, pack8(x));
                }
            } else {
#pragma unroll
                for (uint32_t j = 0; j < 8; j++)
                    if (!(skip >> j & 1u)) out.put(at + j, x[j]);
            }
        }
        /* listed tokens: left as they were until here (out may be the input) */
#pragma unroll 1
        for (uint32_t i0 = 0; i0 < (uint32_t)a.q.biases; i0 += 32) {
            const uint32_t i = i0 + lane;
            const int2 e = i < (uint32_t)a.q.biases ? __ldcg(a.bias + i) : make_int2(-1, 0);
            const uint32_t at = (uint32_t)e.x + out.lo;
            const bool here = (uint32_t)e.x < V && at >= w0 && at < w1;
            uint32_t w = 0;
            if (room) {
                if (here) w = ctr[at - w0];
            } else {
                const uint32_t k = here ? at - w0 : 0u;
#pragma unroll
                for (uint32_t j = 0; j < 8; j++) {
                    const uint32_t o = __shfl_sync(GPUOS_FULL, mine[j], (int)(k >> 3));
                    if ((k & 7u) == j) w = o;
                }
            }
            if (!__any_sync(GPUOS_FULL, here)) continue;
            const bool again = adjust_again(a, i, e.x); /* (i0 is alike in the lanes, and a multiple of 32) */
            if (here && !again) {
                const float y = fmaf(__int_as_float(e.y), a.plain, adjust_penalty(a, in.one(at + shift), w));
                out.put(at, adjust_allowed(a, (uint32_t)e.x) ? y : -INFINITY);
            }
        }
        __syncwarp();
    }
    return GPUOS_ST_OK;
}
DEV int adjust_op(const gpuos_devdesc *d, uint32_t tile)
{
    const uint32_t *m = d->dims;
    if (m[0] == 0 || m[1] == 0) return GPUOS_ST_OK;
    if (!gpuos_adjust_ok(d->dtype, d->a, d->b, d->out, d->aux0, d->aux1, d->aux2, m) ||
        (uint64_t)m[0] * gpuos_adjust_chunks(m[1]) != d->ntiles)
        return GPUOS_ST_BAD_ARGS;
    const int st = d->dtype == GPUOS_F32 ? adjust_tile<true>(d, tile) : adjust_tile<false>(d, tile);
    /* the counters were written by ordinary stores: the buffer's next user may
     * be an asynchronous copy */
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    return st;
}

/* ---------------------------------------------------------------------------
 * The best tokens of a row, with the row's log-sum-exp. One pass over the row:
 * a warp holds the K best so far in its lanes, in order, and the softmax's
 * running maximum and sum; a group of eight elements whose largest is not above
 * the K-th best costs one comparison. Executor: one row of 32,000, K = 1, 9.7 us;
 * 64 of 128,000 in bf16, K = 20, 86; 509 of 128,000 in f32, K = 5, 176.
 *
 * An entry is one 64-bit number: the value's place among the floats, then the
 * token's from above, so that one comparison orders by value, then by token.
 * 0 stands for no entry.
 * ------------------------------------------------------------------------- */
DEV uint64_t top_entry(float x, uint32_t token) { return (uint64_t)choose_key(x) << 32 | (GPUOS_FULL - token); }
DEV uint64_t shfl64(uint64_t v, int src)
{
    const uint32_t lo = __shfl_sync(GPUOS_FULL, (uint32_t)v, src), hi = __shfl_sync(GPUOS_FULL, (uint32_t)(v >> 32), src);
    return (uint64_t)hi << 32 | lo;
}
template <int KL> /* 32 KL >= K */
struct TopList {
    uint64_t e[KL]; /* lane i: the best but i, but 32 + i */
    uint64_t last;  /* the K-th best, or a lower bound of what will be */
    float floor;    /* its value */
    DEV void clear()
    {
#pragma unroll
        for (int k = 0; k < KL; k++) e[k] = 0;
        last = 0;
        floor = -INFINITY;
    }
    DEV void bound(uint64_t l)
    {
        last = l;
        floor = l >> 32 ? choose_unkey((uint32_t)(l >> 32)) : -INFINITY;
    }
    /* every lane, with the same x > last */
    DEV void insert(uint64_t x, uint32_t K)
    {
        const uint32_t lane = lane_id();
        uint32_t at = (uint32_t)__popc(__ballot_sync(GPUOS_FULL, e[0] > x));
        if (KL > 1) at += (uint32_t)__popc(__ballot_sync(GPUOS_FULL, e[KL - 1] > x));
        const uint64_t carry = KL > 1 ? shfl64(e[0], 31) : 0;
#pragma unroll
        for (int k = 0; k < KL; k++) {
            const uint32_t place = lane + 32u * k;
            uint64_t up = shfl64(e[k], (int)(lane ? lane - 1u : 0u));
            if (k && lane == 0) up = carry;
            if (place > at) e[k] = up;
            if (place == at) e[k] = x;
        }
        const uint64_t l = shfl64(e[KL > 1 && K > 32u ? KL - 1 : 0], (int)((K - 1u) & 31u));
        if (l > last) bound(l);
    }
};
/* The n-th largest (1 <= n <= 32) of the lanes' keys. */
DEV uint32_t top_nth(uint32_t key, uint32_t n)
{
    const uint32_t lane = lane_id();
#pragma unroll
    for (uint32_t size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (uint32_t o = size >> 1; o; o >>= 1) {
            const uint32_t other = __shfl_xor_sync(GPUOS_FULL, key, (int)o);
            const bool down = (lane & size) == 0 || size == 32, first = (lane & o) == 0;
            key = down == first ? max(key, other) : min(key, other);
        }
    return __shfl_sync(GPUOS_FULL, key, (int)(n - 1u));
}

template <int KL>
struct TopState {
    TopList<KL> list;
    float m, s; /* each lane's own */
};
#define GPUOS_TOP_UNIT 4 /* groups of eight elements a lane has in flight */

/* Places [from, to) of a row, `from` a multiple of eight, into the state. */
template <bool F32, int KL>
DEV void top_run(const ChooseRow<F32> &r, uint32_t from, uint32_t to, uint32_t K, TopState<KL> &st)
{
    const uint32_t lane = lane_id(), lo = max(from, r.lo), hi = min(to, r.hi);
    const float none = __int_as_float(0x7FFFFFFF); /* NaN: not an element */
    st.list.clear();
    st.m = -FLT_MAX;
    st.s = 0.0f;
    bool first = true;
#pragma unroll 1
    for (uint32_t u0 = from; u0 < hi; u0 += 256u * GPUOS_TOP_UNIT) {
        float x[GPUOS_TOP_UNIT][8], most[GPUOS_TOP_UNIT], unit = -INFINITY;
#pragma unroll
        for (uint32_t u = 0; u < GPUOS_TOP_UNIT; u++) {
            const uint32_t at = u0 + u * 256u + lane * 8u;
            choose_load8(r, at, lo, hi, none, x[u]);
            if (at >= lo && at + 8u <= hi) { /* a NaN among the logits counts as -infinity */
#pragma unroll
                for (uint32_t j = 0; j < 8; j++) x[u][j] = fmaxf(x[u][j], -INFINITY);
            } else {
#pragma unroll
                for (uint32_t j = 0; j < 8; j++)
                    if (at + j >= lo && at + j < hi) x[u][j] = fmaxf(x[u][j], -INFINITY);
            }
        }
#pragma unroll
        for (uint32_t u = 0; u < GPUOS_TOP_UNIT; u++) {
            most[u] = x[u][0];
#pragma unroll
            for (uint32_t j = 1; j < 8; j++) most[u] = fmaxf(most[u], x[u][j]); /* (NaN if nothing is there) */
            unit = fmaxf(unit, most[u]);
        }
        if (unit > st.m) {
            const float m = fminf(unit, FLT_MAX); /* (an infinite maximum: the sum is infinite) */
            st.s *= choose_exp(st.m - m);
            st.m = m;
        }
        float sum[GPUOS_TOP_UNIT]; /* (sums of sums: a rounding for each unit, not for each element) */
#pragma unroll
        for (uint32_t u = 0; u < GPUOS_TOP_UNIT; u++) {
            sum[u] = 0.0f;
#pragma unroll
            for (uint32_t j = 0; j < 8; j++) {
                /* the difference first: the lowest of the type's values is a mask too */
                float e;
                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"((fmaxf(x[u][j], -INFINITY) - st.m) * 1.4426950408889634f));
                sum[u] += e;
            }
        }
        st.s += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        if (first) {
            /* K different lanes' (or halves of lanes') largest are a bound from below */
            first = false;
            uint32_t k;
            if (K <= 32u) {
                k = top_nth(choose_key(unit), K);
            } else {
                float a = -INFINITY, b = -INFINITY;
#pragma unroll
                for (uint32_t u = 0; u < GPUOS_TOP_UNIT; u++) (u < GPUOS_TOP_UNIT / 2 ? a : b) = fmaxf(u < GPUOS_TOP_UNIT / 2 ? a : b, most[u]);
                k = min(top_nth(choose_key(a), 32u), top_nth(choose_key(b), K - 32u));
            }
            st.list.bound((uint64_t)k << 32);
            if (!__any_sync(GPUOS_FULL, unit >= st.list.floor)) continue;
        } else if (!__any_sync(GPUOS_FULL, unit > st.list.floor)) {
            continue; /* (an equal one later in the row is not among the best) */
        }
#pragma unroll
        for (uint32_t u = 0; u < GPUOS_TOP_UNIT; u++) {
#pragma unroll 1
            while (true) {
                /* each lane's best of its eight that are left, the first of equal ones */
                uint32_t j0 = 0;
#pragma unroll
                for (int j = 7; j >= 0; j--)
                    if (x[u][j] == most[u]) j0 = (uint32_t)j;
                const uint32_t token = u0 + u * 256u + lane * 8u + j0 - r.lo;
                const uint64_t mine = most[u] == most[u] ? top_entry(most[u], token) : 0ull;
                uint32_t left = __ballot_sync(GPUOS_FULL, mine > st.list.last);
                if (!left) break;
                if (mine > st.list.last) {
#pragma unroll
                    for (uint32_t j = 0; j < 8; j++)
                        if (j == j0) x[u][j] = none;
                    most[u] = x[u][0];
#pragma unroll
                    for (uint32_t j = 1; j < 8; j++) most[u] = fmaxf(most[u], x[u][j]);
                }
                while (left) {
                    const int src = __ffs((int)left) - 1;
                    left &= left - 1u;
                    const uint64_t c = shfl64(mine, src);
                    if (c > st.list.last) st.list.insert(c, K);
                }
            }
        }
    }
}
/* The lanes' maxima and sums as the warp's, alike in every lane. */
DEV void top_softmax(float &m, float &s)
{
    const float M = warp_max(m);
    s = warp_sum(s * choose_exp(m - M));
    m = M;
}
/* Write the row's answer from its list, maximum and sum. */
template <int KL>
DEV void top_write(const gpuos_devdesc *d, uint32_t row, const TopList<KL> &list, float m, float s)
{
    const uint32_t K = d->dims[3], lane = lane_id();
    const float ls = logf(s); /* (-infinity if nothing but -infinity was there) */
#pragma unroll
    for (int k = 0; k < KL; k++) {
        const uint32_t i = lane + 32u * k;
        if (i >= K) continue;
        const float x = choose_unkey((uint32_t)(list.e[k] >> 32));
        __stcg(reinterpret_cast<uint32_t *>(d->out) + (uint64_t)row * K + i, GPUOS_FULL - (uint32_t)list.e[k]);
        __stcg(reinterpret_cast<float *>(d->aux0) + (uint64_t)row * K + i, x == -INFINITY ? x : x - m - ls);
    }
    if (d->aux1 && lane == 0) __stcg(reinterpret_cast<float *>(d->aux1) + row, m + ls);
}
DEV unsigned char *top_part(const gpuos_devdesc *d, uint32_t tile)
{
    return reinterpret_cast<unsigned char *>(d->aux2) + GPUOS_CHOOSE_COUNTERS + (uint64_t)tile * GPUOS_TOP_PART;
}
template <bool F32, int KL>
DEV int top_tile(const gpuos_devdesc *d, uint32_t tile)
{
    const uint32_t V = d->dims[1], K = d->dims[3], S = gpuos_top_split(d->dims[0], V), lane = lane_id();
    const uint32_t row = tile / S, part = tile - row * S;
    if (row >= d->dims[0]) return GPUOS_ST_OK;
    const ChooseRow<F32> r(d->a, row, d->dims[2], V);
    const uint32_t run = ((V + 7u + S - 1u) / S + 255u) & ~255u;
    TopState<KL> st;
    top_run<F32, KL>(r, part * run, (part + 1u) * run, K, st);
    top_softmax(st.m, st.s);
    if (S == 1) {
        top_write(d, row, st.list, st.m, st.s);
        return GPUOS_ST_OK;
    }
    /* the row's last warp joins the runs' states */
    unsigned char *p = top_part(d, tile);
#pragma unroll
    for (int k = 0; k < KL; k++) __stcg(reinterpret_cast<unsigned long long *>(p + 16) + lane + 32 * k, st.list.e[k]);
    if (lane == 0) __stcg(reinterpret_cast<float2 *>(p), make_float2(st.m, st.s));
    __syncwarp();
    uint32_t last = 0;
    if (lane == 0) {
        uint32_t *ctr = reinterpret_cast<uint32_t *>(d->aux2) + row;
        last = atom_add_acq_rel_gpu32(ctr, 1u) == S - 1u;
        if (last) *ctr = 0; /* left zero for the next call */
    }
    if (!__shfl_sync(GPUOS_FULL, last, 0)) return GPUOS_ST_OK;
    __syncwarp();
    float m = -FLT_MAX, s = 0.0f;
#pragma unroll 1
    for (uint32_t i = lane; i < S; i += 32) {
        const float2 ms = __ldcg(reinterpret_cast<const float2 *>(top_part(d, row * S + i)));
        const float M = fmaxf(m, ms.x);
        s = s * choose_exp(m - M) + ms.y * choose_exp(ms.x - M);
        m = M;
    }
    top_softmax(m, s);
    constexpr uint32_t LISTS = 8 / KL; /* whose loads are out together */
#pragma unroll 1
    for (uint32_t i0 = 0; i0 < S; i0 += LISTS) {
        uint64_t e[LISTS][KL];
#pragma unroll
        for (uint32_t i = 0; i < LISTS; i++) {
            const bool here = i0 + i < S && i0 + i != part;
            const unsigned long long *q = reinterpret_cast<const unsigned long long *>(top_part(d, row * S + (here ? i0 + i : part)) + 16);
#pragma unroll
            for (int k = 0; k < KL; k++) e[i][k] = here && lane + 32u * k < K ? __ldcg(q + lane + 32 * k) : 0ull;
        }
#pragma unroll
        for (uint32_t i = 0; i < LISTS; i++)
#pragma unroll
            for (int k = 0; k < KL; k++) {
                uint32_t left = __ballot_sync(GPUOS_FULL, e[i][k] > st.list.last);
#pragma unroll 1
                while (left) {
                    const int src = __ffs((int)left) - 1;
                    left &= left - 1u;
                    const uint64_t c = shfl64(e[i][k], src);
                    if (c <= st.list.last) break; /* (they come in order) */
                    st.list.insert(c, K);
                }
            }
    }
    top_write(d, row, st.list, m, s);
    return GPUOS_ST_OK;
}
DEV int top_op(const gpuos_devdesc *d, uint32_t tile)
{
    const uint32_t *m = d->dims;
    if (m[0] == 0) return GPUOS_ST_OK;
    if (!gpuos_top_ok(d->dtype, d->a, d->out, d->aux0, d->aux1, d->aux2, m) ||
        (uint64_t)m[0] * gpuos_top_split(m[0], m[1]) != d->ntiles)
        return GPUOS_ST_BAD_ARGS;
    if (m[3] <= 32) return d->dtype == GPUOS_F32 ? top_tile<true, 1>(d, tile) : top_tile<false, 1>(d, tile);
    return d->dtype == GPUOS_F32 ? top_tile<true, 2>(d, tile) : top_tile<false, 2>(d, tile);
}

/* ---------------------------------------------------------------------------
 * The experts of a token. A warp holds a token's scores, expert e in lane
 * e % 32. Choices are made in fp32 and are those of 64-bit arithmetic: where
 * two values that a choice hangs on are nearer than their errors allow, the
 * token's choice is made again in 64 bits.
 * ------------------------------------------------------------------------- */
struct RouteArgs {
    uint32_t N, E, ld, K, G, keep, flags, size; /* (size: experts of a group) */
    const float *bias;
    const int32_t *rows;
    uint32_t *ids;
    float *weights;
    float scale;
};
DEV void route_args(const gpuos_devdesc *d, RouteArgs &a)
{
    a.N = d->dims[0], a.E = d->dims[1], a.ld = d->dims[2], a.K = d->dims[3];
    a.G = d->dims[4] & 0xFFFFu, a.keep = d->dims[4] >> 16, a.flags = d->dims[5];
    a.size = a.E / a.G;
    a.bias = reinterpret_cast<const float *>(d->b);
    a.rows = reinterpret_cast<const int32_t *>(d->aux1);
    a.ids = reinterpret_cast<uint32_t *>(d->out);
    a.weights = reinterpret_cast<float *>(d->aux0);
    a.scale = d->fparam[0];
}
DEV uint64_t route_key(double x)
{
    const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}
DEV double route_value(uint64_t k)
{
    return __longlong_as_double((long long)(k ^ ((uint64_t)((int64_t)~k >> 63) | 0x8000000000000000ull)));
}
DEV uint32_t route_max(uint32_t v) { return __reduce_max_sync(GPUOS_FULL, v); }
DEV uint64_t route_max(uint64_t v)
{
    const uint32_t hi = route_max((uint32_t)(v >> 32));
    return (uint64_t)hi << 32 | route_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
}
DEV float route_logit(const gpuos_devdesc *d, const RouteArgs &a, uint32_t n, uint32_t e)
{
    const uint64_t at = (uint64_t)n * a.ld + e;
    const float x = d->dtype == GPUOS_F32 ? __ldcg(reinterpret_cast<const float *>(d->a) + at)
                                          : bf1(__ldcg(reinterpret_cast<const uint16_t *>(d->a) + at));
    return fmaxf(x, -INFINITY); /* (a NaN counts as -infinity) */
}
/* Scores from a logit, the row's largest and 1 / the row's sum. The upper
 * limits keep an infinite logit's share, and sums of 1024, finite. */
DEV float route_exp(float x) { return choose_exp(fminf(x, 80.0f)); }
/* Two groups' values that fp32 holds as one infinity, where sums of two finite
 * values (none larger than `wide`) may be what is infinite: 64 bits tell them apart. */
DEV bool route_beyond(float edge, float next, float wide) { return wide > 0x1p126f && edge == next && fabsf(edge) > FLT_MAX; }
DEV float route_score(bool sigmoid, float x, float most, float inv)
{
    if (x == -INFINITY) return 0.0f;
    return sigmoid ? 1.0f / (1.0f + route_exp(-x)) : route_exp(x - most) * inv;
}
DEV double route_score(bool sigmoid, double x, double most, double inv)
{
    if (x == -INFINITY) return 0.0;
    return sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(fmin(x - most, 700.0)) * inv;
}
/* A chosen expert's score: as above, but for the difference's own rounding,
 * which is up to 2^-18 of the score of a logit 64 to 80 below the largest. */
DEV float route_weight(bool sigmoid, float x, float most, float inv)
{
    if (sigmoid) return route_score(true, x, most, inv);
    const float w = route_score(false, x, most, inv), h = x - most, z = h - x, l = (x - (h - z)) + (-most - z); /* h + l = x - most (Knuth) */
    return fabsf(h) <= 80.0f ? fmaf(w, l, w) : w;
}
/* Lane k's chosen expert and score -> the token's answer. */
template <typename T>
DEV void route_write(const RouteArgs &a, uint32_t n, uint32_t id, T got)
{
    T w = got;
    if (a.flags & GPUOS_ROUTE_NORM) {
        T sum = got;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(GPUOS_FULL, sum, o);
        if (sum != (T)0) w = got / sum;
    }
    if (lane_id() < a.K) {
        __stcg(a.ids + (uint64_t)n * a.K + lane_id(), id);
        __stcg(a.weights + (uint64_t)n * a.K + lane_id(), (float)(w * (T)a.scale));
    }
}
/* The groups to choose from, by lane g's value of group g. `edge`: the last
 * one's; `mine` is left 0 in the lanes of those kept. */
template <typename Key>
DEV uint32_t route_groups(const RouteArgs &a, Key &mine, Key &edge)
{
    uint32_t kept = 0;
    edge = 0;
#pragma unroll 1
    for (uint32_t k = 0; k < a.keep; k++) {
        edge = route_max(mine);
        const uint32_t owner = (uint32_t)__ffs((int)__ballot_sync(GPUOS_FULL, mine == edge && lane_id() < a.G && !(kept >> lane_id() & 1u))) - 1u;
        kept |= 1u << owner;
        if (lane_id() == owner) mine = 0;
    }
    return kept;
}
/* One token's choice and weights in 64 bits. Few tokens come here, but a
 * launch ends with the last of them: its exponentials run side by side. */
template <int VPL>
__device__ __noinline__ void op_y_sure(const gpuos_devdesc *d, uint32_t n)
{
    RouteArgs a;
    route_args(d, a);
    const uint32_t lane = lane_id();
    const bool sigmoid = a.flags & GPUOS_ROUTE_SIGMOID, top2 = a.flags & GPUOS_ROUTE_TOP2, scored = a.bias || top2;
    uint64_t key[VPL]; /* what groups go by, in order; 0: no expert */
    float most = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; i++)
        if (lane + 32u * i < a.E) most = fmaxf(most, route_logit(d, a, n, lane + 32u * i));
    most = fminf(warp_max(most), FLT_MAX);
    double inv = 0.0;
    if (!sigmoid) {
        double total = 0.0;
#pragma unroll 4
        for (int i = 0; i < VPL; i++)
            total += lane + 32u * i < a.E ? route_score(false, (double)route_logit(d, a, n, lane + 32u * i), (double)most, 1.0) : 0.0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(GPUOS_FULL, total, o);
        inv = total > 0.0 ? 1.0 / total : 0.0;
    }
#pragma unroll
    for (int i = 0; i < VPL; i++) {
        const uint32_t e = lane + 32u * i;
        const bool here = e < a.E;
        double c = here ? (double)route_logit(d, a, n, e) : 0.0; /* without a bias the scores' order is the logits' */
        if (scored) c = route_score(sigmoid, c, (double)most, inv);
        if (a.bias && here) c += (double)fmaxf(__ldcg(a.bias + e), -INFINITY);
        key[i] = here ? route_key(c) : 0ull;
    }
    if (a.G > 1) {
        uint64_t mine = 0, edge;
#pragma unroll 1
        for (uint32_t g = 0; g < a.G; g++) {
            uint64_t one = 0, two = 0;
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                const uint64_t k = lane + 32u * i - g * a.size < a.size ? key[i] : 0ull;
                two = max(two, min(one, k));
                one = max(one, k);
            }
            uint64_t best = route_max(one);
            if (top2) {
                const uint32_t owner = (uint32_t)__ffs((int)__ballot_sync(GPUOS_FULL, one == best)) - 1u;
                const uint64_t next = route_max(lane == owner ? two : one);
                best = route_key(route_value(best) + route_value(next));
            }
            if (lane == g) mine = best;
        }
        const uint32_t kept = route_groups(a, mine, edge);
#pragma unroll
        for (int i = 0; i < VPL; i++)
            if (lane + 32u * i < a.E && !(kept >> ((lane + 32u * i) / a.size) & 1u)) key[i] = 0ull;
    }
    if (top2 && !a.bias) {
#pragma unroll
        for (int i = 0; i < VPL; i++)
            if (key[i]) key[i] = route_key((double)route_logit(d, a, n, lane + 32u * i));
    }
    uint32_t id = 0;
#pragma unroll 1
    for (uint32_t k = 0; k < a.K; k++) {
        uint64_t best = 0;
        uint32_t at = 0;
#pragma unroll
        for (int i = VPL - 1; i >= 0; i--)
            if (key[i] >= best) best = key[i], at = (uint32_t)i;
        const uint64_t win = route_max(best);
        const uint32_t e = __reduce_min_sync(GPUOS_FULL, best == win ? lane + 32u * at : GPUOS_FULL);
        if (lane == (e & 31u)) {
#pragma unroll
            for (int i = 0; i < VPL; i++)
                if (i == (int)(e >> 5)) key[i] = 0ull;
        }
        if (lane == k) id = e;
    }
    const double got = lane < a.K ? route_score(sigmoid, (double)route_logit(d, a, n, id), (double)most, inv) : 0.0;
    route_write(a, n, id, got);
}
/* One token's choice and weights in fp32; false, with nothing written, if the
 * choice is not sure. */
template <int VPL>
DEV bool route_token(const gpuos_devdesc *d, const RouteArgs &a, uint32_t n)
{
    const uint32_t lane = lane_id();
    const bool sigmoid = a.flags & GPUOS_ROUTE_SIGMOID, top2 = a.flags & GPUOS_ROUTE_TOP2;
    uint32_t key[VPL]; /* what is chosen by, in order; 0: not to be chosen */
    float most = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; i++) {
        const uint32_t e = lane + 32u * i;
        const float x = e < a.E ? route_logit(d, a, n, e) : -INFINITY;
        key[i] = e < a.E ? choose_key(x) : 0u; /* without a bias the scores' order is the logits' */
        most = fmaxf(most, x);
    }
    most = fminf(warp_max(most), FLT_MAX); /* (infinite logits share the whole weight) */
    float inv = 0.0f;
    if (!sigmoid) {
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; i++)
            if (lane + 32u * i < a.E) total += route_score(false, choose_unkey(key[i]), most, 1.0f);
        total = warp_sum(total);
        inv = total > 0.0f ? 1.0f / total : 0.0f;
    }
    float wide = 0.0f; /* the largest value */
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            const uint32_t e = lane + 32u * i;
            if (e >= a.E) continue;
            const float c = fmaxf(route_score(sigmoid, choose_unkey(key[i]), most, inv) + __ldcg(a.bias + e), -INFINITY);
            key[i] = choose_key(c);
            if (fabsf(c) <= FLT_MAX) wide = fmaxf(wide, fabsf(c));
        }
    }
    wide = warp_max(wide);
    /* A sigmoid is off by less than 2^-21 of itself (ex2 2^-22, three roundings),
     * a softmax by less than 2^-19 (its sum's errors too; farther than 32 below the
     * largest by 2^-18, of next to nothing), the sum with the bias
     * by 2^-24 more; two values may swap within twice that. Scores of logits
     * below -80 are cut off (route_exp), which is nothing beside a larger one. */
    const float unsure = route_score(sigmoid, most, most, inv) * (sigmoid ? 0x1p-20f : 0x1p-18f) + wide * 0x1p-22f;
    bool sure = !sigmoid || most >= -60.0f || most == -INFINITY;
    if (a.G > 1) {
        uint32_t mine = 0, edge; /* lane g: group g's value */
        uint32_t one = 0, two = 0, g = 0;
        auto close = [&]() { /* the group's value from the lanes' two best of it */
            uint32_t best = route_max(one);
            if (top2) {
                const uint32_t owner = (uint32_t)__ffs((int)__ballot_sync(GPUOS_FULL, one == best)) - 1u;
                float v1 = choose_unkey(best), v2 = choose_unkey(route_max(lane == owner ? two : one));
                if (!a.bias) v1 = route_score(sigmoid, v1, most, inv), v2 = route_score(sigmoid, v2, most, inv);
                best = choose_key(v1 + v2);
            }
            if (lane == g) mine = best;
            one = two = 0, g++;
        };
        if (a.size % 32u == 0) { /* a group is whole rounds of the lanes */
            uint32_t left = a.size / 32u;
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                if (32u * i >= a.E) break;
                two = max(two, min(one, key[i]));
                one = max(one, key[i]);
                if (--left == 0) close(), left = a.size / 32u;
            }
        } else {
#pragma unroll 1
            while (g < a.G) {
#pragma unroll
                for (int i = 0; i < VPL; i++) {
                    const uint32_t k = lane + 32u * i - g * a.size < a.size ? key[i] : 0u;
                    two = max(two, min(one, k));
                    one = max(one, k);
                }
                close();
            }
        }
        const uint32_t kept = route_groups(a, mine, edge);
        if (a.keep < a.G && (a.bias || top2)) {
            const float last = choose_unkey(edge), next = choose_unkey(route_max(mine));
            if (last - next <= 2.0f * unsure || route_beyond(last, next, wide)) sure = false;
        }
#pragma unroll
        for (int i = 0; i < VPL; i++)
            if (lane + 32u * i < a.E && !(kept >> ((lane + 32u * i) / a.size) & 1u)) key[i] = 0u;
    }
    uint32_t id = 0, before = 0, e_before = 0;
    const uint32_t rounds = a.K + (a.bias ? 1u : 0u);
#pragma unroll 1
    for (uint32_t k = 0; k < rounds; k++) {
        uint32_t best = 0, at = 0;
#pragma unroll
        for (int i = VPL - 1; i >= 0; i--)
            if (key[i] >= best) best = key[i], at = (uint32_t)i;
        const uint32_t win = route_max(best);
        if (win == 0) break; /* (only after the K-th) */
        const uint32_t e = __reduce_min_sync(GPUOS_FULL, best == win ? lane + 32u * at : GPUOS_FULL);
        if (lane == (e & 31u)) {
#pragma unroll
            for (int i = 0; i < VPL; i++)
                if (i == (int)(e >> 5)) key[i] = 0u;
        }
        if (a.bias) {
            /* values that may have swapped, unless they are of equal logits and biases */
            if (k && choose_unkey(before) - choose_unkey(win) <= unsure) {
                const float x = route_logit(d, a, n, e_before), b = __ldcg(a.bias + e_before);
                if (!(route_logit(d, a, n, e) == x && __ldcg(a.bias + e) == b)) {
                    sure = false;
                } else if (k == a.K) { /* the last one's like is not chosen: what else is near comes behind it */
                    bool other = false;
#pragma unroll
                    for (int i = 0; i < VPL; i++)
                        if (key[i] && choose_unkey(before) - choose_unkey(key[i]) <= unsure)
                            other |= !(route_logit(d, a, n, lane + 32u * i) == x && __ldcg(a.bias + lane + 32u * i) == b);
                    if (__any_sync(GPUOS_FULL, other)) sure = false;
                }
            }
            before = win, e_before = e;
        }
        if (lane == k && k < a.K) id = e;
    }
    const float x = lane < a.K ? route_logit(d, a, n, id) : -INFINITY;
    /* (a chosen score below e^-80, that floats do not hold: its share may be all
     * that is seen. Without a bias a softmax's largest is among the chosen.) */
    if ((sigmoid || a.bias) && __any_sync(GPUOS_FULL, x - (sigmoid ? 0.0f : most) < -80.0f && x != -INFINITY)) sure = false;
    if (!sure) return false;
    route_write(a, n, id, route_weight(sigmoid, x, most, inv));
    return true;
}
/* A tile's tokens (at most 32); bit k of the result: token first + k is not sure. */
template <int VPL>
DEV uint32_t route_tile(const gpuos_devdesc *d, uint32_t first, uint32_t count)
{
    RouteArgs a;
    route_args(d, a);
    const uint32_t lane = lane_id(), end = min(first + count, a.N);
    const uint32_t rows = a.rows ? (uint32_t)max(__ldcg(a.rows), 0) : a.N;
    uint32_t again = 0;
#pragma unroll 1
    for (uint32_t n = first; n < end; n++) {
        if (n >= rows) { /* padding */
            if (lane < a.K) {
                __stcg(a.ids + (uint64_t)n * a.K + lane, GPUOS_FULL);
                __stcg(a.weights + (uint64_t)n * a.K + lane, 0.0f);
            }
        } else if (!route_token<VPL>(d, a, n)) {
            again |= 1u << (n - first);
        }
    }
    return again;
}
template <int VPL>
DEV void route_again(const gpuos_devdesc *d, uint32_t first, uint32_t again)
{
#pragma unroll 1
    for (; again; again &= again - 1u) op_y_sure<VPL>(d, first + (uint32_t)__ffs((int)again) - 1u);
}
/* Out of line, and done before its tokens go the sure way, so that no frame lies
 * on another: the executor's stack is 952 bytes a thread so. With all in line it
 * was 1,280, beyond the 1,024 that a context keeps for each thread, and its
 * launch had the device's local memory made larger (86 MB, once it is idle). */
template <int VPL>
__device__ __noinline__ uint32_t op_y_tile(const gpuos_devdesc *d, uint32_t first, uint32_t count)
{
    return route_tile<VPL>(d, first, count);
}
DEV int route_op(const gpuos_devdesc *d, uint32_t tile)
{
    const uint32_t *m = d->dims;
    if (m[0] == 0) return GPUOS_ST_OK;
    if (!gpuos_route_ok(d->dtype, d->a, d->b, d->out, d->aux0, d->aux1, m) ||
        (m[0] - 1u) / gpuos_route_rows(m[0]) + 1u != d->ntiles)
        return GPUOS_ST_BAD_ARGS;
    if (tile >= d->ntiles) return GPUOS_ST_OK;
    const uint32_t rows = gpuos_route_rows(m[0]), first = tile * rows;
    if (m[1] <= 256) route_again<8>(d, first, op_y_tile<8>(d, first, rows));
    else route_again<32>(d, first, op_y_tile<32>(d, first, rows));
    return GPUOS_ST_OK;
}

/* ---------------------------------------------------------------------------
 * The experts' order: a stable counting sort of the pairs. Runs of pairs are
 * counted by expert; a run's pairs of an expert then go behind those of the
 * earlier runs, in their order (whole numbers throughout, nothing hangs on
 * which warp comes first).
 * ------------------------------------------------------------------------- */
static_assert(GPUOS_PLAN_OFFSET + 2u * GPUOS_PLAN_TILES * GPUOS_ROUTE_MAX_E * 4u <= GPUOS_CHOOSE_WORKSPACE, "workspace");
struct PlanRun {
    uint32_t P, E, T, lo, hi; /* pairs, experts, runs; this run's pairs */
    const int32_t *ids;
    uint32_t *counts; /* [T][E], in the workspace */
};
DEV void plan_run(const gpuos_devdesc *d, uint32_t tile, PlanRun &p)
{
    p.P = d->dims[0], p.E = d->dims[1], p.T = gpuos_plan_tiles(p.P);
    const uint32_t n = ((p.P + p.T - 1u) / p.T + 31u) & ~31u;
    p.lo = min(tile * n, p.P);
    p.hi = min(p.lo + n, p.P);
    p.ids = reinterpret_cast<const int32_t *>(d->a);
    p.counts = reinterpret_cast<uint32_t *>(reinterpret_cast<unsigned char *>(d->aux2) + GPUOS_PLAN_OFFSET);
}
/* A warp's counters: in its staging buffer if they fit, else in the run's own
 * row of the workspace, where adds go through L2. */
DEV uint32_t *plan_counters(const PlanRun &p, uint32_t tile, bool &shared)
{
    shared = stage_hdr()->stage_bytes >= 4u * p.E;
    return shared ? reinterpret_cast<uint32_t *>(warp_stage_buf()) : p.counts + (uint64_t)tile * p.E;
}
/* Adds to counters from a warp: every add of an earlier call is seen. Returns the old value. */
DEV uint32_t plan_add(uint32_t *c, uint32_t n, bool shared)
{
    if (shared) {
        const uint32_t old = *c;
        *c = old + n;
        return old;
    }
    return atomicAdd(c, n);
}
DEV void plan_count(const PlanRun &p, uint32_t *ctr, bool shared)
{
    const uint32_t lane = lane_id();
    for (uint32_t e = lane; e < p.E; e += 32) {
        if (shared) ctr[e] = 0;
        else __stcg(ctr + e, 0u);
    }
    __threadfence_block();
    __syncwarp();
#pragma unroll 1
    for (uint32_t i = p.lo; i < p.hi; i += 256) {
        int32_t id[8];
#pragma unroll
        for (uint32_t k = 0; k < 8; k++) id[k] = i + 32u * k + lane < p.hi ? __ldcg(p.ids + i + 32u * k + lane) : -1;
#pragma unroll
        for (uint32_t k = 0; k < 8; k++)
            if ((uint32_t)id[k] < p.E) atomicAdd(ctr + id[k], 1u);
    }
    __threadfence_block();
    __syncwarp();
}
DEV int plan_count_op(const gpuos_devdesc *d, uint32_t tile)
{
    if (!gpuos_plan_ok(false, d->a, d->b, d->out, d->aux0, d->aux2, d->dims) || gpuos_plan_tiles(d->dims[0]) != d->ntiles)
        return GPUOS_ST_BAD_ARGS;
    PlanRun p;
    plan_run(d, tile, p);
    if (p.T == 1 || tile >= p.T) return GPUOS_ST_OK;
    bool shared;
    uint32_t *ctr = plan_counters(p, tile, shared);
    plan_count(p, ctr, shared);
    if (shared) {
        for (uint32_t e = lane_id(); e < p.E; e += 32) __stcg(p.counts + (uint64_t)tile * p.E + e, ctr[e]);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
    }
    return GPUOS_ST_OK;
}
DEV int plan_place_op(const gpuos_devdesc *d, uint32_t tile)
{
    if (!gpuos_plan_ok(true, d->a, d->b, d->out, d->aux0, d->aux2, d->dims) || gpuos_plan_tiles(d->dims[0]) != d->ntiles)
        return GPUOS_ST_BAD_ARGS;
    PlanRun p;
    plan_run(d, tile, p);
    if (tile >= p.T) return GPUOS_ST_OK;
    const uint32_t lane = lane_id();
    int32_t *const order = reinterpret_cast<int32_t *>(d->out), *const place = reinterpret_cast<int32_t *>(d->b);
    uint32_t *const offsets = reinterpret_cast<uint32_t *>(d->aux0);
    bool shared;
    uint32_t *ctr = plan_counters(p, p.T + tile, shared); /* (its own second row: the first is read by the others) */
    if (p.T == 1) plan_count(p, ctr, shared);
    /* where the run's pairs of each expert begin */
    uint32_t begin = 0; /* of the expert, over all runs */
#pragma unroll 1
    for (uint32_t e0 = 0; e0 < p.E; e0 += 32) {
        const uint32_t e = e0 + lane;
        uint32_t all = 0, mine = 0;
        if (e < p.E) {
            if (p.T == 1) {
                all = shared ? ctr[e] : __ldcg(ctr + e);
            } else {
#pragma unroll 8
                for (uint32_t t = 0; t < p.T; t++) {
                    if (t == tile) mine = all;
                    all += __ldcg(p.counts + (uint64_t)t * p.E + e);
                }
            }
        }
        uint32_t incl = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(GPUOS_FULL, incl, o);
            if (lane >= (uint32_t)o) incl += v;
        }
        if (e < p.E) {
            const uint32_t at = begin + incl - all;
            if (shared) ctr[e] = at + mine;
            else __stcg(ctr + e, at + mine);
            if (tile == 0) __stcg(offsets + e, at);
        }
        begin += __shfl_sync(GPUOS_FULL, incl, 31);
    }
    if (tile == 0 && lane == 0) __stcg(offsets + p.E, begin);
    __threadfence_block();
    __syncwarp();
    int32_t ahead[8] = {-1, -1, -1, -1, -1, -1, -1, -1};
#pragma unroll 1
    for (uint32_t i0 = p.lo; i0 < p.hi; i0 += 32) {
        const uint32_t i = i0 + lane, step = (i0 - p.lo) / 32u % 8u;
        if (step == 0) { /* eight steps' ids at a time */
#pragma unroll
            for (uint32_t k = 0; k < 8; k++) ahead[k] = i + 32u * k < p.hi ? __ldcg(p.ids + i + 32u * k) : -1;
        }
        const int32_t id = ahead[0];
#pragma unroll
        for (uint32_t k = 0; k < 7; k++) ahead[k] = ahead[k + 1];
        const bool here = (uint32_t)id < p.E;
        const uint32_t peers = __match_any_sync(GPUOS_FULL, here ? id : -1);
        const uint32_t lead = (uint32_t)__ffs((int)peers) - 1u;
        uint32_t at = 0;
        if (here && lane == lead) at = plan_add(ctr + id, (uint32_t)__popc(peers), shared);
        at = __shfl_sync(GPUOS_FULL, at, (int)lead) + (uint32_t)__popc(peers & ((1u << lane) - 1u));
        if (here && at < p.P) __stcg(order + at, (int32_t)i); /* (counts that are not of these pairs: nothing outside is written) */
        if (i < p.hi) __stcg(place + i, here ? (int32_t)at : -1);
        if (i < p.hi && i >= begin) __stcg(order + i, -1); /* (places behind the last pair) */
        __syncwarp();
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    return GPUOS_ST_OK;
}

#ifndef GPUOS_EXECUTOR_ONLY
#define GPUOS_ADJUSTB_THREADS 256u
/* From which length of history on (the tokens' row, which the host knows) eight
 * blocks share it: direct and shared, us, bf16:
 *   tokens       8,000        12,000       16,000       24,000        48,000
 *   8 x 32,000   5.0   6.3    6.4   6.4    7.7   6.4    10.5   6.6    18.4   6.7
 *   1 x 128,000  5.0   6.3    6.4   6.4    7.7   6.4    10.4   6.4    18.3   6.7
 *   8 x 128,000  6.2  12.0    7.6  12.1    9.0  12.1    11.9  12.3    20.0  12.6
 * (64, 32 and 256 blocks that share; 2,048 of them, 64 x 128,000 with 16,000
 * tokens, take 69 us against 18). A row with room for more than 229,376 tokens
 * is not shared, as its 16-bit counters could overflow: 8 x 32,000 with 20,000
 * to 131,071 tokens in it 47 us against 8. With at most 100 tokens in a row of
 * 12,289 or more the shared way takes 5.9 us where the direct one took 2.5. */
#define GPUOS_ADJUSTL_LONG 12288u   /* as long as each block has an SM ... */
#define GPUOS_ADJUSTL_LONGER 24576u /* ... or half of one */
#define GPUOS_ADJUSTL_FEW 152u
/* Elements from which on a thread takes three eights (f32) or four (bf16)
 * instead of two: two and more, us, rows of 128,000:
 *   rows   4            16           32           64             128
 *   f32    4.9   5.0    6.0   6.3    9.1   8.9    17.6   17.7    28.8   28.3   (256: 57, 53)
 *   bf16   4.7   5.6    6.0   6.1    7.6   7.0    13.5   13.3    23.5   22.2 */
#define GPUOS_ADJUSTB_MANY 4000000u
/* As kv4_launch, with a grid of two dimensions and clusters. */
static int choose_launch(void (*kernel)(const gpuos_devdesc), dim3 blocks, uint32_t threads, uint32_t smem, void *stream, const gpuos_devdesc &d,
                         uint32_t cluster = 1)
{
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = blocks;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = (cudaStream_t)stream;
    c.attrs = at;
    c.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&c, kernel, d) == cudaSuccess) return 0;
    (void)cudaGetLastError(); /* reported here */
    return -1;
}
/* Let a kernel have more shared memory than 48 KB, once for each device. */
static int choose_smem(const void *kernel, uint32_t bytes, std::atomic<bool> (&known)[64])
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
    if (known[dev].load(std::memory_order_relaxed)) return 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) return -1;
    known[dev].store(true, std::memory_order_relaxed);
    return 0;
}
/* ---------------------------------------------------------------------------
 * Logits adjusted, launched: a block takes 16 places of one row for each of its
 * threads, or more in large calls (below). A thread's logits, the first tokens
 * and the record are on their way at once, so that a block waits for memory
 * about twice: for those, and for the mask's words.
 *
 * 256 rows of 128,000 in f32 (up to 4,000 tokens, 16 biases, masks for three in
 * four) 53 us, 5.0 TB/s; without tokens, biases and masks 42.5, 6.2 TB/s; 512
 * rows in bf16 63 us, 4.2 TB/s: beside memory it is then bound by instructions
 * (23 for an element, issue slots 60 % used) and by blocks that wait for their
 * slowest warp's tokens. One row of 128,000 3.2 us, 33 rows of 50,001 whose
 * input lies otherwise than the output 5.1: latency.
 * ------------------------------------------------------------------------- */
template <bool F32, bool SAME>
struct AdjustRaw {
    /* vectors that eight elements lie in: whole ones (SAME: the input's rows lie
     * as the output's do), or whatever their start */
    static constexpr int N = (F32 ? 2 : 1) + (SAME ? 0 : 1);
    uint4 v[N];
};
/* The vectors of the input from place `from`, the first of which has `r`
 * elements that are not wanted. */
template <bool F32, bool SAME>
DEV void adjust_raw(const ChooseRow<F32> &in, uint32_t from, uint32_t r, bool here, AdjustRaw<F32, SAME> &raw)
{
    constexpr uint32_t PER = F32 ? 4u : 8u;
#pragma unroll
    for (int k = 0; k < AdjustRaw<F32, SAME>::N; k++) {
        const uint32_t first = from + PER * k;
        /* the last vector is needed only if the elements do not start at a boundary */
        const bool need = here && (SAME || k + 1 < AdjustRaw<F32, SAME>::N || r) && first < in.hi;
        raw.v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (!need) continue;
        if (first >= in.lo && first + PER <= in.hi) {
            raw.v[k] = *in.vec(first);
        } else { /* the row's ends: nothing outside is read */
            uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (uint32_t j = 0; j < PER; j++) {
                if (first + j < in.lo || first + j >= in.hi) continue;
                if (F32) w[j & 3u] = reinterpret_cast<const uint32_t *>(in.base)[first + j];
                else w[(j >> 1) & 3u] |= (uint32_t)reinterpret_cast<const uint16_t *>(in.base)[first + j] << 16 * (j & 1u);
            }
            raw.v[k] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}
template <bool F32, bool SAME>
DEV void adjust_unpack(const AdjustRaw<F32, SAME> &raw, uint32_t r, float (&x)[8])
{
    constexpr int N = AdjustRaw<F32, SAME>::N;
    uint32_t w[4 * N];
#pragma unroll
    for (int k = 0; k < N; k++) w[4 * k] = raw.v[k].x, w[4 * k + 1] = raw.v[k].y, w[4 * k + 2] = raw.v[k].z, w[4 * k + 3] = raw.v[k].w;
    if (!SAME) {
        if (!F32 && r & 4u)
#pragma unroll
            for (int i = 0; i + 2 < 4 * N; i++) w[i] = w[i + 2];
        if (r & 2u)
#pragma unroll
            for (int i = 0; i + (F32 ? 2 : 1) < 4 * N; i++) w[i] = w[i + (F32 ? 2 : 1)];
        if (r & 1u)
#pragma unroll
            for (int i = 0; i + 1 < 4 * N; i++) w[i] = F32 ? w[i + 1] : __funnelshift_r(w[i], w[i + 1], 16);
    }
    if (F32) {
#pragma unroll
        for (int i = 0; i < 8; i++) x[i] = __uint_as_float(w[i % (4 * N)]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) x[2 * i] = bf_lo(w[i]), x[2 * i + 1] = bf_hi(w[i]);
    }
}

/* The vectors of a thread's eight places at `at`. */
template <bool F32, bool SAME>
DEV void adjust_load(const ChooseRow<F32> &in, uint32_t at, uint32_t shift, uint32_t r, uint32_t lo, uint32_t hi, AdjustRaw<F32, SAME> &raw)
{
    if (SAME && at >= lo && at + 8u <= hi) {
#pragma unroll
        for (uint32_t v = 0; v < AdjustRaw<F32, SAME>::N; v++) raw.v[v] = in.vec(at)[v];
    } else {
        adjust_raw(in, at + shift - r, r, at < hi, raw); /* (places before 0 wrap round, and are not in the row) */
    }
}
/* Eight places with their counters and mask bits, done and written but for
 * those that are listed or not in [lo, hi). */
template <bool F32, bool SAME>
DEV void adjust_eight(const AdjustArgs &a, const ChooseRow<F32> &out, const AdjustRaw<F32, SAME> &raw, uint32_t r, const uint4 &w0, const uint4 &w1,
                      uint32_t bits, uint32_t at, uint32_t lo, uint32_t hi)
{
    float x[8];
    adjust_unpack(raw, r, x);
    const uint32_t any = (w0.x | w0.y | w0.z | w0.w) | (w1.x | w1.y | w1.z | w1.w);
    if (any) {
        const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (uint32_t j = 0; j < 8; j++) x[j] = adjust_penalty(a, x[j], w[j]);
    } else {
#pragma unroll
        for (uint32_t j = 0; j < 8; j++) x[j] *= a.plain;
    }
    if (a.mask) {
#pragma unroll
        for (uint32_t j = 0; j < 8; j++) x[j] = bits & 1u << j ? x[j] : -INFINITY;
    }
    if (!(any & GPUOS_ADJUST_LISTED) && at >= lo && at + 8u <= hi) {
        uint4 *o = const_cast<uint4 *>(out.vec(at));
        if (F32) {
            o[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
            o[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
        } else {
            o[0] = pack8(x);
        }
    } else {
        const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (uint32_t j = 0; j < 8; j++)
            if (!(w[j] & GPUOS_ADJUST_LISTED) && at + j >= lo && at + j < hi) out.put(at + j, x[j]);
    }
}
DEV uint32_t adjust_mask(const AdjustArgs &a, uint32_t at, uint32_t lo, uint32_t V)
{
    if (!a.mask) return 0xFFu;
    return lo == 0 ? a.mask[at >> 5] >> (at & 31u) : adjust_bits(a, (int32_t)at - (int32_t)lo, V);
}
/* The listed tokens of places [from, to): nobody has written them (out may be
 * the input). `listed`: the entries' tokens; counter(place). */
template <bool F32, int THREADS, typename Counter>
DEV void adjust_listed(const AdjustArgs &a, const ChooseRow<F32> &in, const ChooseRow<F32> &out, uint32_t V, uint32_t shift, uint32_t from, uint32_t to,
                       const int32_t *listed, const Counter &counter)
{
    for (uint32_t i = threadIdx.x; i < (uint32_t)a.q.biases; i += THREADS) {
        const int2 e = a.bias[i];
        const uint32_t at = (uint32_t)e.x + out.lo;
        if ((uint32_t)e.x >= V || at < from || at >= to) continue;
        bool again = false; /* listed again further on: the later entry counts */
        for (uint32_t k = i + 1; k < (uint32_t)a.q.biases; k++) again |= listed[k] == e.x;
        if (again) continue;
        const float y = fmaf(__int_as_float(e.y), a.plain, adjust_penalty(a, in.one(at + shift), counter(at)));
        out.put(at, adjust_allowed(a, (uint32_t)e.x) ? y : -INFINITY);
    }
}
template <bool F32, bool SAME, int VECS>
__global__ void __launch_bounds__(GPUOS_ADJUSTB_THREADS, (VECS == 2 ? 1280 : 1024) / GPUOS_ADJUSTB_THREADS)
    gpuos_adjust_kernel(const __grid_constant__ gpuos_devdesc d)
{
    constexpr uint32_t THREADS = GPUOS_ADJUSTB_THREADS, CHUNK = THREADS * VECS * 8u;
    __shared__ __align__(16) uint32_t ctr[CHUNK];
    __shared__ int32_t listed[GPUOS_ADJUST_MAX_BIAS];
    kv4_after_previous();
    const uint32_t V = d.dims[1], b = blockIdx.y, t = threadIdx.x;
    const ChooseRow<F32> in(d.a, b, d.dims[2], V), out(d.out, b, d.dims[3], V);
    const uint32_t from = blockIdx.x * CHUNK, lo = max(from, out.lo), hi = min(from + CHUNK, out.hi);
    const uint32_t shift = in.lo - out.lo, r = SAME ? 0u : shift & (F32 ? 3u : 7u); /* (modulo 2^32, like the places) */
    AdjustRaw<F32, SAME> raw[VECS];
#pragma unroll
    for (uint32_t k = 0; k < VECS; k++) adjust_load(in, from + (k * THREADS + t) * 8u, shift, r, lo, hi, raw[k]);
    /* the first tokens too, whether the request has had them or not: their loads
     * need not wait for the record's */
    constexpr uint32_t EARLY = 4;
    const uint32_t Lcap = d.dims[4];
    int32_t early[EARLY];
#pragma unroll
    for (uint32_t k = 0; k < EARLY; k++)
        early[k] = k * THREADS + t < Lcap ? reinterpret_cast<const int32_t *>(d.b)[(uint64_t)b * Lcap + k * THREADS + t] : -1;
    AdjustArgs a;
    if (!adjust_args(&d, b, a)) return; /* (all of a row's blocks) */
    uint32_t bits[VECS];
#pragma unroll
    for (uint32_t k = 0; k < VECS; k++) {
        const uint32_t at = from + (k * THREADS + t) * 8u;
        bits[k] = at < hi ? adjust_mask(a, at, out.lo, V) : 0u;
    }
    const bool counted = a.penal || a.q.biases > 0;
    if (counted) {
#pragma unroll
        for (uint32_t k = 0; k < 2 * VECS; k++) reinterpret_cast<uint4 *>(ctr)[k * THREADS + t] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        if (a.penal) {
            const uint32_t n = (uint32_t)a.q.length, prompt = (uint32_t)a.q.prompt;
            auto mark = [&](int32_t token, uint32_t i) {
                const uint32_t at = (uint32_t)token + out.lo - from;
                if ((uint32_t)token >= V || at >= CHUNK || i >= n) return;
                if (i < prompt) atomicOr(ctr + at, GPUOS_ADJUST_HAD);
                else atomicAdd(ctr + at, 1u);
            };
#pragma unroll
            for (uint32_t k = 0; k < EARLY; k++) mark(early[k], k * THREADS + t);
#pragma unroll 1
            for (uint32_t i0 = EARLY * THREADS + t; i0 < n; i0 += 8u * THREADS) {
                int32_t tok[8];
#pragma unroll
                for (uint32_t k = 0; k < 8; k++) tok[k] = i0 + k * THREADS < n ? a.tokens[i0 + k * THREADS] : -1;
#pragma unroll
                for (uint32_t k = 0; k < 8; k++) mark(tok[k], i0 + k * THREADS);
            }
        }
        for (uint32_t i = t; i < (uint32_t)a.q.biases; i += THREADS) {
            const uint32_t token = (uint32_t)a.bias[i].x, at = token + out.lo - from;
            listed[i] = (int32_t)token;
            if (token < V && at < CHUNK) atomicOr(ctr + at, GPUOS_ADJUST_LISTED);
        }
        __syncthreads();
    }
#pragma unroll
    for (uint32_t k = 0; k < VECS; k++) {
        const uint32_t at = from + (k * THREADS + t) * 8u;
        if (at >= hi) continue;
        uint4 w0 = make_uint4(0u, 0u, 0u, 0u), w1 = w0;
        if (counted) w0 = reinterpret_cast<const uint4 *>(ctr)[2 * (k * THREADS + t)], w1 = reinterpret_cast<const uint4 *>(ctr)[2 * (k * THREADS + t) + 1];
        adjust_eight(a, out, raw[k], r, w0, w1, bits[k], at, lo, hi);
    }
    adjust_listed<F32, (int)THREADS>(a, in, out, V, shift, lo, hi, listed, [&](uint32_t at) { return ctr[at - from]; });
}
/* Long histories: eight blocks of neighbouring chunks, a cluster, share them.
 * Each counts an eighth of the tokens, for all eight chunks, in 16 bits (15 and
 * the prompt's flag); a thread then adds up its places' eight counters out of
 * the eight blocks' shared memory. Eight requests of 20,000 to 131,071 tokens
 * over 32,000: 8.1 us; blocks of 1,024 threads that each look at all tokens
 * 15 to 18; adds to the other blocks' counters from afar, instead of sums, 57. */
#define GPUOS_ADJUSTL_BLOCKS 8u
#define GPUOS_ADJUSTL_THREADS 512u
DEV void choose_cluster_sync()
{
    /* (not the aligned form: it follows loops whose lanes end apart) */
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
template <bool F32, bool SAME>
__global__ void __launch_bounds__(GPUOS_ADJUSTL_THREADS) gpuos_adjust_long_kernel(const __grid_constant__ gpuos_devdesc d)
{
    constexpr uint32_t THREADS = GPUOS_ADJUSTL_THREADS, CHUNK = THREADS * 8u, N = GPUOS_ADJUSTL_BLOCKS;
    extern __shared__ __align__(16) uint32_t adjust_half[]; /* N CHUNK counters of 16 bits */
    __shared__ uint32_t has_bias[CHUNK / 32]; /* of this block's chunk */
    __shared__ int32_t listed[GPUOS_ADJUST_MAX_BIAS];
    kv4_after_previous();
    const uint32_t V = d.dims[1], b = blockIdx.y, t = threadIdx.x, rank = blockIdx.x % N;
    const ChooseRow<F32> in(d.a, b, d.dims[2], V), out(d.out, b, d.dims[3], V);
    const uint32_t from = blockIdx.x * CHUNK, lo = max(from, out.lo), hi = min(from + CHUNK, out.hi); /* (a cluster's last may be empty) */
    const uint32_t shift = in.lo - out.lo, r = SAME ? 0u : shift & (F32 ? 3u : 7u);
    AdjustArgs a;
    if (!adjust_args(&d, b, a)) return; /* (all of a row's blocks) */
    const uint32_t at = from + t * 8u, begin = from - rank * CHUNK; /* (the cluster's first place) */
    AdjustRaw<F32, SAME> raw;
    adjust_load(in, at, shift, r, lo, hi, raw);
    const uint32_t bits = at < hi ? adjust_mask(a, at, out.lo, V) : 0u;
#pragma unroll
    for (uint32_t k = 0; k < N; k++) reinterpret_cast<uint4 *>(adjust_half)[k * THREADS + t] = make_uint4(0u, 0u, 0u, 0u);
    if (t < CHUNK / 32) has_bias[t] = 0u;
    __syncthreads();
    if (a.penal) {
        const uint32_t n = (uint32_t)a.q.length, prompt = (uint32_t)a.q.prompt;
#pragma unroll 1
        for (uint32_t i0 = rank * THREADS + t; i0 < n; i0 += 16u * THREADS * N) {
            int32_t tok[16];
#pragma unroll
            for (uint32_t k = 0; k < 16; k++) tok[k] = i0 + k * THREADS * N < n ? a.tokens[i0 + k * THREADS * N] : -1;
#pragma unroll
            for (uint32_t k = 0; k < 16; k++) {
                const uint32_t p = (uint32_t)tok[k] + out.lo - begin;
                if ((uint32_t)tok[k] >= V || p >= CHUNK * N) continue;
                if (i0 + k * THREADS * N < prompt) atomicOr(adjust_half + (p >> 1), 0x8000u << 16 * (p & 1u));
                else atomicAdd(adjust_half + (p >> 1), 1u << 16 * (p & 1u));
            }
        }
    }
    for (uint32_t i = t; i < (uint32_t)a.q.biases; i += THREADS) {
        const uint32_t token = (uint32_t)a.bias[i].x, p = token + out.lo - from;
        listed[i] = (int32_t)token;
        if (token < V && p < CHUNK) atomicOr(has_bias + (p >> 5), 1u << (p & 31u));
    }
    choose_cluster_sync();
    const uint32_t mine = smem_addr(adjust_half) + (rank * CHUNK + t * 8u) * 2u;
    uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
    for (uint32_t k = 0; k < N; k++) {
        uint32_t remote;
        uint4 v;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(mine), "r"(k));
        asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(remote) : "memory");
        const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (uint32_t j = 0; j < 8; j++) {
            const uint32_t c = h[j >> 1] >> 16 * (j & 1u);
            w[j] = (w[j] + (c & 0x7FFFu)) | (c & 0x8000u) << 16;
        }
    }
    /* nobody reads another block's counters from here on: the sums go in their place */
    choose_cluster_sync();
    const uint32_t flags = at < hi ? has_bias[t >> 2] >> 8 * (t & 3u) : 0u;
    uint32_t *const sums = adjust_half;
#pragma unroll
    for (uint32_t j = 0; j < 8; j++) sums[t * 8u + j] = w[j];
#pragma unroll
    for (uint32_t j = 0; j < 8; j++) w[j] |= flags >> j & 1u ? GPUOS_ADJUST_LISTED : 0u;
    if (at < hi) adjust_eight(a, out, raw, r, make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]), bits, at, lo, hi);
    __syncthreads();
    adjust_listed<F32, (int)THREADS>(a, in, out, V, shift, lo, hi, listed, [&](uint32_t p) { return sums[p - from]; });
}
/* A kernel whose blocks take `chunk` places each, and of a row a multiple of `cluster`. */
static int adjust_launch(void (*kernel)(const gpuos_devdesc), uint32_t threads, uint32_t chunk, uint32_t smem, uint32_t cluster, uint32_t size,
                         const gpuos_devdesc &d, void *stream)
{
    uint32_t chunks = (uint32_t)(((uint64_t)d.dims[1] + 7u + chunk - 1u) / chunk);
    chunks = (chunks + cluster - 1u) / cluster * cluster;
    gpuos_devdesc e = d;
    /* (rows beyond the grid's second dimension: launches of their own) */
    for (uint32_t row = 0; row < d.dims[0]; row += 65535u) {
        e.dims[0] = min(d.dims[0] - row, 65535u);
        e.a = d.a + (uint64_t)row * d.dims[2] * size;
        e.out = d.out + (uint64_t)row * d.dims[3] * size;
        e.b = d.b + (uint64_t)row * d.dims[4] * 4u;
        e.aux0 = d.aux0 + (uint64_t)row * sizeof(gpuos_logits_request);
        e.aux2 = d.aux2 + (uint64_t)row * (d.dims[5] >> 16) * sizeof(gpuos_logits_bias);
        if (choose_launch(kernel, dim3(chunks, e.dims[0]), threads, smem, stream, e, cluster) != 0) return -1;
    }
    return 0;
}
template <bool F32, bool SAME>
static int adjust_launch_by(const gpuos_devdesc &d, void *stream)
{
    constexpr int MANY = F32 ? 3 : 4; /* eights a thread of a large call: what registers hold */
    constexpr uint32_t T = GPUOS_ADJUSTB_THREADS, TL = GPUOS_ADJUSTL_THREADS, N = GPUOS_ADJUSTL_BLOCKS, size = F32 ? 4u : 2u;
    const uint64_t sharing = (uint64_t)d.dims[0] * ((d.dims[1] + 7u) / (TL * 8u) + 1u); /* blocks */
    const bool longer = sharing <= GPUOS_ADJUSTL_FEW ? d.dims[4] > GPUOS_ADJUSTL_LONG : sharing <= 2u * GPUOS_ADJUSTL_FEW && d.dims[4] > GPUOS_ADJUSTL_LONGER;
    if (longer && d.dims[4] <= 0x7000u * N) { /* (a block's share is an eighth and 512 more at most: below 2^15) */
        static std::atomic<bool> known[64];
        constexpr uint32_t smem = TL * 8u * N * 2u;
        if (choose_smem((const void *)gpuos_adjust_long_kernel<F32, SAME>, smem, known) != 0) return -1;
        return adjust_launch(gpuos_adjust_long_kernel<F32, SAME>, TL, TL * 8u, smem, N, size, d, stream);
    }
    if ((uint64_t)d.dims[0] * d.dims[1] > GPUOS_ADJUSTB_MANY) return adjust_launch(gpuos_adjust_kernel<F32, SAME, MANY>, T, T * 8u * MANY, 0, 1, size, d, stream);
    return adjust_launch(gpuos_adjust_kernel<F32, SAME, 2>, T, T * 16u, 0, 1, size, d, stream);
}
template <bool F32>
static int adjust_launch_of(const gpuos_devdesc &d, void *stream)
{
    const uint64_t size = F32 ? 4u : 2u;
    const bool same = ((d.a ^ d.out) & 15u) == 0 && (((uint64_t)d.dims[2] - d.dims[3]) * size & 15u) == 0;
    return same ? adjust_launch_by<F32, true>(d, stream) : adjust_launch_by<F32, false>(d, stream);
}

/* ---------------------------------------------------------------------------
 * The best tokens, launched. The rows one behind the other are cut into equal
 * runs, one for each block, so that all end together; a row, or what a run has
 * of it, is a piece. Bulk copies bring a run into a ring of shared memory, 4,096
 * elements a unit. A piece's first unit gives a bar that at least K of its elements
 * reach; what reaches it is gathered, a few times K elements, and ranked by
 * comparing all with all; now and then the K best so far give a better bar.
 * Warps wait for copies, not for each other, between units. The softmax's sum
 * is kept in base 2 under a maximum of the thread's own: one multiply-add, one
 * exponential and one sum an element.
 *
 * Bound by memory while units stream (a block's 16 KB in 2,050 cycles with three
 * blocks an SM, 7 TB/s); a piece's start and end take it about 5 us (first copy
 * 1, bar 1, ranks 0.5, sums 0.5, a part's way to the row's last block 1 to 2,
 * joining 2), which the SM's other two blocks cover only in part. 456 rows of
 * 128,000 in f32, K = 5: 42.3 us, 5.5 TB/s (K = 1: 40.5); 509 rows, whose runs
 * cross rows, 53, 4.9 TB/s (three equal runs for each row, 4 waves: 62 where this
 * took 56); 64 rows in bf16, K = 20: 16; one row of 32,000, K = 1: 6.2. Units
 * that are whole are read without a look at each place (56.8 us without that). Loads to registers
 * instead of the ring took the same time while they were the only change.
 * ------------------------------------------------------------------------- */
#define GPUOS_TOPB_THREADS 256
#define GPUOS_TOPB_WARPS (GPUOS_TOPB_THREADS / 32)
#define GPUOS_TOPB_SLOTS 456u /* blocks that run at a time: three for each SM */
#define GPUOS_TOPB_FIXED 48u /* cells (of 256 elements) that a piece's start and end cost as much as */
#define GPUOS_TOPB_UNIT 4096u /* elements: sixteen a thread */
#define GPUOS_TOPB_STAGES 3u
#define GPUOS_TOPB_FEW 256u
#define GPUOS_TOPB_PLAIN 192u /* entries that are ranked without a bar before */
#define GPUOS_TOPB_SOME 512u /* ... that a bar lets pass (lists: K, and 56 more of eight) */
static_assert(2u * GPUOS_TOPB_SLOTS <= GPUOS_TOP_TILES, "two pieces of each block in the workspace");
/* (the slow gathering: a unit adds at most K threads' 16 elements to the few before it) */
#define GPUOS_TOPB_ROOM (GPUOS_TOPB_FEW + GPUOS_TOP_MAX_K * 16u)
#define GPUOS_TOPB_JOIN (35u * GPUOS_TOP_MAX_K) /* entries of a row's pieces */
static_assert(GPUOS_TOPB_JOIN >= GPUOS_TOPB_ROOM, "one array for both");
template <bool F32>
struct TopUnit {
    static constexpr uint32_t PER = F32 ? 4u : 8u; /* elements of a vector */
    static constexpr uint32_t N = GPUOS_TOPB_UNIT, BYTES = N * (F32 ? 4u : 2u);
    static constexpr int G = N / GPUOS_TOPB_THREADS / 8; /* eights of a thread */
    /* the place of a thread's element (u, j) from the unit's first: neighbouring
     * threads have neighbouring vectors */
    static DEV uint32_t at(uint32_t u, uint32_t j) { return (((8u / PER) * u + j / PER) * GPUOS_TOPB_THREADS + threadIdx.x) * PER + j % PER; }
};

struct TopBlock {
    /* (eight more of each: a list's end is filled with entries below all others) */
    __align__(16) uint64_t got[GPUOS_TOPB_JOIN + 8u];
    __align__(16) uint64_t few[GPUOS_TOPB_SOME + 8u];
    __align__(16) uint64_t best[GPUOS_TOPB_THREADS];
    uint64_t sorted[GPUOS_TOP_MAX_K];
    uint64_t bar; /* an entry has to be above it */
    float2 part[GPUOS_TOPB_WARPS];
    uint32_t count, left, last;
};
/* How many of n entries (a multiple of eight) are above x. */
DEV uint32_t top_rank(const uint64_t *e, uint32_t n, uint64_t x)
{
    uint32_t r = 0;
#pragma unroll 4
    for (uint32_t i = 0; i < n; i += 8) {
        ulonglong2 v[4];
#pragma unroll
        for (int k = 0; k < 4; k++) v[k] = reinterpret_cast<const ulonglong2 *>(e + i)[k];
#pragma unroll
        for (int k = 0; k < 4; k++) r += (v[k].x > x) + (v[k].y > x);
    }
    return r;
}
DEV uint32_t top_fill(uint64_t *e, uint32_t n) /* (before a barrier) */
{
    if (threadIdx.x < 8u) e[n + threadIdx.x] = 0;
    return (n + 7u) & ~7u;
}
/* (The bars and the sort are functions of their own: inlined at each of their
 * places, 509 x 128,000 took 57.8 us where they take 56.6. A launch runs them from a cold
 * instruction cache.)
 *
 * A bar that at least K of the threads' entries are above (0: there are not
 * K): the K-th of them less one; or, for few, the K-th of the warps' best few
 * less one, which takes a third of the time. Every thread. */
__device__ __noinline__ uint64_t top_bar_exact(TopBlock &s, uint64_t mine, uint32_t K)
{
    const uint32_t t = threadIdx.x;
    __syncthreads(); /* (the last use of best and bar is over) */
    s.best[t] = mine;
    if (t == 0) s.bar = 0;
    __syncthreads();
    if (mine && top_rank(s.best, GPUOS_TOPB_THREADS, mine) == K - 1u) s.bar = mine - 1u;
    __syncthreads();
    return s.bar;
}
__device__ __noinline__ uint64_t top_bar(TopBlock &s, uint64_t mine, uint32_t K)
{
    if (K > 32u) return top_bar_exact(s, mine, K); /* (the warps' eight best are 64: their K-th lets far too many pass) */
    const uint32_t t = threadIdx.x, lane = lane_id();
    uint64_t keep = 0;
#pragma unroll 1
    for (uint32_t i = 0; i < min(K, (K + 23u) / 8u); i++) {
        const uint32_t hi = __reduce_max_sync(GPUOS_FULL, (uint32_t)(mine >> 32));
        const uint32_t lo = __reduce_max_sync(GPUOS_FULL, (uint32_t)(mine >> 32) == hi ? (uint32_t)mine : 0u);
        const uint64_t top = (uint64_t)hi << 32 | lo;
        if (mine == top) mine = 0;
        if (lane == i) keep = top;
    }
    __syncthreads();
    if (lane < 8) s.best[(t >> 5) * 8u + lane] = keep;
    if (t == 0) s.bar = 0;
    __syncthreads();
    if (t < GPUOS_TOPB_WARPS * 8u) {
        const uint64_t x = s.best[t];
        if (x && top_rank(s.best, GPUOS_TOPB_WARPS * 8u, x) == K - 1u) s.bar = x - 1u;
    }
    __syncthreads();
    return s.bar;
}
/* The K best of the n gathered ones, in order, into `sorted` (0 where there
 * are none); every thread, after a barrier. `lists`: they are so many lists of K
 * in order (0: they are in none). */
__device__ __noinline__ void top_sort(TopBlock &s, uint32_t n, uint32_t K, uint32_t lists = 0)
{
    const uint32_t t = threadIdx.x;
    uint64_t *from = s.got;
    if (n > GPUOS_TOPB_PLAIN) { /* first those that reach a bar of their own */
        uint64_t mine = 0, bar;
        if (t == 0) s.left = 0;
        if (lists) { /* of the lists' first 256 entries: their K-th lets little more pass than K (one row of
                      * 128,000, 32 lists, K = 64: 13 us; the best of every 256th entry instead: 107) */
            const uint32_t f = t % lists, k = t / lists;
            if (k < min(K, GPUOS_TOPB_THREADS / lists)) mine = s.got[f * K + k];
            bar = top_bar_exact(s, mine, K);
        } else {
            for (uint32_t i = t; i < n; i += GPUOS_TOPB_THREADS) mine = max(mine, s.got[i]);
            bar = top_bar(s, mine, K);
        }
        for (uint32_t i = t; i < n; i += GPUOS_TOPB_THREADS) {
            const uint64_t x = s.got[i];
            if (x <= bar) continue;
            const uint32_t at = atomicAdd(&s.left, 1u);
            if (at < GPUOS_TOPB_SOME) s.few[at] = x;
        }
        __syncthreads();
        if (s.left <= GPUOS_TOPB_SOME) n = s.left, from = s.few;
    }
    if (t < K) s.sorted[t] = 0;
    const uint32_t n8 = top_fill(from, n);
    __syncthreads();
    for (uint32_t i = t; i < n; i += GPUOS_TOPB_THREADS) {
        const uint64_t x = from[i];
        const uint32_t r = top_rank(from, n8, x);
        if (r < K && x) s.sorted[r] = x;
    }
    __syncthreads();
}
/* The block's row state from the threads' (m, l); every thread has it after. */
DEV void top_block_softmax(TopBlock &s, float &m, float &l)
{
    top_softmax(m, l);
    if (lane_id() == 0) s.part[threadIdx.x >> 5] = make_float2(m, l);
    __syncthreads();
    const uint32_t w = lane_id() & (GPUOS_TOPB_WARPS - 1u);
    m = s.part[w].x, l = lane_id() < GPUOS_TOPB_WARPS ? s.part[w].y : 0.0f;
    top_softmax(m, l);
    __syncthreads();
}
DEV void top_block_write(const gpuos_devdesc &d, uint32_t row, const TopBlock &s, float m, float l)
{
    const uint32_t K = d.dims[3], t = threadIdx.x;
    const float ls = logf(l); /* (-infinity if nothing but -infinity was there; next to 1 the hardware's is off by 2^-22) */
    if (t < K) {
        const float x = choose_unkey((uint32_t)(s.sorted[t] >> 32));
        reinterpret_cast<uint32_t *>(d.out)[(uint64_t)row * K + t] = GPUOS_FULL - (uint32_t)s.sorted[t];
        reinterpret_cast<float *>(d.aux0)[(uint64_t)row * K + t] = x == -INFINITY ? x : x - m - ls;
    }
    if (d.aux1 && t == 0) reinterpret_cast<float *>(d.aux1)[row] = m + ls;
}
/* A vector as a thread's elements from i on. */
template <bool F32>
DEV void top_vector(const uint4 &v, float (&x)[TopUnit<F32>::G][8], uint32_t i)
{
    if (F32) {
        const uint32_t u = i >> 3, j = i & 4u;
        x[u][j] = __uint_as_float(v.x), x[u][j + 1] = __uint_as_float(v.y), x[u][j + 2] = __uint_as_float(v.z), x[u][j + 3] = __uint_as_float(v.w);
    } else {
        unpack8(v, x[i >> 3]);
    }
}
/* A unit's elements in this thread, -infinity outside [lo, hi): those at places
 * [b0, b1) (whole vectors) out of `stage`, which begins at u0 (or, not STAGED,
 * from the row); the others, of which a row's ends have a few, from the row. */
template <bool F32, bool STAGED>
DEV void top_load(const ChooseRow<F32> &r, const unsigned char *stage, uint32_t u0, uint32_t b0, uint32_t b1, uint32_t lo, uint32_t hi,
                  float (&x)[TopUnit<F32>::G][8])
{
    using U = TopUnit<F32>;
#pragma unroll
    for (uint32_t u = 0; u < U::G; u++)
#pragma unroll
        for (uint32_t j = 0; j < 8; j += U::PER) {
            const uint32_t p = u0 + U::at(u, j);
            if (p >= b0 && p < b1) {
                top_vector<F32>(STAGED ? *reinterpret_cast<const uint4 *>(stage + U::at(u, j) * (F32 ? 4u : 2u)) : __ldcg(r.vec(p)), x, 8u * u + j);
            } else {
#pragma unroll
                for (uint32_t k = 0; k < U::PER; k++) x[u][(j + k) & 7u] = p + k >= lo && p + k < hi ? r.one(p + k) : -INFINITY;
            }
        }
}
/* The thread's best of a unit (0: it has none). */
template <bool F32>
DEV uint64_t top_mine(const float (&x)[TopUnit<F32>::G][8], uint32_t u0, uint32_t lo, uint32_t hi, uint32_t row_lo)
{
    using U = TopUnit<F32>;
    float most = -INFINITY;
#pragma unroll
    for (uint32_t u = 0; u < U::G; u++)
#pragma unroll
        for (uint32_t j = 0; j < 8; j++) most = fmaxf(most, x[u][j]);
    uint32_t at = GPUOS_FULL; /* the first of equal ones (places rise with u and j) */
#pragma unroll
    for (int i = 8 * U::G - 1; i >= 0; i--)
        if (x[i >> 3][i & 7] == most) at = u0 + U::at((uint32_t)i >> 3, (uint32_t)i & 7u);
    if (most == -INFINITY) { /* which stands for what is not there too */
        at = GPUOS_FULL;
#pragma unroll 1
        for (uint32_t i = 0; i < 8u * U::G; i++) {
            const uint32_t p = u0 + U::at(i >> 3, i & 7u);
            if (p >= lo && p < hi) {
                at = p;
                break;
            }
        }
    }
    return at == GPUOS_FULL ? 0ull : top_entry(most, at - row_lo);
}
DEV void top_push(TopBlock &s, uint64_t bar, float x, uint32_t p, uint32_t lo, uint32_t hi, uint32_t row_lo)
{
    const uint64_t e = top_entry(fmaxf(x, -INFINITY), p - row_lo);
    if (e <= bar || p < lo || p >= hi) return;
    const uint32_t at = atomicAdd(&s.count, 1u);
    if (at < GPUOS_TOPB_ROOM) s.got[at] = e;
}
/* Gathering when the bar let more pass than there is room for (rows that rise,
 * or lie in few places): the bar rises with each unit, exactly, so that no
 * more than K threads' elements pass, and what is gathered is cut to the K
 * best. Returns how many there are; every thread. */
template <bool F32>
__device__ __noinline__ uint32_t top_gather_slow(TopBlock &s, const ChooseRow<F32> r, uint32_t from, uint32_t lo, uint32_t hi, uint32_t K)
{
    using U = TopUnit<F32>;
    const uint32_t t = threadIdx.x;
    uint64_t bar = 0;
    __syncthreads();
    if (t == 0) s.count = 0;
#pragma unroll 1
    for (uint32_t u0 = from; u0 < hi; u0 += TopUnit<F32>::N) {
        float x[TopUnit<F32>::G][8];
        top_load<F32, false>(r, nullptr, u0, (lo + U::PER - 1u) & ~(U::PER - 1u), hi & ~(U::PER - 1u), lo, hi, x);
        const uint64_t mine = top_mine<F32>(x, u0, lo, hi, r.lo);
        const uint32_t above = (uint32_t)__syncthreads_count(mine > bar);
        if (above == 0) continue;
        if (above > K) {
            s.best[t] = mine;
            __syncthreads();
            if (mine > bar && top_rank(s.best, GPUOS_TOPB_THREADS, mine) == K) s.bar = mine; /* (K others' are above it) */
            __syncthreads();
            bar = s.bar;
        }
        if (mine > bar)
#pragma unroll
            for (uint32_t u = 0; u < TopUnit<F32>::G; u++)
#pragma unroll
                for (uint32_t j = 0; j < 8; j++) top_push(s, bar, x[u][j], u0 + TopUnit<F32>::at(u, j), lo, hi, r.lo);
        __syncthreads();
        const uint32_t n = s.count;
        if (n > GPUOS_TOPB_FEW) { /* the K best so far, and the bar at the last of them */
            top_sort(s, n, K);
            if (t < K) s.got[t] = s.sorted[t];
            if (t == 0) s.count = K;
            bar = max(bar, s.sorted[K - 1]);
        }
    }
    __syncthreads();
    return s.count;
}
DEV float top_ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
/* The rows' cells (256 elements each; their number is below 2^32) in runs: S
 * runs of each row, or runs across rows that differ by one at most, of which
 * the first `more` have one more. */
struct TopRuns {
    uint32_t S, base, more, cells;
    DEV TopRuns(const gpuos_devdesc &d, uint32_t cells_of_a_row)
        : S((uint32_t)d.dep[0]), base((uint32_t)d.dep[1]), more((uint32_t)(d.dep[1] >> 32)), cells(cells_of_a_row)
    {
    }
    DEV uint32_t start(uint32_t run) const
    {
        if (S == 0) return run * base + min(run, more);
        const uint32_t row = run / S;
        return row * cells + (run - row * S) * cells / S; /* (a row has fewer than 2^23 cells, and S is at most 32) */
    }
    DEV uint32_t run_of(uint32_t u) const /* (only across rows) */
    {
        const uint32_t cut = more * (base + 1u);
        return u < cut ? u / (base + 1u) : more + (u - cut) / base;
    }
};
/* A place in a run: a row and, of it, the units from u0 on, up to `end`. */
struct TopCursor {
    uint32_t cell; /* the piece's first */
    uint32_t row, u0, end;
};
template <bool F32>
struct TopWork {
    const gpuos_devdesc &d;
    uint32_t V, cells; /* of a row */
    uint32_t last;     /* the run's end */
    /* the piece that begins at a cell */
    DEV void piece(uint32_t cell, TopCursor &c) const
    {
        c.cell = cell;
        c.row = cell / cells;
        const uint32_t begin = c.row * cells;
        c.u0 = (cell - begin) * 256u;
        c.end = min(cells, last - begin) * 256u;
    }
    /* the next unit; false: the run is over */
    DEV bool next(TopCursor &c) const
    {
        c.u0 += TopUnit<F32>::N;
        if (c.u0 < c.end) return true;
        const uint32_t cell = c.row * cells + c.end / 256u;
        if (cell >= last) return false;
        piece(cell, c);
        return true;
    }
};
template <bool F32>
__global__ void __launch_bounds__(GPUOS_TOPB_THREADS, 3) gpuos_top_kernel(const __grid_constant__ gpuos_devdesc d)
{
    using U = TopUnit<F32>;
    constexpr uint32_t ST = GPUOS_TOPB_STAGES, SIZE = F32 ? 4u : 2u;
    extern __shared__ __align__(128) unsigned char top_ring[];
    __shared__ TopBlock s;
    __shared__ __align__(8) unsigned long long full[ST], empty[ST];
    const uint32_t V = d.dims[1], K = d.dims[3], t = threadIdx.x;
    constexpr float L2E = 1.44269504f; /* (its error is the same for every element: 1e-8 of their distance from the maximum) */
    const uint32_t cells = (V + 7u + 255u) / 256u; /* (a row may begin seven elements behind its first vector) */
    const TopRuns runs(d, cells);
    const TopWork<F32> work{d, V, cells, runs.start(blockIdx.x + 1u)};
    /* the whole vectors of a unit, [first, second) */
    auto whole = [&](const ChooseRow<F32> &r, uint32_t u0, uint32_t lo, uint32_t hi) {
        const uint32_t b0 = max(u0, (lo + U::PER - 1u) & ~(U::PER - 1u));
        return make_uint2(b0, max(b0, min(u0 + U::N, hi & ~(U::PER - 1u))));
    };
    auto copy = [&](const TopCursor &c, uint32_t at) { /* one thread */
        const ChooseRow<F32> r(d.a, c.row, d.dims[2], V);
        const uint2 b = whole(r, c.u0, max(c.u0, r.lo), min(c.end, r.hi));
        const uint32_t bytes = (b.y - b.x) * SIZE;
        if (bytes == 0) {
            asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&full[at])) : "memory");
            return;
        }
        mbar_expect(&full[at], bytes);
        bulk_g2s(top_ring + at * U::BYTES + (b.x - c.u0) * SIZE, r.vec(b.x), bytes, &full[at]);
    };
    if (t == 0) {
#pragma unroll
        for (uint32_t k = 0; k < ST; k++) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(&full[k])) : "memory");
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(&empty[k])), "n"(GPUOS_TOPB_WARPS) : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    kv4_after_previous();
    TopCursor c, ahead; /* the unit that is worked on, and the one whose copy is issued next */
    work.piece(runs.start(blockIdx.x), c);
    ahead = c;
    bool more = true; /* there is such a one */
#pragma unroll
    for (uint32_t k = 0; k < ST; k++) {
        if (more && t == 32u * k) copy(ahead, k);
        more = more && work.next(ahead);
    }
    uint32_t at = 0, turn = 0, n_unit = 0; /* the ring's position */
    bool lost = false; /* a copy did not arrive (bounded, like every wait): the numbers are NaN from there on */
#pragma unroll 1
    while (true) {
        const ChooseRow<F32> r(d.a, c.row, d.dims[2], V);
        const uint32_t from = c.u0, lo = max(from, r.lo), hi = min(c.end, r.hi), row = c.row;
        const uint32_t first = c.cell;
        /* sum of 2^(L2E x - ml), ml = L2E m rounded; and, of units whose largest is
         * so far from 0 that rounding would tell, the sum of e^(x - far_m) */
        float m = -2e6f, ml = -2e6f * L2E, l = 0.0f, far_m = -FLT_MAX, far_l = 0.0f;
        uint64_t bar = 0;
        float barf = -INFINITY;
        __syncthreads(); /* (the last piece is done with what it gathered) */
        if (t == 0) s.count = 0;
        bool again; /* this piece has a further unit */
#pragma unroll 1
        do {
            const uint32_t u0 = c.u0;
            const uint2 b = whole(r, u0, lo, hi);
            float x[U::G][8], unit = -INFINITY;
            if (!mbar_wait(&full[at], turn)) lost = true;
            if (b.x == u0 && b.y == u0 + U::N) {
#pragma unroll
                for (uint32_t i = 0; i < 8u * U::G; i += U::PER)
                    top_vector<F32>(*reinterpret_cast<const uint4 *>(top_ring + at * U::BYTES + U::at(i >> 3, i & 7u) * SIZE), x, i);
            } else { /* a row's first or last */
                top_load<F32, true>(r, top_ring + at * U::BYTES, u0, b.x, b.y, lo, hi, x);
            }
#pragma unroll
            for (uint32_t i = 0; i < 8u * U::G; i += 2) unit = choose_max3(unit, x[i >> 3][i & 7u], x[i >> 3][(i & 7u) + 1]);
            if (fabsf(unit) <= 1e6f) {
                if (unit > m) {
                    const float to = unit * L2E;
                    l *= top_ex2(ml - to);
                    m = unit, ml = to;
                }
                float all = 0.0f; /* (sums of sums: a rounding for each unit, not for each element) */
#pragma unroll
                for (uint32_t u = 0; u < U::G; u++) {
                    float sum = 0.0f;
#pragma unroll
                    for (uint32_t j = 0; j < 8; j++) sum += top_ex2(fmaf(x[u][j], L2E, -ml));
                    all += sum;
                }
                if (!(all == all)) { /* a NaN among the logits counts as -infinity */
                    all = 0.0f;
#pragma unroll
                    for (uint32_t u = 0; u < U::G; u++)
#pragma unroll
                        for (uint32_t j = 0; j < 8; j++) all += top_ex2(fmaf(fmaxf(x[u][j], -INFINITY), L2E, -ml));
                }
                l += all;
            } else if (unit != -INFINITY) {
                const float to = fmaxf(far_m, fminf(unit, FLT_MAX)); /* (an infinite maximum: the sum is infinite) */
                far_l *= choose_exp(far_m - to);
                far_m = to;
#pragma unroll
                for (uint32_t u = 0; u < U::G; u++)
#pragma unroll
                    for (uint32_t j = 0; j < 8; j++) far_l += top_ex2((fmaxf(x[u][j], -INFINITY) - far_m) * L2E);
            }
            if (u0 == from) {
                bar = top_bar(s, top_mine<F32>(x, u0, lo, hi, r.lo), K);
                barf = bar ? choose_unkey((uint32_t)(bar >> 32)) : -INFINITY; /* (that bar's value itself may pass) */
            }
            const bool strict = u0 != from && bar != 0; /* (an equal one in a later unit comes after) */
            if (strict ? unit > barf : unit >= barf) {
                uint32_t reach = 0;
#pragma unroll
                for (uint32_t i = 0; i < 8u * U::G; i++) reach |= x[i >> 3][i & 7u] > barf ? 1u << i : 0u;
                if (!strict) {
#pragma unroll
                    for (uint32_t i = 0; i < 8u * U::G; i++) reach |= !(x[i >> 3][i & 7u] < barf) ? 1u << i : 0u;
                }
#pragma unroll 1
                for (; reach; reach &= reach - 1u) { /* (few: read again, so that no array needs an index) */
                    const uint32_t k = (uint32_t)__ffs((int)reach) - 1u, o = U::at(k >> 3, k & 7u), p = u0 + o;
                    float v = 0.0f;
                    if (p >= b.x && p < b.y) {
                        const unsigned char *e = top_ring + at * U::BYTES + o * SIZE;
                        v = F32 ? *reinterpret_cast<const float *>(e) : bf1(*reinterpret_cast<const uint16_t *>(e));
                    } else if (p >= lo && p < hi) {
                        v = r.one(p);
                    }
                    top_push(s, bar, v, p, lo, hi, r.lo);
                }
            }
            __syncwarp(); /* this warp is done with its elements */
            if (lane_id() == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&empty[at])) : "memory");
            /* the unit's place takes the unit ahead, once all warps have left it; the warps take turns at that */
            if (more) {
                if (t == 32u * (n_unit % GPUOS_TOPB_WARPS)) {
                    if (!mbar_wait(&empty[at], turn)) lost = true;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    copy(ahead, at);
                }
                more = work.next(ahead);
            }
            __syncwarp();
            if (++at == ST) at = 0, turn ^= 1u;
            n_unit++;
            again = u0 + U::N < c.end;
            c.u0 = u0 + U::N;
            const uint32_t nth = (u0 - from) / U::N;
            if (again && ((nth == 3u && c.end - u0 > 8u * U::N) || (nth & 7u) == 7u)) { /* a better bar, if some were gathered */
                __syncthreads();
                const uint32_t n = s.count;
                if (n > K && n <= GPUOS_TOPB_ROOM && (nth == 3u || n > 64u + K)) {
                    top_sort(s, n, K);
                    if (t < K) s.got[t] = s.sorted[t];
                    if (t == 0) s.count = K;
                    bar = max(bar, s.sorted[K - 1u]);
                    barf = choose_unkey((uint32_t)(bar >> 32));
                }
                __syncthreads();
            }
        } while (again);
        if (l > 0.0f) { /* both sums under one maximum */
            l *= top_ex2(-fmaf(m, L2E, -ml));
            const float M = fmaxf(m, far_m);
            l = l * choose_exp(m - M) + far_l * choose_exp(far_m - M);
            m = M;
        } else {
            m = far_m, l = far_l;
        }
        if (__syncthreads_or(lost)) l = __int_as_float(0x7FFFFFFF);
        uint32_t n = s.count;
        if (n > GPUOS_TOPB_ROOM) n = top_gather_slow(s, r, from, lo, hi, K);
        top_sort(s, n, K);
        top_block_softmax(s, m, l);
        const uint32_t row0 = row * cells, end = row0 + c.end / 256u;
        if (first == row0 && end == row0 + cells) {
            top_block_write(d, row, s, m, l);
        } else {
            /* the row's last block joins the pieces: a block's first piece is in its
             * place 0, a later one (which begins a row) in 1; they are counted at
             * the row's first block */
            const uint32_t blk0 = runs.S ? row * runs.S : runs.run_of(row0), F = runs.S ? runs.S : runs.run_of(row0 + cells - 1u) - blk0 + 1u;
            unsigned char *p = top_part(&d, blockIdx.x * 2u + (blockIdx.x == blk0 ? 1u : 0u));
            if (t < K) __stcg(reinterpret_cast<unsigned long long *>(p + 16) + t, (unsigned long long)s.sorted[t]);
            if (t == 0) __stcg(reinterpret_cast<float2 *>(p), make_float2(m, l));
            __syncthreads();
            if (t == 0) {
                uint32_t *ctr = reinterpret_cast<uint32_t *>(d.aux2) + blk0;
                s.last = atom_add_acq_rel_gpu32(ctr, 1u) == F - 1u;
                if (s.last) *ctr = 0; /* left zero for the next call */
            }
            __syncthreads();
            if (s.last) {
                auto part = [&](uint32_t f) { return top_part(&d, (blk0 + f) * 2u + (f == 0 ? 1u : 0u)); };
                m = -FLT_MAX, l = 0.0f;
                if (t < F) {
                    const float2 ms = __ldcg(reinterpret_cast<const float2 *>(part(t)));
                    m = ms.x, l = ms.y;
                }
                for (uint32_t i = t; i < F * K; i += GPUOS_TOPB_THREADS) /* (entries that are not there are 0, and below all others) */
                    s.got[i] = __ldcg(reinterpret_cast<const unsigned long long *>(part(i / K) + 16) + i % K);
                __syncthreads();
                top_sort(s, F * K, K, F);
                top_block_softmax(s, m, l);
                top_block_write(d, row, s, m, l);
            }
        }
        if (end >= work.last) break;
        work.piece(end, c);
    }
}

template <bool F32>
static int top_launch(const gpuos_devdesc &d, void *stream)
{
    /* Runs: as many as run at a time, and none below a unit or a 32nd of a row
     * (what a row's last block can join). Whole rows, or as many equal runs of
     * each as fit, are one piece for each block; other runs balance better but
     * have more pieces, each of which has a start and an end. */
    const uint64_t B = d.dims[0], cells = ((uint64_t)d.dims[1] + 7u + 255u) / 256u, unit = GPUOS_TOPB_UNIT / 256u;
    const uint64_t most = min(min((uint64_t)GPUOS_TOPB_SLOTS, 32u * B), B * ((cells + unit - 1u) / unit));
    if (B * cells >= 1ull << 32) return -1; /* (elements for 500 GB) */
    gpuos_devdesc e = d;
    uint64_t grid = most;
    e.dep[0] = 0;
    if (B <= most) {
        const uint64_t S = most / B, even = cells / S + GPUOS_TOPB_FIXED, uneven = B * cells / most + 2u * GPUOS_TOPB_FIXED;
        if (even <= uneven) grid = B * S, e.dep[0] = S;
    }
    e.dep[1] = B * cells / grid | (B * cells % grid) << 32;
    static std::atomic<bool> known[64];
    if (choose_smem((const void *)gpuos_top_kernel<F32>, GPUOS_TOPB_STAGES * TopUnit<F32>::BYTES, known) != 0) return -1;
    return choose_launch(gpuos_top_kernel<F32>, dim3((uint32_t)grid), GPUOS_TOPB_THREADS, GPUOS_TOPB_STAGES * TopUnit<F32>::BYTES, stream, e);
}

/* ---------------------------------------------------------------------------
 * The experts of a token, launched: eight or sixteen lanes a token, neighbouring
 * experts in a lane, so that a group is one lane's or a few neighbours'. What
 * may be among the K best are the values that reach a bar which K + 1 of the
 * lanes' best three reach; they are gathered, and ranked by comparing
 * all with all. Values are floats to the end; NaN is what may not be chosen.
 *
 * 32,768 tokens of 256 experts (f32, sigmoid, bias, four of eight groups by their
 * two best, K = 8): 31 us against 5.3 of memory: 1,060 warp instructions for two
 * tokens, issue slots 63 % used, the half-rate pipe of minima, maxima and
 * comparisons 50 %. Without bias and groups 18 us. 65,536 of 64 experts 16.1 us.
 * (A warp's next rows asked for ahead: 30.7; 1,024 to 4,096 blocks: 32 to 35.)
 * Where values are near, 1 token in 1,000 here, sums of two floats tell them
 * apart (with 64-bit arithmetic instead the launch took 45 us, its last tokens
 * 15 of them). A kernel for each kind of score and bias would save 6 % of it.
 * ------------------------------------------------------------------------- */
#define GPUOS_ROUTEB_THREADS 128
#define GPUOS_ROUTEB_ROOM 64u /* gathered values of a token at most; more: the token goes the sure way */
#define GPUOS_ROUTEB_MAX_K 15u
#define GPUOS_ROUTEB_BLOCKS 1216u /* at most, eight for each SM: as many as run at a time */
struct RouteToken {
    uint64_t got[GPUOS_ROUTEB_ROOM]; /* value and expert, as one number to compare by */
    float2 fine[GPUOS_ROUTEB_ROOM];  /* the value as a sum of two floats */
    uint64_t best[16];
    float logit[GPUOS_ROUTEB_ROOM], best_logit[16];
    uint16_t id[GPUOS_ROUTEB_ROOM];
};
/* Over a token's L lanes. */
template <int L>
DEV float lanes_max(float v)
{
#pragma unroll
    for (int o = 1; o < L; o <<= 1) v = fmaxf(v, __shfl_xor_sync(GPUOS_FULL, v, o));
    return v;
}
template <int L>
DEV float lanes_sum(float v)
{
#pragma unroll
    for (int o = 1; o < L; o <<= 1) v += __shfl_xor_sync(GPUOS_FULL, v, o);
    return v;
}
/* The lanes' values from the largest down: runs of a size are merged by a
 * comparison of each lane with its mirror image, then with lanes ever nearer;
 * the larger always goes to the lower lane. */
template <int L>
DEV float lanes_sort(float v)
{
    const uint32_t lane = lane_id();
#pragma unroll
    for (uint32_t size = 2; size <= L; size <<= 1)
#pragma unroll
        for (uint32_t o = size >> 1; o; o >>= 1) {
            const float other = __shfl_xor_sync(GPUOS_FULL, v, (int)(o == size >> 1 ? size - 1u : o));
            v = lane & o ? fminf(v, other) : fmaxf(v, other);
        }
    return v;
}
/* For choosing only: few instructions, and off by at most 2^-21 of itself and
 * |x| 2^-23 of itself where x is negative. */
DEV float route_sigmoid_fast(float x)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.44269504f)); /* (infinite below -88: 0) */
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}
/* Sums of two floats, x = h + l: Dekker's and Knuth's error-free sums, and
 * products with the fused multiply-add ("double-double" arithmetic). */
DEV float2 pair_sum(float a, float b)
{
    const float h = __fadd_rn(a, b), z = __fsub_rn(h, a);
    return make_float2(h, __fadd_rn(__fsub_rn(a, __fsub_rn(h, z)), __fsub_rn(b, z)));
}
DEV float2 pair_add(float2 a, float2 b)
{
    const float2 s = pair_sum(a.x, b.x);
    return pair_sum(s.x, __fadd_rn(s.y, __fadd_rn(a.y, b.y)));
}
DEV float2 pair_mul(float2 a, float2 b)
{
    const float h = __fmul_rn(a.x, b.x);
    const float l = __fmaf_rn(a.x, b.y, __fmaf_rn(a.y, b.x, __fmaf_rn(a.x, b.x, -h)));
    return pair_sum(h, l);
}
/* 1 / (1 + e^-x) for |x| <= 80, off by less than 2^-42: e^-x = 2^n e^r with
 * |r| <= ln 2 / 2, e^r by its power series (terms from r^7 / 7! on, below 2^-22,
 * in one float), the quotient by one step of Newton's. */
DEV float2 route_sigmoid_fine(float x)
{
    const float t = fminf(fmaxf(-x, -80.0f), 80.0f), n = rintf(t * 1.44269504f);
    /* ln 2 = 0x1.62ep-1 + 0x1.0bfbe8p-15 + 0x1.cf79acp-40 - ...: the first product is exact */
    float2 r = pair_sum(__fmaf_rn(-n, 0x1.62ep-1f, t), 0.0f);
    const float m = __fmul_rn(-n, 0x1.0bfbe8p-15f);
    r = pair_add(r, make_float2(m, __fmaf_rn(-n, 0x1.cf79acp-40f, __fmaf_rn(-n, 0x1.0bfbe8p-15f, -m))));
    const float y = r.x;
    float tail = 1.0f / 479001600.0f;
    tail = fmaf(tail, y, 1.0f / 39916800.0f);
    tail = fmaf(tail, y, 1.0f / 3628800.0f);
    tail = fmaf(tail, y, 1.0f / 362880.0f);
    tail = fmaf(tail, y, 1.0f / 40320.0f);
    tail = fmaf(tail, y, 1.0f / 5040.0f);
    /* 1 / 720, 1 / 120, 1 / 24, 1 / 6 as sums of two floats */
    float2 p = pair_add(make_float2(0x1.6c16c2p-10f, -0x1.27d27ep-35f), pair_sum(__fmul_rn(tail, y), 0.0f));
    p = pair_add(make_float2(0x1.111112p-7f, -0x1.dddddep-32f), pair_mul(p, r));
    p = pair_add(make_float2(0x1.555556p-5f, -0x1.555556p-30f), pair_mul(p, r));
    p = pair_add(make_float2(0x1.555556p-3f, -0x1.555556p-28f), pair_mul(p, r));
    p = pair_add(make_float2(0.5f, 0.0f), pair_mul(p, r));
    p = pair_add(make_float2(1.0f, 0.0f), pair_mul(p, r));
    p = pair_add(make_float2(1.0f, 0.0f), pair_mul(p, r));
    const float f = kv4_pow2((int)n);
    const float2 q = pair_add(make_float2(1.0f, 0.0f), make_float2(p.x * f, p.y * f));
    const float g = __frcp_rn(q.x);
    const float e = __fmaf_rn(-g, q.y, __fmaf_rn(-g, q.x, 1.0f));
    return pair_sum(g, __fmul_rn(g, e));
}
/* What two values of that kind, or sums of two, may differ by and yet be the
 * other way round. */
DEV float pair_unsure(float wide) { return (1.0f + wide) * 0x1p-39f; }
DEV float pair_less(float2 a, float2 b) { return (a.x - b.x) + (a.y - b.y); } /* a - b, to a part in 2^24 */
struct RouteGathered {
    const float *bias; /* (in shared memory, none NaN) */
    uint32_t have, lanes;
    float wide;
};
/* A token whose groups are sure, but not its experts: all that may be among
 * them are gathered, and are ranked again by finer values (sigmoid scores and
 * biases). Every lane of the token; false if that does not tell either. Only
 * values of equal logits and biases may be equal, and infinite ones. */
__device__ __noinline__ bool op_y_fine(RouteToken *s, uint32_t sub, uint32_t L, const RouteGathered q)
{
#pragma unroll 1
    for (uint32_t i = sub; i < q.have; i += L) {
        const float x = s->logit[i], b = q.bias[s->id[i]];
        s->fine[i] = x == -INFINITY ? make_float2(b, 0.0f) : (fabsf(b) <= FLT_MAX ? pair_add(route_sigmoid_fine(x), make_float2(b, 0.0f)) : make_float2(b, 0.0f));
    }
    __syncwarp(q.lanes);
    bool told = true;
#pragma unroll 1
    for (uint32_t i = sub; i < q.have; i += L) {
        const float2 v = s->fine[i];
        const uint32_t id = s->id[i];
        const float x = s->logit[i], b = q.bias[id];
        uint32_t rank = 0;
#pragma unroll 1
        for (uint32_t k = 0; k < q.have; k++) {
            if (k == i) continue;
            const float2 o = s->fine[k];
            const float more = pair_less(o, v);
            /* (infinite values are equal whatever their logits; their difference is NaN) */
            const bool alike = (s->logit[k] == x && q.bias[s->id[k]] == b) || (o.x == v.x && fabsf(v.x) > FLT_MAX);
            if (alike ? s->id[k] < id : more > 0.0f || o.x > v.x) rank++;
            if (!alike && fabsf(more) <= pair_unsure(q.wide)) told = false;
        }
        if (rank < 16u) s->best[rank] = s->got[i], s->best_logit[rank] = x;
    }
    __syncwarp(q.lanes);
    return told;
}
/* VPL >= values a lane; VEC: as many, and whole 16-byte vectors */
template <bool F32, int L, int VPL, bool VEC>
__global__ void __launch_bounds__(GPUOS_ROUTEB_THREADS, VPL <= 16 ? 8 : 7) gpuos_route_kernel(const __grid_constant__ gpuos_devdesc d)
{
    __shared__ RouteToken tokens[GPUOS_ROUTEB_THREADS / L];
    __shared__ __align__(16) float biases[L][VPL + 4]; /* (four more: the lanes' vectors lie in different banks) */
    __shared__ float flat[L * VPL]; /* ... in the experts' order */
    constexpr uint32_t TOKENS = 32 / L; /* of a warp */
    const float none = __int_as_float(0x7FFFFFFF);
    const uint32_t lane = lane_id(), sub = lane & (L - 1), own = lane & ~(uint32_t)(L - 1), warp = threadIdx.x >> 5;
    const uint32_t lanes = ((1u << L) - 1u) << own;
    RouteToken &s = tokens[threadIdx.x / L];
    kv4_after_previous();
    RouteArgs a;
    route_args(&d, a);
    const uint32_t rows = a.rows ? (uint32_t)max(*a.rows, 0) : a.N;
    const uint32_t P = VEC ? (uint32_t)VPL : (a.E + L - 1u) / L, first = sub * P; /* this lane's experts */
    const bool sigmoid = a.flags & GPUOS_ROUTE_SIGMOID, summed = a.G > 1 && a.flags & GPUOS_ROUTE_TOP2, biased = a.bias != nullptr;
    const bool norm = a.flags & GPUOS_ROUTE_NORM;
    const uint32_t span = L / a.G, group = sub / span; /* lanes of a group */
    /* of K + 1 that reach the bar, how many are lanes' best, second and third
     * best (in random order six of nine are the first, and two the second) */
    const uint32_t live = a.keep * span, ones = min(live, (2u * a.K + 4u) / 3u), twos = min(live, a.K + 1u - ones), threes = a.K + 1u - ones - twos;
    float wide = 0.0f;
    if (biased) {
        for (uint32_t i = threadIdx.x; i < L * P; i += GPUOS_ROUTEB_THREADS) {
            const float b = i < a.E ? fmaxf(a.bias[i], -INFINITY) : 0.0f;
            biases[i / P][i % P] = flat[i] = b;
        }
        __syncthreads();
        for (uint32_t i = sub; i < a.E; i += L) wide = fmaxf(wide, fabsf(flat[i]) <= FLT_MAX ? fabsf(flat[i]) : 0.0f);
        wide = lanes_max<L>(wide) + 1.0f; /* no value is larger */
    }
    const uint32_t step = gridDim.x * (GPUOS_ROUTEB_THREADS / L);
#pragma unroll 1
    for (uint32_t n0 = (blockIdx.x * (GPUOS_ROUTEB_THREADS / 32u) + warp) * TOKENS; n0 < a.N; n0 += step) {
        const uint32_t n = min(n0 + lane / L, a.N - 1u); /* (the last token may be done twice) */
        const bool pad = n >= rows;
        const unsigned char *row = reinterpret_cast<const unsigned char *>(d.a) + ((uint64_t)n * a.ld + first) * (F32 ? 4u : 2u);
        float c[VPL]; /* what is chosen by */
        if (VEC) {
#pragma unroll
            for (int i = 0; i < VPL; i += F32 ? 4 : 8) {
                const uint4 v = reinterpret_cast<const uint4 *>(row)[i / (F32 ? 4 : 8)];
                if (F32) {
                    c[i] = __uint_as_float(v.x), c[i + 1] = __uint_as_float(v.y), c[i + 2] = __uint_as_float(v.z), c[i + 3] = __uint_as_float(v.w);
                } else {
                    float f[8];
                    unpack8(v, f);
#pragma unroll
                    for (int j = 0; j < 8 && i + j < VPL; j++) c[i + j] = f[j];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                c[i] = -INFINITY;
                if (i < (int)P && first + i < a.E)
                    c[i] = F32 ? reinterpret_cast<const float *>(row)[i] : bf1(reinterpret_cast<const uint16_t *>(row)[i]);
            }
        }
        float most = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; i += 2) asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(most) : "f"(c[i]), "f"(c[i + 1]));
        if (__any_sync(GPUOS_FULL, most != most)) { /* a NaN counts as -infinity */
            most = -INFINITY;
#pragma unroll
            for (int i = 0; i < VPL; i++) c[i] = fmaxf(c[i], -INFINITY), most = fmaxf(most, c[i]);
        }
        most = fminf(lanes_max<L>(most), FLT_MAX);
        float inv = 1.0f; /* (a softmax whose scores are only divided by one another does without its sum) */
        if (!sigmoid && (biased || summed || !norm)) {
            float total = 0.0f;
#pragma unroll
            for (int i = 0; i < VPL; i++) total += route_score(false, c[i], most, 1.0f);
            total = lanes_sum<L>(total);
            inv = total > 0.0f ? 1.0f / total : 0.0f;
        }
        if (biased) {
#pragma unroll
            for (int i = 0; i < VPL; i++) c[i] = (sigmoid ? route_sigmoid_fast(c[i]) : route_score(false, c[i], most, inv)) + biases[sub][i];
        }
        /* What two values may differ by and yet be the other way round: twice a
         * value's error. A sigmoid's is 2^-21 of itself (ex2 2^-22, the reciprocal
         * and a sum) and, where x < 0, 1.5 |x| 2^-24 of itself (its argument's
         * rounding); |x| s(x) is at most (1 + |most|) s(most) there. A softmax's
         * 2^-19 (its sum's errors too). A sum with the bias: 2^-24 more of itself. */
        const float low = fmaxf(fminf(most, 0.0f), -256.0f); /* (s(most) is 0 before that) */
        const float unsure = (sigmoid ? route_sigmoid_fast(most) * (0x1.8p-20f - low * 0x1p-21f) : inv * 0x1p-18f) + wide * 0x1p-22f;
        bool sure = !sigmoid || most >= -60.0f || most == -INFINITY;
        if (!VEC) {
#pragma unroll
            for (int i = 0; i < VPL; i++)
                if (i >= (int)P || first + i >= a.E) c[i] = none;
        }
        /* the lane's best three, or nearly: of its even and its odd values the best two */
        float one, two, three;
        {
            float p1 = -INFINITY, p2 = -INFINITY, q1 = -INFINITY, q2 = -INFINITY;
            auto v = [&](int k) { return VEC || c[k] == c[k] ? c[k] : -INFINITY; };
            auto two_more = [](float &best, float &second, float x, float y) {
                const float more = fmaxf(x, y);
                second = choose_max3(second, fminf(x, y), fminf(best, more));
                best = fmaxf(best, more);
            };
#pragma unroll
            for (int i = 0; i < VPL; i += 4) {
                two_more(p1, p2, v(i), v(i + 2));
                two_more(q1, q2, v(i + 1), v(i + 3));
            }
            one = fmaxf(p1, q1);
            const float r = fminf(p1, q1), t = fmaxf(p2, q2);
            two = fmaxf(r, t);
            three = fmaxf(fminf(r, t), fminf(p2, q2));
        }
        bool shut = false;
        if (a.G > 1) {
            float g1 = one, g2 = two;
            for (uint32_t o = 1; o < span; o <<= 1) {
                const float o1 = __shfl_xor_sync(GPUOS_FULL, g1, (int)o), o2 = __shfl_xor_sync(GPUOS_FULL, g2, (int)o);
                g2 = fmaxf(fminf(g1, o1), fmaxf(g2, o2));
                g1 = fmaxf(g1, o1);
            }
            float mine = g1;
            if (summed) mine = biased ? g1 + g2 : route_score(sigmoid, g1, most, inv) + route_score(sigmoid, g2, most, inv);
            uint32_t rank = 0;
            float next = -INFINITY; /* the best behind this group */
#pragma unroll 4
            for (uint32_t k = 0; k < a.G; k++) {
                const float v = __shfl_sync(GPUOS_FULL, mine, (int)(own + k * span));
                const bool ahead = v > mine || (v == mine && k < group);
                rank += ahead;
                if (!ahead && k != group) next = fmaxf(next, v);
            }
            const bool edge = (biased || summed) && rank == a.keep - 1u && a.keep < a.G, near = edge && mine - next <= 2.0f * unsure;
            if (edge && route_beyond(mine, next, wide)) sure = false;
            if (__any_sync(GPUOS_FULL, near)) {
                if (sigmoid && biased) {
                    /* the groups' values again, finer: of what may be their best, which are few */
                    float2 f1 = make_float2(-INFINITY, 0.0f), f2 = f1;
                    const float from = (summed ? g2 : g1) - unsure;
#pragma unroll 1
                    for (uint32_t i = 0; i < P; i++) {
                        if (first + i >= a.E) break;
                        const uint64_t at = (uint64_t)n * a.ld + first + i;
                        const float x = fmaxf(F32 ? reinterpret_cast<const float *>(d.a)[at] : bf1(reinterpret_cast<const uint16_t *>(d.a)[at]), -INFINITY);
                        const float b = biases[sub][i];
                        if (!(route_sigmoid_fast(x) + b >= from)) continue;
                        float2 v = make_float2(b, 0.0f);
                        if (x != -INFINITY && fabsf(b) <= FLT_MAX) v = pair_add(route_sigmoid_fine(x), v);
                        if (v.x > f1.x || (v.x == f1.x && v.y > f1.y)) f2 = f1, f1 = v;
                        else if (v.x > f2.x || (v.x == f2.x && v.y > f2.y)) f2 = v;
                    }
                    __syncwarp();
                    auto more = [](float2 p, float2 q) { return p.x > q.x || (p.x == q.x && p.y > q.y); };
                    for (uint32_t o = 1; o < span; o <<= 1) {
                        float2 o1 = make_float2(__shfl_xor_sync(GPUOS_FULL, f1.x, (int)o), __shfl_xor_sync(GPUOS_FULL, f1.y, (int)o));
                        float2 o2 = make_float2(__shfl_xor_sync(GPUOS_FULL, f2.x, (int)o), __shfl_xor_sync(GPUOS_FULL, f2.y, (int)o));
                        if (more(o1, f1)) {
                            const float2 x1 = f1, x2 = f2;
                            f1 = o1, f2 = o2, o1 = x1, o2 = x2;
                        }
                        if (more(o1, f2)) f2 = o1;
                    }
                    float2 value = f1;
                    if (summed) value = f2.x == -INFINITY || fabsf(f1.x) > FLT_MAX ? make_float2(f1.x + f2.x, 0.0f) : pair_add(f1, f2);
                    rank = 0;
                    bool told = true;
                    for (uint32_t k = 0; k < a.G; k++) {
                        const float2 v = make_float2(__shfl_sync(GPUOS_FULL, value.x, (int)(own + k * span)), __shfl_sync(GPUOS_FULL, value.y, (int)(own + k * span)));
                        if (k == group) continue;
                        rank += more(v, value) || (v.x == value.x && v.y == value.y && k < group);
                        if (fabsf(pair_less(v, value)) <= 2.0f * pair_unsure(wide)) told = false;
                    }
                    if (!told) sure = false;
                } else if (near) {
                    sure = false;
                }
            }
            shut = rank >= a.keep;
            if (shut) one = two = three = -INFINITY;
        }
        float bar = __shfl_sync(GPUOS_FULL, lanes_sort<L>(one), (int)(own + ones - 1u));
        if (twos) bar = fminf(bar, __shfl_sync(GPUOS_FULL, lanes_sort<L>(two), (int)(own + twos - 1u)));
        if (threes) {
            const float b = __shfl_sync(GPUOS_FULL, lanes_sort<L>(three), (int)(own + min(threes, (uint32_t)L) - 1u));
            bar = threes <= live ? fminf(bar, b) : -INFINITY;
        }
        if (biased) bar -= unsure; /* (what may be the other way round is gathered too) */
        uint32_t reach = 0; /* this lane's that reach it */
#pragma unroll
        for (int i = 0; i < VPL; i++) reach |= c[i] >= bar ? 1u << i : 0u;
        if (shut) reach = 0;
        const uint32_t count = (uint32_t)__popc(reach);
        uint32_t have = count;
#pragma unroll
        for (int o = 1; o < L; o <<= 1) {
            const uint32_t v = __shfl_up_sync(GPUOS_FULL, have, o, L);
            if (sub >= (uint32_t)o) have += v;
        }
        uint32_t at = have - count;
        have = __shfl_sync(GPUOS_FULL, have, L - 1, L);
        if (have > GPUOS_ROUTEB_ROOM) sure = false, have = GPUOS_ROUTEB_ROOM;
        for (; reach; reach &= reach - 1u, at++)
            if (at < GPUOS_ROUTEB_ROOM) s.id[at] = (uint16_t)(first + (uint32_t)__ffs((int)reach) - 1u);
        __syncwarp();
        /* (their values again: cheaper than to keep a lane's values in reach of any index) */
        for (uint32_t i = sub; i < have; i += L) {
            const uint32_t id = s.id[i];
            const uint64_t k = (uint64_t)n * a.ld + id;
            const float x = fmaxf(F32 ? reinterpret_cast<const float *>(d.a)[k] : bf1(reinterpret_cast<const uint16_t *>(d.a)[k]), -INFINITY);
            float v = x;
            if (biased) v = (sigmoid ? route_sigmoid_fast(x) : route_score(false, x, most, inv)) + flat[id];
            s.got[i] = top_entry(v, id);
            s.logit[i] = x;
        }
        __syncwarp();
        for (uint32_t i = sub; i < have; i += L) {
            const uint64_t e = s.got[i];
            uint32_t rank = 0;
#pragma unroll 4
            for (uint32_t k = 0; k < have; k++) rank += s.got[k] > e;
            if (rank <= a.K) s.best[rank] = e, s.best_logit[rank] = s.logit[i]; /* (K <= 15) */
        }
        __syncwarp();
        const bool chosen = sub < a.K;
        const uint32_t mine = chosen ? sub : 0u;
        if (biased) {
            bool near = false;
            if (chosen && sub + 1u < have) {
                /* values that may have swapped, unless they are of equal logits and biases */
                const uint64_t e = s.best[sub], o = s.best[sub + 1u];
                const float v = choose_unkey((uint32_t)(e >> 32));
                near = v - choose_unkey((uint32_t)(o >> 32)) <= unsure;
                if (near && s.best_logit[sub] == s.best_logit[sub + 1u] && flat[GPUOS_FULL - (uint32_t)e] == flat[GPUOS_FULL - (uint32_t)o]) {
                    near = false;
                    if (sub + 1u == a.K) { /* the last one's like is not chosen: what else is near comes behind it */
#pragma unroll 1
                        for (uint32_t k = 0; k < have; k++) {
                            const uint64_t g = s.got[k];
                            if (g < o && v - choose_unkey((uint32_t)(g >> 32)) <= unsure)
                                near |= !(s.logit[k] == s.best_logit[sub] && flat[s.id[k]] == flat[GPUOS_FULL - (uint32_t)e]);
                        }
                    }
                }
            }
            const uint32_t who = __ballot_sync(GPUOS_FULL, near);
            if (who & lanes) {
                if (sigmoid) {
                    __syncwarp(lanes); /* (best has been read) */
                    if (!op_y_fine(&s, sub, L, RouteGathered{flat, have, lanes, wide})) sure = false;
                } else {
                    sure = false;
                }
            }
            __syncwarp();
        }
        const uint32_t id = GPUOS_FULL - (uint32_t)s.best[mine];
        const float x = s.best_logit[mine];
        if ((sigmoid || biased) && chosen && x - (sigmoid ? 0.0f : most) < -80.0f && x != -INFINITY) sure = false; /* (see route_token) */
        float w = chosen ? route_weight(sigmoid, x, most, inv) : 0.0f;
        if (norm) {
            const float sum = lanes_sum<L>(w);
            if (sum != 0.0f) w = __fdividef(w, sum); /* (two units in the last place, as a score's own error; sums lie within 2^-116 to 32) */
        }
        uint32_t again = __ballot_sync(GPUOS_FULL, !sure && !pad);
        if (chosen && !(again & lanes)) {
            a.ids[(uint64_t)n * a.K + sub] = pad ? GPUOS_FULL : id;
            a.weights[(uint64_t)n * a.K + sub] = pad ? 0.0f : w * a.scale;
        }
#pragma unroll 1
        for (uint32_t k = 0; again && k < TOKENS; k++, again >>= L)
            if (again & ((1u << L) - 1u) && n0 + k < a.N) op_y_sure<L * VPL <= 256 ? 8 : 32>(&d, n0 + k);
        __syncwarp();
    }
}
/* The general way: a warp a token. */
template <int VPL>
__global__ void __launch_bounds__(GPUOS_ROUTEB_THREADS) gpuos_route_any_kernel(const __grid_constant__ gpuos_devdesc d)
{
    kv4_after_previous();
    const uint32_t step = gridDim.x * (GPUOS_ROUTEB_THREADS / 32u);
    for (uint32_t n = blockIdx.x * (GPUOS_ROUTEB_THREADS / 32u) + (threadIdx.x >> 5); n < d.dims[0]; n += step)
        route_again<VPL>(&d, n, route_tile<VPL>(&d, n, 1u));
}

template <bool F32, int L, int VPL>
static int route_launch(const gpuos_devdesc &d, void *stream)
{
    const uint32_t tokens = GPUOS_ROUTEB_THREADS / L, size = F32 ? 4u : 2u;
    const uint64_t blocks = ((uint64_t)d.dims[0] + tokens - 1u) / tokens;
    const uint32_t grid = (uint32_t)min(blocks, (uint64_t)GPUOS_ROUTEB_BLOCKS);
    const bool vec = d.dims[1] == L * VPL && (VPL * size) % 16u == 0 && (d.a & 15u) == 0 && ((uint64_t)d.dims[2] * size & 15u) == 0;
    if (vec) return choose_launch(gpuos_route_kernel<F32, L, VPL, true>, dim3(grid), GPUOS_ROUTEB_THREADS, 0, stream, d);
    return choose_launch(gpuos_route_kernel<F32, L, VPL, false>, dim3(grid), GPUOS_ROUTEB_THREADS, 0, stream, d);
}
template <bool F32>
static int route_launch_of(const gpuos_devdesc &d, void *stream)
{
    const uint32_t E = d.dims[1], K = d.dims[3], G = d.dims[4] & 0xFFFFu, keep = d.dims[4] >> 16;
    /* a token's lanes have to hold whole groups or equal parts of one, and three
     * values of each open lane have to be enough for a bar, or all fit */
    auto fits = [&](uint32_t L) {
        return (G == 1u || (L % G == 0 && E % L == 0)) && (K + 1u <= 3u * keep * (L / G) || keep * (E / G) <= GPUOS_ROUTEB_ROOM);
    };
    /* eight lanes and sixteen, us, no bias, one group:
     *   tokens      64           4,096        65,536
     *   E = 32      3.2   3.4    3.9   4.5    14.9   34.0
     *   E = 64      3.5   3.6    4.5   5.1    16.1   34.9
     *   E = 128     4.1   4.1    5.7   5.6    21.6   39.0
     *   E = 256 (32,768 tokens)               19.1   18.1, with bias and groups 43 and 32 */
    if (K <= 8u && E <= 128u && fits(8)) {
        if (E <= 64u) return route_launch<F32, 8, 8>(d, stream);
        return route_launch<F32, 8, 16>(d, stream);
    }
    if (K <= GPUOS_ROUTEB_MAX_K && E <= 512u && fits(16)) {
        if (E <= 256u) return route_launch<F32, 16, 16>(d, stream);
        return route_launch<F32, 16, 32>(d, stream);
    }
    const uint32_t grid = (uint32_t)min(((uint64_t)d.dims[0] + 3u) / 4u, (uint64_t)GPUOS_ROUTEB_BLOCKS);
    if (E <= 256u) return choose_launch(gpuos_route_any_kernel<8>, dim3(grid), GPUOS_ROUTEB_THREADS, 0, stream, d);
    return choose_launch(gpuos_route_any_kernel<32>, dim3(grid), GPUOS_ROUTEB_THREADS, 0, stream, d);
}

/* ---------------------------------------------------------------------------
 * The experts' order, launched: a block takes a run, 4,096 pairs at a time, a
 * warp up to 128 of them. Within a warp's 32 pairs, equal ids find each other
 * by votes on their bits; over its steps, over the warps and over the runs,
 * counts say what comes before. Latency: 512 pairs of 256 experts 3.4 us, one
 * launch; 262,144 pairs 9.4, two launches of 96 blocks (64 runs: 9.5 where these
 * took 8.8), of which the second reads the counts of all runs (96 KB a block).
 * ------------------------------------------------------------------------- */
#define GPUOS_PLANB_THREADS 1024u
#define GPUOS_PLANB_WARPS 32u
#define GPUOS_PLANB_STEPS 4u
#define GPUOS_PLANB_PAIRS (GPUOS_PLANB_THREADS * GPUOS_PLANB_STEPS)
static_assert(GPUOS_PLANB_PAIRS >= GPUOS_PLAN_ONE, "a plan of one run is one turn");

__global__ void __launch_bounds__(GPUOS_PLANB_THREADS) gpuos_plan_count_kernel(const __grid_constant__ gpuos_devdesc d)
{
    __shared__ uint32_t count[GPUOS_ROUTE_MAX_E];
    PlanRun p;
    plan_run(&d, blockIdx.x, p);
    const uint32_t t = threadIdx.x;
    count[t] = 0;
    kv4_after_previous();
    __syncthreads();
#pragma unroll 1
    for (uint32_t i = p.lo + t; i < p.hi; i += GPUOS_PLANB_PAIRS) {
        int32_t id[GPUOS_PLANB_STEPS];
#pragma unroll
        for (uint32_t k = 0; k < GPUOS_PLANB_STEPS; k++) id[k] = i + k * GPUOS_PLANB_THREADS < p.hi ? p.ids[i + k * GPUOS_PLANB_THREADS] : -1;
#pragma unroll
        for (uint32_t k = 0; k < GPUOS_PLANB_STEPS; k++)
            if ((uint32_t)id[k] < p.E) atomicAdd(count + id[k], 1u);
    }
    __syncthreads();
    if (t < p.E) p.counts[blockIdx.x * p.E + t] = count[t];
}
/* The sum of the threads' values before this one's, and of all. */
DEV uint32_t plan_scan(uint32_t v, uint32_t *warps, uint32_t &total)
{
    const uint32_t lane = lane_id(), w = threadIdx.x >> 5;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(GPUOS_FULL, incl, o);
        if (lane >= (uint32_t)o) incl += x;
    }
    if (lane == 31) warps[w] = incl;
    __syncthreads();
    uint32_t s = warps[lane];
    const uint32_t own = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(GPUOS_FULL, s, o);
        if (lane >= (uint32_t)o) s += x;
    }
    total = __shfl_sync(GPUOS_FULL, s, 31);
    return __shfl_sync(GPUOS_FULL, s - own, (int)w) + incl - v;
}
__global__ void __launch_bounds__(GPUOS_PLANB_THREADS) gpuos_plan_place_kernel(const __grid_constant__ gpuos_devdesc d)
{
    extern __shared__ __align__(16) uint16_t plan_before[]; /* [32 warps][E]: the warps' pairs, then those of the warps before */
    __shared__ uint32_t base[GPUOS_ROUTE_MAX_E], warps[32], part[2][GPUOS_PLANB_THREADS];
    PlanRun p;
    plan_run(&d, blockIdx.x, p);
    const uint32_t t = threadIdx.x, lane = lane_id(), w = t >> 5;
    int32_t *const order = reinterpret_cast<int32_t *>(d.out), *const place = reinterpret_cast<int32_t *>(d.b);
    uint32_t *const offsets = reinterpret_cast<uint32_t *>(d.aux0);
    uint16_t *const mine = plan_before + w * p.E;
    kv4_after_previous();
    uint32_t total = 0;
    if (p.T > 1) {
        /* pairs of each expert in the runs before this one, and in all */
        const uint32_t parts = GPUOS_PLANB_THREADS / p.E, q = t / p.E, e = t - q * p.E;
        uint32_t all = 0, before = 0;
        if (q < parts) {
#pragma unroll 8
            for (uint32_t k = q; k < p.T; k += parts) {
                const uint32_t c = __ldcg(p.counts + k * p.E + e);
                all += c;
                before += k < blockIdx.x ? c : 0u;
            }
        }
        part[0][t] = all, part[1][t] = before;
        __syncthreads();
        all = before = 0;
        if (t < p.E)
            for (uint32_t k = 0; k < parts; k++) all += part[0][k * p.E + t], before += part[1][k * p.E + t];
        const uint32_t at = plan_scan(all, warps, total);
        if (t < p.E) {
            base[t] = at + before;
            if (blockIdx.x == 0) offsets[t] = at;
        }
    }
#pragma unroll 1
    for (uint32_t i0 = p.lo; i0 < p.hi || (p.T == 1 && i0 == 0); i0 += GPUOS_PLANB_PAIRS) {
        int32_t id[GPUOS_PLANB_STEPS];
        uint32_t rank[GPUOS_PLANB_STEPS];
        /* the warps' parts are of one length, whole steps */
        const uint32_t turn = min(p.hi - i0, GPUOS_PLANB_PAIRS), steps = (turn + GPUOS_PLANB_THREADS - 1u) / GPUOS_PLANB_THREADS;
        const uint32_t i = i0 + w * steps * 32u + lane;
#pragma unroll
        for (uint32_t k = 0; k < GPUOS_PLANB_STEPS; k++) id[k] = k < steps && i + 32u * k < p.hi ? p.ids[i + 32u * k] : -1;
        for (uint32_t k = t; k < GPUOS_PLANB_WARPS * p.E / 2u; k += GPUOS_PLANB_THREADS) reinterpret_cast<uint32_t *>(plan_before)[k] = 0u;
        __syncthreads();
#pragma unroll
        for (uint32_t k = 0; k < GPUOS_PLANB_STEPS; k++) {
            if (k >= steps) break;
            const bool here = (uint32_t)id[k] < p.E;
            uint32_t peers = __ballot_sync(GPUOS_FULL, here); /* (with __match_any_sync a plan of 262,144 pairs took 11.9 us, so 9.4) */
#pragma unroll 1
            for (uint32_t bit = 1; bit < p.E; bit <<= 1) {
                const uint32_t set = __ballot_sync(GPUOS_FULL, (uint32_t)id[k] & bit);
                peers &= (uint32_t)id[k] & bit ? set : ~set;
            }
            const uint32_t below = (uint32_t)__popc(peers & ((1u << lane) - 1u));
            rank[k] = here ? mine[id[k]] + below : 0u;
            __syncwarp();
            if (here && below == 0) mine[id[k]] = (uint16_t)(rank[k] + (uint32_t)__popc(peers));
            __syncwarp();
        }
        __syncthreads();
        uint32_t sum = 0;
        if (t < p.E) {
#pragma unroll
            for (uint32_t k = 0; k < GPUOS_PLANB_WARPS; k++) {
                const uint32_t c = plan_before[k * p.E + t];
                plan_before[k * p.E + t] = (uint16_t)sum;
                sum += c;
            }
        }
        if (p.T == 1) { /* (one turn: its counts are all) */
            const uint32_t at = plan_scan(sum, warps, total);
            if (t < p.E) base[t] = offsets[t] = at;
        }
        __syncthreads();
#pragma unroll
        for (uint32_t k = 0; k < GPUOS_PLANB_STEPS; k++) {
            const uint32_t at = i + 32u * k;
            if (k >= steps || at >= p.hi) continue;
            const bool here = (uint32_t)id[k] < p.E;
            const uint32_t to = here ? base[id[k]] + mine[id[k]] + rank[k] : 0u;
            place[at] = here ? (int32_t)to : -1;
            if (here && to < p.P) order[to] = (int32_t)at; /* (counts that are not of these pairs: nothing outside is written) */
            if (at >= total) order[at] = -1; /* (behind the last pair) */
        }
        __syncthreads();
        if (t < p.E) base[t] += sum;
    }
    if (blockIdx.x == 0 && t == 0) offsets[p.E] = total;
}

static int plan_launch(const gpuos_devdesc &d, void *stream)
{
    if (d.op_id == GPUOS_OP_EXPERT_COUNT)
        return d.ntiles == 1 ? 0 : choose_launch(gpuos_plan_count_kernel, dim3(d.ntiles), GPUOS_PLANB_THREADS, 0, stream, d);
    const uint32_t smem = (GPUOS_PLANB_WARPS * d.dims[1] * 2u + 15u) & ~15u;
    static std::atomic<bool> known[64];
    if (smem > 32768u && choose_smem((const void *)gpuos_plan_place_kernel, GPUOS_PLANB_WARPS * GPUOS_ROUTE_MAX_E * 2u, known) != 0) return -1;
    return choose_launch(gpuos_plan_place_kernel, dim3(d.ntiles), GPUOS_PLANB_THREADS, smem, stream, d);
}
static int choose_eager_launch(const gpuos_devdesc &d, void *stream)
{
    const bool f32 = d.dtype == GPUOS_F32;
    if (d.op_id == GPUOS_OP_EXPERT_COUNT || d.op_id == GPUOS_OP_EXPERT_PLACE) return plan_launch(d, stream);
    if (d.dims[0] == 0 || d.dims[1] == 0) return 0;
    switch (d.op_id) {
    case GPUOS_OP_LOGITS_ADJUST: return f32 ? adjust_launch_of<true>(d, stream) : adjust_launch_of<false>(d, stream);
    case GPUOS_OP_LOGITS_TOP: return f32 ? top_launch<true>(d, stream) : top_launch<false>(d, stream);
    default: return f32 ? route_launch_of<true>(d, stream) : route_launch_of<false>(d, stream);
    }
}
/* Load the kernels (see gpuos_dev_preload). */
static int choose_preload()
{
    const void *const all[] = {
        (const void *)gpuos_adjust_kernel<true, true, 2>, (const void *)gpuos_adjust_kernel<true, true, 3>, (const void *)gpuos_adjust_long_kernel<true, true>,
        (const void *)gpuos_adjust_kernel<true, false, 2>, (const void *)gpuos_adjust_kernel<true, false, 3>, (const void *)gpuos_adjust_long_kernel<true, false>,
        (const void *)gpuos_adjust_kernel<false, true, 2>, (const void *)gpuos_adjust_kernel<false, true, 4>, (const void *)gpuos_adjust_long_kernel<false, true>,
        (const void *)gpuos_adjust_kernel<false, false, 2>, (const void *)gpuos_adjust_kernel<false, false, 4>, (const void *)gpuos_adjust_long_kernel<false, false>,
        (const void *)gpuos_top_kernel<true>, (const void *)gpuos_top_kernel<false>,
        (const void *)gpuos_route_kernel<true, 8, 8, true>, (const void *)gpuos_route_kernel<true, 8, 8, false>,
        (const void *)gpuos_route_kernel<true, 8, 16, true>, (const void *)gpuos_route_kernel<true, 8, 16, false>,
        (const void *)gpuos_route_kernel<true, 16, 16, true>, (const void *)gpuos_route_kernel<true, 16, 16, false>,
        (const void *)gpuos_route_kernel<true, 16, 32, true>, (const void *)gpuos_route_kernel<true, 16, 32, false>,
        (const void *)gpuos_route_kernel<false, 8, 8, true>, (const void *)gpuos_route_kernel<false, 8, 8, false>,
        (const void *)gpuos_route_kernel<false, 8, 16, true>, (const void *)gpuos_route_kernel<false, 8, 16, false>,
        (const void *)gpuos_route_kernel<false, 16, 16, true>, (const void *)gpuos_route_kernel<false, 16, 16, false>,
        (const void *)gpuos_route_kernel<false, 16, 32, true>, (const void *)gpuos_route_kernel<false, 16, 32, false>,
        (const void *)gpuos_route_any_kernel<8>, (const void *)gpuos_route_any_kernel<32>,
        (const void *)gpuos_plan_count_kernel, (const void *)gpuos_plan_place_kernel};
    for (const void *f : all) {
        cudaFuncAttributes at;
        if (cudaFuncGetAttributes(&at, f) != cudaSuccess) return -1;
    }
    return 0;
}
#endif /* GPUOS_EXECUTOR_ONLY */
#endif /* GPUOS_CHOOSE_CUH */
