/*
 * What a decode step chooses (included by gpuos_device.cu, whose memory, bf16
 * and staging helpers it uses): logits adjusted for the next token, the best
 * tokens of a row, the experts of a token, and the experts' order.
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
DEV float choose_unkey(uint32_t k) { return __uint_as_float(k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u)); }

/* ---------------------------------------------------------------------------
 * Logits adjusted. One pass: each logit is read once and written once, so it
 * is bound by memory; what a token's penalty needs, its count among the
 * request's tokens, comes from counters of the tile's window of the
 * vocabulary in shared memory, filled by one look at the request's tokens.
 * A counter holds the count after the prompt and two flags.
 * ------------------------------------------------------------------------- */
#define GPUOS_ADJUST_HAD 0x80000000u    /* in the prompt */
#define GPUOS_ADJUST_LISTED 0x40000000u /* has a bias: written after the others */
#define GPUOS_ADJUST_COUNT 0x3FFFFFFFu

struct AdjustArgs {
    gpuos_logits_request q;
    const int32_t *tokens;
    const uint32_t *mask; /* its row; null: none */
    const int2 *bias;
    float inv_rep, inv_temp;
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
    a.inv_rep = 1.0f / a.q.repetition;
    a.inv_temp = a.q.temperature > 0.0f ? 1.0f / a.q.temperature : 1.0f;
    a.penal = a.q.length > 0 && !(a.q.repetition == 1.0f && a.q.presence == 0.0f && a.q.frequency == 0.0f);
    return (uint32_t)a.q.length <= Lcap && (uint32_t)a.q.prompt <= (uint32_t)a.q.length && (a.q.mask < 0 || (uint32_t)a.q.mask < M) &&
           (uint32_t)a.q.biases <= Nb;
}
/* (A product with 1 / repetition or 1 / temperature, rounded, is off by 2^-23
 * of itself where the quotient is by 2^-24: a division is ten times the code,
 * and a rounding to bf16 costs 2^-8 afterwards.) */
DEV float adjust_penalty(const AdjustArgs &a, float x, uint32_t w)
{
    const uint32_t c = w & GPUOS_ADJUST_COUNT;
    float y = w & (GPUOS_ADJUST_COUNT | GPUOS_ADJUST_HAD) ? (x > 0.0f ? x * a.inv_rep : x * a.q.repetition) : x;
    if (c) y -= fmaf(a.q.frequency, (float)c, a.q.presence);
    return y;
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
/* Entry i's token is listed again behind it: the later entry counts. */
DEV bool adjust_again(const AdjustArgs &a, uint32_t i, int32_t token)
{
    for (uint32_t k = i + 1; k < (uint32_t)a.q.biases; k++)
        if (__ldcg(&a.bias[k].x) == token) return true;
    return false;
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
                for (uint32_t i0 = 0; i0 < n; i0 += 256) {
                    int32_t t[8];
#pragma unroll
                    for (uint32_t k = 0; k < 8; k++) {
                        const uint32_t i = i0 + k * 32u + lane;
                        t[k] = i < n ? __ldcg(a.tokens + i) : -1;
                    }
#pragma unroll
                    for (uint32_t k = 0; k < 8; k++)
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
                x[j] = bits >> j & 1u ? adjust_penalty(a, x[j], w) * a.inv_temp : -INFINITY;
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
            if (here && !adjust_again(a, i, e.x)) {
                const float y = (adjust_penalty(a, in.one(at + shift), w) + __int_as_float(e.y)) * a.inv_temp;
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
 * the K-th best costs one comparison.
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
#pragma unroll 1
    for (uint32_t i = 0; i < S; i++) {
        if (i == part) continue;
        const unsigned long long *q = reinterpret_cast<const unsigned long long *>(top_part(d, row * S + i) + 16);
        uint64_t e[KL];
#pragma unroll
        for (int k = 0; k < KL; k++) e[k] = lane + 32u * k < K ? __ldcg(q + lane + 32 * k) : 0ull;
#pragma unroll
        for (int k = 0; k < KL; k++) {
            uint32_t left = __ballot_sync(GPUOS_FULL, e[k] > st.list.last);
            while (left) {
                const int src = __ffs((int)left) - 1;
                left &= left - 1u;
                const uint64_t c = shfl64(e[k], src);
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
/* One token's choice and weights in 64 bits. Few tokens come here, so it is
 * short: values in local memory, loops that are not unrolled. */
__device__ __noinline__ void op_y_sure(const gpuos_devdesc *d, uint32_t n)
{
    RouteArgs a;
    route_args(d, a);
    const uint32_t lane = lane_id(), V = (a.E + 31u) / 32u;
    const bool sigmoid = a.flags & GPUOS_ROUTE_SIGMOID, top2 = a.flags & GPUOS_ROUTE_TOP2;
    double c[GPUOS_ROUTE_MAX_E / 32];
    float most = -INFINITY;
#pragma unroll 1
    for (uint32_t i = 0; i < V; i++)
        if (lane + 32u * i < a.E) most = fmaxf(most, route_logit(d, a, n, lane + 32u * i));
    most = fminf(warp_max(most), FLT_MAX);
    double inv = 0.0;
    if (!sigmoid) {
        double total = 0.0;
#pragma unroll 1
        for (uint32_t i = 0; i < V; i++)
            if (lane + 32u * i < a.E) total += route_score(false, (double)route_logit(d, a, n, lane + 32u * i), (double)most, 1.0);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(GPUOS_FULL, total, o);
        inv = total > 0.0 ? 1.0 / total : 0.0;
    }
#pragma unroll 1
    for (uint32_t i = 0; i < V; i++) {
        const uint32_t e = lane + 32u * i;
        c[i] = 0.0;
        if (e >= a.E) continue;
        c[i] = (double)route_logit(d, a, n, e); /* without a bias the scores' order is the logits' */
        if (a.bias || top2) c[i] = route_score(sigmoid, c[i], (double)most, inv);
        if (a.bias) c[i] += (double)__ldcg(a.bias + e);
        if (!(c[i] == c[i])) c[i] = -INFINITY;
    }
    uint32_t kept = GPUOS_FULL;
    if (a.G > 1) {
        uint64_t mine = 0, edge;
#pragma unroll 1
        for (uint32_t g = 0; g < a.G; g++) {
            uint64_t one = 0, two = 0;
#pragma unroll 1
            for (uint32_t i = 0; i < V; i++) {
                const uint32_t e = lane + 32u * i - g * a.size;
                const uint64_t k = e < a.size ? route_key(c[i]) : 0;
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
        kept = route_groups(a, mine, edge);
    }
    uint32_t id = 0, taken = 0;
#pragma unroll 1
    for (uint32_t k = 0; k < a.K; k++) {
        uint64_t best = 0;
        uint32_t at = 0;
#pragma unroll 1
        for (uint32_t i = 0; i < V; i++) {
            const uint32_t e = lane + 32u * i;
            if (e >= a.E || taken >> i & 1u || !(kept >> (a.G > 1 ? e / a.size : 0u) & 1u)) continue;
            const uint64_t key = a.bias || !top2 ? route_key(c[i]) : route_key((double)route_logit(d, a, n, e));
            if (key > best) best = key, at = i;
        }
        const uint64_t win = route_max(best);
        const uint32_t e = __reduce_min_sync(GPUOS_FULL, best == win ? lane + 32u * at : GPUOS_FULL);
        if (lane == (e & 31u)) taken |= 1u << (e >> 5);
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
    /* A sigmoid is off by less than 2^-21 of itself (ex2 2^-22, three roundings),
     * a softmax by less than 2^-19 (its sum's errors too), the sum with the bias
     * by 2^-24 more; two values may swap within twice that. Scores of logits
     * below -80 are cut off (route_exp), which is nothing beside a larger one. */
    const float unsure = route_score(sigmoid, most, most, inv) * (sigmoid ? 0x1p-20f : 0x1p-18f) + warp_max(wide) * 0x1p-22f;
    bool sure = !sigmoid || most >= -60.0f || most == -INFINITY;
    if (a.G > 1) {
        uint32_t mine = 0, edge; /* lane g: group g's value */
#pragma unroll 1
        for (uint32_t g = 0; g < a.G; g++) {
            uint32_t one = 0, two = 0;
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                const uint32_t e = lane + 32u * i - g * a.size;
                const uint32_t k = e < a.size ? key[i] : 0u;
                two = max(two, min(one, k));
                one = max(one, k);
            }
            uint32_t best = route_max(one);
            if (top2) {
                const uint32_t owner = (uint32_t)__ffs((int)__ballot_sync(GPUOS_FULL, one == best)) - 1u;
                float v1 = choose_unkey(best), v2 = choose_unkey(route_max(lane == owner ? two : one));
                if (!a.bias) v1 = route_score(sigmoid, v1, most, inv), v2 = route_score(sigmoid, v2, most, inv);
                best = choose_key(v1 + v2);
            }
            if (lane == g) mine = best;
        }
        const uint32_t kept = route_groups(a, mine, edge);
        if (a.keep < a.G && (a.bias || top2) && choose_unkey(edge) - choose_unkey(route_max(mine)) <= 2.0f * unsure) sure = false;
#pragma unroll
        for (int i = 0; i < VPL; i++)
            if (lane + 32u * i < a.E && !(kept >> ((lane + 32u * i) / a.size) & 1u)) key[i] = 0u;
    }
    uint32_t id = 0, before = 0;
    float xb = 0.0f, bb = 0.0f; /* the last one's logit and bias */
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
                if (!(route_logit(d, a, n, e) == xb && __ldcg(a.bias + e) == bb)) sure = false;
            }
            before = win, xb = route_logit(d, a, n, e), bb = __ldcg(a.bias + e);
        }
        if (lane == k && k < a.K) id = e;
    }
    const float x = lane < a.K ? route_logit(d, a, n, id) : -INFINITY;
    /* (a chosen logit below -80: its weight may be all that is seen) */
    if (sigmoid && __any_sync(GPUOS_FULL, x < -80.0f && x != -INFINITY)) sure = false;
    if (!sure) return false;
    route_write(a, n, id, route_score(sigmoid, x, most, inv));
    return true;
}
template <int VPL>
DEV void route_tile(const gpuos_devdesc *d, uint32_t first, uint32_t count)
{
    RouteArgs a;
    route_args(d, a);
    const uint32_t lane = lane_id(), end = min(first + count, a.N);
    const uint32_t rows = a.rows ? (uint32_t)max(__ldcg(a.rows), 0) : a.N;
#pragma unroll 1
    for (uint32_t n = first; n < end; n++) {
        if (n >= rows) { /* padding */
            if (lane < a.K) {
                __stcg(a.ids + (uint64_t)n * a.K + lane, GPUOS_FULL);
                __stcg(a.weights + (uint64_t)n * a.K + lane, 0.0f);
            }
        } else if (!route_token<VPL>(d, a, n)) {
            op_y_sure(d, n);
        }
    }
}
DEV int route_op(const gpuos_devdesc *d, uint32_t tile)
{
    const uint32_t *m = d->dims;
    if (m[0] == 0) return GPUOS_ST_OK;
    if (!gpuos_route_ok(d->dtype, d->a, d->b, d->out, d->aux0, d->aux1, m) ||
        (m[0] - 1u) / GPUOS_ROUTE_ROWS + 1u != d->ntiles)
        return GPUOS_ST_BAD_ARGS;
    if (tile >= d->ntiles) return GPUOS_ST_OK;
    if (m[1] <= 256) route_tile<8>(d, tile * GPUOS_ROUTE_ROWS, GPUOS_ROUTE_ROWS);
    else route_tile<32>(d, tile * GPUOS_ROUTE_ROWS, GPUOS_ROUTE_ROWS);
    return GPUOS_ST_OK;
}

/* ---------------------------------------------------------------------------
 * The experts' order: a stable counting sort of the pairs. Runs of pairs are
 * counted by expert; a run's pairs of an expert then go behind those of the
 * earlier runs, in their order (whole numbers throughout, nothing hangs on
 * which warp comes first).
 * ------------------------------------------------------------------------- */
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
#pragma unroll 1
    for (uint32_t i0 = p.lo; i0 < p.hi; i0 += 32) {
        const uint32_t i = i0 + lane;
        const int32_t id = i < p.hi ? __ldcg(p.ids + i) : -1;
        const bool here = (uint32_t)id < p.E;
        const uint32_t peers = __match_any_sync(GPUOS_FULL, here ? id : -1);
        const uint32_t lead = (uint32_t)__ffs((int)peers) - 1u;
        uint32_t at = 0;
        if (here && lane == lead) at = plan_add(ctr + id, (uint32_t)__popc(peers), shared);
        at = __shfl_sync(GPUOS_FULL, at, (int)lead) + (uint32_t)__popc(peers & ((1u << lane) - 1u));
        if (here) __stcg(order + at, (int32_t)i);
        if (i < p.hi) __stcg(place + i, here ? (int32_t)at : -1);
        if (i < p.hi && i >= begin) __stcg(order + i, -1); /* (places behind the last pair) */
        __syncwarp();
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    return GPUOS_ST_OK;
}

#ifndef GPUOS_EXECUTOR_ONLY
template <int OP>
__global__ void __launch_bounds__(32) gpuos_choose_eager_kernel(const __grid_constant__ gpuos_devdesc d)
{
    stage_init(16384);
    kv4_after_previous();
    if (OP == GPUOS_OP_LOGITS_ADJUST) (void)adjust_op(&d, blockIdx.x);
    if (OP == GPUOS_OP_LOGITS_TOP) (void)top_op(&d, blockIdx.x);
    if (OP == GPUOS_OP_EXPERT_ROUTE) (void)route_op(&d, blockIdx.x);
    if (OP == GPUOS_OP_EXPERT_COUNT) (void)plan_count_op(&d, blockIdx.x);
    if (OP == GPUOS_OP_EXPERT_PLACE) (void)plan_place_op(&d, blockIdx.x);
}
template <int OP>
static int choose_tiles_launch(const gpuos_devdesc &d, void *stream)
{
    return kv4_launch(gpuos_choose_eager_kernel<OP>, d.ntiles, 32, gpuos_dev_dyn_smem(1, 16384), stream, d);
}
static int choose_eager_launch(const gpuos_devdesc &d, void *stream)
{
    switch (d.op_id) {
    case GPUOS_OP_LOGITS_ADJUST: return choose_tiles_launch<GPUOS_OP_LOGITS_ADJUST>(d, stream);
    case GPUOS_OP_LOGITS_TOP: return choose_tiles_launch<GPUOS_OP_LOGITS_TOP>(d, stream);
    case GPUOS_OP_EXPERT_ROUTE: return choose_tiles_launch<GPUOS_OP_EXPERT_ROUTE>(d, stream);
    case GPUOS_OP_EXPERT_COUNT: return choose_tiles_launch<GPUOS_OP_EXPERT_COUNT>(d, stream);
    default: return choose_tiles_launch<GPUOS_OP_EXPERT_PLACE>(d, stream);
    }
}
/* Load the kernels (see gpuos_dev_preload). */
static int choose_preload()
{
    const void *const all[] = {
        (const void *)gpuos_choose_eager_kernel<GPUOS_OP_LOGITS_ADJUST>, (const void *)gpuos_choose_eager_kernel<GPUOS_OP_LOGITS_TOP>,
        (const void *)gpuos_choose_eager_kernel<GPUOS_OP_EXPERT_ROUTE>, (const void *)gpuos_choose_eager_kernel<GPUOS_OP_EXPERT_COUNT>,
        (const void *)gpuos_choose_eager_kernel<GPUOS_OP_EXPERT_PLACE>};
    for (const void *f : all) {
        cudaFuncAttributes at;
        if (cudaFuncGetAttributes(&at, f) != cudaSuccess) return -1;
    }
    return 0;
}
#endif /* GPUOS_EXECUTOR_ONLY */
#endif /* GPUOS_CHOOSE_CUH */
