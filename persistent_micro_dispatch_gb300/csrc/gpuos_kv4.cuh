/*
 * The 4-bit paged key/value cache: attention, write, read back and page copy
 * (included by gpuos_device.cu, whose memory, bf16 and staging helpers it
 * uses).
 *
 * Page layout (one page = GPUOS_KV4_PAGE = 32 tokens of every cache head; the
 * pool is [npages][Hkv][34 D] bytes, G = D / 32 scale groups per token):
 *
 *   keys          [key>>4][key>>2 & 3][key & 1][c>>3][key>>1 & 1][g][c>>1 & 3]   16 D bytes
 *   values        [key>>4][c>>2][key>>2 & 3][key & 3][g][c>>1 & 1]               16 D bytes
 *   key scales    [key][g]                                                          D bytes
 *   value scales  [key>>4][key>>2 & 3][g][key & 3]                                  D bytes
 *
 * (c = channel within its group g; two neighbouring channels to a byte, the
 * even one low). A code is e2m1: sign, and {0, .5, 1, 1.5, 2, 3, 4, 6}; a
 * scale byte is an exponent + 127 (255: the group held a NaN or infinity).
 * 4.25 bits an element.
 *
 * The order is that of the matrix fragments. mma.m16n8k16 is used with the
 * cache as its A operand (S^T = K q^T and O^T = V^T p^T): 16 keys or 16
 * channels against 8 query rows, so up to eight query rows that share a cache
 * head cost one pass over it, and a lane's codes of a 16-key tile are 8 G
 * contiguous bytes of keys and of values: one or two 16-byte loads, the whole
 * warp's contiguous. Row m of S^T (and k of O^T's product) stands for key
 * 4 (m>>1 & 3) + (m & 1) + 2 (m >> 3): then lane (i = lane / 4, j = lane % 4)
 * needs keys 4 j .. 4 j + 3 of the values.
 */
#ifndef GPUOS_KV4_CUH
#define GPUOS_KV4_CUH

#include <cuda_fp16.h>
#include <float.h>

#include <atomic>

#define GPUOS_KV4_SCRATCH 768u /* bytes of a warp's converted scales */
#define GPUOS_KV4_WIDE 0x80000000u

DEV constexpr uint32_t kv4_page_bytes(uint32_t D) { return 34u * D; }

/* 2^e for an exponent in [-126, 127] */
DEV float kv4_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

/* Four bytes of code pairs -> four f16x2 (exact); low nibble in the low half. */
DEV void kv4_decode4(uint32_t w, uint32_t (&o)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]) : "r"(w));
}
/* Eight values -> eight codes, value 0 in the lowest nibble; nearest, ties to
 * the even code (|x| <= 6 but for a clamped scale, where 6 is the answer). */
DEV uint32_t kv4_encode8(const float (&x)[8])
{
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return w;
}
DEV void kv4_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
DEV uint32_t kv4_trans8x8(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
DEV uint32_t kv4_pack_h2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
DEV uint32_t kv4_hmul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
DEV float kv4_ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

/* ---------------------------------------------------------------------------
 * Attention: o[r] = sum_n softmax_n(scale q[r].K[n]) V[n] over the keys that
 * row r sees. The T g query rows of a request that share a cache head
 * (g = H / Hkv; row r = t g + hh) are cut into row tiles of 8 NT rows.
 *
 * An item is one (request, head, row tile). Work is counted in units of one
 * page of an item (a request of length 0: one unit), with GPUOS_KV4_LEAD more
 * before its first page for what an item costs of itself (a warp fetches page
 * ids, queries and a first page one after another: about 4 us, against 0.6 us
 * for each further page); the units are numbered in that order and cut into
 * equal runs, one per warp, whatever the requests' lengths. Without, 16 ragged
 * requests of 2 to 4,099 tokens took 32.5 us, 256 of 30 to 60 tokens 20.6, in
 * an early form; now, with 3, 4, 6, 8, 12 units, the same two (32 heads over
 * 4) 12.3, 12.3, 12.4, 12.2, 11.5 and 12.8, 14.5, 14.0, 12.6, 11.6 us; 64 of
 * 200 to 1,500 (32 over 8) 22.3, 22.1, 22.5, 22.9, 24.0; one of 100 7.7, 7.8,
 * 8.0, 5.5, 7.1; 33 of 1 to 3,001 (14 over 2, D = 64) 10.0, 10.0, 10.4, 10.1,
 * 9.8; 8 of 20,000 38.0, 38.2, 38.1, 38.5, 38.4. Six is in the middle, not a
 * best: short requests want more, medium ones fewer. A run that ends inside an
 * item leaves a partial state, merged with its neighbours' (below).
 *
 * Numerics. q is scaled by a power of two for each row to [128, 256) and held
 * in f16: exact for the bf16 values within 2^-21 of the row's largest, and off
 * by at most 2^-32 of it below. If a group of 32 channels has its largest
 * 2^14 below the row's, every page goes the slow way (below), where each group
 * has a power of its own; what is lost is 2^-18 of a group's largest at most.
 * Codes are exact in f16; the products are summed in fp32 for each scale
 * group, and the groups' sums are scaled and added in fp32. Weights p, the
 * largest 2^14 to 2^15, are rounded to f16 (11 bits; bf16's 8 would show in a
 * bf16 output; one 2^-28 of the largest still has them all) and multiplied
 * there by 2^(b - E), b the value's scale byte and E a byte of the group's
 * choosing, which is also the accumulators' unit. A page is taken that way
 * only if E - 12 <= b <= E for all its keys. Then the product is off by 2^-25
 * at most where it is not exact, and the key that set the softmax's reference
 * weighs 2^14 with b >= E - 12: what is lost is 6 * 2^-27 of the largest p 2^b
 * that the row has met, for each key, whatever the other rows and the hidden
 * keys hold. Any other page goes the slow way (op_x_slow): it multiplies
 * p 2^(b - x) in fp32, x the row's own largest p 2^b in the page, before it
 * rounds to f16, and sets E anew. The softmax's reference and sum and the
 * output accumulators are fp32.
 * ------------------------------------------------------------------------- */
struct Kv4Args {
    const uint16_t *q;
    const unsigned char *pool;
    const int32_t *lens;
    const int32_t *table;
    uint16_t *out;
    uint32_t B, H, Hkv, T, g, RT, P, npages, rows; /* (rows: of a row tile) */
    float scale; /* times log2 e */
    float inv_g; /* 1 / g */
};
DEV void kv4_args(const gpuos_devdesc *d, uint32_t rows_per_tile, Kv4Args &a)
{
    a.q = reinterpret_cast<const uint16_t *>(d->a);
    a.pool = reinterpret_cast<const unsigned char *>(d->b);
    a.lens = reinterpret_cast<const int32_t *>(d->aux0);
    a.table = reinterpret_cast<const int32_t *>(d->aux1);
    a.out = reinterpret_cast<uint16_t *>(d->out);
    a.B = d->dims[0];
    a.H = d->dims[1] & 0xFFFFu;
    a.Hkv = d->dims[1] >> 16;
    a.T = d->dims[2] >> 16;
    a.g = a.H / a.Hkv;
    a.inv_g = 1.0f / (float)a.g;
    a.rows = rows_per_tile;
    a.RT = (a.T * a.g + rows_per_tile - 1) / rows_per_tile;
    a.P = d->dims[3];
    a.npages = d->dims[4];
    a.scale = d->fparam[0] * 1.4426950408889634f;
}
/* Query row r of a cache head: token t = floor(r / g), query head h g + hh.
 * In floats, without a division's code: r is below 2^21 + 16, so (r + 1/2) / g
 * is off by less than the 1 / (2 g) that parts it from an integer. */
DEV void kv4_token(const Kv4Args &a, uint32_t r, uint32_t &t, uint32_t &hh)
{
    t = (uint32_t)(((float)r + 0.5f) * a.inv_g);
    hh = r - t * a.g;
}
/* Pages of a request; a length that its table row cannot hold counts as one
 * unit that does nothing (bad). */
DEV uint32_t kv4_pages(const Kv4Args &a, int32_t len, bool &bad)
{
    bad = len < 0 || (uint32_t)len > a.P * GPUOS_KV4_PAGE;
    return bad || len == 0 ? 1u : ((uint32_t)len + GPUOS_KV4_PAGE - 1u) / GPUOS_KV4_PAGE;
}
DEV uint32_t kv4_pages(const Kv4Args &a, int32_t len)
{
    bool bad;
    return kv4_pages(a, len, bad);
}

/* A warp's place in the work. */
struct Kv4Pos {
    uint32_t b, h, r0; /* request, head, first row of the row tile */
    uint32_t off, np; /* next unit of the item; its pages */
    int32_t len;
    uint32_t first; /* the unit of the item's first page */
};
/* The next units of an item up to `left`: pages [begin, end), none in the lead. */
DEV uint32_t kv4_take(const Kv4Pos &p, uint32_t left, uint32_t &begin, uint32_t &end)
{
    const uint32_t span = p.np + GPUOS_KV4_LEAD - p.off, n = min(left, span);
    begin = p.off > GPUOS_KV4_LEAD ? p.off - GPUOS_KV4_LEAD : 0u;
    end = p.off + n > GPUOS_KV4_LEAD ? p.off + n - GPUOS_KV4_LEAD : 0u;
    return n;
}
/* All units of the call, and (every lane) the length of request `lane`. */
DEV uint32_t kv4_units(const Kv4Args &a, int32_t &len0)
{
    const uint32_t lane = lane_id();
    uint32_t n = 0; /* (the host keeps the units that the table can hold below 2^32) */
    len0 = 0;
#pragma unroll 1
    for (uint32_t i = lane; i < a.B; i += 128) { /* four loads in flight */
        int32_t len[4];
#pragma unroll
        for (int k = 0; k < 4; k++) len[k] = i + 32u * k < a.B ? __ldcg(a.lens + i + 32u * k) : 0;
        if (i == lane) len0 = len[0];
#pragma unroll
        for (int k = 0; k < 4; k++) n += i + 32u * k < a.B ? kv4_pages(a, len[k]) + GPUOS_KV4_LEAD : 0u;
    }
    return __reduce_add_sync(0xFFFFFFFFu, n) * a.Hkv * a.RT;
}
/* W units in n runs that differ by one unit at most: the first W mod n have
 * one more than the others. */
struct Kv4Runs {
    uint32_t base, more; /* units of a run; runs with one more */
    DEV Kv4Runs(uint32_t W, uint32_t n) : base(W / n) { more = W - base * n; }
    DEV uint32_t start(uint32_t run) const { return run * base + min(run, more); }
    DEV uint32_t run_of(uint32_t u) const
    {
        const uint32_t cut = more * (base + 1u);
        return u < cut ? u / (base + 1u) : more + (u - cut) / base;
    }
};
/* The place of unit u (u < the number of units). */
DEV void kv4_seek(const Kv4Args &a, uint32_t u, int32_t len0, Kv4Pos &p)
{
    const uint32_t lane = lane_id(), HR = a.Hkv * a.RT;
    const uint32_t pg = u / HR; /* pages of all requests before u's request: at most this */
    uint32_t base = 0;
#pragma unroll 1
    for (uint32_t i0 = 0; i0 < a.B; i0 += 32) {
        const uint32_t i = i0 + lane;
        const int32_t len = i0 == 0 ? len0 : (i < a.B ? __ldcg(a.lens + i) : 0);
        const uint32_t cnt = i < a.B ? kv4_pages(a, len) + GPUOS_KV4_LEAD : 0u;
        uint32_t incl = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= (uint32_t)o) incl += v;
        }
        const uint32_t bal = __ballot_sync(0xFFFFFFFFu, pg < base + incl);
        if (bal) {
            const int src = __ffs(bal) - 1;
            p.b = i0 + (uint32_t)src;
            p.len = __shfl_sync(0xFFFFFFFFu, len, src);
            p.np = kv4_pages(a, p.len);
            const uint32_t span = p.np + GPUOS_KV4_LEAD;
            const uint32_t lo_b = (base + __shfl_sync(0xFFFFFFFFu, incl, src) - span) * HR;
            const uint32_t off = u - lo_b;
            const uint32_t item = off / span;
            p.off = off - item * span;
            p.first = lo_b + item * span + GPUOS_KV4_LEAD;
            p.h = a.RT == 1 ? item : item / a.RT;
            p.r0 = (item - p.h * a.RT) * a.rows;
            return;
        }
        base += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    p.b = a.B; /* not reached for u < kv4_units() */
    p.len = 0;
    p.np = 1;
    p.h = p.r0 = p.off = 0;
    p.first = u;
}
/* The next item. */
DEV void kv4_next(const Kv4Args &a, Kv4Pos &p)
{
    p.first += p.np;
    p.off = 0;
    p.r0 += a.rows;
    if (p.r0 < a.T * a.g) {
        p.first += GPUOS_KV4_LEAD;
        return;
    }
    p.r0 = 0;
    if (++p.h >= a.Hkv) {
        p.h = 0;
        if (++p.b >= a.B) return;
        p.len = __ldcg(a.lens + p.b);
        p.np = kv4_pages(a, p.len);
    }
    p.first += GPUOS_KV4_LEAD;
}

/* One item's running state in a warp: lane (i, j) holds query rows
 * 8 nt + 2 j + {0, 1} (index r) and channels 32 g + 4 i + {0..3} of O^T. */
template <int G, int NT>
struct Kv4State {
    uint32_t q[NT][G][4]; /* f16x2 of row 8 nt + i: channels 32 g + 8 j + {0..7} */
    float f[NT][2];       /* score factor of rows 2 j, 2 j + 1: |scale| log2(e) 2^k, positive */
    float m[NT][2];       /* the reference that scores are taken against, equal in the lanes of a row */
    float l[NT][2];       /* this lane's part of the running sum */
    float acc[NT][G][2][4];
    uint32_t E[G]; /* the unit of each group's accumulators: 2^(E - 127) */
    uint32_t open; /* bit g: group g's window of scales is in use (a row may have no weight that bears it out);
                      GPUOS_KV4_WIDE: none is, whatever the other bits say */
    uint32_t nlo, factor; /* of group lane % G: 12 - E in both halves (closed: no byte passes); 15 - E in both f16 exponents */
    uint32_t nan; /* bit 2 NT g + 2 nt + c: row (nt, c) saw a NaN among group g's values */
    uint32_t lim[NT][2]; /* keys that the row sees */
    uint32_t min_lim;    /* least of them over the tile's rows */
};

DEV uint32_t kv4_row_limit(const Kv4Args &a, int32_t len, uint32_t r)
{
    if (r >= a.T * a.g) return (uint32_t)len;
    uint32_t t, hh;
    kv4_token(a, r, t, hh);
    return (uint32_t)max(len - (int32_t)(a.T - 1u - t), 0);
}

/* The lane's part of the window of scales, from E and open. */
template <int G, int NT>
DEV void kv4_window(Kv4State<G, NT> &s)
{
    const uint32_t mine = lane_id() % G;
    uint32_t e = s.E[0];
#pragma unroll
    for (int g = 1; g < G; g++) e = mine == (uint32_t)g ? s.E[g] : e;
    const uint32_t lo = s.open >> mine & ~(s.open / GPUOS_KV4_WIDE) & 1u ? (12u - e) & 0xFFFFu : 0x4000u;
    s.nlo = lo | lo << 16;
    s.factor = (15u - e) * 0x04000400u;
}

/* Where the lane's part of a tile's query row begins (channel 8 j); null
 * behind the last row. */
template <int G>
DEV const uint16_t *kv4_q_row(const Kv4Args &a, const Kv4Pos &p, uint32_t row)
{
    const uint32_t r = p.r0 + row;
    uint32_t t, hh;
    kv4_token(a, r, t, hh);
    return r < a.T * a.g
               ? a.q + (((uint64_t)p.b * a.T + t) * a.H + (uint64_t)p.h * a.g + hh) * (32u * G) + 8u * (lane_id() & 3u)
               : nullptr;
}
/* The item's query rows, as they lie in memory. */
template <int G, int NT>
struct Kv4Query {
    uint4 raw[NT][G]; /* row 8 nt + i: channels 32 g + 8 j + {0..7} */
};
template <int G, int NT>
DEV void kv4_load_q(const Kv4Args &a, const Kv4Pos &p, Kv4Query<G, NT> &x)
{
    constexpr uint32_t D = 32u * G;
    const uint32_t lane = lane_id(), i = lane >> 2, j = lane & 3u;
    const uint32_t h = p.h, r0 = p.r0;
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
        const uint32_t r = r0 + 8u * nt + i;
        const bool have = r < a.T * a.g;
        uint32_t t, hh;
        kv4_token(a, r, t, hh);
        const uint16_t *qr = a.q + (((uint64_t)p.b * a.T + t) * a.H + (uint64_t)h * a.g + hh) * D + 8u * j;
#pragma unroll
        for (int g = 0; g < G; g++)
            x.raw[nt][g] = have ? __ldcg(reinterpret_cast<const uint4 *>(qr + 32 * g)) : make_uint4(0, 0, 0, 0);
    }
}
/* An item's first state. */
template <int G, int NT>
DEV void kv4_begin(const Kv4Args &a, const Kv4Pos &p, const Kv4Query<G, NT> &qx, Kv4State<G, NT> &s)
{
    const uint32_t j = lane_id() & 3u, r0 = p.r0;
    bool wide = false;
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
        const uint4(&raw)[G] = qx.raw[nt];
        /* each group's largest magnitude (two groups a word), as bf16 bits:
         * those of positive numbers are in order, infinity and NaN (the row
         * is left as it is) on top */
        uint32_t w = 0, least = 0xFFFFFFFFu; /* (less one, so that an empty group is the most) */
#pragma unroll
        for (int g = 0; g < G; g += 2) {
            uint32_t m[2];
#pragma unroll
            for (int h = 0; h < 2; h++)
                m[h] = __vmaxu2(__vmaxu2(raw[g + h].x & 0x7FFF7FFFu, raw[g + h].y & 0x7FFF7FFFu),
                                __vmaxu2(raw[g + h].z & 0x7FFF7FFFu, raw[g + h].w & 0x7FFF7FFFu));
            uint32_t top = __vmaxu2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
            top = __vmaxu2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = __vmaxu2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            w = __vmaxu2(w, top);
            least = __viaddmin_u16x2(top, 0xFFFFFFFFu, least);
        }
        w = max(w & 0xFFFFu, w >> 16);
        least = min(least & 0xFFFFu, least >> 16) + 1u;
        /* k: the largest times 2^-k is in [128, 256); both 2^k and 2^-k stay normal numbers */
        const int k = w == 0 || w >= 0x7F80u ? 0 : max(-126, (int)(w >> 7) - 127 - 7);
        /* the factor stays positive: a negative scale turns q, one of zero
         * empties it */
        float down = kv4_pow2(-k), f = fabsf(a.scale) * kv4_pow2(k);
        /* a group 2^14 below the largest has lost bits in f16, a factor that
         * is no normal number has too, and under a large one the least keys
         * count: every page goes the slow way */
        wide |= least + (14u << 7) < w || ((f < FLT_MIN || f > 0x1p80f) && a.scale != 0.0f);
        if (a.scale < 0.0f) down = -down;
        if (f == 0.0f) {
            down = 0.0f;
            f = 1.0f;
        }
#pragma unroll
        for (int g = 0; g < G; g++) {
            const uint32_t x[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
#pragma unroll
            for (int c = 0; c < 4; c++) s.q[nt][g][c] = kv4_pack_h2(bf_lo(x[c]) * down, bf_hi(x[c]) * down);
        }
        s.f[nt][0] = __shfl_sync(0xFFFFFFFFu, f, 8 * j);
        s.f[nt][1] = __shfl_sync(0xFFFFFFFFu, f, 8 * j + 4);
#pragma unroll
        for (int c = 0; c < 2; c++) {
            s.m[nt][c] = -FLT_MAX;
            s.l[nt][c] = 0.0f;
            s.lim[nt][c] = kv4_row_limit(a, p.len, r0 + 8u * nt + 2u * j + c);
        }
#pragma unroll
        for (int g = 0; g < G; g++)
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
                for (int c = 0; c < 4; c++) s.acc[nt][g][u][c] = 0.0f;
    }
#pragma unroll
    for (int g = 0; g < G; g++) s.E[g] = 0;
    s.nan = 0;
    s.open = __any_sync(0xFFFFFFFFu, wide) ? GPUOS_KV4_WIDE : (1u << G) - 1u;
    kv4_window(s);
    s.min_lim = kv4_row_limit(a, p.len, r0); /* rows come in order of t */
}

template <bool GLOBAL>
DEV uint4 kv4_ld16(const unsigned char *p)
{
    if (GLOBAL) return __ldcg(reinterpret_cast<const uint4 *>(p));
    return *reinterpret_cast<const uint4 *>(p);
}
template <bool GLOBAL>
DEV uint32_t kv4_ld4(const unsigned char *p)
{
    if (GLOBAL) return __ldcg(reinterpret_cast<const uint32_t *>(p));
    return *reinterpret_cast<const uint32_t *>(p);
}
/* The bytes of a word of four keys from key0 on that are below n. */
DEV uint32_t kv4_keep(uint32_t key0, uint32_t n)
{
    if (key0 + 4u <= n) return 0xFFFFFFFFu;
    if (key0 >= n) return 0u;
    return (1u << (8u * (n - key0))) - 1u;
}

/* 2^n for |n| up to 250 in two factors, as 2^n itself may leave fp32's range. */
DEV float2 kv4_pow2x2(int n)
{
    n = min(max(n, -250), 250);
    return make_float2(kv4_pow2(n / 2), kv4_pow2(n - n / 2));
}
/* x 2^n of a number x >= 0 (0 below 2^-126), by its exponent; NaN stays */
DEV float kv4_shift(float x, int n)
{
    const uint32_t u = __float_as_uint(x);
    const int e = (int)(u >> 23);
    return e != 0 && e + n > 0 || e >= 255 ? __uint_as_float(e >= 255 ? u : u + ((uint32_t)n << 23)) : 0.0f;
}
/* floor(log2 |x|) of a number's bits, sign taken off; below 2^-126: -127 */
DEV int kv4_log2(uint32_t bits) { return (int)(bits >> 23) - 127; }
/* A word or byte of a page, which lies in shared or global memory (volatile:
 * never from L1, which other ops' writes pass by). */
DEV uint32_t kv4_any32(const unsigned char *p) { return *reinterpret_cast<const volatile uint32_t *>(p); }
DEV uint32_t kv4_any8(const unsigned char *p) { return *reinterpret_cast<const volatile unsigned char *>(p); }
/* Largest of the lanes that hold a row's keys. */
DEV int kv4_max_keys(int x)
{
    x = max(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
    x = max(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
    return max(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
}

/* The lane's word of value scales, keys key0 .. key0 + 3: what lies behind the
 * page's nv keys becomes the window's largest byte (its weights are zero). */
template <int G, int NT>
DEV uint32_t kv4_fill(uint32_t vw, uint32_t key0, uint32_t nv, const Kv4State<G, NT> &s)
{
    const uint32_t keep = kv4_keep(key0, nv);
    return (vw & keep) | (min(12u - (uint32_t)(int)(int16_t)s.nlo, 255u) * 0x01010101u & ~keep);
}
/* Does any lane's word hold a byte outside E - 12 .. E (the larger of byte -
 * (E - 12), mod 2^16, and 12, is 12 for the others), or its key a scale too
 * large (far), or has the page not come for it (here)? */
template <int G, int NT>
DEV bool kv4_outside(uint32_t vw, uint32_t far, bool here, const Kv4State<G, NT> &s)
{
    const uint32_t lo = __viaddmax_u16x2(__byte_perm(vw, 0u, 0x4140), s.nlo, 0x000C000Cu);
    const uint32_t x = __viaddmax_u16x2(__byte_perm(vw, 0u, 0x4342), s.nlo, lo) ^ 0x000C000Cu;
    return __any_sync(0xFFFFFFFFu, (x | far) != 0u || !here);
}

/* A page holds value scales outside its groups' windows (vw: the lane's word
 * of them), or key scales too large (far). Before the first weight the windows
 * are free: each is laid four octaves above the largest scale of the keys that
 * every row sees (of all keys, where that is none), and its twelve octaves
 * hold most pages. False if the page does not fit all the same. */
template <int G, int NT>
DEV bool kv4_fit(uint32_t base, uint32_t nv, uint32_t key0, uint32_t &vw, uint32_t far, bool here, Kv4State<G, NT> &s)
{
    float any = 0.0f;
#pragma unroll
    for (int nt = 0; nt < NT; nt++) any = fmaxf(any, fmaxf(s.l[nt][0], s.l[nt][1]));
    if (__any_sync(0xFFFFFFFFu, any != 0.0f)) return false;
    const uint32_t lane = lane_id();
    const uint32_t all = s.min_lim > base ? min(nv, s.min_lim - base) : nv;
    const uint32_t x = vw & kv4_keep(key0, all);
    const uint32_t top = max(max(x & 255u, x >> 8 & 255u), max(x >> 16 & 255u, x >> 24));
#pragma unroll
    for (int g = 0; g < G; g++) {
        const uint32_t t = __reduce_max_sync(0xFFFFFFFFu, lane % G == (uint32_t)g ? top : 0u);
        if (t != 0u && t != 255u) s.E[g] = t + 4u; /* (acc is zero) */
    }
    kv4_window(s);
    vw = kv4_fill(vw, key0, nv, s);
    return !kv4_outside(vw, far, here, s);
}

/* A page whose value scales lie too far apart, or too far from what the rows
 * have met, for weights in f16 under one unit, or whose keys are so large that
 * their products with a query scaled to 128 may leave fp32 although the scores
 * do not, or a query whose groups lie far apart (s->q[nt][0] says where it
 * lies): as kv4_page, but each group of a query row has its own power of
 * two, which meets the key's scale and the factor's in one exponent, and each
 * row's products p 2^b are formed in fp32 and rounded to f16 against their own
 * largest, 2^x. Then the window of scales is laid anew: four octaves above the
 * scale of what the page's heaviest keys hold, but never so high that its unit
 * is more than 2^12 above what some row has weighed (cap), because that is
 * what bounds the error of the pages that follow; if the accumulators' range
 * asks for more, the window is closed and every page comes here. (Rows of one
 * tile that heed values more than 2^150 apart in one group: the smaller are
 * lost.) A call whose every page comes here took 740 us instead of 81 (64
 * requests of 2,000 to 16,383 tokens, scales random over 40 octaves); out of
 * line, so that the common path keeps its registers, and named for its place
 * among the cache's ops behind the others (see op_xwrite). */
template <int G, int NT>
__device__ __noinline__ void op_x_slow(const unsigned char *pg, uint32_t base, uint32_t nv, uint32_t rows, float scale, Kv4State<G, NT> *s)
{
    constexpr uint32_t D = 32u * G;
    constexpr int NONE = -100000;
    const uint32_t lane = lane_id(), i = lane >> 2, j = lane & 3u;
    const uint32_t k0 = 4u * (i >> 1) + (i & 1u); /* keys 16 t + k0 + {0, 2} */
    float sc[2][NT][4];
    uint32_t lim[NT][2]; /* (behind the last row: sees nothing) */
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
#pragma unroll
        for (int r = 0; r < 2; r++) lim[nt][r] = 8u * nt + 2u * j + r < rows ? s->lim[nt][r] : 0u;
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int c = 0; c < 4; c++) sc[t][nt][c] = 0.0f;
    }
    const uint16_t *row[NT];
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
        row[nt] = reinterpret_cast<const uint16_t *>((uint64_t)s->q[nt][0][1] << 32 | s->q[nt][0][0]);
    /* scale = rest 2^es; an infinity or NaN is all rest, zero all exponent */
    const uint32_t sb = __float_as_uint(scale) & 0x7FFFFFFFu;
    const int es = sb == 0u ? -4096 : (sb >= 0x7F800000u ? 0 : max(kv4_log2(sb), -126));
    const float rest = sb == 0u ? 1.0f : scale * kv4_pow2(-max(es, -126));
#pragma unroll 1
    for (uint32_t g = 0; g < G; g++) {
        uint32_t q[NT][4];
        int kg[NT][2]; /* of rows 2 j, 2 j + 1 */
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            const uint4 raw = row[nt] ? __ldcg(reinterpret_cast<const uint4 *>(row[nt] + 32u * g)) : make_uint4(0, 0, 0, 0);
            const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
            uint32_t w = 0;
#pragma unroll
            for (int c = 0; c < 4; c++) w = __vmaxu2(w, x[c] & 0x7FFF7FFFu);
            w = max(w & 0xFFFFu, w >> 16);
            w = max(w, __shfl_xor_sync(0xFFFFFFFFu, w, 1));
            w = max(w, __shfl_xor_sync(0xFFFFFFFFu, w, 2));
            const int k = w == 0 || w >= 0x7F80u ? 0 : max(-126, (int)(w >> 7) - 127 - 7);
            const float down = kv4_pow2(-k);
#pragma unroll
            for (int c = 0; c < 4; c++) q[nt][c] = kv4_pack_h2(bf_lo(x[c]) * down, bf_hi(x[c]) * down);
            kg[nt][0] = __shfl_sync(0xFFFFFFFFu, k, 8 * j) + es - 127;
            kg[nt][1] = __shfl_sync(0xFFFFFFFFu, k, 8 * j + 4) + es - 127;
        }
#pragma unroll
        for (int t = 0; t < 2; t++) {
            const unsigned char *kp = pg + (uint32_t)t * 8u * D + lane * 8u * G + 4u * g;
            const unsigned char *ks = pg + 32u * D + (16u * t + k0) * G + g;
            uint32_t x0[4], x1[4];
            kv4_decode4(kv4_any32(kp), x0);
            kv4_decode4(kv4_any32(kp + 4u * G), x1);
            const uint32_t b[2] = {kv4_any8(ks), kv4_any8(ks + 2u * G)};
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                kv4_mma(c, x0[0], x1[0], x0[1], x1[1], q[nt][0], q[nt][1]);
                kv4_mma(c, x0[2], x1[2], x0[3], x1[3], q[nt][2], q[nt][3]);
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const float2 f = kv4_pow2x2((int)b[k >> 1] + kg[nt][k & 1]);
                    sc[t][nt][k] += b[k >> 1] == 255u ? NAN : c[k] * f.x * f.y;
                }
            }
        }
    }
    /* weights, and for each row: whether it had weight before this page, the
     * octaves that its reference rose and what that leaves of what is
     * accumulated, its largest weight here */
    float rise[NT][2], fall[NT][2];
    bool before[NT][2], lost[NT][2]; /* lost: not a number */
    int heavy[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int r = 0; r < 2; r++) {
            float mx = -INFINITY;
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const uint32_t key = 16u * t + k0 + 2u * h;
                    float &x = sc[t][nt][r + 2 * h];
                    x = key < nv && base + key < lim[nt][r] ? x * rest : -INFINITY;
                    mx = fmaxf(mx, x);
                }
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
            const float m0 = s->m[nt][r], m = mx - 15.0f > m0 ? mx - 14.0f : m0;
            const float alpha = kv4_ex2(m0 - m), l0 = s->l[nt][r];
            before[nt][r] = kv4_max_keys(l0 != 0.0f) != 0;
            lost[nt][r] = kv4_max_keys(l0 != l0) != 0;
            rise[nt][r] = m - m0;
            float l = l0 * alpha;
            uint32_t top = 0;
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    float &x = sc[t][nt][r + 2 * h];
                    x = kv4_ex2(x - m);
                    l += x;
                    top = max(top, __float_as_uint(x) & 0x7FFFFFFFu);
                }
            heavy[nt][r] = kv4_log2((uint32_t)kv4_max_keys((int)top));
            s->m[nt][r] = m;
            s->l[nt][r] = l;
            fall[nt][r] = alpha;
        }
#pragma unroll 1
    for (uint32_t g = 0; g < G; g++) {
        uint32_t b[2][2]; /* scale bytes of the lane's keys */
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const uint32_t key = 16u * t + k0 + 2u * h;
                b[t][h] = kv4_any8(pg + 33u * D + (key >> 2) * 4u * G + (key & 3u) + 4u * g);
            }
        int x[NT][2], cap = -NONE, top = NONE, like = NONE;
        uint32_t pb[2][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            float w[2][4];
#pragma unroll
            for (int r = 0; r < 2; r++) {
                int most = NONE, nan = 0;
#pragma unroll
                for (int t = 0; t < 2; t++)
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const uint32_t key = 16u * t + k0 + 2u * h, p = __float_as_uint(sc[t][nt][r + 2 * h]);
                        const bool see = key < nv && base + key < lim[nt][r];
                        if (b[t][h] == 255u) nan |= see;
                        else if (p != 0u && p < 0x7F800000u) most = max(most, kv4_log2(p) + (int)b[t][h]);
                    }
                x[nt][r] = most = kv4_max_keys(most);
                if (kv4_max_keys(nan)) s->nan |= 1u << (2u * NT * g + 2u * nt + r);
#pragma unroll
                for (int t = 0; t < 2; t++)
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const float p = sc[t][nt][r + 2 * h];
                        w[t][r + 2 * h] = b[t][h] == 255u ? 0.0f : (most == NONE ? p : kv4_shift(p, (int)b[t][h] - most + 14));
                    }
                /* the largest p 2^b that the row is known to have met is at
                 * least 2^(E - 12) if the window was open, and 2^(x - 14) */
                if (lim[nt][r] == 0u || lost[nt][r] || !(before[nt][r] || most != NONE)) continue;
                const int old = before[nt][r] && (s->open >> g & 1u) ? (int)s->E[g] - (int)fminf(ceilf(rise[nt][r]), 4096.0f) : NONE;
                cap = min(cap, max(old, most == NONE ? NONE : most - 2));
                top = max(top, most);
                if (most != NONE) like = max(like, most - heavy[nt][r]);
            }
#pragma unroll
            for (int t = 0; t < 2; t++) {
                pb[t][nt][0] = kv4_trans8x8(kv4_pack_h2(w[t][0], w[t][1]));
                pb[t][nt][1] = kv4_trans8x8(kv4_pack_h2(w[t][2], w[t][3]));
            }
        }
        float c[NT][2][4];
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
                for (int k = 0; k < 4; k++) c[nt][u][k] = 0.0f;
#pragma unroll
        for (int t = 0; t < 2; t++) {
            /* two neighbouring channels a byte: 16 bits of the word that holds groups g & ~1 and g | 1 */
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; k++)
                v[k] = kv4_any32(pg + 16u * D + (uint32_t)t * 8u * D + lane * 8u * G + (k * (G / 2) + (g >> 1)) * 4u) >> (16u * (g & 1u));
            uint32_t e01[4], o01[4], e23[4], o23[4];
            kv4_decode4((v[0] & 0x0F0Fu) | ((v[1] << 4) & 0xF0F0u), e01);
            kv4_decode4(((v[0] >> 4) & 0x0F0Fu) | (v[1] & 0xF0F0u), o01);
            kv4_decode4((v[2] & 0x0F0Fu) | ((v[3] << 4) & 0xF0F0u), e23);
            kv4_decode4(((v[2] >> 4) & 0x0F0Fu) | (v[3] & 0xF0F0u), o23);
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                kv4_mma(c[nt][0], e01[0], o01[0], e23[0], o23[0], pb[t][nt][0], pb[t][nt][1]);
                kv4_mma(c[nt][1], e01[1], o01[1], e23[1], o23[1], pb[t][nt][0], pb[t][nt][1]);
            }
        }
        /* over the rows: the lanes j of each i */
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            cap = min(cap, __shfl_xor_sync(0xFFFFFFFFu, cap, o));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            like = max(like, __shfl_xor_sync(0xFFFFFFFFu, like, o));
        }
        float acc[NT][2][4];
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
                for (int k = 0; k < 4; k++) acc[nt][u][k] = s->acc[nt][g][u][k] * fall[nt][k & 1];
        const int E = (int)s->E[g];
        int unit = E;
        if (top != NONE) {
            /* accumulators of 2^-90 to 2^90 leave room for what follows */
            uint32_t big = 0;
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    const uint32_t a = __float_as_uint(acc[nt][k >> 2][k & 3]) & 0x7FFFFFFFu;
                    big = max(big, a < 0x7F800000u ? a : 0u);
                }
            big = __reduce_max_sync(0xFFFFFFFFu, big);
            int least = top - 74;
            if (big != 0u) least = max(least, E + kv4_log2(big) - 90);
            unit = min(like + 4, cap);
            unit = min(max(unit < least ? max(E, least) : unit, 1), 300);
            s->E[g] = (uint32_t)unit;
            s->open = unit <= cap ? s->open | 1u << g : s->open & ~(1u << g);
        }
        const float2 old = kv4_pow2x2(E - unit);
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const float2 add = kv4_pow2x2(x[nt][r] == NONE ? 0 : x[nt][r] - 14 - unit);
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const int u = k >> 1, v = r + 2 * (k & 1);
                    s->acc[nt][g][u][v] = acc[nt][u][v] * old.x * old.y + c[nt][u][v] * add.x * add.y;
                }
            }
    }
    kv4_window(*s);
}

/* The state in a copy, so that it stays in registers where this is not called. */
template <int G, int NT>
DEV void kv4_page_rare(const Kv4Args &a, const Kv4Pos &p, const unsigned char *pg, uint32_t base, uint32_t nv, Kv4State<G, NT> &s)
{
    Kv4State<G, NT> copy = s;
#pragma unroll
    for (int nt = 0; nt < NT; nt++) { /* (the page's path reads the query itself) */
        const uint64_t at = (uint64_t)kv4_q_row<G>(a, p, 8u * nt + (lane_id() >> 2));
        copy.q[nt][0][0] = (uint32_t)at;
        copy.q[nt][0][1] = (uint32_t)(at >> 32);
    }
    op_x_slow<G, NT>(pg, base, nv, a.T * a.g - p.r0, a.scale, &copy);
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int g = 0; g < G; g++)
#pragma unroll
            for (int c = 0; c < 4; c++) copy.q[nt][g][c] = s.q[nt][g][c];
    s = copy;
}
/* Existing keys of the page that begins with key `base`. */
DEV uint32_t kv4_existing(uint32_t base, uint32_t valid)
{
    return valid > base ? min(valid - base, (uint32_t)GPUOS_KV4_PAGE) : 0u;
}

/* One page: keys [base, base + 32) of the item, of which those below `valid`
 * exist (the rest of a request's last page holds anything). `scratch` (768
 * bytes of the warp's) passes the scales from the lane that converts a word
 * of them to the lanes that use them; without it (GLOBAL: the page is in
 * global memory, there is no staging) they pass by shuffles. False: nothing is
 * done, as the page has to go the slow way (kv4_page_rare), or has not come
 * (here, as each lane found it: the limit of their waits may part them). */
template <int G, int NT, bool GLOBAL>
DEV bool kv4_page(const unsigned char *pg, unsigned char *scratch, uint32_t base, uint32_t valid, bool here, Kv4State<G, NT> &s)
{
    constexpr uint32_t D = 32u * G;
    const uint32_t lane = lane_id(), i = lane >> 2, j = lane & 3u;
    const uint32_t nv = kv4_existing(base, valid);

    /* ---- scales. Key scales: lane = key, G bytes -> G floats 2^(byte - 127)
     * (byte 0 gives 0: with a factor up to 2^80 such a group would add 2^-30
     * to a score). Above 191 (255 among them) the page goes the slow way;
     * below, a sum of D products with queries up to 256 stays under 2^82.
     * Value scales: lane = word ((key / 4) G + group) -> four f16, 2^(byte -
     * E): exponent field byte - E + 15, 3 to 15 for the bytes of the window;
     * with any other byte the page goes the slow way. ---- */
    float kf[G];
    uint32_t far;
    {
        const uint32_t w = G == 4 ? kv4_ld4<GLOBAL>(pg + 32u * D + 4u * lane)
                                  : kv4_ld4<GLOBAL>(pg + 32u * D + 4u * (lane >> 1)) >> (16u * (lane & 1u));
#pragma unroll
        for (int g = 0; g < G; g++)
            kf[g] = __uint_as_float((g < 3 ? w << (23 - 8 * g) : w >> 1) & 0x7F800000u);
        far = lane < nv ? w & w << 1 & (G == 4 ? 0x80808080u : 0x8080u) : 0u;
    }
    uint2 vs;
    {
        const uint32_t word = lane % (8u * G), key0 = word / G * 4u;
        uint32_t vw = kv4_ld4<GLOBAL>(pg + 33u * D + 4u * word);
        if (nv < GPUOS_KV4_PAGE) vw = kv4_fill(vw, key0, nv, s);
        if (kv4_outside(vw, far, here, s) && !kv4_fit<G, NT>(base, nv, key0, vw, far, here, s)) return false;
        vs.x = __byte_perm(vw, 0u, 0x4140) * 1024u + s.factor;
        vs.y = __byte_perm(vw, 0u, 0x4342) * 1024u + s.factor;
    }
    if (!GLOBAL) {
        __syncwarp(); /* the last page's readers are done */
        if (G == 4) *reinterpret_cast<float4 *>(scratch + 16u * lane) = make_float4(kf[0], kf[1], kf[G - 2], kf[G - 1]);
        else *reinterpret_cast<float2 *>(scratch + 8u * lane) = make_float2(kf[0], kf[1]);
        *reinterpret_cast<uint2 *>(scratch + 512u + 8u * (lane % (8u * G))) = vs; /* (G == 2: both halves of the warp alike) */
        __syncwarp();
    }

    /* ---- scores: S^T tile t = keys 16 t .. 16 t + 15 against the rows ---- */
    float sc[2][NT][4];
#pragma unroll
    for (int t = 0; t < 2; t++) {
        const uint32_t k0 = 16u * t + 4u * (i >> 1) + (i & 1u); /* the lane's keys: k0 (c 0, 1) and k0 + 2 (c 2, 3) */
        uint32_t kw[2][G];
        float f0[G], f1[G];
        const unsigned char *kp = pg + (uint32_t)t * 8u * D + lane * 8u * G;
        if (G == 4) {
            const uint4 x = kv4_ld16<GLOBAL>(kp), y = kv4_ld16<GLOBAL>(kp + 16);
            kw[0][0] = x.x; kw[0][1] = x.y; kw[0][G - 2] = x.z; kw[0][G - 1] = x.w;
            kw[1][0] = y.x; kw[1][1] = y.y; kw[1][G - 2] = y.z; kw[1][G - 1] = y.w;
        } else {
            const uint4 x = kv4_ld16<GLOBAL>(kp);
            kw[0][0] = x.x; kw[0][1] = x.y;
            kw[1][0] = x.z; kw[1][1] = x.w;
        }
        if (GLOBAL) {
#pragma unroll
            for (int g = 0; g < G; g++) {
                f0[g] = __shfl_sync(0xFFFFFFFFu, kf[g], k0);
                f1[g] = __shfl_sync(0xFFFFFFFFu, kf[g], k0 + 2u);
            }
        } else if (G == 4) {
            const float4 x = *reinterpret_cast<const float4 *>(scratch + 16u * k0);
            const float4 y = *reinterpret_cast<const float4 *>(scratch + 16u * (k0 + 2u));
            f0[0] = x.x; f0[1] = x.y; f0[G - 2] = x.z; f0[G - 1] = x.w;
            f1[0] = y.x; f1[1] = y.y; f1[G - 2] = y.z; f1[G - 1] = y.w;
        } else {
            const float2 x = *reinterpret_cast<const float2 *>(scratch + 8u * k0);
            const float2 y = *reinterpret_cast<const float2 *>(scratch + 8u * (k0 + 2u));
            f0[0] = x.x; f0[1] = x.y;
            f1[0] = y.x; f1[1] = y.y;
        }
#pragma unroll
        for (int g = 0; g < G; g++) {
            uint32_t x0[4], x1[4];
            kv4_decode4(kw[0][g], x0);
            kv4_decode4(kw[1][g], x1);
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                kv4_mma(c, x0[0], x1[0], x0[1], x1[1], s.q[nt][g][0], s.q[nt][g][1]);
                kv4_mma(c, x0[2], x1[2], x0[3], x1[3], s.q[nt][g][2], s.q[nt][g][3]);
                if (g == 0) {
                    sc[t][nt][0] = c[0] * f0[g]; sc[t][nt][1] = c[1] * f0[g];
                    sc[t][nt][2] = c[2] * f1[g]; sc[t][nt][3] = c[3] * f1[g];
                } else {
                    sc[t][nt][0] = fmaf(c[0], f0[g], sc[t][nt][0]); sc[t][nt][1] = fmaf(c[1], f0[g], sc[t][nt][1]);
                    sc[t][nt][2] = fmaf(c[2], f1[g], sc[t][nt][2]); sc[t][nt][3] = fmaf(c[3], f1[g], sc[t][nt][3]);
                }
            }
        }
    }
    if (base + GPUOS_KV4_PAGE > s.min_lim || nv < GPUOS_KV4_PAGE) { /* the same in every lane */
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    const uint32_t key = 16u * t + 4u * (i >> 1) + (i & 1u) + (c & 2u);
                    if (key >= nv || base + key >= s.lim[nt][c & 1]) sc[t][nt][c] = -INFINITY;
                }
    }

    /* ---- online softmax. Weights are 2^(score - m), m a reference 14 below
     * the largest score when it was last set: it is set anew (and what is
     * accumulated rescaled) only when a score comes 15 above it. ---- */
    float high[NT][2];
    bool over = false;
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int r = 0; r < 2; r++) {
            high[nt][r] = fmaxf(fmaxf(sc[0][nt][r], sc[0][nt][r + 2]), fmaxf(sc[1][nt][r], sc[1][nt][r + 2]));
            over |= fmaf(high[nt][r], s.f[nt][r], -15.0f) > s.m[nt][r];
        }
    if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int r = 0; r < 2; r++) {
                float mx = high[nt][r] * s.f[nt][r];
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
                const float mn = fmaxf(s.m[nt][r], mx - 14.0f);
                const float alpha = kv4_ex2(s.m[nt][r] - mn); /* 0 from the first reference, -FLT_MAX */
                s.m[nt][r] = mn;
                s.l[nt][r] *= alpha;
#pragma unroll
                for (int g = 0; g < G; g++)
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        s.acc[nt][g][u][r] *= alpha;
                        s.acc[nt][g][u][r + 2] *= alpha;
                    }
            }
    }
    uint32_t pb[2][NT][2]; /* p^T: B fragments of the second product */
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int t = 0; t < 2; t++) {
#pragma unroll
            for (int c = 0; c < 4; c++)
                sc[t][nt][c] = kv4_ex2(fmaf(sc[t][nt][c], s.f[nt][c & 1], -s.m[nt][c & 1]));
            s.l[nt][0] += sc[t][nt][0] + sc[t][nt][2];
            s.l[nt][1] += sc[t][nt][1] + sc[t][nt][3];
            pb[t][nt][0] = kv4_trans8x8(kv4_pack_h2(sc[t][nt][0], sc[t][nt][1]));
            pb[t][nt][1] = kv4_trans8x8(kv4_pack_h2(sc[t][nt][2], sc[t][nt][3]));
        }
    /* ---- O^T += V^T p^T ---- */
#pragma unroll
    for (int t = 0; t < 2; t++) {
        const unsigned char *vp = pg + 16u * D + (uint32_t)t * 8u * D + lane * 8u * G;
        uint32_t w[4][G / 2]; /* key 4 j + slot: groups 2 w, 2 w + 1 */
        if (G == 4) {
            const uint4 x = kv4_ld16<GLOBAL>(vp), y = kv4_ld16<GLOBAL>(vp + 16);
            w[0][0] = x.x; w[0][G / 2 - 1] = x.y; w[1][0] = x.z; w[1][G / 2 - 1] = x.w;
            w[2][0] = y.x; w[2][G / 2 - 1] = y.y; w[3][0] = y.z; w[3][G / 2 - 1] = y.w;
        } else {
            const uint4 x = kv4_ld16<GLOBAL>(vp);
            w[0][0] = x.x; w[1][0] = x.y; w[2][0] = x.z; w[3][0] = x.w;
        }
        uint32_t s01[G], s23[G];
        if (GLOBAL) {
#pragma unroll
            for (int g = 0; g < G; g++) {
                s01[g] = __shfl_sync(0xFFFFFFFFu, vs.x, ((uint32_t)t * 4u + j) * G + g);
                s23[g] = __shfl_sync(0xFFFFFFFFu, vs.y, ((uint32_t)t * 4u + j) * G + g);
            }
        } else {
#pragma unroll
            for (int x = 0; x < G / 2; x++) {
                const uint4 y = *reinterpret_cast<const uint4 *>(scratch + 512u + (((uint32_t)t * 4u + j) * G + 2 * x) * 8u);
                s01[2 * x] = y.x; s23[2 * x] = y.y;
                s01[2 * x + 1] = y.z; s23[2 * x + 1] = y.w;
            }
        }
#pragma unroll
        for (int x = 0; x < G / 2; x++) {
            /* bytes of (key, key + 1) pairs of one channel: even channels, odd channels */
            uint32_t e01[4], o01[4], e23[4], o23[4];
            kv4_decode4((w[0][x] & 0x0F0F0F0Fu) | ((w[1][x] << 4) & 0xF0F0F0F0u), e01);
            kv4_decode4(((w[0][x] >> 4) & 0x0F0F0F0Fu) | (w[1][x] & 0xF0F0F0F0u), o01);
            kv4_decode4((w[2][x] & 0x0F0F0F0Fu) | ((w[3][x] << 4) & 0xF0F0F0F0u), e23);
            kv4_decode4(((w[2][x] >> 4) & 0x0F0F0F0Fu) | (w[3][x] & 0xF0F0F0F0u), o23);
#pragma unroll
            for (int gg = 0; gg < 2; gg++) {
                const int g = 2 * x + gg;
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    const uint32_t b0 = kv4_hmul2(pb[t][nt][0], s01[g]), b1 = kv4_hmul2(pb[t][nt][1], s23[g]);
                    kv4_mma(s.acc[nt][g][0], e01[2 * gg], o01[2 * gg], e23[2 * gg], o23[2 * gg], b0, b1);
                    kv4_mma(s.acc[nt][g][1], e01[2 * gg + 1], o01[2 * gg + 1], e23[2 * gg + 1], o23[2 * gg + 1], b0, b1);
                }
            }
        }
    }
    return true;
}

/* End of a run within an item: l summed over the lanes of a row, acc brought
 * to the mean of the values under this run's weights. */
template <int G, int NT>
DEV void kv4_finish(Kv4State<G, NT> &s)
{
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
        float inv[2];
#pragma unroll
        for (int r = 0; r < 2; r++) {
            float l = s.l[nt][r];
            l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
            l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
            l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
            s.l[nt][r] = l;
            inv[r] = l != 0.0f ? 1.0f / l : 0.0f;
        }
#pragma unroll
        for (int g = 0; g < G; g++) {
            /* 2^(E - 127) in two factors (E may be 0, or above 254) */
            const int e = (int)s.E[g] - 127, e1 = e / 2;
            const float p2 = kv4_pow2(e - e1);
#pragma unroll
            for (int c = 0; c < 4; c++) {
                const float x = inv[c & 1] * kv4_pow2(e1);
                s.acc[nt][g][0][c] = s.acc[nt][g][0][c] * x * p2;
                s.acc[nt][g][1][c] = s.acc[nt][g][1][c] * x * p2;
            }
        }
    }
    if (__any_sync(0xFFFFFFFFu, s.nan != 0u)) {
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int g = 0; g < G; g++)
#pragma unroll
                for (int c = 0; c < 4; c++)
                    if (s.nan >> (2 * NT * g + 2 * nt + (c & 1)) & 1u) s.acc[nt][g][0][c] = s.acc[nt][g][1][c] = NAN;
    }
}
/* Rows that see no key are zero; the sum of a row that sees some is zero only
 * when no score is a number. */
DEV float kv4_empty(uint32_t lim) { return lim ? NAN : 0.0f; }

template <int G, int NT>
DEV void kv4_store(const Kv4Args &a, const Kv4Pos &p, const Kv4State<G, NT> &s)
{
    constexpr uint32_t D = 32u * G;
    const uint32_t lane = lane_id(), i = lane >> 2, j = lane & 3u;
    const uint32_t h = p.h, r0 = p.r0;
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int c = 0; c < 2; c++) {
            const uint32_t r = r0 + 8u * nt + 2u * j + c;
            if (r >= a.T * a.g) continue;
            uint32_t t, hh;
            kv4_token(a, r, t, hh);
            uint16_t *o = a.out + (((uint64_t)p.b * a.T + t) * a.H + (uint64_t)h * a.g + hh) * D + 4u * i;
            const bool none = s.l[nt][c] == 0.0f;
            const float z = kv4_empty(s.lim[nt][c]);
#pragma unroll
            for (int g = 0; g < G; g++) {
                uint2 w;
                w.x = pack_bf2(none ? z : s.acc[nt][g][0][c], none ? z : s.acc[nt][g][0][c + 2]);
                w.y = pack_bf2(none ? z : s.acc[nt][g][1][c], none ? z : s.acc[nt][g][1][c + 2]);
                *reinterpret_cast<uint2 *>(o + 32 * g) = w;
            }
        }
}

/* A partial state in memory: NT x 4 float4 {m0, l0, m1, l1} (by j), then the
 * accumulators [nt][g][r][lane] as float4 of the lane's four channels. */
template <int G, int NT>
struct Kv4Part {
    static constexpr uint32_t floats = NT * 16u + NT * G * 256u;
};
static_assert(4u * (GPUOS_KV4_MAX_TILES + 2u * GPUOS_KV4_TILES * Kv4Part<4, 1>::floats) <= GPUOS_KV4_WORKSPACE &&
                  4u * (GPUOS_KV4_MAX_TILES + 2u * GPUOS_KV4_MAX_BLOCKS * Kv4Part<4, 2>::floats) <= GPUOS_KV4_WORKSPACE &&
                  4u * GPUOS_KV4_MAX_TILES == GPUOS_KV4_COUNTERS && GPUOS_KV4_TILES <= GPUOS_KV4_MAX_TILES && GPUOS_KV4_MAX_BLOCKS <= GPUOS_KV4_MAX_TILES,
              "the workspace holds every tile's and block's states and counters");
template <bool GLOBAL, int G, int NT>
DEV void kv4_part_store(void *part, const Kv4State<G, NT> &s)
{
    const uint32_t lane = lane_id();
    float4 *p4 = reinterpret_cast<float4 *>(part);
    auto put = [&](uint32_t at, float4 v) {
        if (GLOBAL) __stcg(p4 + at, v);
        else p4[at] = v;
    };
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
        if (lane < 4) put(nt * 4 + lane, make_float4(s.m[nt][0], s.l[nt][0], s.m[nt][1], s.l[nt][1]));
#pragma unroll
        for (int g = 0; g < G; g++)
#pragma unroll
            for (int r = 0; r < 2; r++)
                put(NT * 4 + ((nt * G + g) * 2 + r) * 32 + lane,
                    make_float4(s.acc[nt][g][0][r], s.acc[nt][g][0][r + 2], s.acc[nt][g][1][r], s.acc[nt][g][1][r + 2]));
    }
}

/* A request's head and row tile. */
struct Kv4Item {
    uint32_t b, h, r0, np;
};
/* Four channels of the output: element idx of a state's accumulators. */
template <int G, int NT>
DEV void kv4_out4(const Kv4Args &a, const Kv4Item &it, uint32_t idx, float l, float4 v)
{
    constexpr uint32_t D = 32u * G;
    const uint32_t lane = idx & 31u, r2 = idx >> 5 & 1u, g = idx >> 6 & (G - 1u), nt = idx / (64u * G);
    const uint32_t r = it.r0 + 8u * nt + 2u * (lane & 3u) + r2;
    if (r >= a.T * a.g) return;
    uint32_t t, hh;
    kv4_token(a, r, t, hh);
    if (l == 0.0f) {
        const float z = kv4_empty(kv4_row_limit(a, __ldcg(a.lens + it.b), r));
        v = make_float4(z, z, z, z);
    }
    uint2 w;
    w.x = pack_bf2(v.x, v.y);
    w.y = pack_bf2(v.z, v.w);
    *reinterpret_cast<uint2 *>(a.out + (((uint64_t)it.b * a.T + t) * a.H + (uint64_t)it.h * a.g + hh) * D + 32u * g + 4u * (lane >> 2)) = w;
}
/* Two stored states, the left one's keys first, into a third place or (dst
 * null) the output. Nothing of a state stays in registers: this is the
 * executor's path, whose worker keeps what a tile leaves it. */
template <int G, int NT>
DEV void kv4_part_merge(const Kv4Args &a, const Kv4Item &it, const float *left, const float *right, float *dst)
{
    const uint32_t lane = lane_id(), j = lane & 3u;
    const float4 *x4 = reinterpret_cast<const float4 *>(left), *y4 = reinterpret_cast<const float4 *>(right);
    float4 *d4 = reinterpret_cast<float4 *>(dst);
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
        const float4 p = __ldcg(x4 + nt * 4 + j), q = __ldcg(y4 + nt * 4 + j);
        __syncwarp(); /* dst may be one of them: every lane has read its rows' (m, l) */
        float wx[2], wy[2], m[2], l[2];
#pragma unroll
        for (int r = 0; r < 2; r++) {
            const float mx = r ? p.z : p.x, lx = r ? p.w : p.y, my = r ? q.z : q.x, ly = r ? q.w : q.y;
            m[r] = fmaxf(mx, my);
            wx[r] = lx * kv4_ex2(mx - m[r]);
            wy[r] = ly * kv4_ex2(my - m[r]);
            l[r] = wx[r] + wy[r];
            const float inv = l[r] != 0.0f ? 1.0f / l[r] : 0.0f;
            wx[r] *= inv;
            wy[r] *= inv;
        }
        if (dst && lane < 4) __stcg(d4 + nt * 4 + j, make_float4(m[0], l[0], m[1], l[1]));
#pragma unroll
        for (int g0 = 0; g0 < G; g0 += 2) {
            float4 x[4], y[4]; /* both states of two groups in flight (the stores may be to one of them) */
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const uint32_t idx = ((uint32_t)(nt * G + g0) * 2u + k) * 32u + lane;
                x[k] = __ldcg(x4 + NT * 4 + idx);
                y[k] = __ldcg(y4 + NT * 4 + idx);
            }
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const uint32_t idx = ((uint32_t)(nt * G + g0) * 2u + k) * 32u + lane;
                const int r = k & 1;
                const float4 v = make_float4(fmaf(y[k].x, wy[r], x[k].x * wx[r]), fmaf(y[k].y, wy[r], x[k].y * wx[r]),
                                             fmaf(y[k].z, wy[r], x[k].z * wx[r]), fmaf(y[k].w, wy[r], x[k].w * wx[r]));
                if (dst) __stcg(d4 + NT * 4 + idx, v);
                else kv4_out4<G, NT>(a, it, idx, l[r], v);
            }
        }
    }
}

/* The pages of one run within an item, [first, end): into the state, up to one
 * that has to go the slow way; first is then that page, and end otherwise (the
 * call that the slow way takes is the caller's: within this loop it cost 3 %).
 * With staging the pages arrive by bulk copies into the two halves of the
 * warp's buffer in turn. */
template <int G, int NT>
DEV int kv4_run(const Kv4Args &a, const Kv4Pos &p, uint32_t &first, uint32_t end, Kv4State<G, NT> &s)
{
    constexpr uint32_t PB = kv4_page_bytes(32u * G);
    const uint32_t lane = lane_id(), h = p.h;
    const int32_t *row = a.table + (uint64_t)p.b * a.P;
    const uint64_t stride = (uint64_t)a.Hkv * PB;
    const unsigned char *pool = a.pool + (uint64_t)h * PB;
    const uint32_t begin = first;
    const bool staged = stage_hdr()->stage_bytes >= 2u * PB + GPUOS_KV4_SCRATCH;
    WarpStage *w = warp_stage();
    unsigned char *buf = warp_stage_buf();
    int status = GPUOS_ST_OK;
    uint32_t phs = staged ? w->phase[0] | w->phase[1] << 1 : 0u;
    /* page ids, 32 at a time in the warp's lanes; one that is not in the pool
     * stands for no keys (page 0 is read and masked) */
    const uint32_t n = end - begin;
    int32_t ids = 0, ids_next = 0;
    first = end;
    auto load_ids = [&](uint32_t k) { return begin + k + lane < end ? __ldcg(row + begin + k + lane) : 0; };
    ids = load_ids(0);
    auto issue = [&](uint32_t k, int32_t id) {
        if (lane == 0) {
            mbar_expect(&w->mbar[k & 1u], PB);
            bulk_g2s(buf + (k & 1u) * PB, pool + (uint64_t)((uint32_t)id < a.npages ? (uint32_t)id : 0u) * stride, PB,
                     &w->mbar[k & 1u]);
        }
    };
    if (staged) {
        asm volatile("fence.proxy.async;" ::: "memory"); /* pages written by other ops, slots read by the last run */
        issue(0, __shfl_sync(0xFFFFFFFFu, ids, 0));
        if (n > 1) issue(1, __shfl_sync(0xFFFFFFFFu, ids, 1));
    }
#pragma unroll 1
    for (uint32_t k = 0; k < n; k++) {
        if ((k & 31u) == 0) {
            if (k) ids = ids_next;
            ids_next = load_ids(k + 32);
        }
        const int32_t id = __shfl_sync(0xFFFFFFFFu, ids, k & 31u);
        const bool there = (uint32_t)id < a.npages;
        if (!there) status = GPUOS_ST_BAD_ARGS;
        const uint32_t base = (begin + k) * GPUOS_KV4_PAGE, valid = there ? (uint32_t)p.len : 0u;
        if (staged) {
            const uint32_t hb = k & 1u;
            const bool here = mbar_wait(&w->mbar[hb], phs >> hb & 1u);
            phs ^= 1u << hb;
            if (!kv4_page<G, NT, false>(buf + hb * PB, buf + 2u * PB, base, valid, here, s)) {
                /* leave no copy in flight: wait (once more, bounded) for this
                 * half if its copy has not landed, and for the other one if
                 * it has a copy out */
                bool lost = __any_sync(0xFFFFFFFFu, !here);
                if (lost) (void)mbar_wait(&w->mbar[hb], ~(phs >> hb) & 1u);
                if (k + 1 < n) {
                    const uint32_t ph = phs >> (hb ^ 1u) & 1u;
                    if (!mbar_wait(&w->mbar[hb ^ 1u], ph) && !mbar_wait(&w->mbar[hb ^ 1u], ph)) lost = true;
                    phs ^= 1u << (hb ^ 1u);
                }
                lost = __any_sync(0xFFFFFFFFu, lost);
                if (lost) status = GPUOS_ST_COPY_TIMEOUT;
                else first = begin + k;
                break;
            }
            if (k + 2 < n) {
                const int32_t nx = (k & 31u) < 30u ? __shfl_sync(0xFFFFFFFFu, ids, (k + 2) & 31u)
                                                   : __shfl_sync(0xFFFFFFFFu, ids_next, (k + 2) & 31u);
                __syncwarp(); /* every lane is done with this half */
                if (lane == 0) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                issue(k + 2, nx);
            }
        } else {
            if (!kv4_page<G, NT, true>(pool + (uint64_t)(there ? (uint32_t)id : 0u) * stride, nullptr, base, valid, true, s)) {
                first = begin + k;
                break;
            }
        }
    }
    if (staged) {
        __syncwarp();
        if (lane == 0) {
            w->phase[0] = phs & 1u;
            w->phase[1] = phs >> 1 & 1u;
        }
        __syncwarp();
    }
    return status;
}

/* The workspace: GPUOS_KV4_MAX_TILES counters, then two partial states for
 * each tile (an item that began before the tile, an item that ends after it). */
DEV uint32_t *kv4_counters(const gpuos_devdesc *d) { return reinterpret_cast<uint32_t *>(d->aux2); }
template <int G, int NT>
DEV float *kv4_slot(const gpuos_devdesc *d, uint32_t tile, uint32_t which)
{
    return reinterpret_cast<float *>(d->aux2) + GPUOS_KV4_MAX_TILES + ((uint64_t)tile * 2u + which) * Kv4Part<G, NT>::floats;
}

/* One executor tile: a warp's run of units. Partial states of an item meet in
 * a binary tree over its tiles, numbered from the item's first: at the node
 * that splits at s the second to arrive merges the two halves and goes on, so
 * the merge's depth is the logarithm of the tiles and no tile waits. */
template <int G, int NT>
DEV int kv4_sdpa_tile(const gpuos_devdesc *d, uint32_t tile)
{
    Kv4Args a;
    kv4_args(d, 8u * NT, a);
    int32_t len0;
    const uint32_t W = kv4_units(a, len0);
    const uint32_t nt = min(min(d->ntiles, W), (uint32_t)GPUOS_KV4_TILES); /* (what the workspace holds) */
    if (tile >= nt) return GPUOS_ST_OK;
    const Kv4Runs runs(W, nt);
    uint32_t u = runs.start(tile);
    const uint32_t u1 = runs.start(tile + 1u);
    Kv4Pos p;
    kv4_seek(a, u, len0, p);
    int status = GPUOS_ST_OK;
#pragma unroll 1
    while (u < u1) {
        uint32_t begin, end;
        u += kv4_take(p, u1 - u, begin, end);
        bool bad;
        (void)kv4_pages(a, p.len, bad);
        if (bad) {
            status = GPUOS_ST_BAD_ARGS; /* the request's rows are left as they were */
        } else if (begin < end) {
            Kv4State<G, NT> s;
            Kv4Query<G, NT> qx;
            kv4_load_q(a, p, qx);
            kv4_begin(a, p, qx, s);
#pragma unroll 1
            for (uint32_t at = begin; p.len && at < end;) {
                const int st = kv4_run(a, p, at, end, s);
                if (st) status = st;
                if (at < end) {
                    const uint32_t id = (uint32_t)__ldcg(a.table + (uint64_t)p.b * a.P + at), base = at * GPUOS_KV4_PAGE;
                    kv4_page_rare(a, p, a.pool + ((uint64_t)(id < a.npages ? id : 0u) * a.Hkv + p.h) * kv4_page_bytes(32u * G), base,
                                  kv4_existing(base, id < a.npages ? (uint32_t)p.len : 0u), s);
                    at++;
                }
            }
            kv4_finish(s);
            if (begin != 0 || end != p.np) {
                const uint32_t first = runs.run_of(p.first);
                const uint32_t F = runs.run_of(p.first + p.np - 1) - first + 1;
                auto slot = [&](uint32_t at) { return kv4_slot<G, NT>(d, first + at, at == 0); };
                uint32_t c = tile - first;
                kv4_part_store<true>(slot(c), s);
#pragma unroll 1
                for (uint32_t step = 1; step < F; step <<= 1) {
                    const uint32_t other = c ^ step;
                    if (other < F) {
                        uint32_t *cnt = kv4_counters(d) + first + (c | step);
                        __syncwarp();
                        uint32_t old = 0;
                        if (lane_id() == 0) old = atom_add_acq_rel_gpu32(cnt, 1u);
                        old = __shfl_sync(0xFFFFFFFFu, old, 0);
                        if (old == 0) break; /* the other half's last tile goes on */
                        __syncwarp();
                        if (lane_id() == 0) *cnt = 0; /* left zero for the next call */
                        kv4_part_merge<G, NT>(a, Kv4Item{p.b, p.h, p.r0, p.np}, slot(c & ~step), slot(c | step),
                                              step << 1 < F ? slot(c & ~step) : nullptr);
                    }
                    c &= ~step;
                }
            } else {
                kv4_store(a, p, s);
            }
        }
        kv4_next(a, p);
    }
    return status;
}

/* The executor's entries check sizes and alignment again: an alias of an op (a
 * user op id) is not checked on the host. */
DEV bool kv4_aligned(uint64_t p, uint32_t to) { return p != 0 && (p & (to - 1u)) == 0; }
DEV int kv4_sdpa_op(const gpuos_devdesc *d, uint32_t tile)
{
    if (d->dims[0] == 0) return GPUOS_ST_OK;
    const uint32_t H = d->dims[1] & 0xFFFFu, Hkv = d->dims[1] >> 16, D = d->dims[2] & 0xFFFFu, T = d->dims[2] >> 16;
    const uint32_t P = d->dims[3], npages = d->dims[4];
    if (Hkv == 0 || H == 0 || H % Hkv || T == 0 || T > GPUOS_KV4_MAX_T || P == 0 || P > GPUOS_KV4_MAX_PAGES ||
        npages == 0 || npages > GPUOS_KV4_MAX_PAGES || (D != 64 && D != 128))
        return GPUOS_ST_BAD_ARGS;
    if (!kv4_aligned(d->a, 16) || !kv4_aligned(d->b, 16) || !kv4_aligned(d->out, 16) || !kv4_aligned(d->aux2, 16) ||
        !kv4_aligned(d->aux0, 4) || !kv4_aligned(d->aux1, 4))
        return GPUOS_ST_BAD_ARGS;
    const uint32_t HR = Hkv * ((T * (H / Hkv) + GPUOS_KV4_ROWS - 1u) / GPUOS_KV4_ROWS); /* below 2^31 */
    if ((uint64_t)d->dims[0] * HR >= (1ull << 32) / (P + GPUOS_KV4_LEAD)) return GPUOS_ST_BAD_ARGS;
    return D == 128 ? kv4_sdpa_tile<4, 1>(d, tile) : kv4_sdpa_tile<2, 1>(d, tile);
}

/* ---------------------------------------------------------------------------
 * Write and read back. Row (n, h) is token n's head h: keys and values of a
 * row go to (come from) slot slots[n] = page * 32 + key. A negative slot is a
 * hole: not written, read as zeros.
 *
 * A warp takes eight neighbouring tokens of one head at a time, because
 * neighbours in a prompt are neighbours in a page, and lanes in the order of
 * the page: for keys lane (token, j) holds channels 32 g + 8 j .. + 7 of every
 * group g, 4 G contiguous bytes of codes; for values, four tokens at a time,
 * lane (token, i) holds channels 32 g + 4 i .. + 3, 2 G contiguous bytes. Then
 * two keys' (four values') pieces fill a 32-byte sector and a row's channels
 * are moved 64 bytes at a time. Both ops move the rows' bytes: 512 of a bf16
 * row of 128 channels, keys and values, against 136 of codes. 8,192 tokens of
 * 8 heads are written in 9.6 us (4.4 TB/s; 192,512 of them in 134: no one
 * thing is full there, the ALU pipe 72 %, issue 70 %, memory 54 %, with 40 %
 * of the warps that an SM holds; 580 instructions for eight rows), 163,840
 * read back in 154 us (6.26 TB/s, memory).
 *
 * Scale: the least e >= -127 with max |x| <= 6 2^e (at most 125, so that
 * 6 2^e is finite: above it the largest code stands for what is larger).
 * x 2^-e is exact, so a code is the correctly rounded one.
 * ------------------------------------------------------------------------- */
/* The codes of a lane of keys (j) or values (i) of a slot, after the page's. */
template <int G>
DEV uint32_t kv4_k_at(uint32_t key, uint32_t j)
{
    return (key >> 4) * 256u * G + ((((key >> 2 & 3u) * 2u + (key & 1u)) * 4u + j) * 2u + (key >> 1 & 1u)) * 4u * G;
}
template <int G>
DEV uint32_t kv4_v_at(uint32_t key, uint32_t i)
{
    return 512u * G + (key >> 4) * 256u * G + ((i * 4u + (key >> 2 & 3u)) * 4u + (key & 3u)) * 2u * G;
}
/* The value scale byte of group 0 of a slot; group g: + 4 g. */
template <int G>
DEV uint32_t kv4_vs_at(uint32_t key) { return 33u * 32u * G + (key >> 2) * 4u * G + (key & 3u); }

/* A tile's tokens: the host's tiles are blocks of tokens (a multiple of
 * eight) by head. False if the tile has none. */
DEV bool kv4_tokens(const gpuos_devdesc *d, uint32_t tile, uint32_t &h, uint32_t &n0, uint32_t &n1)
{
    const uint32_t N = d->dims[0], H = d->dims[1], blocks = d->ntiles / H;
    const uint32_t per = (uint32_t)(((uint64_t)N + blocks - 1) / blocks + 7u) & ~7u;
    const uint32_t blk = tile / H;
    h = tile - blk * H;
    if ((uint64_t)blk * per >= N) return false;
    n0 = blk * per;
    n1 = N - n0 < per ? N : n0 + per;
    return true;
}
/* C neighbouring values of a row (4 or 8), as they lie in memory. */
template <int C, bool F32>
struct Kv4Raw {
    static constexpr int N = F32 ? C : C / 2;
    uint32_t w[N];
    DEV void load(const void *base, uint64_t e)
    {
        const unsigned char *p = reinterpret_cast<const unsigned char *>(base) + e * (F32 ? 4u : 2u);
        if (N == 2) {
            const uint2 v = __ldcg(reinterpret_cast<const uint2 *>(p));
            w[0] = v.x; w[1] = v.y;
        } else {
#pragma unroll
            for (int c = 0; c < N; c += 4) {
                const uint4 v = __ldcg(reinterpret_cast<const uint4 *>(p) + c / 4);
                w[c] = v.x; w[c + 1] = v.y; w[(c + 2) % N] = v.z; w[(c + 3) % N] = v.w;
            }
        }
    }
    DEV float value(int c) const
    {
        if (F32) return __uint_as_float(w[c % N]);
        return c & 1 ? bf_hi(w[c / 2]) : bf_lo(w[c / 2]);
    }
    /* The largest magnitude, as the bits of an fp32 number: those of positive
     * numbers are in order, infinity and NaN on top. */
    DEV uint32_t top() const
    {
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < N; c++) m = F32 ? max(m, w[c] & 0x7FFFFFFFu) : __vmaxu2(m, w[c] & 0x7FFF7FFFu);
        return F32 ? m : max(m << 16, m & 0xFFFF0000u);
    }
};
template <int C, bool F32>
DEV void kv4_store_row(void *base, uint64_t e, const float (&x)[C])
{
    if (F32) {
        float4 *p = reinterpret_cast<float4 *>(reinterpret_cast<float *>(base) + e);
#pragma unroll
        for (int c = 0; c < C / 4; c++) p[c] = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
    } else if (C == 8) {
        *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(base) + e) =
            make_uint4(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]), pack_bf2(x[C - 4], x[C - 3]), pack_bf2(x[C - 2], x[C - 1]));
    } else {
        *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(base) + e) =
            make_uint2(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]));
    }
}
/* The scales of a row's G groups, C values of each in every one of LANES
 * neighbouring lanes: byte is that of the lane's group (lane % LANES) * G /
 * LANES, down[g] what values of group g are multiplied by (0: a group with a
 * NaN or infinity). The maxima are split among the lanes as they are reduced,
 * so that a lane works out one scale, not G. */
template <int C, int LANES, int G, bool F32>
DEV void kv4_scales(const Kv4Raw<C, F32> (&v)[G], uint32_t &byte, float (&down)[G])
{
    const uint32_t lane = lane_id();
    uint32_t t[G];
#pragma unroll
    for (int g = 0; g < G; g++) t[g] = v[g].top();
    int o = LANES;
#pragma unroll
    for (int n = G; n > 1; n >>= 1) { /* the upper half of the groups goes to the lanes with bit o */
        o >>= 1;
        const bool up = lane & (uint32_t)o;
#pragma unroll
        for (int g = 0; g < n / 2; g++) {
            const uint32_t keep = up ? t[g + n / 2] : t[g], give = up ? t[g] : t[g + n / 2];
            t[g] = max(keep, __shfl_xor_sync(0xFFFFFFFFu, give, o));
        }
    }
#pragma unroll
    for (o >>= 1; o > 0; o >>= 1) t[0] = max(t[0], __shfl_xor_sync(0xFFFFFFFFu, t[0], o));
    /* e = floor(log2 top) - 2, and one more above 1.5 * 2^floor(log2 top) */
    const uint32_t x = (t[0] + 0x3FFFFFu) >> 23;
    const bool none = t[0] >= 0x7F800000u;
    byte = none ? 255u : min(max(x, 2u) - 2u, 252u);
    const float mine = none ? 0.0f : __uint_as_float((254u - byte) << 23); /* 2^-e */
#pragma unroll
    for (int g = 0; g < G; g++) down[g] = __shfl_sync(0xFFFFFFFFu, mine, (lane & ~(LANES - 1u)) + (uint32_t)g * (LANES / G));
}
/* Values of C codes (from the lowest nibble of w on) under a scale byte. */
template <int C>
DEV void kv4_dequantise(uint32_t w, uint32_t byte, float (&x)[C])
{
    uint32_t h[4];
    kv4_decode4(w, h);
    float s = __uint_as_float(byte ? byte << 23 : 0x00400000u); /* 2^-127 is a subnormal number */
    if (byte == 255u) s = NAN;
#pragma unroll
    for (int c = 0; c < C / 2; c++) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[c]));
        x[2 * c] = f.x * s;
        x[2 * c + 1] = f.y * s;
    }
}
/* G words (G == 4: 16 bytes; G == 2: 8) */
template <int G>
DEV void kv4_ld_words(const unsigned char *p, uint32_t (&w)[G])
{
    if (G == 4) {
        const uint4 x = __ldcg(reinterpret_cast<const uint4 *>(p));
        w[0] = x.x; w[1] = x.y; w[G - 2] = x.z; w[G - 1] = x.w;
    } else {
        const uint2 x = __ldcg(reinterpret_cast<const uint2 *>(p));
        w[0] = x.x; w[1] = x.y;
    }
}
template <int G, bool F32>
DEV int kv4_write_tile(const gpuos_devdesc *d, uint32_t tile)
{
    constexpr uint32_t D = 32u * G;
    const uint32_t H = d->dims[1], lane = lane_id(), j = lane & 3u, i = lane & 7u;
    const int32_t *slots = reinterpret_cast<const int32_t *>(d->aux0);
    const uint32_t nslots = d->dims[3] * GPUOS_KV4_PAGE;
    const void *const ksrc = reinterpret_cast<const void *>(d->a), *const vsrc = reinterpret_cast<const void *>(d->b);
    unsigned char *const pool = reinterpret_cast<unsigned char *>(d->out);
    uint32_t h, n0, n1;
    if (!kv4_tokens(d, tile, h, n0, n1)) return GPUOS_ST_OK;
    bool bad = false;
#pragma unroll 1
    for (uint32_t n = n0; n < n1; n += 8) {
        const uint32_t left = n1 - n;
        const int32_t mine = (lane & 7u) < left ? __ldcg(slots + n + (lane & 7u)) : -1; /* token lane % 8 */
        bad |= mine >= 0 && (uint32_t)mine >= nslots;
        Kv4Raw<8, F32> xk[G];
        Kv4Raw<4, F32> xv[2][G];
#pragma unroll
        for (int g = 0; g < G; g++) { /* rows behind the last: the last again */
            xk[g].load(ksrc, ((uint64_t)(n + min(lane >> 2, left - 1u)) * H + h) * D + 32u * g + 8u * j);
#pragma unroll
            for (int t = 0; t < 2; t++)
                xv[t][g].load(vsrc, ((uint64_t)(n + min(4u * t + (lane >> 3), left - 1u)) * H + h) * D + 32u * g + 4u * i);
        }
        {
            const int32_t slot = __shfl_sync(0xFFFFFFFFu, mine, lane >> 2);
            uint32_t w[G], byte;
            float down[G];
            kv4_scales<8, 4, G, F32>(xk, byte, down);
#pragma unroll
            for (int g = 0; g < G; g++) {
                float x[8];
#pragma unroll
                for (int c = 0; c < 8; c++) x[c] = xk[g].value(c) * down[g];
                w[g] = down[g] != 0.0f ? kv4_encode8(x) : 0u;
            }
            if ((uint32_t)slot < nslots) {
                unsigned char *pg = pool + ((uint64_t)((uint32_t)slot / GPUOS_KV4_PAGE) * H + h) * kv4_page_bytes(D);
                const uint32_t key = (uint32_t)slot % GPUOS_KV4_PAGE;
                if (G == 4) *reinterpret_cast<uint4 *>(pg + kv4_k_at<G>(key, j)) = make_uint4(w[0], w[1], w[G - 2], w[G - 1]);
                else *reinterpret_cast<uint2 *>(pg + kv4_k_at<G>(key, j)) = make_uint2(w[0], w[1]);
                if (j % (4u / G) == 0) pg[32u * D + key * G + j / (4u / G)] = (unsigned char)byte;
            }
        }
#pragma unroll
        for (int t = 0; t < 2; t++) {
            const int32_t slot = __shfl_sync(0xFFFFFFFFu, mine, 4u * t + (lane >> 3));
            uint32_t w[G / 2], byte;
            float down[G];
            kv4_scales<4, 8, G, F32>(xv[t], byte, down);
#pragma unroll
            for (int g = 0; g < G; g += 2) {
                float x[8];
#pragma unroll
                for (int c = 0; c < 8; c++) x[c] = xv[t][g + c / 4].value(c % 4) * down[g + c / 4];
                const uint32_t c2 = kv4_encode8(x);
                w[g / 2] = (down[g] != 0.0f ? c2 & 0xFFFFu : 0u) | (down[g + 1] != 0.0f ? c2 & 0xFFFF0000u : 0u);
            }
            if ((uint32_t)slot < nslots) {
                unsigned char *pg = pool + ((uint64_t)((uint32_t)slot / GPUOS_KV4_PAGE) * H + h) * kv4_page_bytes(D);
                const uint32_t key = (uint32_t)slot % GPUOS_KV4_PAGE;
                if (G == 4) *reinterpret_cast<uint2 *>(pg + kv4_v_at<G>(key, i)) = make_uint2(w[0], w[G / 2 - 1]);
                else *reinterpret_cast<uint32_t *>(pg + kv4_v_at<G>(key, i)) = w[0];
                if (i % (8u / G) == 0) pg[kv4_vs_at<G>(key) + 4u * (i / (8u / G))] = (unsigned char)byte;
            }
        }
    }
    return __any_sync(0xFFFFFFFFu, bad) ? GPUOS_ST_BAD_ARGS : GPUOS_ST_OK;
}
template <int G, bool F32>
DEV int kv4_read_tile(const gpuos_devdesc *d, uint32_t tile)
{
    constexpr uint32_t D = 32u * G;
    const uint32_t H = d->dims[1], lane = lane_id(), j = lane & 3u, i = lane & 7u;
    const int32_t *slots = reinterpret_cast<const int32_t *>(d->aux0);
    const uint32_t nslots = d->dims[3] * GPUOS_KV4_PAGE;
    const unsigned char *const pool = reinterpret_cast<const unsigned char *>(d->a);
    void *const kdst = reinterpret_cast<void *>(d->out), *const vdst = reinterpret_cast<void *>(d->aux1);
    uint32_t h, n0, n1;
    if (!kv4_tokens(d, tile, h, n0, n1)) return GPUOS_ST_OK;
    bool bad = false;
    int32_t mine = n0 + (lane & 7u) < n1 ? __ldcg(slots + n0 + (lane & 7u)) : -1; /* token lane % 8 */
#pragma unroll 1
    for (uint32_t n = n0; n < n1; n += 8) {
        bad |= mine >= 0 && (uint32_t)mine >= nslots;
        /* every load of the eight tokens is out before the first is used */
        const int32_t ks = __shfl_sync(0xFFFFFFFFu, mine, lane >> 2);
        const bool kin = (uint32_t)ks < nslots;
        uint32_t kw[G], ksc = 0, vw[2][G / 2], vsc[2][G];
        {
            const uint32_t slot = kin ? (uint32_t)ks : 0u, key = slot % GPUOS_KV4_PAGE;
            const unsigned char *pg = pool + ((uint64_t)(slot / GPUOS_KV4_PAGE) * H + h) * kv4_page_bytes(D);
            kv4_ld_words<G>(pg + kv4_k_at<G>(key, j), kw);
            ksc = G == 4 ? __ldcg(reinterpret_cast<const uint32_t *>(pg + 32u * D + key * G))
                         : (uint32_t)__ldcg(reinterpret_cast<const uint16_t *>(pg + 32u * D + key * G));
        }
        bool vin[2];
        uint32_t vkey[2];
#pragma unroll
        for (int t = 0; t < 2; t++) {
            const int32_t vs = __shfl_sync(0xFFFFFFFFu, mine, 4u * t + (lane >> 3));
            vin[t] = (uint32_t)vs < nslots;
            const uint32_t slot = vin[t] ? (uint32_t)vs : 0u;
            vkey[t] = slot % GPUOS_KV4_PAGE;
            const unsigned char *pg = pool + ((uint64_t)(slot / GPUOS_KV4_PAGE) * H + h) * kv4_page_bytes(D);
            if (G == 4) {
                const uint2 x = __ldcg(reinterpret_cast<const uint2 *>(pg + kv4_v_at<G>(vkey[t], i)));
                vw[t][0] = x.x;
                vw[t][G / 2 - 1] = x.y;
            } else {
                vw[t][0] = __ldcg(reinterpret_cast<const uint32_t *>(pg + kv4_v_at<G>(vkey[t], i)));
            }
            kv4_ld_words<G>(pg + kv4_vs_at<G>(vkey[t] & ~3u), vsc[t]); /* four keys' bytes of each group */
        }
        mine = n + 8u + (lane & 7u) < n1 ? __ldcg(slots + n + 8u + (lane & 7u)) : -1;
        const uint32_t left = n1 - n;
        if (lane >> 2 < left) {
#pragma unroll
            for (int g = 0; g < G; g++) {
                float x[8];
                kv4_dequantise<8>(kin ? kw[g] : 0u, kin ? ksc >> (8 * g) & 255u : 127u, x);
                kv4_store_row<8, F32>(kdst, ((uint64_t)(n + (lane >> 2)) * H + h) * D + 32u * g + 8u * j, x);
            }
        }
#pragma unroll
        for (int t = 0; t < 2; t++) {
            if (4u * t + (lane >> 3) >= left) continue;
#pragma unroll
            for (int g = 0; g < G; g++) {
                float x[4];
                const uint32_t w = vw[t][g / 2] >> (16 * (g & 1));
                kv4_dequantise<4>(vin[t] ? w : 0u, vin[t] ? vsc[t][g] >> (8u * (vkey[t] & 3u)) & 255u : 127u, x);
                kv4_store_row<4, F32>(vdst, ((uint64_t)(n + 4u * t + (lane >> 3)) * H + h) * D + 32u * g + 4u * i, x);
            }
        }
    }
    return __any_sync(0xFFFFFFFFu, bad) ? GPUOS_ST_BAD_ARGS : GPUOS_ST_OK;
}
DEV bool kv4_rows_ok(const gpuos_devdesc *d, uint64_t second)
{
    return kv4_aligned(d->a, 16) && kv4_aligned(second, 16) && kv4_aligned(d->out, 16) && kv4_aligned(d->aux0, 4) &&
           d->dims[0] <= GPUOS_KV4_MAX_ROWS && d->dims[1] != 0 && d->dims[1] <= 0xFFFFu &&
           (d->dims[2] == 64 || d->dims[2] == 128) && d->dims[3] != 0 && d->dims[3] <= GPUOS_KV4_MAX_PAGES &&
           d->dtype <= GPUOS_BF16 && d->ntiles >= d->dims[1];
}
DEV int kv4_write_op(const gpuos_devdesc *d, uint32_t tile)
{
    if (d->dims[0] == 0) return GPUOS_ST_OK;
    if (!kv4_rows_ok(d, d->b)) return GPUOS_ST_BAD_ARGS;
    const bool f32 = d->dtype == GPUOS_F32;
    if (d->dims[2] == 128) return f32 ? kv4_write_tile<4, true>(d, tile) : kv4_write_tile<4, false>(d, tile);
    return f32 ? kv4_write_tile<2, true>(d, tile) : kv4_write_tile<2, false>(d, tile);
}
DEV int kv4_read_op(const gpuos_devdesc *d, uint32_t tile)
{
    if (d->dims[0] == 0) return GPUOS_ST_OK;
    if (!kv4_rows_ok(d, d->aux1)) return GPUOS_ST_BAD_ARGS;
    const bool f32 = d->dtype == GPUOS_F32;
    if (d->dims[2] == 128) return f32 ? kv4_read_tile<4, true>(d, tile) : kv4_read_tile<4, false>(d, tile);
    return f32 ? kv4_read_tile<2, true>(d, tile) : kv4_read_tile<2, false>(d, tile);
}

/* ---------------------------------------------------------------------------
 * Page copy: pool[layer][dst] = pool[layer][src] for every (src, dst) pair and
 * layer, GPUOS_PAGE_CHUNK bytes a tile, eight 16-byte loads in flight a lane.
 * Bound by memory: 611 pages of 128 KB in 4 layers 87.5 us, 6.6 TB/s; 15 of
 * 34 KB in 32 layers 5.7 us, a launch and its ramp.
 * ------------------------------------------------------------------------- */
DEV int page_copy_op(const gpuos_devdesc *d, uint32_t tile)
{
    const uint32_t n = d->dims[0], p16 = d->dims[1], npages = d->dims[2], layers = d->dims[3];
    if (n == 0) return GPUOS_ST_OK;
    if (p16 == 0 || layers == 0 || !kv4_aligned(d->a, 16) || !kv4_aligned(d->aux0, 8)) return GPUOS_ST_BAD_ARGS;
    constexpr uint32_t C = GPUOS_PAGE_CHUNK / 16u;
    const uint32_t nc = p16 / C + (p16 % C != 0);
    const uint32_t pair = tile / nc, c0 = (tile - pair * nc) * C;
    const uint32_t layer = pair / n, k = pair - layer * n;
    if (layer >= layers) return GPUOS_ST_OK;
    const int2 sd = __ldcg(reinterpret_cast<const int2 *>(d->aux0) + k);
    if (sd.x < 0 || sd.y < 0) return GPUOS_ST_OK;
    if ((uint32_t)sd.x >= npages || (uint32_t)sd.y >= npages) return GPUOS_ST_BAD_ARGS;
    if (sd.x == sd.y) return GPUOS_ST_OK;
    uint4 *pool = reinterpret_cast<uint4 *>(d->a) + (uint64_t)layer * npages * p16 + c0;
    const uint4 *src = pool + (uint64_t)sd.x * p16;
    uint4 *dst = pool + (uint64_t)sd.y * p16;
    const uint32_t m = p16 - c0 < C ? p16 - c0 : C;
    constexpr int U = 8;
#pragma unroll 1
    for (uint32_t i0 = lane_id(); i0 < m; i0 += 32u * U) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; u++)
            if (i0 + 32u * u < m) v[u] = __ldcg(src + i0 + 32u * u);
#pragma unroll
        for (int u = 0; u < U; u++)
            if (i0 + 32u * u < m) __stcg(dst + i0 + 32u * u, v[u]);
    }
    return GPUOS_ST_OK;
}

#ifndef GPUOS_EXECUTOR_ONLY /* the relocatable build holds the executor and its ops alone */
/* ---------------------------------------------------------------------------
 * Attention as a launch of its own (gpuos_eager_run). The runs are those of
 * the executor's tiles, one for each warp, but a block has an SM to itself:
 * NS pages in flight a warp, and the partial states of an item that warps of
 * one block share meet in shared memory. An item that spans blocks leaves one
 * partial state for each of them in the workspace; the last block to arrive
 * merges them in the order of the keys.
 *
 * Bound by memory while pages stream: 64 requests of 2,000 to 16,383 tokens
 * (32 heads over 8, D = 128) 81 us, 5.4 TB/s over the launch and 6.7 in its
 * middle (a page's 517 instructions take 150 of the 187 cycles that its bytes
 * take an SM); one of 131,071 (64 heads over 8) 34.8 us; one of 1,000 8.4 us,
 * which is a chain of loads (lengths, page ids, page) and merges. Twelve warps
 * of 168 registers: sixteen of 128 were 2 to 10 % slower, eight 16 % on the
 * long case; they only win where latency is all (1,000 tokens: 8.0 us).
 * ------------------------------------------------------------------------- */
/* These kernels are launched with programmatic stream serialisation: their
 * blocks may start as soon as those of the stream's previous kernel have
 * ended, and wait here, before anything else, until its writes are visible.
 * That takes 2 us off a launch that follows another in a stream. Every
 * thread of every block waits, whether it has work or not: a kernel that ended
 * without would let the next one pass the one before it. */
DEV void kv4_after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
static int kv4_launch(void (*kernel)(const gpuos_devdesc), uint32_t blocks, uint32_t threads, uint32_t smem, void *stream,
                      const gpuos_devdesc &d)
{
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(blocks);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = (cudaStream_t)stream;
    c.attrs = &at;
    c.numAttrs = 1;
    if (cudaLaunchKernelEx(&c, kernel, d) == cudaSuccess) return 0;
    (void)cudaGetLastError(); /* reported here */
    return -1;
}

template <int G, int NT>
struct Kv4Block {
    static constexpr uint32_t WARPS = NT == 1 ? 12 : 8; /* 168 and 255 registers a thread */
    static constexpr uint32_t NS = 2; /* (three: 0.5 to 2 % slower; a page is 4,352 bytes, 104 KB in flight an SM) */
    static constexpr uint32_t PB = 34u * 32u * G;
    static constexpr uint32_t FRAG = Kv4Part<G, NT>::floats * 4u;
    static constexpr uint32_t WARP_BYTES = NS * PB + GPUOS_KV4_SCRATCH;
    static constexpr uint32_t SMEM = WARPS * (WARP_BYTES + FRAG);
    static_assert(FRAG <= NS * PB, "a warp's last partial state takes the place of its pages");
    static_assert(WARP_BYTES % 16 == 0 && FRAG % 16 == 0, "alignment");
};
/* What a warp leaves: the state of the item it began in the middle of, and of
 * the item that it does not finish (none: ~0). */
struct Kv4Left {
    uint32_t head, tail; /* the units of the items' first pages */
    Kv4Item hitem, titem;
};

template <int G, int NT>
__global__ void __launch_bounds__(Kv4Block<G, NT>::WARPS * 32, 1) gpuos_kv4_attend_kernel(const __grid_constant__ gpuos_devdesc d)
{
    using C = Kv4Block<G, NT>;
    constexpr uint32_t PB = C::PB, NS = C::NS;
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ __align__(8) unsigned long long bars[C::WARPS][C::NS];
    __shared__ Kv4Left left[C::WARPS];
    __shared__ float weight[2][C::WARPS][8 * NT]; /* of the warps' heads and tails in their items */
    __shared__ float2 total[2][C::WARPS][8 * NT]; /* those items' (m, l) */
    __shared__ struct {
        uint32_t first;
        Kv4Item it;
        uint32_t blk0, last; /* the item's first block; its blocks, if all are here */
    } shared[2];
    const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
    unsigned char *mine = sm + warp * C::WARP_BYTES;
    kv4_after_previous();
    if (lane == 0) {
        for (uint32_t k = 0; k < NS; k++)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(&bars[warp][k])) : "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        left[warp].head = left[warp].tail = ~0u;
    }
    __syncwarp();
    Kv4Args a;
    kv4_args(&d, 8u * NT, a);
    int32_t len0;
    const uint32_t W = kv4_units(a, len0);
    /* Little work: no more warps than units, and as many blocks for each
     * item, so that with equal lengths none spans more. Few items: the last
     * block of one merges the states of all, so no more of them than the
     * square root of its units (0.1 us each, against 0.1 us for each page of
     * the twelve warps; a single head over 131,072 tokens: 152 blocks 29.6
     * us, 70 blocks 23.5). */
    const uint32_t items = a.B * a.Hkv * a.RT; /* < W */
    uint32_t nblk = min(gridDim.x, items * ((uint32_t)sqrtf((float)(W / items)) + 1u));
    if (W < C::WARPS * nblk) {
        nblk = (W + C::WARPS - 1) / C::WARPS;
        if (nblk > items) nblk = min((nblk + items - 1) / items * items, gridDim.x);
    }
    if (blockIdx.x >= nblk) return;
    const Kv4Runs runs(W, nblk); /* the blocks' runs, then the warps' */
    const uint32_t b0 = runs.start(blockIdx.x), b1 = runs.start(blockIdx.x + 1u);
    const Kv4Runs mine_of(b1 - b0, C::WARPS);
    uint32_t u = b0 + mine_of.start(warp);
    const uint32_t u1 = b0 + mine_of.start(warp + 1u);
    Kv4Pos p;
    uint32_t slot = 0, parity = 0; /* the ring's position */
    bool lost = false; /* a page did not arrive: what this warp has yet to do is NaN */
    if (u < u1) kv4_seek(a, u, len0, p);
#pragma unroll 1
    while (u < u1) {
        uint32_t begin, end;
        u += kv4_take(p, u1 - u, begin, end);
        bool bad;
        (void)kv4_pages(a, p.len, bad);
        if (!bad && begin < end) { /* (bad: the request's rows are left as they were) */
            Kv4State<G, NT> s;
            const uint32_t n = p.len && !lost ? end - begin : 0u;
            const int32_t *row = a.table + (uint64_t)p.b * a.P + begin;
            const uint64_t stride = (uint64_t)a.Hkv * PB;
            const unsigned char *pool = a.pool + (uint64_t)p.h * PB;
            /* page ids, 32 at a time in the lanes; one that is not in the
             * pool stands for no keys (page 0 is read and masked) */
            int32_t ids = lane < n ? __ldcg(row + lane) : 0, ids_next = 0;
            Kv4Query<G, NT> qx;
            kv4_load_q(a, p, qx); /* used after the first pages are on their way */
            auto issue = [&](uint32_t at, int32_t id) {
                if (lane == 0) {
                    mbar_expect(&bars[warp][at], PB);
                    bulk_g2s(mine + at * PB, pool + ((uint32_t)id < a.npages ? (uint32_t)id : 0u) * stride, PB, &bars[warp][at]);
                }
            };
            /* every lane is done with the last item's pages, whose slots these
             * copies take (ordinary reads, then asynchronous writes) */
            __syncwarp();
            if (lane == 0) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
#pragma unroll
            for (uint32_t k = 0; k < NS; k++) {
                const int32_t id = __shfl_sync(0xFFFFFFFFu, ids, k);
                if (k < n) issue(slot + k < NS ? slot + k : slot + k - NS, id);
            }
            kv4_begin(a, p, qx, s);
            uint32_t k = 0;
            /* the page's slot takes the next page but one */
            auto follow = [&]() {
                if (k + NS < n) {
                    const uint32_t kn = k + NS;
                    const int32_t nx = __shfl_sync(0xFFFFFFFFu, kn >> 5 != k >> 5 ? ids_next : ids, kn & 31u);
                    __syncwarp(); /* every lane is done with this slot */
                    if (lane == 0) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    issue(slot, nx);
                }
                if (++slot == NS) {
                    slot = 0;
                    parity ^= 1u;
                }
                k++;
            };
#pragma unroll 1
            while (k < n) { /* (the slow way's call stands outside the loop over pages: 2 % of the batch case) */
                uint32_t base, valid;
                bool done = true;
#pragma unroll 1
                do {
                    if ((k & 31u) == 0) {
                        if (k) ids = ids_next;
                        ids_next = k + 32u + lane < n ? __ldcg(row + k + 32u + lane) : 0;
                    }
                    const int32_t id = __shfl_sync(0xFFFFFFFFu, ids, k & 31u);
                    base = (begin + k) * GPUOS_KV4_PAGE;
                    valid = (uint32_t)id < a.npages ? (uint32_t)p.len : 0u;
                    /* bounded, like every wait; lanes poll for themselves, and the limit may part them */
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bars[warp][slot], parity))) {
                        lost = true;
                        break;
                    }
                    done = kv4_page<G, NT, false>(mine + slot * PB, mine + NS * PB, base, valid, true, s);
                    if (done) follow();
                } while (done && k < n);
                if (lost) {
                    /* no copy is left in flight: each is waited for once
                     * more, and none is issued again */
                    for (uint32_t c = 0; c < NS && k + c < n; c++) {
                        (void)mbar_wait(&bars[warp][slot], parity);
                        if (++slot == NS) {
                            slot = 0;
                            parity ^= 1u;
                        }
                    }
                    break;
                }
                if (!done) {
                    kv4_page_rare(a, p, mine + slot * PB, base, kv4_existing(base, valid), s);
                    follow();
                }
            }
            if (lost) {
#pragma unroll
                for (int nt = 0; nt < NT; nt++) s.l[nt][0] = s.l[nt][1] = NAN;
            }
            kv4_finish(s);
            if (begin == 0 && end == p.np) {
                kv4_store(a, p, s);
            } else {
                /* the item goes on in the next warp: its state ends this
                 * warp's run, and takes the place of the pages */
                const bool tail = begin == 0;
                __syncwarp();
                kv4_part_store<false>(tail ? mine : sm + C::WARPS * C::WARP_BYTES + warp * C::FRAG, s);
                if (lane == 0) {
                    (tail ? left[warp].tail : left[warp].head) = p.first;
                    (tail ? left[warp].titem : left[warp].hitem) = Kv4Item{p.b, p.h, p.r0, p.np};
                }
            }
        }
        kv4_next(a, p);
    }
    __syncthreads();
    /* The items that warps of this block share, in order: the state that
     * begins one (a warp's tail; or the block's first head, of an item that
     * an earlier block began) and the heads that follow it. Lane w looks at
     * warp w's. First each warp finds the weights of its own two states, row
     * by row, against the others of their items; then a thread for each four
     * channels adds the states' means. */
    constexpr uint32_t NE = NT * G * 64u; /* float4s of a state's accumulators */
    const uint32_t head = lane < C::WARPS ? left[lane].head : ~0u, tail = lane < C::WARPS ? left[lane].tail : ~0u;
#pragma unroll 1
    for (uint32_t k = 0; k < 2; k++) {
        const uint32_t first = __shfl_sync(0xFFFFFFFFu, k ? tail : head, warp);
        if (first == ~0u) continue;
        const uint32_t heads = __ballot_sync(0xFFFFFFFFu, head == first), own = __ballot_sync(0xFFFFFFFFu, tail == first);
        /* lane (q, r): row r of the states of warps q, q + Q, ... */
        constexpr uint32_t Q = 32u / (8u * NT);
        static_assert(C::WARPS % Q == 0, "warps in the lanes' turns");
        const uint32_t r = lane % (8u * NT), q = lane / (8u * NT);
        auto ml_of = [&](uint32_t w, bool t) {
            return reinterpret_cast<const float2 *>(t ? sm + w * C::WARP_BYTES : sm + C::WARPS * C::WARP_BYTES + w * C::FRAG)[r];
        };
        float2 x[C::WARPS / Q + 1];
#pragma unroll
        for (uint32_t w = 0; w < C::WARPS / Q; w++)
            x[w] = heads >> (w * Q + q) & 1u ? ml_of(w * Q + q, false) : make_float2(-FLT_MAX, 0.0f);
        x[C::WARPS / Q] = own && q == 0 ? ml_of((uint32_t)__ffs((int)own) - 1u, true) : make_float2(-FLT_MAX, 0.0f);
        const float2 me = ml_of(warp, k);
        float M = -FLT_MAX, l = 0.0f;
#pragma unroll
        for (uint32_t w = 0; w <= C::WARPS / Q; w++) M = fmaxf(M, x[w].x);
#pragma unroll
        for (uint32_t o = 8u * NT; o < 32u; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
#pragma unroll
        for (uint32_t w = 0; w <= C::WARPS / Q; w++) l = fmaf(x[w].y, kv4_ex2(x[w].x - M), l);
#pragma unroll
        for (uint32_t o = 8u * NT; o < 32u; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        if (q == 0) {
            weight[k][warp][r] = l != 0.0f ? me.y * kv4_ex2(me.x - M) / l : 0.0f;
            /* 2^-46: a weight is 2^15 at most and the keys are 2^31, so that
             * the blocks' sum of values under such weights stays in fp32
             * where the values do (scaled here, not there: that code runs
             * cold, and one more instruction in its loop cost 0.3 to 1 us) */
            total[k][warp][r] = make_float2(M, l * 0x1p-46f);
        }
    }
    __syncthreads();
    const uint32_t orphan = __ballot_sync(0xFFFFFFFFu, head < b0), tails = __ballot_sync(0xFFFFFFFFu, tail != ~0u);
    float4 *const ws = reinterpret_cast<float4 *>(reinterpret_cast<float *>(d.aux2) + GPUOS_KV4_MAX_TILES);
    uint32_t out = 0; /* bit 0: a state of an item that began earlier is in the workspace; bit 1: of one that goes on */
    uint32_t todo = tails << 1 | (orphan ? 1u : 0u); /* bit 0: the orphan; bit 1 + w: warp w's tail */
#pragma unroll 1
    while (todo) {
        const uint32_t c = (uint32_t)__ffs((int)todo) - 1u;
        todo &= todo - 1u;
        const bool begins = c != 0;
        const uint32_t w0 = begins ? c - 1u : (uint32_t)__ffs((int)orphan) - 1u;
        const uint32_t first = __shfl_sync(0xFFFFFFFFu, begins ? tail : head, w0);
        const uint32_t heads = __ballot_sync(0xFFFFFFFFu, head == first);
        const Kv4Item it = begins ? left[w0].titem : left[w0].hitem;
        const bool whole = begins && first + it.np <= b1;
        for (uint32_t idx = threadIdx.x; idx < NE; idx += C::WARPS * 32u) {
            const uint32_t r = idx / (64u * G) * 8u + 2u * (idx & 3u) + (idx >> 5 & 1u); /* the element's row */
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (begins) {
                const float wt = weight[1][w0][r];
                const float4 x = reinterpret_cast<const float4 *>(sm + w0 * C::WARP_BYTES)[NT * 4 + idx];
                v = make_float4(x.x * wt, x.y * wt, x.z * wt, x.w * wt);
            }
#pragma unroll 4
            for (uint32_t w = 0; w < C::WARPS; w++) {
                if (!(heads >> w & 1u)) continue;
                const float wt = weight[0][w][r];
                const float4 x = reinterpret_cast<const float4 *>(sm + C::WARPS * C::WARP_BYTES + w * C::FRAG)[NT * 4 + idx];
                v.x = fmaf(x.x, wt, v.x);
                v.y = fmaf(x.y, wt, v.y);
                v.z = fmaf(x.z, wt, v.z);
                v.w = fmaf(x.w, wt, v.w);
            }
            const float2 ml = total[begins][w0][r];
            if (whole) {
                kv4_out4<G, NT>(a, it, idx, ml.y, v);
            } else {
                float4 *st = ws + ((uint64_t)blockIdx.x * 2u + (begins ? 1u : 0u)) * (C::FRAG / 16u);
                __stcg(st + NT * 4 + idx, v);
                if ((idx & 31u) < 4u && (idx >> 6 & (G - 1u)) == 0u) /* the row's (m, l), once */
                    __stcg(reinterpret_cast<float2 *>(st) + r, ml);
            }
        }
        if (!whole) {
            out |= begins ? 2u : 1u;
            if (threadIdx.x == 0) {
                shared[begins].first = first;
                shared[begins].it = it;
            }
        }
    }
    if (out == 0) return;
    __syncthreads();
    if (lane == 0 && warp < 2u) {
        /* the blocks of an item count at the counter of its first block */
        uint32_t last = 0;
        if (out >> warp & 1u) {
            const uint32_t first = shared[warp].first;
            const uint32_t blk0 = runs.run_of(first);
            const uint32_t F = runs.run_of(first + shared[warp].it.np - 1) - blk0 + 1;
            uint32_t *cnt = kv4_counters(&d) + blk0;
            if (atom_add_acq_rel_gpu32(cnt, 1u) == F - 1) {
                *cnt = 0; /* left zero for the next call */
                last = F;
            }
            shared[warp].blk0 = blk0;
        }
        shared[warp].last = last;
    }
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < 2; k++) {
        const uint32_t F = shared[k].last;
        if (F == 0) continue;
        const uint32_t blk0 = shared[k].blk0;
#pragma unroll
        for (uint32_t idx = threadIdx.x; idx < NE; idx += C::WARPS * 32u) {
            const uint32_t r = idx / (64u * G) * 8u + 2u * (idx & 3u) + (idx >> 5 & 1u);
            float M = -FLT_MAX, l = 0.0f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            /* two states at a time: this code runs once, from an instruction
             * cache that does not hold it, and is faster short (unrolled 2,
             * 4, 6, 10, 20 times, 64 long requests: 79.2, 80.1, 79.7, 80.3,
             * 84.4 us) */
            constexpr uint32_t U = 2;
            for (uint32_t f0 = 0; f0 < F; f0 += U) {
                float2 ml[U];
                float4 x[U];
#pragma unroll
                for (uint32_t f = 0; f < U; f++) {
                    const uint32_t ff = min(f0 + f, F - 1);
                    const float4 *st = ws + ((uint64_t)(blk0 + ff) * 2u + (ff == 0 ? 1u : 0u)) * (C::FRAG / 16u);
                    ml[f] = __ldcg(reinterpret_cast<const float2 *>(st) + r);
                    x[f] = __ldcg(st + NT * 4 + idx);
                }
                float mb = M;
#pragma unroll
                for (uint32_t f = 0; f < U; f++) mb = fmaxf(mb, ml[f].x);
                const float sc = kv4_ex2(M - mb);
                l *= sc;
                v = make_float4(v.x * sc, v.y * sc, v.z * sc, v.w * sc);
                M = mb;
#pragma unroll
                for (uint32_t f = 0; f < U; f++) {
                    if (f0 + f >= F) continue; /* duplicates */
                    const float wt = ml[f].y * kv4_ex2(ml[f].x - M);
                    l += wt;
                    v.x = fmaf(x[f].x, wt, v.x);
                    v.y = fmaf(x[f].y, wt, v.y);
                    v.z = fmaf(x[f].z, wt, v.z);
                    v.w = fmaf(x[f].w, wt, v.w);
                }
            }
            const float inv = l != 0.0f ? 1.0f / l : 0.0f;
            kv4_out4<G, NT>(a, shared[k].it, idx, l, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
        }
    }
}

template <int G, int NT>
static int kv4_attend_launch(const gpuos_devdesc &d, void *stream)
{
    using C = Kv4Block<G, NT>;
    /* once per device: its SMs, and the kernel's shared memory there */
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
    int sms = known[dev].load(std::memory_order_relaxed);
    if (sms == 0) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
        if (cudaFuncSetAttribute(gpuos_kv4_attend_kernel<G, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)C::SMEM) != cudaSuccess)
            return -1;
        known[dev].store(sms, std::memory_order_relaxed);
    }
    /* no more blocks than the longest requests can fill */
    const uint64_t g = (d.dims[1] & 0xFFFFu) / (d.dims[1] >> 16), T = d.dims[2] >> 16;
    const uint64_t units =
        (uint64_t)d.dims[0] * (d.dims[3] + GPUOS_KV4_LEAD) * (d.dims[1] >> 16) * ((T * g + 8 * NT - 1) / (8 * NT));
    uint64_t grid = (units + C::WARPS - 1) / C::WARPS;
    if (grid > (uint64_t)sms) grid = (uint64_t)sms;
    if (grid > GPUOS_KV4_MAX_BLOCKS) grid = GPUOS_KV4_MAX_BLOCKS;
    return kv4_launch(gpuos_kv4_attend_kernel<G, NT>, (uint32_t)grid, C::WARPS * 32, C::SMEM, stream, d);
}

/* The other ops: one warp a tile, as in the executor; four warps a block, so
 * that a block's limit of 32 an SM leaves room for 64 warps; a kernel for each
 * type and head dimension, so that each has its own registers. */
#define GPUOS_KV4_EAGER_WARPS 4u
template <int OP, int G, bool F32>
__global__ void __launch_bounds__(GPUOS_KV4_EAGER_WARPS * 32) gpuos_kv4_eager_kernel(const __grid_constant__ gpuos_devdesc d)
{
    const uint32_t tile = blockIdx.x * GPUOS_KV4_EAGER_WARPS + (threadIdx.x >> 5);
    kv4_after_previous();
    if (tile >= d.ntiles) return;
    if (OP == GPUOS_OP_KV4_WRITE) (void)kv4_write_tile<G, F32>(&d, tile);
    if (OP == GPUOS_OP_KV4_READ) (void)kv4_read_tile<G, F32>(&d, tile);
    if (OP == GPUOS_OP_PAGE_COPY) (void)page_copy_op(&d, tile);
}
template <int OP, int G, bool F32>
static int kv4_tiles_launch(const gpuos_devdesc &d, void *stream)
{
    const uint32_t blocks = (d.ntiles + GPUOS_KV4_EAGER_WARPS - 1) / GPUOS_KV4_EAGER_WARPS;
    return kv4_launch(gpuos_kv4_eager_kernel<OP, G, F32>, blocks, GPUOS_KV4_EAGER_WARPS * 32, 0, stream, d);
}
template <int OP>
static int kv4_rows_launch(const gpuos_devdesc &d, void *stream)
{
    if (d.dims[0] == 0) return 0;
    if (d.dims[2] == 128)
        return d.dtype == GPUOS_F32 ? kv4_tiles_launch<OP, 4, true>(d, stream) : kv4_tiles_launch<OP, 4, false>(d, stream);
    return d.dtype == GPUOS_F32 ? kv4_tiles_launch<OP, 2, true>(d, stream) : kv4_tiles_launch<OP, 2, false>(d, stream);
}
static int kv4_eager_launch(const gpuos_devdesc &d, void *stream)
{
    switch (d.op_id) {
    case GPUOS_OP_KV4_WRITE: return kv4_rows_launch<GPUOS_OP_KV4_WRITE>(d, stream);
    case GPUOS_OP_KV4_READ: return kv4_rows_launch<GPUOS_OP_KV4_READ>(d, stream);
    case GPUOS_OP_PAGE_COPY: return kv4_tiles_launch<GPUOS_OP_PAGE_COPY, 4, false>(d, stream);
    default: break;
    }
    if (d.dims[0] == 0) return 0;
    /* Row tiles of eight or of sixteen rows. Sixteen read and convert a page
     * half as often; eight leave room for twelve warps an SM instead of eight
     * (D = 128) and waste less of a last tile. Device us by eights, by
     * sixteens, 4 cache heads:
     *   D    rows  4 x 1,000    4 x 3,000    8 x 8,000    8 x 20,000   32 x 8,000
     *   64   16     8.3   8.0    9.8   9.4   15.6  14.8   27.0  23.1   38.1  30.7
     *   64   24     8.5   8.5   10.3  11.0   19.5  19.7   36.2  36.2   53.5  53.0
     *   64   40     9.3   9.5   11.7  11.4   27.1  25.7   54.7  49.3   83.4  74.9
     *   64   128   13.2  11.5   20.1  17.4   68.7  53.1    157   117    247   185
     *   128  16     8.7  10.4   11.3  12.4   20.2  20.9   37.2  34.0   54.4  46.2
     *   128  24     9.1  10.7   12.2  14.9   26.0  28.4   50.8  53.7   77.1  80.4
     *   128  32    10.4  10.7   13.3  15.3   31.4  28.6   64.7  54.2   99.3  80.8
     *   128  56    11.6  12.7   16.7  17.9   48.7  45.2    106  95.8    167   150
     * So three tiles of eight (four halves of two sixteens) are by eights; D =
     * 64 by sixteens; D = 128 by sixteens from about nine pages for each of
     * 1,824 warps on. The lengths are on the device, so the table's width
     * stands for them: requests much shorter than their table allows are taken
     * for long ones (16 of 2 to 4,099 tokens, 32 rows: 17.3 us, 16.2 by eights). */
    const uint32_t rows = (d.dims[2] >> 16) * ((d.dims[1] & 0xFFFFu) / (d.dims[1] >> 16)), tiles = (rows + 7u) / 8u;
    const uint64_t pages = (uint64_t)d.dims[0] * d.dims[3] * (d.dims[1] >> 16) * tiles;
    const bool eights = tiles == 1u || tiles == 3u || ((d.dims[2] & 0xFFFFu) == 128u && pages < 16384u);
    if ((d.dims[2] & 0xFFFFu) == 128) return eights ? kv4_attend_launch<4, 1>(d, stream) : kv4_attend_launch<4, 2>(d, stream);
    return eights ? kv4_attend_launch<2, 1>(d, stream) : kv4_attend_launch<2, 2>(d, stream);
}
/* Load the kernels (see gpuos_dev_preload). */
static int kv4_preload()
{
    const void *const all[] = {
        (const void *)gpuos_kv4_attend_kernel<4, 1>, (const void *)gpuos_kv4_attend_kernel<4, 2>,
        (const void *)gpuos_kv4_attend_kernel<2, 1>, (const void *)gpuos_kv4_attend_kernel<2, 2>,
        (const void *)gpuos_kv4_eager_kernel<GPUOS_OP_KV4_WRITE, 4, false>,
        (const void *)gpuos_kv4_eager_kernel<GPUOS_OP_KV4_WRITE, 4, true>,
        (const void *)gpuos_kv4_eager_kernel<GPUOS_OP_KV4_WRITE, 2, false>,
        (const void *)gpuos_kv4_eager_kernel<GPUOS_OP_KV4_WRITE, 2, true>,
        (const void *)gpuos_kv4_eager_kernel<GPUOS_OP_KV4_READ, 4, false>,
        (const void *)gpuos_kv4_eager_kernel<GPUOS_OP_KV4_READ, 4, true>,
        (const void *)gpuos_kv4_eager_kernel<GPUOS_OP_KV4_READ, 2, false>,
        (const void *)gpuos_kv4_eager_kernel<GPUOS_OP_KV4_READ, 2, true>,
        (const void *)gpuos_kv4_eager_kernel<GPUOS_OP_PAGE_COPY, 4, false>};
    for (const void *f : all) {
        cudaFuncAttributes at;
        if (cudaFuncGetAttributes(&at, f) != cudaSuccess) return -1;
    }
    return 0;
}
#endif /* GPUOS_EXECUTOR_ONLY */
#endif /* GPUOS_KV4_CUH */
