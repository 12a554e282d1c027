// Appending keys and values to a paged cache, with the position rotation applied on the way.
//
// Token i of sequence b stands at position p = cache_len[b] + i, in slot p % page of page
// page_table[b][p / page]; the cache is [n_pages][H][page][D].  The first R dimensions of every query
// and key head are rotated in pairs (x1, x2), j < R / 2, by the angle a = p inv_freq[j]:
//     y1 = x1 cos a - x2 sin a,   y2 = x2 cos a + x1 sin a
// (pairs (j, j + R/2), or neighbours (2j, 2j + 1)).  At positions of a million an fp32 product would
// leave the angle off by up to 0.06: the half turns p inv_freq / pi are formed and reduced to [-1, 1] in fp64;
// sincospif takes their fp32 value, and what that left off is put back to first order.  The rotated value is rounded
// once to the cache's type.
//
// An E4M3 cache holds one scale per page, head and tensor.  The scale is a power of two, so moving the
// page's earlier codes to a larger scale is exact except where they become subnormal; the least one
// with amax <= 448 scale leaves the largest value in the top two binades of E4M3.  A page that already
// holds tokens keeps its scale unless the new ones need a larger one.
//
// The work is one pass over the data and bound by HBM; a unit is 16 elements of a row (both partners of
// eight pairs), so no thread needs another's values.  Rows that are stored as they are read go by token
// (append_rows); an E4M3 page and head is one CTA (its scale needs all its new values, held in
// registers, and nobody else touches the page).  Both kinds of CTA share one launch.  16384 tokens of 64 + 16 heads of
// 128 into a bf16 cache: 140 us, 5.6 TB/s; 8 ragged chunks into an E4M3 cache, 32 query heads: 74 us, 3.5 TB/s (bound by
// instruction issue: the angles of a page's keys are formed for every head).
#pragma once
#include "common.cuh"

namespace lsa {

constexpr unsigned ERRF_PAGE = 32u;  // device error word (common.cuh): a page number outside the cache

struct AppendArgs {
    const void *q, *k, *v;          // [N][heads][D], rows of a token contiguous
    int64_t q_stride, k_stride, v_stride;  // elements from one token to the next
    const int64_t *q_offsets;       // [B + 1]
    const int32_t *cache_len;       // [B]
    const int32_t *page_table;      // [B][max_pages]
    const float *inv_freq;          // [rot / 2]
    void *q_out, *k_cache, *v_cache;
    float *k_scale, *v_scale;       // [n_pages][H], E4M3 only
    int64_t N, n_pages;
    int B, max_pages, Hq, H, D, page, rot, interleaved;
    int tokens;                     // tokens of a CTA's rows
    int row_ctas_per_token;         // CTAs of them
    int64_t row_ctas;               // CTAs [0, row_ctas) go by token, the others by page
};

// Elements of unit u of a row: two runs of 8 starting at a and b.
__device__ __forceinline__ void unit_runs(const AppendArgs &A, int u, int &a, int &b)
{
    if (!A.interleaved && u < A.rot / 16) {
        a = u * 8;
        b = a + A.rot / 2;
    } else {
        a = u * 16;
        b = a + 8;
    }
}

template <int DT>
__device__ __forceinline__ void load_run8(const void *row, int64_t e, float (&x)[8])
{
    if constexpr (DT == DT_F32) {
        const float4 a = __ldg((const float4 *)((const float *)row + e));
        const float4 b = __ldg((const float4 *)((const float *)row + e) + 1);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        const uint4 w = __ldg((const uint4 *)((const __nv_bfloat16 *)row + e));
        const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            x[2 * i] = __uint_as_float(r[i] << 16);
            x[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
        }
    }
}

template <int DT>
__device__ __forceinline__ void store_run8(void *row, int64_t e, const float (&x)[8])
{
    if constexpr (DT == DT_F32) {
        float4 *p = (float4 *)((float *)row + e);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            r[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        *(uint4 *)((__nv_bfloat16 *)row + e) = make_uint4(r[0], r[1], r[2], r[3]);
    }
}

// cos and sin of pos * inv_freq: of the reduced angle's fp32 value, then corrected by what that rounding left off
// (d, to first order: h is within 2^-25 half turns of t, so d is below pi 2^-25 and what is left off, d^2 / 2, below 2^-47).
__device__ __forceinline__ void turn(int64_t pos, float inv_freq, float &c, float &s)
{
    double t = (double)pos * (double)inv_freq * 0.31830988618379067154;  // 1 / pi: half turns
    t -= 2.0 * rint(0.5 * t);
    const float h = (float)t, d = (float)(t - (double)h) * 3.14159265f;
    float s0, c0;
    sincospif(h, &s0, &c0);
    s = fmaf(c0, d, s0);
    c = fmaf(-s0, d, c0);
}

// Rotate the eight pairs of a unit: x runs a and b (halves: a[i] with b[i]; neighbours: within a, within b).
__device__ __forceinline__ void rotate_unit(bool interleaved, const float (&c)[8], const float (&s)[8], float (&a)[8],
                                            float (&b)[8])
{
    if (!interleaved) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float x1 = a[i], x2 = b[i];
            a[i] = x1 * c[i] - x2 * s[i];
            b[i] = x2 * c[i] + x1 * s[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float x1 = a[2 * i], x2 = a[2 * i + 1], z1 = b[2 * i], z2 = b[2 * i + 1];
            a[2 * i] = x1 * c[i] - x2 * s[i];
            a[2 * i + 1] = x2 * c[i] + x1 * s[i];
            b[2 * i] = z1 * c[4 + i] - z2 * s[4 + i];
            b[2 * i + 1] = z2 * c[4 + i] + z1 * s[4 + i];
        }
    }
}

// What a CTA needs to know of a sequence.
struct SeqOf {
    int64_t off, n;  // first token, tokens
    int b, len;      // b = -1: none
};

// The sequences of tokens n .. n + many - 1 (b = -1: none, a row behind the last sequence) into slots.  Every thread
// of the block calls it; one round of loads.  Where offsets decrease (flagged), sequences overlap: a token then is the
// last one's that has it.
__device__ __forceinline__ void block_seqs_of_tokens(const int64_t *q_offsets, const int32_t *cache_len, int B, int64_t N, int64_t n,
                                                     int many, SeqOf *slots)
{
    if ((int)threadIdx.x < many) slots[threadIdx.x].b = -1;
    int overlap = 0;
    __syncthreads();
    for (int b = threadIdx.x; b < B; b += blockDim.x) {
        const int64_t lo = __ldg(q_offsets + b), hi = __ldg(q_offsets + b + 1);
        const int len = __ldg(cache_len + b);
        if (lo < 0 || hi < lo || hi > N) {
            flag(ERRF_OFFSETS);
        } else {
            for (int64_t i = max(lo, n); i < min(hi, n + many); i++) {
                SeqOf &s = slots[i - n];
                overlap |= atomicMax(&s.b, b) >= 0;
                s.off = lo;
                s.n = hi - lo;
                s.len = len;
            }
        }
    }
    if (!__syncthreads_or(overlap)) return;
    for (int b = threadIdx.x; b < B; b += blockDim.x) {  // (several have written a slot: now the one whose it is)
        const int64_t lo = __ldg(q_offsets + b), hi = __ldg(q_offsets + b + 1);
        if (lo < 0 || hi < lo || hi > N) continue;
        for (int64_t i = max(lo, n); i < min(hi, n + many); i++) {
            SeqOf &s = slots[i - n];
            if (s.b != b) continue;
            s.off = lo;
            s.n = hi - lo;
            s.len = __ldg(cache_len + b);
        }
    }
    __syncthreads();
}

// Page of position pos of sequence b, or -1 (flagged) where the table has none.
__device__ __forceinline__ int32_t page_of(const int32_t *page_table, int max_pages, int64_t n_pages, int b, int64_t pi)
{
    if (pi < 0 || pi >= max_pages) {
        flag(ERRF_COUNT);
        return -1;
    }
    const int32_t p = __ldg(page_table + (int64_t)b * max_pages + pi);
    if (p < 0 || p >= n_pages) {
        flag(ERRF_PAGE);
        return -1;
    }
    return p;
}

constexpr int APPEND_TOKENS = 8;  // tokens a CTA takes at most

// Rows that are stored in the type they are read in (queries; keys and values of an fp32 or bf16 cache): a CTA has
// A.tokens tokens, or a part of one token's rows.
template <int DT, bool KV>
__device__ __forceinline__ void append_rows(const AppendArgs &A, float2 *cs, SeqOf *slots, int32_t *pages)
{
    const int64_t n0 = (int64_t)(blockIdx.x / A.row_ctas_per_token) * A.tokens;
    const int part = blockIdx.x % A.row_ctas_per_token;
    const int many = (int)min((int64_t)A.tokens, A.N - n0);
    const int nq = A.q ? A.Hq : 0;
    const int rows = nq + (KV ? 2 * A.H : 0);
    const int upr = A.D / 16, units = rows * upr, half = A.rot / 2;
    block_seqs_of_tokens(A.q_offsets, A.cache_len, A.B, A.N, n0, many, slots);
    for (int i = threadIdx.x; i < many * half; i += blockDim.x) {
        const int t = i / half, j = i % half;
        const SeqOf &s = slots[t];
        float c = 0.f, sn = 0.f;
        if (s.b >= 0 && s.len >= 0) turn(s.len + (n0 + t - s.off), __ldg(A.inv_freq + j), c, sn);
        cs[t * half + (j & 7) * (half >> 3) + (j >> 3)] = make_float2(c, sn);  // (units next to one another: no bank twice)
    }
    if ((int)threadIdx.x < many) {
        const SeqOf s = slots[threadIdx.x];
        int32_t page = -1;
        if (s.b >= 0) {
            if (s.len < 0) {
                flag(ERRF_COUNT);
                slots[threadIdx.x].b = -1;  // (nothing of it is touched)
            } else if (KV) {
                page = page_of(A.page_table, A.max_pages, A.n_pages, s.b, (s.len + (n0 + threadIdx.x - s.off)) / A.page);
            }
        }
        pages[threadIdx.x] = page;
    }
    __syncthreads();
    // (units of the CTA's tokens one after another; no divisions: a thread's next unit is `stride` on, of this token or a
    // later one)
    const int stride = A.row_ctas_per_token * blockDim.x, shift = A.D == 128 ? 3 : (A.D == 64 ? 2 : 1);
    for (int t = 0, i = part * blockDim.x + threadIdx.x;; i += stride) {
        while (i >= units && t < many) {
            i -= units;
            t++;
        }
        if (t >= many) break;
        const SeqOf &s = slots[t];
        if (s.b < 0) continue;  // a row behind the last sequence: left as it is
        const int row = i >> shift, u = i & (upr - 1);
        const int64_t n = n0 + t;
        const void *src;
        void *dst;
        int64_t se, de;
        bool rot = u < A.rot / 16;
        if (row < nq) {
            src = A.q; se = n * A.q_stride + (int64_t)row * A.D;
            dst = A.q_out; de = (n * A.Hq + row) * A.D;
        } else {
            const bool is_v = row >= nq + A.H;
            const int h = row - nq - (is_v ? A.H : 0);
            if (pages[t] < 0) continue;
            src = is_v ? A.v : A.k;
            se = n * (is_v ? A.v_stride : A.k_stride) + (int64_t)h * A.D;
            dst = is_v ? A.v_cache : A.k_cache;
            de = (((int64_t)pages[t] * A.H + h) * A.page + ((s.len + (n - s.off)) & (A.page - 1))) * A.D;
            rot = rot && !is_v;
        }
        int ra, rb;
        if (rot) unit_runs(A, u, ra, rb);
        else { ra = u * 16; rb = ra + 8; }
        float xa[8], xb[8];
        load_run8<DT>(src, se + ra, xa);
        load_run8<DT>(src, se + rb, xb);
        if (rot) {
            const float2 *cu = cs + t * half + u;
            float c[8], sn[8];
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float2 v = cu[e * (half >> 3)];
                c[e] = v.x;
                sn[e] = v.y;
            }
            rotate_unit(A.interleaved, c, sn, xa, xb);
        }
        store_run8<DT>(dst, de + ra, xa);
        store_run8<DT>(dst, de + rb, xb);
    }
}

// Power of two 2^e, least with amax <= 448 * 2^e (448 = 1.75 * 2^8), at least 2^-64; amax finite, >= 0.
__device__ __forceinline__ float e4m3_scale(float amax)
{
    const uint32_t bits = __float_as_uint(amax);
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)((e < -64 ? -64 : e) + 127) << 23);
}

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

constexpr int APPEND_THREADS = 256;

// One page and head of an E4M3 cache, keys or values; U units of 16 elements a thread.
template <int DT, int U>
__device__ __forceinline__ void append_page(const AppendArgs &A, int64_t job, SeqOf *slot, int *last, float *red)
{
    const int tensor = (int)(job % 2);
    const int h = (int)((job / 2) % A.H);
    const int64_t pj = job / 2 / A.H;
    // Page jobs of sequence b are numbered from off_b / page + 2b: a sequence of n tokens touches at
    // most n / page + 2 pages, so the ranges do not meet.  Largest b whose range starts at or before pj.
    if (threadIdx.x == 0) *last = -1;
    __syncthreads();
    SeqOf mine = {};
    mine.b = -1;
    for (int b = threadIdx.x; b < A.B; b += blockDim.x) {
        const int64_t lo = __ldg(A.q_offsets + b), hi = __ldg(A.q_offsets + b + 1);
        const int len = __ldg(A.cache_len + b);
        if (lo < 0 || hi < lo || hi > A.N) {
            flag(ERRF_OFFSETS);
        } else if (lo / A.page + 2 * (int64_t)b <= pj) {
            mine.off = lo;
            mine.n = hi - lo;
            mine.len = len;
            mine.b = b;
        }
    }
    if (mine.b >= 0) atomicMax(last, mine.b);
    __syncthreads();
    if (*last < 0) return;
    if (mine.b == *last) *slot = mine;
    __syncthreads();
    const int b = slot->b;
    const int64_t off = slot->off, n = slot->n, len = slot->len;
    if (n == 0) return;
    if (len < 0) {
        if (threadIdx.x == 0) flag(ERRF_COUNT);
        return;
    }
    const int64_t pi = len / A.page + (pj - (off / A.page + 2 * (int64_t)b));
    const int64_t first = max(len, pi * A.page), end = min(len + n, (pi + 1) * A.page);
    if (first >= end) return;
    const int32_t page = page_of(A.page_table, A.max_pages, A.n_pages, b, pi);
    if (page < 0) return;
    const void *src = tensor ? A.v : A.k;
    const int64_t stride = tensor ? A.v_stride : A.k_stride;
    uint8_t *cache = (uint8_t *)(tensor ? A.v_cache : A.k_cache) + ((int64_t)page * A.H + h) * A.page * A.D;
    float *scale = (tensor ? A.v_scale : A.k_scale) + (int64_t)page * A.H + h;
    const int held = (int)(first - pi * A.page);  // tokens that the page holds already
    const int upr = A.D / 16, units = (int)(end - first) * upr;

    float x[U][16];
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < U; k++) {
        const int i = threadIdx.x + k * APPEND_THREADS;
        if (i < units) {
            const int64_t pos = first + i / upr;
            const int u = i % upr;
            int ra, rb;
            const bool rot = !tensor && u < A.rot / 16;
            if (rot) unit_runs(A, u, ra, rb);
            else { ra = u * 16; rb = ra + 8; }
            const int64_t se = (off + pos - len) * stride + (int64_t)h * A.D;
            float xa[8], xb[8];
            load_run8<DT>(src, se + ra, xa);
            load_run8<DT>(src, se + rb, xb);
            if (rot) {
#pragma unroll
                for (int t = 0; t < 8; t++) {  // (a pair at a time: cos and sin of eight would cost 16 registers)
                    float c, s;
                    turn(pos, __ldg(A.inv_freq + u * 8 + t), c, s);
                    float &x1 = !A.interleaved ? xa[t] : (t < 4 ? xa[2 * t] : xb[2 * (t - 4)]);
                    float &x2 = !A.interleaved ? xb[t] : (t < 4 ? xa[2 * t + 1] : xb[2 * (t - 4) + 1]);
                    const float y1 = x1 * c - x2 * s;
                    x2 = x2 * c + x1 * s;
                    x1 = y1;
                }
            }
#pragma unroll
            for (int t = 0; t < 8; t++) {
                x[k][t] = xa[t];
                x[k][8 + t] = xb[t];
                // (infinities and NaN set no scale: the former saturate, the latter are stored as NaN)
                const float ua = fabsf(xa[t]), ub = fabsf(xb[t]);
                if (ua <= 3.4028235e38f) amax = fmaxf(amax, ua);
                if (ub <= 3.4028235e38f) amax = fmaxf(amax, ub);
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
    const float before = held ? *scale : 0.f;
    __syncthreads();  // (also: every thread has read the old scale)
#pragma unroll
    for (int wi = 0; wi < APPEND_THREADS / 32; wi++) amax = fmaxf(amax, red[wi]);
    float now = e4m3_scale(amax);
    if (held) {
        if (!(before >= 0.f) || before > 3.4028235e38f) {  // (what the page's codes mean is not known: nothing is written)
            if (threadIdx.x == 0) flag(ERRF_SCALE);
            return;
        }
        if (before >= now) {
            now = before;
        } else {
            const float f = before / now;
            for (int i = threadIdx.x; i < held * upr; i += APPEND_THREADS) {
                uint4 w = *(uint4 *)(cache + (int64_t)i * 16);
                uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int t = 0; t < 4; t++)
                    r[t] = pack_e4m3x4(f * e4m3_to_float(r[t] & 255), f * e4m3_to_float((r[t] >> 8) & 255),
                                       f * e4m3_to_float((r[t] >> 16) & 255), f * e4m3_to_float(r[t] >> 24));
                *(uint4 *)(cache + (int64_t)i * 16) = make_uint4(r[0], r[1], r[2], r[3]);
            }
        }
    }
    if (threadIdx.x == 0) *scale = now;
    const bool pow2 = (__float_as_uint(now) & 0x7FFFFFu) == 0;
    const float inv = 1.f / now;
#pragma unroll
    for (int k = 0; k < U; k++) {
        const int i = threadIdx.x + k * APPEND_THREADS;
        if (i < units) {
            const int u = i % upr;
            int ra, rb;
            if (!tensor && u < A.rot / 16) unit_runs(A, u, ra, rb);
            else { ra = u * 16; rb = ra + 8; }
            uint8_t *row = cache + (int64_t)(held + i / upr) * A.D;
            // (the reciprocal of a power of two is exact; a scale that the page had need not be one)
            if (!pow2) {
#pragma unroll
                for (int e = 0; e < 16; e++) x[k][e] /= now;
            } else {
#pragma unroll
                for (int e = 0; e < 16; e++) x[k][e] *= inv;
            }
            *(uint2 *)(row + ra) = make_uint2(pack_e4m3x4(x[k][0], x[k][1], x[k][2], x[k][3]), pack_e4m3x4(x[k][4], x[k][5], x[k][6], x[k][7]));
            *(uint2 *)(row + rb) = make_uint2(pack_e4m3x4(x[k][8], x[k][9], x[k][10], x[k][11]), pack_e4m3x4(x[k][12], x[k][13], x[k][14], x[k][15]));
        }
    }
}

// U: units a thread of a page's CTA (0: no E4M3 cache).  A CTA's chain of reads is long against its work, so the CTAs
// that an SM holds count for more than a few spilled registers: five of them (48 registers) took 74 us where three (77)
// took 86 (8 chunks into an E4M3 cache), 143 where four took 158 (16384 tokens into a bf16 one).
template <int DT, int U>
__global__ void __launch_bounds__(APPEND_THREADS, U <= 2 ? 5 : 2) k_kv_append(const AppendArgs A)
{
    extern __shared__ float2 cs[];  // [tokens][rot / 2] cos, sin
    __shared__ SeqOf slots[APPEND_TOKENS];
    __shared__ int32_t pages[APPEND_TOKENS];
    __shared__ int last;
    __shared__ float red[APPEND_THREADS / 32];
    if (U == 0 || (int64_t)blockIdx.x < A.row_ctas) append_rows<DT, U == 0>(A, cs, slots, pages);
    else if constexpr (U > 0) append_page<DT, U>(A, (int64_t)blockIdx.x - A.row_ctas, slots, &last, red);
}

}  // namespace lsa
