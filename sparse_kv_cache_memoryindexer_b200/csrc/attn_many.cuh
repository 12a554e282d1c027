// Core attention for many query rows on tcgen05 (chunks of a prompt, a window's tokens at once), D = 64 or 128,
// bf16 or E4M3 caches.
//
// A CTA holds 256 query rows of one sequence and key/value head (token-major, the G = Hq / H heads of a group
// inside a token) as two MMA tiles of 128, and walks the keys that any of them sees in blocks of 128.  Per block
// and tile: S = Q K^T (M = N = 128) into TMEM; a warpgroup reads its tile's rows (a thread has a whole row, so
// maximum and sum need no exchange), writes the probabilities over S as the A operand of O += P V (M = 128,
// N = D, the values read MN-major as they lie in the cache).  While one warpgroup works on its S, the tensor
// core does the other tile's products.  TMEM: S0 S1 O0 O1, 128 columns each; P takes the first 64 of its S.
// The running maximum is let go stale by up to 2^8: O is brought to a new one only when a row's has grown by
// more, which after the first blocks is rare, so O stays in TMEM.
// What bounds it: a tile's chain of softmax (about 2200 clocks beside the other tile's) and its two products (1000)
// takes 3500 clocks a block, where the MMAs of both tiles take 2048 (2 x 128 x 128 x D multiply-adds each, 4096 a
// clock) and their exponentials as long.  Two chunks of 4096 and 1900 tokens over a window of 4096, 32 heads of 128:
// 566 us, 865 TFLOP/s (the plain form 42 ms); 2048 tokens on an E4M3 history of 14001: 579 us, 870 TFLOP/s.
//
// Probabilities are rounded to the type of the values in the product, bf16 or f16, once (both operands of an MMA have one type);
// their sum is taken before that, in fp32.
//
// Keys and values come by TMA, one box per page (128-byte swizzle); E4M3 pages come as they are and four warps
// decode them exactly to f16 tiles (see attn_few.cuh for how a page's scales enter; the probabilities' factor
// is 2^7 here, so that with a stale maximum they stay below f16's largest: weights under 2^-21 of the maximum in use are
// subnormal in f16 and lose bits, where the few-row kernel, whose maximum is never stale, has 2^-29).
// Value rows that none of the CTA's rows sees (behind its last token, before its first window, on pages that are
// not there) are zeroed: what lies there, stale or never written, must not meet a probability of zero in the
// product.  A key that some rows see and others must not, itself NaN or infinite, makes its tile's rows NaN;
// those rows are done again by attend_row.
//
// Few tiles: their keys are split over CTAs (grid z), the parts joined by k_attn_many_join.
// Every mbarrier wait is bounded; on time-out the CTA flags ERRF_TIMEOUT, waits (bounded) for its copies and MMAs
// in flight, frees its TMEM and returns.
#pragma once
#include "attn_few.cuh"
#include "tc_common.cuh"
#include "train_tc.cuh"

namespace lsa {

namespace many {

constexpr int TILE_ROWS = 128;
constexpr int CTA_ROWS = 256;
constexpr int BLOCK = 128;        // keys per block
constexpr int META = 4;           // blocks whose page data are kept (see the producer)

template <int CT, int D>
struct Cfg {
    static constexpr int NB = D / 64;                     // 64-element boxes of a row
    static constexpr uint32_t TILE_BYTES = NB * 16384u;   // 128 rows of f16 / bf16
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_K = 2 * TILE_BYTES;     // two stages
    static constexpr uint32_t OFF_V = OFF_K + 2 * TILE_BYTES;
    static constexpr uint32_t RAW = CT == DT_FP8 ? BLOCK * D : 0u;
    static constexpr uint32_t OFF_KRAW = OFF_V + 2 * TILE_BYTES;
    static constexpr uint32_t OFF_VRAW = OFF_KRAW + RAW;
    static constexpr uint32_t OFF_META = OFF_VRAW + RAW;  // META x 112 bytes
    static constexpr uint32_t OFF_QF = OFF_META + META * 112;  // row factors [256] (E4M3)
    static constexpr uint32_t OFF_BAR = OFF_QF + (CT == DT_FP8 ? CTA_ROWS * 4 : 0);
    static constexpr uint32_t BARS = 21;
    static constexpr uint32_t OFF_MISC = OFF_BAR + 8 * BARS;
    static constexpr uint32_t SMEM = OFF_MISC + 16 + 1024;
    static constexpr int THREADS = CT == DT_FP8 ? 512 : 384;
    // registers of the softmax warpgroups, the one of producer and issuer, the decoding one: of 3 x 168 (bf16) or 4 x 128
    static constexpr int REGS_SOFTMAX = CT == DT_FP8 ? 184 : 208;
    static constexpr int REGS_ISSUE = CT == DT_FP8 ? 56 : 80;
    static constexpr int REGS_DECODE = 88;
    static_assert(CT == DT_FP8 ? 2 * REGS_SOFTMAX + REGS_ISSUE + REGS_DECODE <= 4 * 128 : 2 * REGS_SOFTMAX + REGS_ISSUE <= 3 * 168, "");
    static constexpr uint32_t IDESC_S = CT == DT_FP8 ? tc::idesc_f16(128, BLOCK) : tc::idesc_bf16(128, BLOCK);
    static constexpr uint32_t IDESC_O = (CT == DT_FP8 ? tc::idesc_f16(128, D) : tc::idesc_bf16(128, D)) | (1u << 16);
    static constexpr float SHIFT = CT == DT_FP8 ? 7.f : 0.f;
};

constexpr float STALE = 8.f;  // log2 of how far a row's maximum may run ahead of the one in use

// Page data of a block: for each 16 keys the key scale, log2 of the value scale and its reciprocal; which are live,
// and which have a value scale of zero.
struct Meta {
    float ks[8], lv[8], inv[8];
    uint32_t live, zero, pad[2];
};
static_assert(sizeof(Meta) == 112, "Meta");

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]) : "r"(a));
}
using tc::fma2;
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// The lowest n bits (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t first_bits(int n) { return n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u); }
// Registers of a warpgroup: the kernel starts with 65536 / threads each; the shares below add up to no more.
template <int N>
__device__ __forceinline__ void setmaxnreg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// The work of a CTA: rows row0 .. of sequence b (rows of them), keys in `blocks` blocks; block i starts at position
// 128 i for i < sb, else 128 (wb0 + i - sb).
struct Job {
    int b, row0, rows;
    int64_t off, len;
    int64_t p_first, last;  // position of the first row's token; last position that any row sees
    int64_t low;            // first position of the first row's window
    int sb, wb0, blocks;
};

// Rows of the block at position p0 that some row of the CTA sees: [0, end) without [gap0, gap1).
__device__ __forceinline__ void seen_rows(const AttnArgs &A, const Job &j, int64_t p0, int &gap0, int &gap1, int &end)
{
    end = (int)min((int64_t)BLOCK, j.last + 1 - p0);
    gap0 = (int)max((int64_t)0, min((int64_t)BLOCK, A.n_sink - p0));
    gap1 = (int)max((int64_t)0, min((int64_t)BLOCK, j.low - p0));
}

template <int CTA>
__device__ __forceinline__ bool load_job(const AttnArgs &A, int64_t x, int *found, Job &j)
{
    const int G = A.Hq / A.H;
    if (threadIdx.x == 0) *found = -1;
    __syncthreads();
    for (int b = threadIdx.x; b < A.B; b += blockDim.x) {
        const int64_t lo = __ldg(A.q_offsets + b), hi = __ldg(A.q_offsets + b + 1);
        if (lo < 0 || hi < lo || hi > A.N) flag(ERRF_OFFSETS);
        else if (hi > lo && lo * G / CTA + b <= x) atomicMax(found, b);
    }
    __syncthreads();
    j.b = *found;
    if (j.b < 0) return false;
    j.off = __ldg(A.q_offsets + j.b);
    const int64_t n = __ldg(A.q_offsets + j.b + 1) - j.off;
    const int64_t tile = x - (j.off * G / CTA + j.b);
    if (tile * CTA >= n * G) return false;
    j.row0 = (int)(tile * CTA);
    j.rows = (int)min((int64_t)CTA, n * G - j.row0);
    j.len = __ldg(A.cache_len + j.b);
    if (j.len < 0) {
        flag(ERRF_COUNT);
        j.len = -n;  // every query stands before position 0: nothing to see
    }
    j.p_first = j.len + j.row0 / G;
    j.last = j.len + (j.row0 + j.rows - 1) / G;
    const int64_t limit = (int64_t)A.max_pages * A.page;
    if (j.last >= limit) {
        flag(ERRF_COUNT);
        j.last = limit - 1;
    }
    j.low = (A.window > 0 && j.p_first + 1 > A.window) ? j.p_first + 1 - A.window : 0;
    j.wb0 = (int)(j.low / BLOCK);
    const int64_t sinks = min((int64_t)A.n_sink, j.low);
    j.sb = (int)min((sinks + BLOCK - 1) / BLOCK, (int64_t)j.wb0);
    const int64_t wend = j.last < 0 ? 0 : j.last / BLOCK + 1;
    if (j.wb0 > wend) {  // (only where the lengths are bad)
        j.sb = min(j.sb, (int)wend);
        j.blocks = j.sb;
    } else {
        j.blocks = j.sb + (int)(wend - j.wb0);
    }
    return true;
}

__device__ __forceinline__ void row_of(const AttnArgs &A, const Job &j, int r, int64_t &n, int64_t &pos, int &g)
{
    const int G = A.Hq / A.H, R = j.row0 + r;
    n = j.off + R / G;
    pos = j.len + R / G;
    g = R % G;
}

// A part in the workspace: maxima (log2, of what the exponents are relative to) and sums of 256 rows, then O.  E4M3: a
// sum is marked where value scales are unusual (marked_sum).
template <int D>
constexpr size_t part_floats() { return 2 * CTA_ROWS + (size_t)CTA_ROWS * D; }

// Bounded waits as tc::mbar_wait and tc::mbar_wait_warp, for barriers that complete every microsecond: the clock
// is read once in 64 tries (each of which the hardware may hold for a while), since reading %globaltimer takes
// longer than most waits here.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    if (tc::mbar_try(bar, parity)) return true;
    uint64_t t0 = 0;
    for (uint32_t i = 1;; i++) {
        if (tc::mbar_try(bar, parity)) return true;
        if ((i & 63) == 0) {
            if (*abort_flag) return false;
            const uint64_t now = tc::gtime();
            if (t0 == 0) t0 = now;
            if (now - t0 > tc::WAIT_NS) {
                *abort_flag = 1;
                flag(ERRF_TIMEOUT);
                return false;
            }
        }
    }
}
// The whole warp waits: every lane polls (one instruction for all of them), and they leave together.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    const bool ok = wait_bar(bar, parity, abort_flag);
    return __all_sync(0xffffffffu, ok);
}

// One arrival for a warp whose lanes have all done (and fenced) what it tells of.
__device__ __forceinline__ void arrive_warp(uint32_t bar)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar);
}

__device__ __forceinline__ bool wait_alone(uint32_t bar, uint32_t parity)
{
    volatile int never = 0;
    return tc::mbar_wait(bar, parity, &never);
}

template <int CT, int D>
__global__ void __launch_bounds__((Cfg<CT, D>::THREADS), 1)
    k_attn_many(const AttnArgs A, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, float *parts)
{
    using namespace tc;
    using C = Cfg<CT, D>;
    constexpr bool FP8 = CT == DT_FP8;
    constexpr int NB = C::NB;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int found;
    uint8_t *base = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = smem_u32(base);
    Meta *meta = (Meta *)(base + C::OFF_META);
    float *qfac = (float *)(base + C::OFF_QF);
    uint32_t *tmem_holder = (uint32_t *)(base + C::OFF_MISC);
    volatile int *abort_flag = (volatile int *)(base + C::OFF_MISC + 4);
    uint32_t *met = (uint32_t *)(base + C::OFF_MISC + 8);  // unusual value scales of the CTA's pages (E4M3; the producer's)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto bar = [&](int i) { return sbase + C::OFF_BAR + 8u * i; };
    auto k_full = [&](int s) { return bar(s); };
    auto k_empty = [&](int s) { return bar(2 + s); };
    auto v_full = [&](int s) { return bar(4 + s); };
    auto v_empty = [&](int s) { return bar(6 + s); };
    auto s_full = [&](int t) { return bar(8 + t); };
    auto p_full = [&](int t) { return bar(10 + t); };
    auto o_done = [&](int t) { return bar(12 + t); };
    const uint32_t landed = bar(14), kraw_full = bar(14), kraw_empty = bar(15), vraw_full = bar(16), vraw_empty = bar(17),
                   drained = bar(18);
    auto p_half = [&](int t) { return bar(19 + t); };

    // later tiles first: with no window they have the most keys
    const int64_t x = (int64_t)gridDim.x - 1 - blockIdx.x;
    const int h = blockIdx.y, Z = gridDim.z, z = blockIdx.z;
    Job j;
    if (!load_job<CTA_ROWS>(A, x, &found, j)) return;
    const int i0 = (int)((int64_t)j.blocks * z / Z), i1 = (int)((int64_t)j.blocks * (z + 1) / Z), nb = i1 - i0;
    float *part = Z > 1 ? parts + ((size_t)((x * A.H + h) * Z + z)) * part_floats<D>() : nullptr;
    const int G = A.Hq / A.H;
    if (nb == 0) {  // no keys here
        if (part) {
            for (int r = tid; r < CTA_ROWS; r += C::THREADS) {
                part[r] = -INFINITY;
                part[CTA_ROWS + r] = 0.f;
            }
        } else {
            for (int i = tid; i < j.rows * (D / 8); i += C::THREADS) {
                int64_t n, pos;
                int g;
                row_of(A, j, i / (D / 8), n, pos, g);
                const int64_t at = n * A.Hq + h * G + g;
                *(uint4 *)((__nv_bfloat16 *)A.out + at * D + (i % (D / 8)) * 8) = make_uint4(0u, 0u, 0u, 0u);
                if (A.lse && i % (D / 8) == 0) A.lse[at] = -INFINITY;
            }
        }
        return;
    }

    if (tid == 0) {
        for (int s = 0; s < 2; s++) {
            mbar_init(k_full(s), FP8 ? 4 : 1);
            mbar_init(k_empty(s), 1);
            mbar_init(v_full(s), FP8 ? 4 : 1);
            mbar_init(v_empty(s), 1);
            mbar_init(s_full(s), 1);
            mbar_init(p_full(s), 4);
            mbar_init(p_half(s), 4);
            mbar_init(o_done(s), 1);
        }
        mbar_init(bar(14), 1);    // (landed, or kraw_full)
        mbar_init(kraw_empty, 4);
        mbar_init(vraw_full, 1);
        mbar_init(vraw_empty, 4);
        mbar_init(drained, 1);
        *abort_flag = 0;
        *met = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    // the query rows, D / 8 lanes a row, into the swizzled tiles, by every warp but the producer's, which starts its loads
    if (warp != 8) {
        constexpr int STAGERS = C::THREADS - 32;
        const int st = tid < 256 ? tid : tid - 32;
        auto row_at = [&](int r) -> int64_t {
            const int R = j.row0 + r;
            return r < j.rows ? (j.off + R / G) * A.q_stride + (int64_t)(h * G + R % G) * D : -1;
        };
        constexpr int PIECES = CTA_ROWS * (D / 8);
        auto q_at = [&](int i) {
            const int r = i / (D / 8), c = i % (D / 8);
            return C::OFF_Q + (uint32_t)(r >> 7) * C::TILE_BYTES + (uint32_t)(c >> 3) * 16384u + train_tc::sw128(r & 127, c & 7);
        };
        if constexpr (!FP8) {
            for (int i = st; i < PIECES; i += STAGERS) {
                const int64_t from = row_at(i / (D / 8));
                few::cp_async16(sbase + q_at(i), (const __nv_bfloat16 *)A.q + (from < 0 ? 0 : from + (i % (D / 8)) * 8), from < 0 ? 0 : 16);
            }
            few::cp_commit();
            few::cp_wait<0>();
            if (A.scale < 0.f) {  // the scores' factor is |scale|: the sign goes to the query
#pragma unroll 1
                for (int i = st; i < PIECES; i += STAGERS) {
                    uint4 *p = (uint4 *)(base + q_at(i));
                    *p = make_uint4(p->x ^ 0x80008000u, p->y ^ 0x80008000u, p->z ^ 0x80008000u, p->w ^ 0x80008000u);
                }
            }
        } else {
            // f16 by a power of two of the row's own: its largest element comes to [2^8, 2^9)
            constexpr int EACH = (PIECES + STAGERS - 1) / STAGERS;  // (whole warps reach or miss the last one: D / 8 lanes a row)
            uint4 v[EACH];
#pragma unroll
            for (int k = 0; k < EACH; k++) {
                const int i = st + k * STAGERS;
                const int64_t from = i < PIECES ? row_at(i / (D / 8)) : -1;
                v[k] = make_uint4(0u, 0u, 0u, 0u);
                if (from >= 0) v[k] = __ldg((const uint4 *)((const __nv_bfloat16 *)A.q + from) + i % (D / 8));
            }
#pragma unroll
            for (int k = 0; k < EACH; k++) {
                const int i = st + k * STAGERS;
                if (i >= PIECES) break;
                uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
                float mx = 0.f;
#pragma unroll
                for (int e = 0; e < 4; e++)
                    mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xFFFF0000u))));
#pragma unroll
                for (int o = 1; o < D / 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                int e = 8 - ((int)(__float_as_uint(mx) >> 23) - 127);
                e = e > 120 ? 120 : (e < -120 ? -120 : e);
                const float up = copysignf(__uint_as_float((uint32_t)(e + 127) << 23), A.scale);  // (the scores' factor is |scale|)
                if (i % (D / 8) == 0) qfac[i / (D / 8)] = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                for (int x2 = 0; x2 < 4; x2++)
                    w[x2] = few::pack_f16x2(__uint_as_float(w[x2] << 16) * up, __uint_as_float(w[x2] & 0xFFFF0000u) * up);
                *(uint4 *)(base + q_at(i)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        fence_async();
        asm volatile("bar.sync 1, %0;" ::"n"(STAGERS) : "memory");
    }
    auto block_pos = [&](int i) -> int64_t { return (int64_t)(i < j.sb ? i : j.wb0 + (i - j.sb)) * BLOCK; };

    if (warp < 8) {
        // ------------------------------------------------------- softmax: warpgroup t has tile t, a thread a row
        setmaxnreg_inc<C::REGS_SOFTMAX>();
        const int t = warp >> 2, rr = tid & 127, r = t * TILE_ROWS + rr;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lanes + (uint32_t)t * 128u, o_addr = tmem + lanes + 256u + (uint32_t)t * 128u;
        int64_t n = 0, pos = -1;
        int g = 0;
        if (r < j.rows) row_of(A, j, r, n, pos, g);
        const int64_t mylow = (A.window > 0 && pos + 1 > A.window) ? pos + 1 - A.window : 0;
        // first and last rows' positions of the tile: a block that all of its rows see whole needs no masks
        const int tr0 = t * TILE_ROWS, tr1 = min(j.rows, tr0 + TILE_ROWS) - 1;
        const int64_t t_first = j.len + (j.row0 + min(tr0, j.rows - 1)) / G, t_last = j.len + (j.row0 + max(tr1, 0)) / G;
        // (a factor of zero would make NaN of a masked -inf)
        const float f = fmaxf(fabsf(A.scale) * 1.4426950408889634f, 1e-30f) * (FP8 ? qfac[r] : 1.f);
        const float fx = FP8 ? 1.f : f;  // from s to log2 units
        float m = -INFINITY, l = 0.f;    // m: the maximum in use, in the units of s
        bool ok = true;
        for (int i = 0; i < nb; i++) {
            const int64_t p0 = block_pos(i0 + i);
            if (!wait_warp(s_full(t), i & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const Meta *me = meta + (i & (META - 1));
            const uint32_t live = me->live;
            float s[4][32];
#pragma unroll
            for (int pc = 0; pc < 4; pc++) {
                tmem_ld32(s_addr + 32 * pc, s[pc]);
                if (pc & 1) tmem_wait_ld();
            }
            if constexpr (FP8) {
#pragma unroll
                for (int pc = 0; pc < 4; pc++)
#pragma unroll
                    for (int gg = 0; gg < 2; gg++) {
                        const float a = f * me->ks[2 * pc + gg], b = me->lv[2 * pc + gg];
#pragma unroll
                        for (int k = 16 * gg; k < 16 * gg + 16; k += 2) {
                            const float2 y = fma2(make_float2(s[pc][k], s[pc][k + 1]), make_float2(a, a), make_float2(b, b));
                            s[pc][k] = y.x;
                            s[pc][k + 1] = y.y;
                        }
                    }
            }
            if (!(live == 0xFFu && p0 + BLOCK - 1 <= t_first &&
                  (A.window == 0 || p0 > t_last - A.window || p0 + BLOCK <= A.n_sink))) {
                // columns [0, hi) and ([lo, ..) or [0, sk)) of the block are visible to this row
                const int hi = (int)max((int64_t)0, min((int64_t)BLOCK, pos + 1 - p0)),
                          lo = (int)max((int64_t)0, min((int64_t)BLOCK, mylow - p0)),
                          sk = (int)max((int64_t)0, min((int64_t)BLOCK, (int64_t)A.n_sink - p0));
#pragma unroll
                for (int pc = 0; pc < 4; pc++) {
                    const uint32_t pages = ((live >> (2 * pc) & 1) ? 0xFFFFu : 0u) | ((live >> (2 * pc + 1) & 1) ? 0xFFFF0000u : 0u);
                    const uint32_t w = first_bits(hi - 32 * pc) & (~first_bits(lo - 32 * pc) | first_bits(sk - 32 * pc)) & pages;
#pragma unroll
                    for (int k = 0; k < 32; k++) s[pc][k] = (w & (1u << k)) ? s[pc][k] : -INFINITY;
                }
            }
            float mx4[4];
#pragma unroll
            for (int pc = 0; pc < 4; pc++) {
                mx4[pc] = s[pc][0];
#pragma unroll
                for (int k = 1; k < 31; k += 2) mx4[pc] = fmaxf(fmaxf(mx4[pc], s[pc][k]), s[pc][k + 1]);
                mx4[pc] = fmaxf(mx4[pc], s[pc][31]);
            }
            const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
            const bool grow = m == -INFINITY ? mx != -INFINITY : (mx - m) * fx > STALE;
            if (__any_sync(0xffffffffu, grow)) {
                const float mn = fmaxf(m, mx);
                const float ff = m == -INFINITY ? 0.f : few::exp2_fast((m - mn) * fx);
                m = mn;
                l *= ff;
                if (i > 0) {
                    if (!wait_warp(o_done(t), (i - 1) & 1, abort_flag)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t u[16];
                        tmem_ld16(o_addr + c, u);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; k++) u[k] = __float_as_uint(__uint_as_float(u[k]) * ff);
                        tmem_st16(o_addr + c, u);
                    }
                    tmem_wait_st();
                }
            }
            const float ref = (m == -INFINITY ? 0.f : m) * fx - C::SHIFT;
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int pc = 0; pc < 4; pc++) {
                uint32_t u[16];
#pragma unroll
                for (int gg = 0; gg < 2; gg++) {
                    if (FP8) sum = make_float2(0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        float2 y = fma2(make_float2(s[pc][16 * gg + k], s[pc][16 * gg + k + 1]), make_float2(fx, fx), make_float2(-ref, -ref));
                        y.x = few::exp2_fast(y.x);
                        y.y = few::exp2_fast(y.y);
                        sum = add2(sum, y);
                        u[8 * gg + k / 2] = FP8 ? few::pack_f16x2(y.x, y.y) : few::pack_b16x2(y.x, y.y);
                    }
                    if (FP8) l = fmaf(sum.x + sum.y, me->inv[2 * pc + gg], l);
                }
                tmem_st16(s_addr + 16 * pc, u);
                if (pc == 1) {  // the product over the first 64 keys can start
                    tmem_wait_st();
                    tc_fence_before();
                    arrive_warp(p_half(t));
                }
            }
            if (!FP8) l += sum.x + sum.y;
            tmem_wait_st();
            tc_fence_before();
            arrive_warp(p_full(t));
        }
        if (ok && !wait_warp(o_done(t), (nb - 1) & 1, abort_flag)) ok = false;
        if (ok) {
            tc_fence_after();
            if (FP8) l = marked_sum(l, *met, 128.f);
            bool bad = !part && r < j.rows && few::from_zero<CT>(l, m, m);
            const float mark = l;
            l = few::sum_of<CT>(l);
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const float ml2 = m * (FP8 ? 1.f : f) - C::SHIFT;
            const int64_t at = n * A.Hq + h * G + g;
#pragma unroll
            for (int pc = 0; pc < D / 32; pc++) {
                float v[32];
                tmem_ld32(o_addr + 32 * pc, v);
                tmem_wait_ld();
                if (r < j.rows) {
                    if (part) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *(float4 *)(part + 2 * CTA_ROWS + (size_t)r * D + 32 * pc + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; k += 8) {
                            uint32_t u[4];
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                const float a = v[k + 2 * e] * inv, b = v[k + 2 * e + 1] * inv;
                                bad |= !(fabsf(a) <= 3.4028235e38f) || !(fabsf(b) <= 3.4028235e38f);
                                u[e] = few::pack_b16x2(a, b);
                            }
                            *(uint4 *)((__nv_bfloat16 *)A.out + at * D + 32 * pc + k) = make_uint4(u[0], u[1], u[2], u[3]);
                        }
                    }
                }
            }
            if (r < j.rows) {
                if (part) {
                    part[r] = m == -INFINITY ? -INFINITY : ml2;
                    part[CTA_ROWS + r] = mark;
                } else if (A.lse) {
                    A.lse[at] = l == 0.f ? -INFINITY : (ml2 + log2f(l)) * 0.6931471805599453f;
                }
            }
            uint32_t again = __ballot_sync(0xffffffffu, bad);
            while (again) {  // (this tile's products are done: its query tile is free for the rows)
                const int src = __ffs(again) - 1;
                again &= again - 1;
                const int64_t n2 = __shfl_sync(0xffffffffu, n, src), pos2 = __shfl_sync(0xffffffffu, pos, src);
                const int g2 = __shfl_sync(0xffffffffu, g, src);
                attend_row<DT_BF16, CT>(A, j.b, pos2, n2, h * G + g2, (float *)(base + C::OFF_Q + t * C::TILE_BYTES) + (warp & 3) * ATTN_MAX_D);
            }
        }
    } else if (warp < 12) {
        setmaxnreg_dec<C::REGS_ISSUE>();
        if (warp == 8) {
            // ------------------------------------------------------- producer: lane x has page x of the block
            const int per_block = BLOCK / A.page;
            const uint32_t page_bytes = (uint32_t)A.page * (FP8 ? D : 128);  // of one box
            const int boxes = FP8 ? 1 : NB;
            int issued = 0;
            int specials = 0;
            bool special = false;
            // Page numbers are read two blocks ahead, an E4M3 page's scales one: with the reads in the loop's way a block of
            // an E4M3 history took 6600 clocks.
            auto read_page = [&](int i) -> int32_t {  // (-1: no query sees it, or there is no such block)
                if (i >= nb) return -1;
                const int64_t pa = block_pos(i0 + i) + (int64_t)lane * A.page;
                if (lane >= per_block || pa > j.last || (pa + A.page <= j.low && pa >= A.n_sink)) return -1;
                const int32_t p = __ldg(A.page_table + (int64_t)j.b * A.max_pages + pa / A.page);
                return p < 0 ? -2 : p;  // (-2: seen, and not there)
            };
            auto good_page = [&](int32_t p) { return p >= 0 && p < A.n_pages; };
            auto read_scale = [&](const float *s, int32_t p) { return FP8 && good_page(p) ? __ldg(s + (int64_t)p * A.H + h) : 1.f; };
            int32_t page1 = read_page(0), page2 = read_page(1);
            float ks1 = read_scale(A.k_scale, page1), vs1 = read_scale(A.v_scale, page1);
            for (int i = 0; i < nb; i++) {
                const int64_t p0 = block_pos(i0 + i);
                int32_t page = page1;
                const float ks = ks1, vs = vs1;
                page1 = page2;
                page2 = read_page(i + 2);
                ks1 = read_scale(A.k_scale, page1);
                vs1 = read_scale(A.v_scale, page1);
                if (page != -1 && !good_page(page)) {
                    flag(ERRF_PAGE);
                    page = -1;
                }
                if (FP8 && page >= 0 && (!good_scale(ks) || !good_scale(vs))) {
                    flag(ERRF_SCALE);
                    page = -1;
                }
                const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
                const uint32_t bytes = (uint32_t)__popc(there) * page_bytes * boxes;
                const int y = (int)(((int64_t)max(page, 0) * A.H + h) * A.page);
                // keys.  (A block's Meta is written once its stage is free, when S of block i - 2 is done: softmax may
                // still be at i - 2, or i - 3 of the E4M3 path, which runs one block further ahead, but no further back.)
                if (!wait_warp(FP8 ? kraw_empty : k_empty(i & 1), FP8 ? (i & 1) ^ 1 : ((i >> 1) & 1) ^ 1, abort_flag)) break;
                Meta *me = meta + (i & (META - 1));
                if (lane < per_block) {
                    const float lv = !FP8 ? 0.f : (page >= 0 && vs > 0.f ? log2f(vs) : ZERO_LV);
                    const float inv = !FP8 ? 1.f : (page >= 0 && vs > 0.f ? 1.f / vs : ZERO_INV);
                    for (int k = 0; k < A.page / 16; k++) {
                        const int at = lane * (A.page / 16) + k;
                        me->ks[at] = page >= 0 ? ks : 0.f;
                        me->lv[at] = lv;
                        me->inv[at] = inv;
                    }
                }
                uint32_t live = 0, zero = 0;
                for (int k = 0; k < 8; k++) live |= (there >> (k * 16 / A.page) & 1u) << k;
                const bool odd = FP8 && page >= 0 && !usual_value_scale(vs);
                if (FP8 && __any_sync(0xffffffffu, odd)) {
                    const uint32_t zs = __ballot_sync(0xffffffffu, odd && vs == 0.f);
                    for (int k = 0; k < 8; k++) zero |= (zs >> (k * 16 / A.page) & 1u) << k;
                    const uint32_t of = __reduce_or_sync(0xffffffffu, odd ? met_of(vs) : 0u);
                    if (lane == 0) *met |= of;
                }
                if (lane == 0) {
                    me->live = live;
                    me->zero = zero;
                }
                __syncwarp();
                const uint32_t kf = FP8 ? kraw_full : k_full(i & 1);
                if (lane == 0) mbar_expect_tx(kf, bytes);
                __syncwarp();
                if (page >= 0) {
                    const uint32_t dst = sbase + (FP8 ? C::OFF_KRAW : C::OFF_K + (uint32_t)(i & 1) * C::TILE_BYTES) + (uint32_t)lane * page_bytes;
                    for (int bx = 0; bx < boxes; bx++) tma_load_2d(dst + bx * 16384u, &kmap, 64 * bx, y, kf);
                }
                __syncwarp();
                // values
                if (!wait_warp(FP8 ? vraw_empty : v_empty(i & 1), FP8 ? (i & 1) ^ 1 : ((i >> 1) & 1) ^ 1, abort_flag)) break;
                const uint32_t vdst = sbase + (FP8 ? C::OFF_VRAW : C::OFF_V + (uint32_t)(i & 1) * C::TILE_BYTES);
                uint32_t vf = FP8 ? vraw_full : v_full(i & 1);
                if constexpr (!FP8) {
                    // rows that no query sees must be zero: on pages that are not loaded, and parts of pages that are (those
                    // after they have landed)
                    uint8_t *vt = base + C::OFF_V + (uint32_t)(i & 1) * C::TILE_BYTES;
                    int gap0, gap1, end;
                    seen_rows(A, j, p0, gap0, gap1, end);
                    auto seen = [&](int row) { return row < end && (row < gap0 || row >= gap1); };
                    auto clear = [&](int from, int to) {
                        for (int e = 8 * from + lane; e < 8 * to; e += 32)
#pragma unroll
                            for (int bx = 0; bx < NB; bx++) *(uint4 *)(vt + bx * 16384 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
                    };
                    const uint32_t real = vf;
                    const bool part_seen = lane < per_block && page >= 0 &&
                                           !(seen(lane * A.page) && seen(lane * A.page + A.page - 1) &&
                                             (gap0 >= gap1 || gap1 <= lane * A.page || gap0 >= lane * A.page + A.page));
                    special = __any_sync(0xffffffffu, part_seen);
                    if (special) vf = landed;
                    if (live != 0xFFu) {
                        for (int q = 0; q < per_block; q++)
                            if (!(there >> q & 1)) clear(q * A.page, (q + 1) * A.page);
                        fence_async();
                        __syncwarp();
                    }
                    if (lane == 0) mbar_expect_tx(vf, bytes);
                    __syncwarp();
                    if (page >= 0)
                        for (int bx = 0; bx < NB; bx++) tma_load_2d(vdst + (uint32_t)lane * page_bytes + bx * 16384u, &vmap, 64 * bx, y, vf);
                    __syncwarp();
                    if (special) {  // (a few blocks of a CTA's: at the ends of the first tokens, the window, the cache)
                        if (!wait_warp(landed, specials & 1, abort_flag)) break;
                        clear(gap0, gap1);
                        clear(end, BLOCK);
                        fence_async();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(real);
                        __syncwarp();
                        special = false;
                        specials++;
                    }
                } else {
                    if (lane == 0) mbar_expect_tx(vf, bytes);
                    __syncwarp();
                    if (page >= 0) tma_load_2d(vdst + (uint32_t)lane * page_bytes, &vmap, 0, y, vf);
                    __syncwarp();
                }
                issued = i + 1;
            }
            if (*abort_flag && lane == 0) {
                // let the copies in flight land before the CTA exits (those of the block that broke off among them)
                for (int i = max(0, issued - 2); i <= min(issued, nb - 1); i++) {
                    if (FP8) {
                        wait_alone(kraw_full, i & 1);
                        wait_alone(vraw_full, i & 1);
                    } else {
                        wait_alone(k_full(i & 1), (i >> 1) & 1);
                        wait_alone(v_full(i & 1), (i >> 1) & 1);
                    }
                }
                if (!FP8 && special) wait_alone(landed, specials & 1);
            }
            __syncwarp();
        } else if (warp == 9) {
            // ------------------------------------------------------- MMA issuer: one thread from here to the end (the
            // tensor core waits for it; warp-wide waits and elections cost it about 100 clocks each)
            if (elect_one()) {
                bool ok = true;
                auto score = [&](int t, int i) {
                    const uint32_t q = sbase + C::OFF_Q + (uint32_t)t * C::TILE_BYTES, k = sbase + C::OFF_K + (uint32_t)(i & 1) * C::TILE_BYTES;
#pragma unroll
                    for (int kk = 0; kk < D / 16; kk++) {
                        const uint32_t o = (uint32_t)(kk >> 2) * 16384u + (uint32_t)(kk & 3) * 32u;
                        mma_bf16(tmem + (uint32_t)t * 128u, sdesc(q + o), sdesc(k + o), C::IDESC_S, kk > 0 ? 1u : 0u);
                    }
                    mma_commit(s_full(t));
                    if (t == 1) mma_commit(k_empty(i & 1));
                };
                auto value = [&](int t, int i, int half) {
                    const uint32_t v = sbase + C::OFF_V + (uint32_t)(i & 1) * C::TILE_BYTES;
#pragma unroll
                    for (int k2 = 0; k2 < BLOCK / 32; k2++) {
                        const int kk = half * (BLOCK / 32) + k2;
                        mma_ts(tmem + 256u + (uint32_t)t * 128u, tmem + (uint32_t)t * 128u + 8u * kk,
                               train_tc::sdesc_mn(v + 2048u * kk, 16384u, 1024u), C::IDESC_O, (i > 0 || kk > 0) ? 1u : 0u);
                    }
                    if (half == 1) {
                        mma_commit(o_done(t));
                        if (t == 1) mma_commit(v_empty(i & 1));
                    }
                };
                ok = wait_bar(k_full(0), 0, abort_flag);
                if (ok) {
                    tc_fence_after();
                    score(0, 0);
                    score(1, 0);
                }
                for (int i = 0; i < nb && ok; i++) {
                    const bool more = i + 1 < nb;
#pragma unroll
                    for (int t = 0; t < 2; t++) {
                        ok = wait_bar(p_half(t), i & 1, abort_flag) && (t == 1 || wait_bar(v_full(i & 1), (i >> 1) & 1, abort_flag));
                        if (!ok) break;
                        tc_fence_after();
                        value(t, i, 0);
                        ok = wait_bar(p_full(t), i & 1, abort_flag) &&
                             (t == 1 || !more || wait_bar(k_full((i + 1) & 1), ((i + 1) >> 1) & 1, abort_flag));
                        if (!ok) break;
                        tc_fence_after();
                        value(t, i, 1);
                        if (more) score(t, i + 1);
                    }
                }
                if (!ok) {  // whatever was issued ends before TMEM and shared memory go
                    mma_commit(drained);
                    wait_alone(drained, 0);
                }
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------- E4M3 pages to f16 tiles (warps 12 .. 15)
        if constexpr (FP8) {
            setmaxnreg_dec<C::REGS_DECODE>();
            const int ct = tid - 384;
            // (What a warp runs once a block is unrolled in full here and in the softmax: with more of it the SM's
            // instruction cache no longer held a block's code, and everything took twice as long.)
            constexpr int PER = D / 16;  // 16-code pieces of a row
            // a thread has piece c of every STEP-th row: the swizzle of its rows is one
            constexpr int STEP = 128 / PER;
            const int c = ct % PER, row0 = ct / PER;
            // (the lanes of the upper box store their halves in the other order: no two on one bank)
            const int odd = (c >> 2) & 1;
            const uint32_t box = (uint32_t)(c >> 2) * 16384u;
            const uint32_t at_a = box + train_tc::sw128(row0, ((2 * c) & 7) + odd), at_b = box + train_tc::sw128(row0, ((2 * c) & 7) + 1 - odd);
            auto convert = [&](uint32_t raw, uint32_t tile, uint32_t live, int gap0, int gap1, int end) {
                const bool all = live == 0xFFu && end == BLOCK && gap0 >= gap1;
#pragma unroll 1
                for (int k0 = 0; k0 < PER; k0 += 4) {
                    const uint8_t *from = base + raw + (uint32_t)(ct + 128 * k0) * 16;
                    uint8_t *to = base + tile + (uint32_t)(k0 * STEP) * 128u;
                    uint4 w[4];
#pragma unroll
                    for (int k = 0; k < 4; k++) w[k] = *(const uint4 *)(from + 2048 * k);
                    if (!all) {
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const int row = row0 + STEP * (k0 + k);
                            if (!(row < end && (row < gap0 || row >= gap1) && (live >> (row >> 4) & 1))) w[k] = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        uint4 lo, hi;
                        few::e4m3x4_to_f16x2(w[k].x, lo.x, lo.y);
                        few::e4m3x4_to_f16x2(w[k].y, lo.z, lo.w);
                        few::e4m3x4_to_f16x2(w[k].z, hi.x, hi.y);
                        few::e4m3x4_to_f16x2(w[k].w, hi.z, hi.w);
                        *(uint4 *)(to + at_a + (uint32_t)(k * STEP) * 128u) = odd ? hi : lo;
                        *(uint4 *)(to + at_b + (uint32_t)(k * STEP) * 128u) = odd ? lo : hi;
                    }
                }
            };
            for (int i = 0; i < nb; i++) {
                const int64_t p0 = block_pos(i0 + i);
                int gap0, gap1, end;
                seen_rows(A, j, p0, gap0, gap1, end);
                bool go = true;
#pragma unroll 1
                for (int v = 0; v < 2 && go; v++) {  // keys, values (one body for both: see below)
                    const uint32_t raw_full = v ? vraw_full : kraw_full, empty = v ? v_empty(i & 1) : k_empty(i & 1);
                    go = wait_warp(raw_full, i & 1, abort_flag) && wait_warp(empty, ((i >> 1) & 1) ^ 1, abort_flag);
                    if (!go) break;
                    const Meta &me = meta[i & (META - 1)];
                    // (values of a page whose scale is zero are zeros: its keys have their share of the sum, no more)
                    convert(v ? C::OFF_VRAW : C::OFF_KRAW, (v ? C::OFF_V : C::OFF_K) + (uint32_t)(i & 1) * C::TILE_BYTES,
                            v ? me.live & ~me.zero : me.live, gap0, gap1, end);
                    fence_async();
                    arrive_warp(v ? v_full(i & 1) : k_full(i & 1));
                    arrive_warp(v ? vraw_empty : kraw_empty);
                }
                if (!go) break;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
}

constexpr int JOIN_WARPS = 8;

// Joins the Z parts of every row.  Grid: (tiles, heads, 256 / JOIN_WARPS); a warp has a row.
template <int CT, int D>
__global__ void __launch_bounds__(32 * JOIN_WARPS) k_attn_many_join(const AttnArgs A, const float *parts, int Z)
{
    __shared__ int found;
    __shared__ float qs[JOIN_WARPS][ATTN_MAX_D];
    const int64_t x = blockIdx.x;
    const int h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.z * JOIN_WARPS + warp;
    Job j;
    const bool work = load_job<CTA_ROWS>(A, x, &found, j);
    pdl_wait();  // (before any return: this launch must not end before the one whose parts it joins)
    if (!work || r >= j.rows) return;
    constexpr size_t PF = part_floats<D>();
    const float *p0 = parts + (size_t)((x * A.H + h) * Z) * PF;
    float M = -INFINITY;
    for (int z = 0; z < Z; z++) M = fmaxf(M, p0[z * PF + r]);
    constexpr int PER = D / 32;
    float acc[PER], L = 0.f;
    bool zero = false;
#pragma unroll
    for (int e = 0; e < PER; e++) acc[e] = 0.f;
    for (int z = 0; z < Z; z++) {
        const float *p = p0 + z * PF;
        const float m = p[r], l = p[CTA_ROWS + r];
        // a part without keys has written nothing else; one whose scores are all NaN has no maximum either, and a sum of NaN
        if (m == -INFINITY && l == 0.f) continue;
        const float f = few::exp2_fast(m - M);
        L = fmaf(few::sum_of<CT>(l), f, L);
        zero |= few::from_zero<CT>(l, m, M);
#pragma unroll
        for (int e = 0; e < PER; e++) acc[e] = fmaf(p[2 * CTA_ROWS + (size_t)r * D + lane + 32 * e], f, acc[e]);
    }
    int64_t n, pos;
    int g;
    const int G = A.Hq / A.H;
    row_of(A, j, r, n, pos, g);
    const int64_t at = n * A.Hq + h * G + g;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    bool bad = zero;
#pragma unroll
    for (int e = 0; e < PER; e++) {
        const float v = acc[e] * inv;
        bad |= !(fabsf(v) <= 3.4028235e38f);
        store_elem<DT_BF16>(A.out, at * D + lane + 32 * e, v);
    }
    if (A.lse && lane == 0) A.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    if (__any_sync(0xffffffffu, bad)) attend_row<DT_BF16, CT>(A, j.b, pos, n, h * G + g, qs[warp]);
}

inline int64_t tiles_of(int64_t N, int B, int G) { return N * G / CTA_ROWS + B; }

// Tiles and heads, were the tokens shared evenly by the sequences.
inline int64_t likely_ctas(int64_t N, int B, int Hq, int H)
{
    const int64_t rows = std::max<int64_t>(N / B, 1) * (Hq / H);
    return B * ((rows + CTA_ROWS - 1) / CTA_ROWS) * H;
}

// The most CTAs that may share one tile's keys: what brings the launch to about two for each SM.
inline int most_splits(int64_t N, int B, int Hq, int H, int sms)
{
    const int64_t ctas = likely_ctas(N, B, Hq, H);
    if (ctas >= sms) return 1;
    return (int)std::min<int64_t>(64, std::max<int64_t>(1, 2 * (int64_t)sms / ctas));
}

// Bytes of one part of every tile and head.
inline size_t part_bytes(int64_t N, int B, int Hq, int H, int D)
{
    return (size_t)tiles_of(N, B, Hq / H) * H * (2 * CTA_ROWS + (size_t)CTA_ROWS * D) * sizeof(float);
}

// CTAs that share one tile's keys, tiles of `blocks` blocks at most: the number with the least time, counted in blocks:
// the waves of CTAs, each its share of the blocks and about four for its start and end, and about eight for the second
// launch.  (128 tiles of 34 blocks: 100 us whole, 140 in two parts, which make two waves.)  No more than the workspace has
// room for, whatever size it was made for (a whole tile needs none).  least: that time.
inline int splits_of(int64_t N, int B, int Hq, int H, int D, int sms, int64_t blocks, size_t workspace_bytes, int64_t *least)
{
    const int64_t ctas = likely_ctas(N, B, Hq, H);
    const int most = (int)std::min<size_t>(most_splits(N, B, Hq, H, sms), workspace_bytes / part_bytes(N, B, Hq, H, D));
    int best = 1;
    *least = INT64_MAX;
    for (int z = 1; z <= std::max(most, 1); z++) {
        const int64_t t = (ctas * z + sms - 1) / sms * ((blocks + z - 1) / z + 4) + (z > 1 ? 8 : 0);
        if (t < *least) {
            *least = t;
            best = z;
        }
    }
    return best;
}

// Keys that a tile sees at most, were the tokens shared evenly.
inline int64_t likely_keys(const AttnArgs &A)
{
    const int64_t limit = (int64_t)A.max_pages * A.page;
    return A.window > 0 ? std::min(limit, A.window + A.N / A.B) : limit;
}

inline size_t parts_bytes(int64_t N, int B, int Hq, int H, int D)
{
    if (Hq % H) return 0;
    const int z = most_splits(N, B, Hq, H, 160);  // (what 148 SMs can use, and a few more)
    if (z == 1) return 0;
    return z * part_bytes(N, B, Hq, H, D);
}

// Tensor map of a cache as rows of D elements, a box of one page (bf16: half rows of 64, 128-byte swizzle).
inline bool make_cache_map(CUtensorMap *m, const void *ptr, bool fp8, int64_t rows, int D, int page)
{
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const int eb = fp8 ? 1 : 2;
    cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)D * eb};
    cuuint32_t box[2] = {(cuuint32_t)(fp8 ? D : 64), (cuuint32_t)page};
    cuuint32_t estr[2] = {1, 1};
    return enc(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides,
               box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, fp8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether this kernel takes the call: its MMAs and tensor maps can hold it, and it is the faster one.  Estimates in
// microseconds from measurements: the few-row kernel 8 and, for each 16-key chunk of a 16-row tile that falls on one of the
// SM's 8 warps, 1.45 (E4M3: 1.12) at D = 128 and 0.8 (0.9) at D = 64; this one 5 and 1.95 (2.2) for each block of its longest
// CTA, whose softmax does not know D.  Measured (few-row kernel : this one; 9000 tokens before, L2 cold):
//                                              D = 128 bf16    E4M3         D = 64 bf16    E4M3
//   32 users, window 4096, 8 heads, 16 rows    121 : 150       83 : 180     74 : 144       60 : 176
//   the same, 32 rows                          207 : 150      143 : 181     95 : 146       98 : 176
//   the same, 64 rows                          326 : 150      258 : 184    165 : 146      172 : 177
//   8 users, window 1024, 8 heads, 64 rows      28 : 31        29 : 37      23 : 31        25 : 35
//   the same, 128 rows                          49 : 31        51 : 37      45 : 31        49 : 35
//   1 user, window 512, 8 heads, 128 rows       17 : 23        17 : 27      14 : 22        15 : 25
//   1 user, 131000 keys, 1 head, 64 rows        51 : 60        58 : 70      43 : 56        45 : 66
//   the same, 128 rows                          70 : 61        74 : 72      53 : 59        55 : 68
//   2 users, 1000 keys, 4 heads, 800 rows       53 : 33        56 : 40      25 : 31        27 : 37
// LSA_ATTN_MANY=0 or 1 in the environment takes the one or the other wherever it can (to check them against one another).
inline bool takes(const AttnArgs &A, int cdt, size_t workspace_bytes, int sms)
{
    if (cdt == DT_F32 || A.k > 0 || (A.D != 64 && A.D != 128)) return false;
    if (A.n_pages * A.H * A.page >= (int64_t)1 << 31 || A.H > 65535) return false;
    const char *env = getenv("LSA_ATTN_MANY");
    if (env && env[0] == '0') return false;
    const int64_t rows = std::max<int64_t>(A.N / A.B, 1) * (A.Hq / A.H), keys = likely_keys(A);
    int64_t blocks;
    splits_of(A.N, A.B, A.Hq, A.H, A.D, sms, keys / BLOCK + 1, workspace_bytes, &blocks);
    const double chunk_us = A.D == 64 ? (cdt == DT_FP8 ? 0.9 : 0.8) : (cdt == DT_FP8 ? 1.12 : 1.45);
    const double few_us = 8 + chunk_us * A.B * ((rows + 15) / 16) * A.H * (keys / 16 + 1) / (8.0 * sms);
    const double many_us = 5 + (cdt == DT_FP8 ? 2.2 : 1.95) * blocks;
    return ((env && env[0] == '1') || many_us < few_us) && tc_available();
}

template <int CT, int D>
cudaError_t launch(const AttnArgs &A, void *workspace, size_t workspace_bytes, int sms, cudaStream_t st, int *launches)
{
    using C = Cfg<CT, D>;
    CUtensorMap km, vm;
    const int64_t rows = A.n_pages * A.H * A.page;
    if (!make_cache_map(&km, A.k_cache, CT == DT_FP8, rows, D, A.page) || !make_cache_map(&vm, A.v_cache, CT == DT_FP8, rows, D, A.page))
        return cudaErrorInvalidValue;
    auto kernel = k_attn_many<CT, D>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kernel, C::SMEM, done);
    if (e != cudaSuccess) return e;
    const int64_t tiles = tiles_of(A.N, A.B, A.Hq / A.H);
    int64_t least;
    const int Z = splits_of(A.N, A.B, A.Hq, A.H, A.D, sms, likely_keys(A) / BLOCK + 1, workspace_bytes, &least);
    k_attn_many<CT, D><<<dim3((unsigned)tiles, (unsigned)A.H, (unsigned)Z), C::THREADS, C::SMEM, st>>>(A, km, vm, (float *)workspace);
    ++*launches;
    if (Z == 1) return cudaSuccess;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)tiles, (unsigned)A.H, CTA_ROWS / JOIN_WARPS), dim3(32 * JOIN_WARPS), 0, st, attr);
    e = cudaLaunchKernelEx(&cfg, k_attn_many_join<CT, D>, A, (const float *)workspace, Z);
    ++*launches;
    return e;
}

}  // namespace many

}  // namespace lsa
