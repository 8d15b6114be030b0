// Attention of one new token per sequence over a paged key-value cache.
//
// Every cached key and value is read once and used by the G = n_heads /
// n_kv_heads queries of its head, so the kernel is a stream over the cache:
// its floor is the cached bytes at the copy rate.
//
// Split. The attended tokens of every (sequence, head tile), a segment, are cut
// into chunks of 8 KB of keys and 8 KB of values. All chunks of the call, numbered
// segment by segment, are dealt out evenly and contiguously to one resident CTA
// per SM and within it to its warps, from the lengths as they stand on the device:
// a ragged batch, one long sequence and thousands of short ones are balanced
// alike, in one launch. A warp that holds a whole segment writes its output; parts
// of a segment that is cut between warps are joined by their CTA at its end, and
// those of one cut between CTAs by the CTA that finishes last, always in order, so
// that results do not depend on which one that is.
//
// A warp copies its chunks by TMA into its own ring of stages (keys and values
// take turns; the swizzle lets ldmatrix read them without bank conflicts) and
// meets no other warp before its end. The copies run ahead over the ends of
// segments: up to 128 KB per SM are in flight, where the copy rate times the
// memory latency asks for 45; more only queues up.
//
// Products. The tokens are the rows of the matrix instruction and the query
// heads its 8 columns (mma m16n8k16), S^T = K Q^T and O^T = V^T P^T: up to 8 heads
// per key-value head cost half of what padding the heads to 16 rows would. P^T is
// turned into the second product's operand by movmatrix. At 2 G FLOP per cached
// byte the legacy tensor path has several times the rate that the copy allows.
// Scores, maxima, sums and outputs are fp32. The weights of a bf16 cache enter the
// second product as two bf16 numbers each, off by 2^-16: rounded to one (2^-8, as much
// as the output's own rounding) they took the output from 1.7e-3 to 2.0e-3 of its norm,
// and the product with the rest is hidden by the stream. (Heads of 256 with more than 8
// queries per key-value head take 10% longer for it, and with a seventh warp 2.5% less.)
// For an e4m3 cache they are rounded once, to fp16 (2^-11, or 2^-39 of the largest
// weight), in which its keys and values are exact, and the queries to 2^-39 of their
// head's largest; the sum is taken before that rounding.
//
// Measured (GB300, inputs larger than L2; copy rate 6.77 TB/s): 131072 tokens of one
// sequence, 48 heads over 8 of 128 channels, 86.5 us, 6.2 TB/s; 64 sequences of up to
// 16384 tokens, pages of 16, 224 us, 6.6 TB/s; 32 windows of 1024 tokens, 16 heads over
// 8 of 256, capped, 38.3 us, 5.3 TB/s; 48 sequences of up to 9001 tokens in 8 bits, 64 heads
// over 4 of 128, 32.6 us, 4.2 TB/s; 17 tokens 5.2 us. What is above the stream's time is the
// chain of reads before the first copy (lengths, block table, keys: 3 us) and the last
// joins (5 to 7 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kv_cache.h"
#include "moe_internal.h"
#include "sm100.cuh"

namespace moe {

namespace {

constexpr int kRing = 16 * 1024;   // bytes of stages per warp
constexpr int kHalf = 8 * 1024;    // of a chunk's keys, or values
constexpr int kMaxCtas = 160;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Compile-time shape of one kernel: head dimension, cache type, query heads / 8.
template <int D_, bool FP8_, int NT_>
struct Cfg {
    static constexpr int D = D_, NT = NT_;
    static constexpr bool FP8 = FP8_;
    static constexpr int RB = D * (FP8 ? 1 : 2);              // bytes of a row
    static constexpr int CT = kHalf / RB;                     // tokens of a chunk
    static constexpr int LINE = RB < 128 ? RB : 128;          // bytes of a shared-memory row (the swizzle's width)
    static constexpr int COLS = RB / LINE;                    // column blocks of a row
    static constexpr int HALF = CT * RB;                      // bytes of a chunk's keys (or values): one stage
    static constexpr int STAGES = kRing / HALF;
    static constexpr int HEADS = 8 * NT;
    static constexpr int MT = CT / 16, KS = D / 16, DT = D / 16;
    static constexpr int UNITS = LINE / 32;                   // 32-byte steps of a line
    static constexpr int STEPS = RB / 32;                     // and of a row
    static constexpr int FRAGS = NT * DT;                     // output fragments of a segment, 32 lanes x float4
    static constexpr int PART = FRAGS * 512;                  // their bytes
    static constexpr int WARPS = FRAGS == 32 ? 7 : 8;         // 7 where the parts of 8 leave no room for their rings
    static constexpr int THREADS = 32 * WARPS;
    // Weights are 2^UP times exp(score - maximum), and so are their sums and outputs: in fp16
    // that leaves 28 octaves below the largest with all 11 bits, where 1 would leave 14.
    static constexpr float UP = FP8 ? 14.f : 0.f, DOWN = FP8 ? 0x1p-14f : 1.f;
    static constexpr size_t smem = 1024 + (size_t)WARPS * kRing + (size_t)(WARPS - 1) * PART;   // the first sets none aside
};

// Every warp comes here once, from the end of its chunks or without any.
template <int THREADS>
__device__ __forceinline__ void warps_meet() {
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

struct AttendArgs {
    moe_kv_attend_args a;
    KvShape s;
    const float *k_scale, *v_scale;
    unsigned* health;
    float4* part_o;     // [CTA][2][FRAGS][32]: unnormalised output fragments
    float4* part_ml;    // [CTA][2][8]: maximum (base two) and sum of two heads
    int* arrived;       // [max_batch * head tiles], zero between calls
    int box_rows;       // tokens of one TMA box
    int boxes_log2;     // boxes of a chunk's column block
    int page_log2;      // of page_size, -1 where it is no power of two
    int G, tiles, HT;   // query heads of a key-value head; head tiles of one, and of all
    int stall;          // MOE_KV_OPT_TEST_STALL
};

__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool FP8>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (FP8)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, "
                     "%9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// two e4m3 values, the lower or upper two bytes of v, as an fp16 pair, exact
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t v) {
    uint32_t d;
    asm("{.reg .b16 h, l; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(d) : "r"(v));
    return d;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t v) {
    uint32_t d;
    asm("{.reg .b16 h, l; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h;}" : "=r"(d) : "r"(v));
    return d;
}
template <bool FP8>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
    if constexpr (FP8) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
// tanh z, off by 8 units of 2^-24 relative to itself: up to 1/2 by an odd polynomial, fitted
// to the least relative error there (1.5e-8), and where PAST, past it, by 1 - 2 / (exp(2 z) +
// 1), whose error of 2^-22 would be the larger the nearer to zero.
template <bool PAST>
__device__ __forceinline__ float tanh_of(float z) {
    const float u = z * z;
    const float r = z * fmaf(fmaf(fmaf(fmaf(0.0172414916f, u, -0.0530454943f), u, 0.13325879f), u, -0.333331439f), u, 1.f);
    if (!PAST || !(fabsf(z) > 0.5f)) return r;
    return 1.f - 2.f * rcp(ex2(z * (2.f * kLog2e)) + 1.f);
}
// Two weights, each as the sum of two bf16 numbers: its upper 16 bits, and the rest
// rounded, 2^-16 of the weight at most. The rest is above zero, so that an infinite value
// times the two is not NaN.
__device__ __forceinline__ void split_pair(float lo, float hi, uint32_t& upper, uint32_t& rest) {
    const uint32_t a = __float_as_uint(lo), b = __float_as_uint(hi);
    upper = __byte_perm(a, b, 0x7632);
    rest = pack_pair<false>(fmaxf(lo - __uint_as_float(a & 0xffff0000u), 0x1p-126f),
                            fmaxf(hi - __uint_as_float(b & 0xffff0000u), 0x1p-126f));
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, int w,
                                            uint32_t bar, uint64_t pol) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
        "l"(tm), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "l"(pol)
        : "memory");
}

// Offset of byte `col` (within one line) of row `row` of a stage: rows of LINE
// bytes, their 16-byte units exchanged as the TMA swizzle does, within 8 of them
// (128-byte lines) or 4 (64-byte lines). Further column blocks follow CT * LINE on.
template <class C>
__device__ __forceinline__ uint32_t line_at(int row, int col) {
    if constexpr (C::LINE == 128) return row * 128 + (col ^ ((row & 7) << 4));
    else return row * 64 + (col ^ (((row >> 1) & 3) << 4));
}

// A segment: sequence b, head tile `tile` of key-value head hk, units [beg, end)
// of the chunk sequence.
struct Place {
    int beg, end, b, hk, tile;
};

// One output fragment (head tile column nt, 16 channels dt) to the output rows
// of `heads` heads from o: called by a whole warp, c and r of heads 2j and 2j + 1.
template <class C>
__device__ __forceinline__ void emit(__nv_bfloat16* o, int heads, int nt, int dt, const float (&c)[4], const float (&r)[2]) {
    const int lane = threadIdx.x % 32, g = lane >> 2, j = lane & 3;
    if constexpr (C::FP8) {   // c[0], c[2]: channels 2g, 2g + 1
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int h = nt * 8 + 2 * j + i;
            if (h < heads)
                *reinterpret_cast<uint32_t*>(o + (int64_t)h * C::D + dt * 16 + 2 * g) =
                    pack_pair<false>(c[i] * r[i], c[i + 2] * r[i]);
        }
    } else {                  // c[0], c[2]: channels g, g + 8
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t v = transpose8(pack_pair<false>(c[2 * i] * r[0], c[2 * i + 1] * r[1]));
            const int h = nt * 8 + g;
            if (h < heads) *reinterpret_cast<uint32_t*>(o + (int64_t)h * C::D + dt * 16 + 8 * i + 2 * j) = v;
        }
    }
}

// One joined output fragment: normalised and written, with the log-sum-exp by the
// warp of a head's first channels.
template <class C>
__device__ __forceinline__ void finish(const AttendArgs& p, int b, int h0, int heads, int nt, int dt, float vs,
                                       const float (&a)[4], const float (&M)[2], const float (&L)[2]) {
    const int lane = threadIdx.x % 32, g = lane >> 2, j = lane & 3;
    const float r[2] = {L[0] == 0.f ? 0.f : vs / L[0], L[1] == 0.f ? 0.f : vs / L[1]};
    const int64_t row = (int64_t)b * p.s.n_heads + h0;
    emit<C>(static_cast<__nv_bfloat16*>(p.a.out) + row * C::D, heads, nt, dt, a, r);
    if (dt == 0 && g == 0 && p.a.lse)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int h = nt * 8 + 2 * j + c;
            if (h < heads) p.a.lse[row + h] = L[c] == 0.f ? -INFINITY : M[c] * kLn2 + logf(L[c] * C::DOWN);
        }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    k_kv_attend(const AttendArgs p, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
    constexpr int NT = C::NT, CT = C::CT, D = C::D, kWarps = C::WARPS, kThreads = C::THREADS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int sm_pre[1025];                // chunks before sequence b
    __shared__ int sm_len[1024];
    __shared__ int sm_wsum[kWarps];
    __shared__ __align__(8) uint64_t sm_bar[kWarps][C::STAGES];
    __shared__ uint32_t sm_rows[kWarps][C::STAGES];  // which groups of 16 rows a stage holds
    __shared__ __align__(16) float2 sm_ml[kWarps][C::HEADS];   // maximum and sum of the parts below
    __shared__ Place sm_cut[2];                      // segments from before and into after the CTA, to be joined here
    __shared__ int sm_on[2], sm_c0[2];               // how many CTAs they have, 0 for none; the first
    __shared__ float2 sm_sum[C::HEADS];
    __shared__ int sm_abort;

    const KvShape& s = p.s;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int g = lane >> 2, j = lane & 3;
    const uint32_t ring0 = (bw::saddr(smem_raw) + 1023) & ~1023u, ring = ring0 + warp * kRing;
    uint32_t bits = 0;

    if (lane < C::STAGES) bw::mbar_init(bw::saddr(&sm_bar[warp][lane]), 1);
    if (threadIdx.x == 0) sm_abort = sm_on[0] = sm_on[1] = 0;
    bw::mbar_fence_init();
    if (threadIdx.x == 0) {
        bw::tma_prefetch_desc(&tm_k);
        bw::tma_prefetch_desc(&tm_v);
    }
    pdl_wait();      // nothing of the caller's is read before the preceding kernel is done
    pdl_trigger();

    // ---- chunks of every sequence, summed ------------------------------------------
    const int G = p.G, tiles = p.tiles, HT = p.HT, B = p.a.B;
    // a sequence attends to tokens [first_of(len), len)
    auto first_of = [&](int len) { return p.a.window > 0 ? max(0, len - p.a.window) : 0; };
    {
        const int most = p.a.max_pages * s.page_size;
        const int per = (B + kThreads - 1) / kThreads;
        const int b0 = threadIdx.x * per, b1 = min(B, b0 + per);
        int mine = 0;
        for (int b = b0; b < b1; ++b) {
            int len = max(p.a.lens[b], 0);
            if (len > most) {
                len = most;
                bits |= MOE_KV_BAD_LENGTH;
            }
            sm_len[b] = len;
            const int n = (len + CT - 1) / CT - first_of(len) / CT;
            sm_pre[b + 1] = n;
            mine += n;
        }
        int incl = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(~0u, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) sm_wsum[warp] = incl;
        __syncthreads();
        int run = incl - mine;
        for (int w = 0; w < warp; ++w) run += sm_wsum[w];
        for (int b = b0; b < b1; ++b) {
            run += sm_pre[b + 1];
            sm_pre[b + 1] = run;
        }
        if (threadIdx.x == 0) sm_pre[0] = 0;
        __syncthreads();
    }
    // Chunks of this CTA, and of its warps. Few chunks go to few CTAs: one or more per
    // warp, and no more CTAs than pay for their join. A chunk costs a CTA about 0.27 us
    // of streaming and each of a segment's parts about 0.045 us of joining (up to 8
    // fragments, 4 KB; in proportion above), so c CTAs on S segments take 0.27 total / c
    // + 0.045 c / S, least at sqrt(6 total S). One sequence of 40189 tokens in 8 bits, 12
    // heads over 1 of 128 (16 fragments): 19.4 us, by the rule for 8 21.6. (Each CTA has
    // some chunks: a segment's CTAs are consecutive.)
    const int total = sm_pre[B] * HT;   // below 2^31: kv_attend_countable
    int ctas = min((int)gridDim.x, (total + kWarps - 1) / kWarps);
    const float sq = 48.f / max(8, C::FRAGS) * total * ((float)B * HT);
    if (sq < (float)ctas * ctas) ctas = (int)ceilf(sqrtf(sq));
    const int me = blockIdx.x;
    const int share = ctas ? total / ctas : 0, rest = total - share * ctas;
    auto cta_beg = [&](int c) { return c * share + min(c, rest); };
    auto cta_of = [&](int u) { return u < rest * (share + 1) ? u / (share + 1) : rest + (u - rest * (share + 1)) / share; };
    const int u0 = me < ctas ? cta_beg(me) : 0, u1 = me < ctas ? cta_beg(me + 1) : 0;
    auto warp_beg = [&](int w) { return u0 + (u1 - u0) * w / kWarps; };
    auto head_of = [&](const Place& q) { return q.hk * G + q.tile * C::HEADS; };
    auto heads_of = [&](const Place& q) { return min(C::HEADS, G - q.tile * C::HEADS); };
    const int w0 = warp_beg(warp), w1 = warp_beg(warp + 1);
    // a warp's part of the segment that began before it; the first warp has none
    float4* part = reinterpret_cast<float4*>(smem_raw + (ring0 - bw::saddr(smem_raw)) + kWarps * kRing);

    // sequences with nothing to attend to
    for (int b = blockIdx.x; b < B; b += gridDim.x) {
        if (sm_pre[b + 1] != sm_pre[b]) continue;
        uint2* o = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.a.out) + (int64_t)b * s.n_heads * D);
        for (int i = threadIdx.x; i < s.n_heads * (D / 4); i += kThreads) o[i] = make_uint2(0, 0);
        if (p.a.lse)
            for (int i = threadIdx.x; i < s.n_heads; i += kThreads) p.a.lse[(int64_t)b * s.n_heads + i] = -INFINITY;
    }

    if (w0 < w1) {
        // the segment of unit w0
        Place at;
        {
            // the first b with sm_pre[b + 1] * HT > w0: the block of `step` it is in, then itself
            const int step = (B + 31) / 32;
            const int blk = __ffs(__ballot_sync(~0u, sm_pre[min(B, (lane + 1) * step)] * HT > w0)) - 1;
            const int lo = blk * step - 1 +
                           __ffs(__ballot_sync(~0u, lane < step && sm_pre[min(B, blk * step + lane + 1)] * HT > w0));
            const int n = sm_pre[lo + 1] - sm_pre[lo], base = sm_pre[lo] * HT, ht = (w0 - base) / n;
            at.b = lo;
            at.hk = tiles == 1 ? ht : ht / tiles;
            at.tile = ht - at.hk * tiles;
            at.beg = base + ht * n;
            at.end = at.beg + n;
        }
        // the next segment
        auto advance = [&](Place& q) {
            const int n = q.end - q.beg;
            q.beg = q.end;
            q.end += n;
            if (++q.tile < tiles) return;
            q.tile = 0;
            if (++q.hk < s.n_kv_heads) return;
            q.hk = 0;
            do ++q.b;
            while (sm_pre[q.b + 1] == sm_pre[q.b]);
            q.end = q.beg + (sm_pre[q.b + 1] - sm_pre[q.b]);
        };

        // ---- the copies of this warp ----------------------------------------------------
        // Stages hold a chunk's keys, then its values, in turn. Box i of either: rows
        // [box * box_rows, ...), one column block; lane i looks its page up a chunk ahead.
        const int boxes = 1 << p.boxes_log2;
        const int bx = lane & (boxes - 1), col = lane >> p.boxes_log2;
        const bool issuer = col < C::COLS;
        // read once, unless further head tiles of the same keys follow
        const uint64_t pol = tiles == 1 ? bw::l2_evict_first() : bw::l2_evict_normal();
        const uint32_t box_bytes = p.box_rows * C::LINE;
        const uint32_t box_at = col * (CT * C::LINE) + bx * box_bytes;
        Place nx = at;             // the chunk whose pages are being looked up
        int nx_page = -1, nx_slot = 0, nx_at = 0;   // of this lane's box; nx_at: its block-table column
        bool nx_live = false, nx_read = false;
        // a segment's queries into L2: the load itself would wait behind the copies in flight
        auto prefetch_q = [&](const Place& q) {
            const int heads = heads_of(q);
            const char* src = reinterpret_cast<const char*>(
                static_cast<const __nv_bfloat16*>(p.a.q) + (int64_t)q.b * p.a.q_stride + (int64_t)head_of(q) * D);
            for (int i = lane * 128; i < heads * D * 2; i += 32 * 128)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(src + i));
        };
        // the pages of unit u: the first one, or the one after the last looked up
        auto lookup = [&](int u, bool start) {
            nx_live = u < w1;
            if (!nx_live) return;
            if (u == nx.end) {
                advance(nx);
                start = true;
            }
            const int len = sm_len[nx.b], first = first_of(len);
            const int tok = (first / CT + u - nx.beg) * CT + bx * p.box_rows;
            if (start) {
                if (u != w0) prefetch_q(nx);
                nx_at = p.page_log2 >= 0 ? tok >> p.page_log2 : tok / s.page_size;
                nx_slot = tok - nx_at * s.page_size;
            } else {
                for (nx_slot += CT; nx_slot >= s.page_size; nx_slot -= s.page_size) ++nx_at;
            }
            // not looked at before the issue, an iteration later
            nx_read = issuer && tok < len && tok + p.box_rows > first;
            nx_page = nx_read ? p.a.block_table[(int64_t)nx.b * p.a.max_pages + nx_at] : -1;
        };
        int ahead = w0;
        int issued = 0, put = 0;   // stages issued, and the stage after them
        auto issue = [&]() {       // the looked-up chunk's keys or values into the next stage
            if (nx_read) nx_page = kv_page(s, nx_page, bits);
            const uint32_t bar = bw::saddr(&sm_bar[warp][put]);
            const unsigned have = __ballot_sync(~0u, nx_page >= 0);
            if (lane == 0) {
                bw::mbar_arrive_tx(bar, __popc(have) * box_bytes);
                uint32_t rows = 0;
                for (int i = 0; i < boxes; ++i)
                    if (have >> i & 1) rows |= ((1u << (p.box_rows / 16)) - 1) << (i * p.box_rows / 16);
                sm_rows[warp][put] = rows;
            }
            __syncwarp();
            if (nx_page >= 0 && nx.b != p.stall)
                tma_load_4d(ring + put * C::HALF + box_at, issued & 1 ? &tm_v : &tm_k, col * (C::FP8 ? 128 : 64), nx_slot,
                            nx.hk, nx_page, bar, pol);
            if (++put == C::STAGES) put = 0;
            if (!(++issued & 1)) lookup(++ahead, false);
        };
        // this lane's rows for ldmatrix: of operand A of K Q^T, and of V^T P^T transposed
        uint32_t ka[C::UNITS], va[C::UNITS];
#pragma unroll
        for (int i = 0; i < C::UNITS; ++i) {
            ka[i] = line_at<C>((lane & 7) + ((lane >> 3) & 1) * 8, i * 32 + (lane >> 4) * 16);
            va[i] = C::FP8 ? ka[i] : line_at<C>((lane & 7) + (lane >> 4) * 8, i * 32 + ((lane >> 3) & 1) * 16);
        }

        // ---- segments ------------------------------------------------------------------
        int take = 0;                    // the stage to be consumed next, and its barrier's phase
        uint32_t phase = 0;
        const float cap2 = fmaxf(p.a.softcap * kLog2e, 1.2e-38f);   // the cap in base two
        int stop = 1;                    // end of the segment's chunks; 0 once a copy did not arrive in time
        auto next_stage = [&]() {        // waits for it; the stage's shared address
            const bool here = bw::mbar_wait(bw::saddr(&sm_bar[warp][take]), phase, &sm_abort, p.health, MOE_KV_TIMEOUT);
            if (!__all_sync(~0u, here)) {
                stop = 0;
                nx_live = false;         // no further copy is started
            }
            return ring + take * C::HALF;
        };
        auto release = [&]() {           // every lane has read it: fill it again
            if (++take == C::STAGES) {
                take = 0;
                phase ^= 1;
            }
            __syncwarp();
            if (nx_live) issue();
        };
        for (int cur = w0;; advance(at)) {
            const int seg_end = min(at.end, w1);
            const int h0 = head_of(at), heads = heads_of(at);
            const int len = sm_len[at.b], first = first_of(len);

            // queries: operand B of S^T = K Q^T (column g of head tile nt)
            uint32_t qf[C::KS][NT][2];
            float coef[NT][2];           // score in base two (or its share of the cap) per accumulator unit, heads 2j and 2j + 1
            float m[NT][2], l[NT][2], o[C::DT][NT][4];
            const float ks_unit = p.k_scale[at.hk], vs = p.v_scale[at.hk];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const bool real = nt * 8 + g < heads;
                const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(p.a.q) + (int64_t)at.b * p.a.q_stride +
                                          (int64_t)(h0 + nt * 8 + g) * D;
#pragma unroll
                for (int ks = 0; ks < C::KS; ++ks) {
                    if constexpr (!C::FP8) {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            qf[ks][nt][i] = real ? *reinterpret_cast<const uint32_t*>(qp + 16 * ks + 2 * j + 8 * i) : 0u;
                    } else {
                        // channels 4j..4j+3 of a step stand at k = 2j, 2j+1, 2j+8, 2j+9, as the
                        // bytes of the keys do
                        const uint2 v = real ? *reinterpret_cast<const uint2*>(qp + 16 * ks + 4 * j) : make_uint2(0, 0);
                        qf[ks][nt][0] = v.x;
                        qf[ks][nt][1] = v.y;
                    }
                }
            }
            // the first copies follow the first queries, which would wait behind them
            if (cur == w0) {
                lookup(w0, true);
                for (int i = 0; i < C::STAGES && nx_live; ++i) issue();
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float unit = 1.f;
                if constexpr (C::FP8) {
                    // a head's queries are scaled by a power of two to below 2^15, where fp16 holds
                    // their 8 bits
                    float top = 0.f;
#pragma unroll
                    for (int ks = 0; ks < C::KS; ++ks)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qf[ks][nt][i] << 16)),
                                                   fabsf(__uint_as_float(qf[ks][nt][i] & 0xffff0000u))));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                    // 2^(14 - e) with e the exponent of top, kept within fp32's normal range
                    const int e = (int)(__float_as_uint(top) >> 23) - 127;
                    const int a = top < INFINITY ? max(-112, min(126, 14 - e)) : 0;
                    const float up = __int_as_float((a + 127) << 23);
                    unit = __int_as_float((127 - a) << 23);
#pragma unroll
                    for (int ks = 0; ks < C::KS; ++ks)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t v = qf[ks][nt][i];
                            qf[ks][nt][i] =
                                pack_pair<true>(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xffff0000u) * up);
                        }
                }
                // a negative scale turns the queries, so that the largest product has the largest score
                if (p.a.scale < 0.f)
#pragma unroll
                    for (int ks = 0; ks < C::KS; ++ks)
#pragma unroll
                        for (int i = 0; i < 2; ++i) qf[ks][nt][i] ^= 0x80008000u;
                const float k = ks_unit * fabsf(p.a.scale);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    coef[nt][c] = k * __shfl_sync(~0u, unit, (2 * j + c) * 4);
                    coef[nt][c] = fmaxf(coef[nt][c] * kLog2e, 1.2e-38f);   // keeps -inf times it -inf
                    if (p.a.softcap != 0.f) coef[nt][c] = fminf(coef[nt][c] / cap2, 3.4e38f);
                    m[nt][c] = -INFINITY;
                    l[nt][c] = 0.f;
                }
#pragma unroll
                for (int dt = 0; dt < C::DT; ++dt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[dt][nt][i] = 0.f;
            }

            if (stop) stop = seg_end;
            for (; cur < stop; ++cur) {
                const int tok0 = (first / CT + cur - at.beg) * CT;
                const uint32_t rows = sm_rows[warp][take];
                const uint32_t kt = next_stage();
                const bool whole = tok0 >= first && tok0 + CT <= len && rows == (1u << C::MT) - 1;

                float sc[C::MT][NT][4];
#pragma unroll
                for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) sc[mt][nt][i] = 0.f;
#pragma unroll
                for (int st = 0; st < C::STEPS; ++st)
#pragma unroll
                    for (int mt = 0; mt < C::MT; ++mt) {
                        uint32_t r[4];
                        ldm4(r, kt + ka[st % C::UNITS] + (st / C::UNITS) * (CT * C::LINE) + mt * 16 * C::LINE);
                        if constexpr (!C::FP8) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma<false>(sc[mt][nt], r, qf[st][nt][0], qf[st][nt][1]);
                        } else {
#pragma unroll
                            for (int k2 = 0; k2 < 2; ++k2) {
                                const uint32_t a[4] = {e4m3_lo(r[2 * k2]), e4m3_lo(r[2 * k2 + 1]), e4m3_hi(r[2 * k2]),
                                                       e4m3_hi(r[2 * k2 + 1])};
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma<true>(sc[mt][nt], a, qf[2 * st + k2][nt][0], qf[2 * st + k2][nt][1]);
                            }
                        }
                    }
                release();

                if (p.a.softcap != 0.f) {   // scores become their share of the cap
                    float most = 0.f;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float x = 0.f;
#pragma unroll
                            for (int mt = 0; mt < C::MT; ++mt)
                                x = fmaxf(x, fmaxf(fabsf(sc[mt][nt][c]), fabsf(sc[mt][nt][c + 2])));
                            most = fmaxf(most, x * coef[nt][c]);
                        }
                    auto cap = [&](auto past) {
#pragma unroll
                        for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int i = 0; i < 4; ++i) sc[mt][nt][i] = tanh_of<past>(sc[mt][nt][i] * coef[nt][i & 1]);
                    };
                    if (__any_sync(~0u, most > 0.5f)) cap(std::true_type{});
                    else cap(std::false_type{});
                }
                // which tokens are attended
                auto seen = [&](int t) {
                    const int tok = tok0 + t;
                    return tok >= first && tok < len && (rows >> (t >> 4) & 1);
                };
                if (!whole) {
#pragma unroll
                    for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {
                            const bool on = seen(mt * 16 + g + i * 4);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int c = 0; c < 2; ++c)
                                    if (!on) sc[mt][nt][i + c] = -INFINITY;
                        }
                }
                // weights: operand B of O^T = V^T P^T; of a bf16 cache the upper halves, and the rest
                uint32_t pf[C::MT][NT][2], pr[C::MT][NT][C::FP8 ? 1 : 2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    // scores in base two are `unit` times sc, unit > 0
                    float unit[2], base[2], low[2], f[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        unit[c] = p.a.softcap != 0.f ? cap2 : coef[nt][c];
                        float x = sc[0][nt][c];
#pragma unroll
                        for (int mt = 0; mt < C::MT; ++mt) x = fmaxf(x, fmaxf(sc[mt][nt][c], sc[mt][nt][c + 2]));
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
                        x = fmaxf(m[nt][c], x * unit[c]);
                        base[c] = x == -INFINITY ? 0.f : x;
                        f[c] = ex2(m[nt][c] - base[c]);
                        low[c] = base[c] - C::UP;
                        m[nt][c] = x;
                        l[nt][c] *= f[c];
                    }
                    if (__any_sync(~0u, f[0] != 1.f || f[1] != 1.f))
#pragma unroll
                        for (int dt = 0; dt < C::DT; ++dt)
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[dt][nt][i] *= f[i & 1];
                    // The base is a rounded product, and the products below are not: past 2^17 that
                    // tells (2^-8 of the weights, and at last their whole range), so that there both are.
                    if (__any_sync(~0u, fabsf(m[nt][0]) > 0x1p17f || fabsf(m[nt][1]) > 0x1p17f)) {
#pragma unroll
                        for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                sc[mt][nt][i] = __fmul_rn(sc[mt][nt][i], unit[i & 1]) - base[i & 1];
                        unit[0] = unit[1] = 1.f;
                        low[0] = low[1] = -C::UP;
                    }
#pragma unroll
                    for (int mt = 0; mt < C::MT; ++mt) {
                        float w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            w[i] = ex2(fmaf(sc[mt][nt][i], unit[i & 1], -low[i & 1]));
                            l[nt][i & 1] += w[i];
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if constexpr (C::FP8) {
                                pf[mt][nt][i] = transpose8(pack_pair<true>(w[2 * i], w[2 * i + 1]));
                            } else {
                                uint32_t u, rest;
                                split_pair(w[2 * i], w[2 * i + 1], u, rest);
                                pf[mt][nt][i] = transpose8(u);
                                pr[mt][nt][i] = transpose8(rest);
                            }
                        }
                    }
                }

                // values: tokens that are not attended may hold anything, so their bits are cleared
                const uint32_t vt = next_stage();
                auto values = [&](auto masked) {
#pragma unroll
                    for (int mt = 0; mt < C::MT; ++mt) {
                        uint32_t keep[2] = {~0u, ~0u};
                        if constexpr (masked)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                keep[i] = (seen(mt * 16 + 8 * i + 2 * j) ? 0xffffu : 0u) |
                                          (seen(mt * 16 + 8 * i + 2 * j + 1) ? 0xffff0000u : 0u);
#pragma unroll
                        for (int st = 0; st < C::STEPS; ++st) {
                            uint32_t r[4];
                            ldm4t(r, vt + va[st % C::UNITS] + (st / C::UNITS) * (CT * C::LINE) + mt * 16 * C::LINE);
                            if constexpr (!C::FP8) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) r[i] &= keep[i >> 1];
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) mma<false>(o[st][nt], r, pf[mt][nt][0], pf[mt][nt][1]);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) mma<false>(o[st][nt], r, pr[mt][nt][0], pr[mt][nt][1]);
                            } else {
#pragma unroll
                                for (int d2 = 0; d2 < 2; ++d2) {
                                    // bytes: channels 2g, 2g + 1 of token 2j, then of token 2j + 1
                                    const uint32_t x = __byte_perm(r[2 * d2], 0, 0x3120);
                                    const uint32_t y = __byte_perm(r[2 * d2 + 1], 0, 0x3120);
                                    const uint32_t a[4] = {e4m3_lo(x) & keep[0], e4m3_hi(x) & keep[0], e4m3_lo(y) & keep[1],
                                                           e4m3_hi(y) & keep[1]};
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt)
                                        mma<true>(o[2 * st + d2][nt], a, pf[mt][nt][0], pf[mt][nt][1]);
                                }
                            }
                        }
                    }
                };
                if (whole) values(std::false_type{});
                else values(std::true_type{});
                release();
            }

            // Without its copies the warp goes through the ends of its segments all the same, so that
            // nothing waits for it, and what it had a part in becomes NaN.
            cur = seg_end;
            if (!stop)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) l[nt][0] = l[nt][1] = NAN;

            // ---- the segment's end ----------------------------------------------------------
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    l[nt][c] += __shfl_xor_sync(~0u, l[nt][c], 4);
                    l[nt][c] += __shfl_xor_sync(~0u, l[nt][c], 8);
                    l[nt][c] += __shfl_xor_sync(~0u, l[nt][c], 16);
                }
            const bool last = at.end >= w1;
            // no copy may land in the rings once the warps have met: every stage's last fill is waited for
            if (last && !stop) {
                int own = 0;
                for (int i = 0; i < C::STAGES && i < issued; ++i)
                    bw::mbar_wait(bw::saddr(&sm_bar[warp][i]), (issued - 1 - i) / C::STAGES & 1, &own, nullptr, 0);
                __syncwarp();
            }
            // A segment that is cut between warps is joined by the first of them, which
            // holds its own part in registers; the others set theirs aside.
            const bool theirs = at.beg < w0 && w0 != u0;
            if (theirs) {
                float4* dst = part + (warp - 1) * (C::FRAGS * 32) + lane;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int dt = 0; dt < C::DT; ++dt)
                        dst[(nt * C::DT + dt) * 32] =
                            make_float4(o[dt][nt][0], o[dt][nt][1], o[dt][nt][2], o[dt][nt][3]);
                    if (g == 0)
                        *reinterpret_cast<float4*>(&sm_ml[warp][nt * 8 + 2 * j]) =
                            make_float4(m[nt][0], l[nt][0], m[nt][1], l[nt][1]);
                }
            }
            if (last) warps_meet<C::THREADS>();
            if (!theirs) {
                // of two CTAs with a segment, this is the second where the other has arrived by now
                int* arrived = p.arrived + (at.b * s.n_kv_heads + at.hk) * tiles + at.tile;
                const int side = at.beg < u0 ? 0 : at.end > u1 ? 1 : -1;
                const int c0 = side < 0 ? me : cta_of(at.beg), n = side < 0 ? 1 : cta_of(at.end - 1) - c0 + 1;
                int before = n == 2 ? *static_cast<volatile int*>(arrived) : 0;
                for (int x = warp + 1; last && x < kWarps && warp_beg(x) < at.end; ++x) {
                    if (warp_beg(x) == warp_beg(x + 1)) continue;
                    const float4* src = part + (x - 1) * (C::FRAGS * 32) + lane;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float4 ml = *reinterpret_cast<const float4*>(&sm_ml[x][nt * 8 + 2 * j]);
                        const float mx[2] = {ml.x, ml.z}, lx[2] = {ml.y, ml.w};
                        float f[2], e[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float top = fmaxf(m[nt][c], mx[c]), base = top == -INFINITY ? 0.f : top;
                            f[c] = ex2(m[nt][c] - base);
                            e[c] = ex2(mx[c] - base);
                            m[nt][c] = top;
                            l[nt][c] = l[nt][c] * f[c] + lx[c] * e[c];
                        }
#pragma unroll
                        for (int dt = 0; dt < C::DT; ++dt) {
                            const float4 v = src[(nt * C::DT + dt) * 32];
                            o[dt][nt][0] = o[dt][nt][0] * f[0] + e[0] * v.x;
                            o[dt][nt][1] = o[dt][nt][1] * f[1] + e[1] * v.y;
                            o[dt][nt][2] = o[dt][nt][2] * f[0] + e[0] * v.z;
                            o[dt][nt][3] = o[dt][nt][3] * f[1] + e[1] * v.w;
                        }
                    }
                }
                before = __shfl_sync(~0u, before, 0);
                bool done = n == 1;
                if (n > 1) {
                    if (before == 0) {
                        float4* dst = p.part_o + (me * 2 + side) * (C::FRAGS * 32) + lane;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                            for (int dt = 0; dt < C::DT; ++dt)
                                __stcg(dst + (nt * C::DT + dt) * 32,
                                       make_float4(o[dt][nt][0], o[dt][nt][1], o[dt][nt][2], o[dt][nt][3]));
                            if (g == 0)
                                __stcg(&p.part_ml[(me * 2 + side) * 8 + nt * 4 + j],
                                       make_float4(m[nt][0], l[nt][0], m[nt][1], l[nt][1]));
                        }
                        __threadfence();
                        __syncwarp();
                        if (lane == 0) before = atomicAdd(arrived, 1);
                        before = __shfl_sync(~0u, before, 0);
                    }
                    if (before == n - 1 && lane == 0) {
                        *arrived = 0;       // for the next call
                        if (n > 2) {        // joined by the whole CTA, below
                            sm_cut[side] = at;
                            sm_on[side] = n;
                            sm_c0[side] = c0;
                        }
                    }
                    // of two CTAs, the warp that comes second adds the other's part
                    if (n == 2) {
                        done = before == 1;
                        if (done) {
                            __threadfence();
                            // the earlier CTA's part is its second, the later one's its first; e0 is the
                            // earlier one's factor, whichever this is
                            const int slot = side ? (me + 1) * 2 : (me - 1) * 2 + 1;
                            const float4* src = p.part_o + slot * (C::FRAGS * 32) + lane;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float4 v[C::DT];
                                const float4 ml = __ldcg(&p.part_ml[slot * 8 + nt * 4 + j]);
#pragma unroll
                                for (int dt = 0; dt < C::DT; ++dt) v[dt] = __ldcg(src + (nt * C::DT + dt) * 32);
                                const float mx[2] = {ml.x, ml.z}, lx[2] = {ml.y, ml.w};
                                float f[2], e[2];
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    const float top = fmaxf(m[nt][c], mx[c]), base = top == -INFINITY ? 0.f : top;
                                    f[c] = ex2(m[nt][c] - base);
                                    e[c] = ex2(mx[c] - base);
                                    m[nt][c] = top;
                                    l[nt][c] = side ? fmaf(lx[c], e[c], l[nt][c] * f[c]) : fmaf(l[nt][c], f[c], lx[c] * e[c]);
                                }
#pragma unroll
                                for (int dt = 0; dt < C::DT; ++dt) {
                                    const float w[4] = {v[dt].x, v[dt].y, v[dt].z, v[dt].w};
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        const float a = o[dt][nt][i], fa = f[i & 1], eb = e[i & 1];
                                        o[dt][nt][i] = side ? fmaf(w[i], eb, a * fa) : fmaf(a, fa, w[i] * eb);
                                    }
                                }
                            }
                        }
                    }
                }
                if (done) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int dt = 0; dt < C::DT; ++dt)
                            finish<C>(p, at.b, h0, heads, nt, dt, vs, o[dt][nt], m[nt], l[nt]);
                    }
                }
            }
            if (last) break;
        }
    } else {
        warps_meet<C::THREADS>();
    }

    // ---- segments of three or more CTAs, by the CTA that finished them -----------------------
    __syncthreads();
    if (sm_on[0] || sm_on[1]) {
        __threadfence();
        for (int side = 0; side < 2; ++side) {
            if (!sm_on[side]) continue;
            const Place q = sm_cut[side];
            const int c0 = sm_c0[side], n = sm_on[side], heads = heads_of(q);
            const float vs = p.v_scale[q.hk];
            // a warp per GO fragments; the first parts are on their way while the warps, a head
            // each, work out the parts' factors
            constexpr int GO = C::FRAGS > kWarps ? 2 : 1, BATCH = 16 / GO, STEP = 2 * C::FRAGS * 32;
            float4 v[GO][BATCH];
            auto fetch = [&](int f0, int i0) {
#pragma unroll
                for (int k = 0; k < GO; ++k) {
                    const int f = f0 + k * kWarps;
                    const float4* src = p.part_o + (c0 + i0) * STEP + f * 32 + lane;
#pragma unroll
                    for (int i = 0; i < BATCH; ++i)
                        if (f < C::FRAGS && i0 + i < n) v[k][i] = __ldcg(src + i * STEP + (i0 + i == 0 ? STEP / 2 : 0));
                }
            };
            fetch(warp, 0);
            float* fac = reinterpret_cast<float*>(smem_raw);   // [n][HEADS]: the rings are idle
#pragma unroll
            for (int h = warp; h < C::HEADS; h += kWarps) {
                float2 ml[kMaxCtas / 32];
                float M = -INFINITY, L = 0.f;
#pragma unroll
                for (int i = 0; i < kMaxCtas / 32; ++i) {
                    const int at = lane + 32 * i;
                    ml[i] = make_float2(-INFINITY, 0.f);
                    if (at < n)
                        ml[i] = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + ((c0 + at) * 2 + (at == 0)) * 16 + h);
                    M = fmaxf(M, ml[i].x);
                }
                for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, x));
                const float mb = M == -INFINITY ? 0.f : M;
#pragma unroll
                for (int i = 0; i < kMaxCtas / 32; ++i) {
                    const float e = ex2(ml[i].x - mb);
                    if (lane + 32 * i < n) fac[(lane + 32 * i) * C::HEADS + h] = e;
                    L += e * ml[i].y;
                }
                for (int x = 16; x; x >>= 1) L += __shfl_xor_sync(~0u, L, x);
                if (lane == 0) sm_sum[h] = make_float2(M, L);
            }
            __syncthreads();
#pragma unroll 1
            for (int f0 = warp; f0 < C::FRAGS; f0 += GO * kWarps) {
                float a[GO][4] = {};
#pragma unroll 1
                for (int i0 = 0; i0 < n; i0 += BATCH) {
                    if (f0 != warp || i0) fetch(f0, i0);
#pragma unroll
                    for (int k = 0; k < GO; ++k) {
                        const float* e = fac + i0 * C::HEADS + (f0 + k * kWarps) % C::FRAGS / C::DT * 8 + 2 * j;
#pragma unroll
                        for (int i = 0; i < BATCH; ++i)
                            if (i0 + i < n) {
                                const float2 x = *reinterpret_cast<const float2*>(e + i * C::HEADS);
                                a[k][0] += x.x * v[k][i].x;
                                a[k][1] += x.y * v[k][i].y;
                                a[k][2] += x.x * v[k][i].z;
                                a[k][3] += x.y * v[k][i].w;
                            }
                    }
                }
#pragma unroll
                for (int k = 0; k < GO; ++k) {
                    const int f = f0 + k * kWarps, h = f / C::DT * 8 + 2 * j;
                    if (f >= C::FRAGS) break;
                    const float M[2] = {sm_sum[h].x, sm_sum[h + 1].x}, L[2] = {sm_sum[h].y, sm_sum[h + 1].y};
                    finish<C>(p, q.b, head_of(q), heads, f / C::DT, f % C::DT, vs, a[k], M, L);
                }
            }
            __syncthreads();   // fac and sm_sum are free again
        }
    }
    if (bits) atomicOr(p.health, bits);
}

template <class C>
cudaError_t launch(const Kv& K, const AttendArgs& p, cudaStream_t stream) {
    return launch_pdl(k_kv_attend<C>, dim3(std::min(K.num_sms, kMaxCtas)), dim3(C::THREADS), C::smem, stream, true, p,
                      K.tm_k, K.tm_v);
}

// The kernel of a cache: more than 8 heads per key-value head share one pass over it
// as 16 columns, more than 16 take further passes.
template <class F>
auto pick(const KvShape& s, F f) {
    const bool two = s.n_heads / s.n_kv_heads > 8;
    if (s.e4m3) {
        if (s.head_dim == 64) return two ? f(Cfg<64, true, 2>{}) : f(Cfg<64, true, 1>{});
        if (s.head_dim == 128) return two ? f(Cfg<128, true, 2>{}) : f(Cfg<128, true, 1>{});
        return two ? f(Cfg<256, true, 2>{}) : f(Cfg<256, true, 1>{});
    }
    if (s.head_dim == 64) return two ? f(Cfg<64, false, 2>{}) : f(Cfg<64, false, 1>{});
    if (s.head_dim == 128) return two ? f(Cfg<128, false, 2>{}) : f(Cfg<128, false, 1>{});
    return two ? f(Cfg<256, false, 2>{}) : f(Cfg<256, false, 1>{});
}

}  // namespace

size_t kv_attend_workspace(const Kv& K, size_t out[3]) {
    const int G = K.s.n_heads / K.s.n_kv_heads;
    const int heads = pick(K.s, [](auto c) { return decltype(c)::HEADS; });
    const size_t part = (size_t)heads * K.s.head_dim * 4;
    out[0] = (size_t)K.num_sms * 2 * part;
    out[1] = (size_t)K.num_sms * 2 * 16 * 8;
    out[2] = (size_t)K.d.max_batch * K.s.n_kv_heads * ((G + heads - 1) / heads) * 4;
    return out[0] + out[1] + out[2];
}

cudaError_t kv_attend_setup(Kv& K) {
    const int ct = pick(K.s, [](auto c) { return decltype(c)::CT; });
    const uint32_t line = pick(K.s, [](auto c) { return decltype(c)::LINE; });
    K.box_rows = 16;
    while (K.box_rows * 2 <= ct && K.s.page_size % (K.box_rows * 2) == 0) K.box_rows *= 2;
    const auto encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const size_t es = K.s.e4m3 ? 1 : 2;
    const cuuint64_t dims[4] = {(cuuint64_t)K.s.head_dim, (cuuint64_t)K.s.page_size, (cuuint64_t)K.s.n_kv_heads,
                                (cuuint64_t)K.s.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)K.s.token_stride * es, (cuuint64_t)K.s.head_stride * es,
                                   (cuuint64_t)K.s.page_stride * es};
    const cuuint32_t box[4] = {(cuuint32_t)(line / es), (cuuint32_t)K.box_rows, 1, 1};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    for (int i = 0; i < 2; ++i)
        if (encode(i ? &K.tm_v : &K.tm_k, K.s.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                   i ? K.v_pages : K.k_pages, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   line == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    return pick(K.s, [](auto c) {
        using C = decltype(c);
        return cudaFuncSetAttribute(k_kv_attend<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::smem);
    });
}

bool kv_attend_countable(const KvShape& s, int B, int max_pages) {
    const int G = s.n_heads / s.n_kv_heads;
    const int ct = pick(s, [](auto c) { return decltype(c)::CT; });
    const int heads = pick(s, [](auto c) { return decltype(c)::HEADS; });
    return ((int64_t)max_pages * s.page_size / ct + 1) * B * s.n_kv_heads * ((G + heads - 1) / heads) <= INT32_MAX;
}

moe_status kv_attend_launch(Kv& K, const moe_kv_attend_args& a, cudaStream_t stream) {
    const int G = K.s.n_heads / K.s.n_kv_heads;
    const int ct = pick(K.s, [](auto c) { return decltype(c)::CT; });
    const int heads = pick(K.s, [](auto c) { return decltype(c)::HEADS; });
    const int tiles = (G + heads - 1) / heads;
    int boxes_log2 = 0, page_log2 = 0;
    while (K.box_rows << boxes_log2 < ct) ++boxes_log2;
    while (1 << page_log2 < K.s.page_size) ++page_log2;
    if (1 << page_log2 != K.s.page_size) page_log2 = -1;
    AttendArgs p{a,         K.s,        K.k_scale, K.v_scale, K.health, K.part_o,               K.part_ml, K.arrived,
                 K.box_rows, boxes_log2, page_log2, G,         tiles,    K.s.n_kv_heads * tiles, K.stall};
    // changes no score below 2^68, and a score's share of it would lose bits
    if (p.a.softcap >= 0x1p80f) p.a.softcap = 0.f;
    const cudaError_t e = pick(K.s, [&](auto c) { return launch<decltype(c)>(K, p, stream); });
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "attend launch");
}

}  // namespace moe
