// Attention of a chunk of new tokens per sequence over a paged key-value cache, on the
// 5th-generation tensor cores.
//
// The rows of a tile are (token, query head) pairs of one key-value head, tokens outermost:
// all G = n_heads / n_kv_heads queries of a head share every key and value that is read, and
// a chunk of few tokens still fills rows. A CTA takes two tiles of 128 rows at a time (heads
// of 256: one) over the same blocks of 128 cached tokens:
//
//   S = Q K^T        both from shared memory, into 128 columns of tensor memory
//   P = exp(S - m)   by a thread per row, its scores in registers, back over S as 16-bit numbers
//   O += P V         P from tensor memory, V from shared memory (rows are K), O stays there
//
// so that the products of one tile run under the softmax of the other. The running maximum
// m is raised only when a row's scores pass it by 2^8: until then the weights are at most
// 2^8 and neither sum nor outputs need a factor. Heads of 256 channels leave room for one
// tile: its two softmax groups take half the columns each, and S has two buffers.
//
// Weights of a bf16 cache enter the second product rounded to bf16 (2^-8 of each at most; the
// sum is taken before the rounding): outputs are 2.0e-3 to 2.3e-3 of their norm from 64 bits,
// of which their own rounding to bf16 is 1.6e-3. Where the handle asks for it (FINE,
// MOE_KV_OPT_CHUNK_WEIGHTS) a second bf16 number holds what the first one left (2^-15), and the
// outputs' own rounding is all: half as many products again, a prompt 733 -> 1020 us, 128 tokens
// far into a document 107 -> 139, drafts 298 -> 433, windows with heads of 256 64 -> 68. Those of an
// 8-bit cache are fp16, in which its keys and values are exact: 1.7e-3, all of it the output's own
// rounding.
//
// Roles. Eight softmax warps; an issuing warp per tile (a wait behind issued products ends only
// when those have left the queue); a warp that walks the CTA's parts for all roles and copies
// keys, one that copies values; four that turn 8-bit stages into 16-bit ones and look through
// values that only some rows see. What bounds a block of two tiles of heads of 128 is its 32
// products at 103 cycles each (64 would be the peak: a product of 128 x 128 x 16 takes 93 at
// least on one CTA) and two hand-overs of 260: 3820 cycles. All loops are kept as loops: the
// first form's 135 KB of instructions were read again and again (13000 misses of the cache for
// them per SM in 41 blocks, 2069 us for a prompt that takes 735).
//
// Split. All blocks of all tiles of the call, numbered tile by tile, are dealt out evenly and
// contiguously to one CTA per SM from the lengths as they stand on the device. A tile that is
// cut between CTAs leaves unnormalised parts in the workspace, which a second, small launch
// joins in order.
//
// Measured (GB300; floors at 1897 TFLOP/s and 6.80 TB/s): a prompt of 8192 tokens, 48 heads
// over 8 of 128, 733 us (1125 TFLOP/s, 59%), in 8 bits 796; 8 x 800 tokens after 7200, 64 heads over
// 4, 1197 TFLOP/s (63%); 128 tokens after 32640 107 us (51%); 64 x 4 tokens after up to 16380, pages
// of 16, 298 us (5.3 TB/s, 78%); 32 ragged chunks in 8 bits 212 us (774 TFLOP/s); 8 chunks of 509 in
// windows of 1024, capped, heads of 256, 64 us; 17 tokens 8.7 us, of which 3.5 before the first copy
// (lengths, the walk, the block table) and most of the rest instructions that run once, where the
// block table holds 512 positions at most, and 11.6 with the second launch where it is wider.
// Heads of 64 do half the operations for the same softmax: a prompt of 8192, 32 over 8, 395 us (37%).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kv_cache.h"
#include "kv_math.cuh"
#include "moe_internal.h"
#include "sm100_more.cuh"

namespace moe {

namespace {

constexpr int kBlk = 128;              // cached tokens of a block
constexpr int kRing = 16;              // blocks whose page flags are kept
constexpr int kParts = 4;              // parts that the roles may be apart
// What a tile's beginning and end cost, in blocks: a prompt of 8192 takes 1047, 855, 727, 733, 743
// and 753 us with 1 to 6, a batch in 8 bits 258, 236, 219, 212, 215 and 218. (About 10000 cycles:
// the last block's edge 2500, the next tile's queries 3500, the outputs 4300; a block is 3800.)
// Other heads have other blocks and other ends, in much the same proportion: with 1, 2, 3, 4, 6 and
// 8 a prompt of 8192 takes 529, 431, 392, 395, 408 and 416 on 32/8 heads of 64, 604, 498, 447, 451, 462
// and 471 on 16/8 of 256, 1221, 1024, 868, 795, 802 and 809 on 48/8 of 128 in 8 bits; windows of heads of
// 256 60, 56, 57, 57, 59 and 60. Four is within 2% of the best of each.
constexpr int kTileCost = 4;

// Compile-time shape of one kernel: head dimension, cache type, capped scores, weights as two
// numbers.
template <int D_, bool FP8_, bool CAP_, bool FINE_ = false>
struct Cfg {
    static constexpr int D = D_;
    static constexpr bool FP8 = FP8_, CAP = CAP_, FINE = FINE_;
    static constexpr int NS = D == 256 ? 1 : 2;          // row tiles in flight
    static constexpr int ROWS = 128 * NS;
    // A block of keys or values of heads of 256 takes two stages: values by tokens, keys by
    // channels, since a product of 128 x 64 takes as long as one of 128 x 128.
    static constexpr int PARTS = D == 256 ? 2 : 1;
    static constexpr int SR = kBlk / PARTS;              // tokens of a stage of values
    static constexpr int KD = D / PARTS;                 // channels of a stage of keys
    static constexpr int PANEL = SR * 128, KPANEL = kBlk * 128;   // a stage is panels of 64 channels
    static constexpr int STAGE = SR * D * 2;
    static constexpr int QPANEL = 128 * 128, QTILE = 128 * D * 2;
    static constexpr int NST = FP8 ? (D == 64 ? 6 : 3) : (D == 64 ? 8 : 4);
    static constexpr int RAW = SR * D, NRAW = FP8 ? 3 : 0;    // 8-bit stages, before conversion
    static constexpr int WARPS = 16, THREADS = 32 * WARPS;
    static constexpr int COLS = NS == 2 ? 128 : 64;      // score columns of a softmax thread
    // Registers of a softmax thread, and of the others: together those of the launch.
    static constexpr int SOFTMAX_REGS = 184, REGS = 72;
    static_assert(256 * SOFTMAX_REGS + (THREADS - 256) * REGS <= THREADS * (65536 / THREADS / 8 * 8), "more registers than launched with");
    static constexpr int O_AT = 256;                     // tensor-memory column of the outputs
    static constexpr int READY = 4;                                // warps that pass a stage on
    // An 8-bit cache is exact in fp16, and so are queries scaled to their row's largest; the
    // weights are 2^7 times their size, at most 2^15: 2^-31 of exp(m) is their smallest step.
    static constexpr float UP = FP8 ? 7.f : 0.f, DOWN = FP8 ? 0x1p-7f : 1.f;
    static constexpr size_t smem = 1024 + (size_t)NS * QTILE + (size_t)NST * STAGE + (size_t)NRAW * RAW;
};

// What a CTA left of a tile that is cut between CTAs.
enum { REC_CUT = 1, REC_FIRST = 2, REC_LAST = 4 };
struct Rec {
    int flags, rows, row0, start, hk, pad[3];
};

// Division of 0 <= x < 2^31 by a number of 1..4096 that the launch knows: the quotient by its
// rounded-up reciprocal 2^k / d, exact since d <= 2^(k - 31). (A division in the kernel is
// twenty instructions, and the cache for those is what the roles wait for.)
struct Div {
    uint32_t m;
    int k, d;
    explicit Div(int by) : m(0), k(31), d(by) {
        while ((1 << (k - 31)) < by) ++k;
        m = (uint32_t)((((uint64_t)1 << k) + by - 1) / by);
    }
    __device__ __forceinline__ int of(int x) const { return (int)((uint64_t)(uint32_t)x * m >> k); }
    __device__ __forceinline__ int rest(int x) const { return x - of(x) * d; }
};

struct ChunkArgs {
    moe_kv_chunk_args a;
    KvShape s;
    const void* v_pages;
    const float *k_scale, *v_scale;
    unsigned* health;
    Rec* recs;          // [CTA][2]
    float2* part_ml;    // [CTA][2][ROWS]: maximum (base two) and sum
    float4* part_o;     // [CTA][2][D / 4][ROWS]
    Div G, page;        // query heads of a key-value head, tokens of a page
    int box_rows, stall;   // MOE_KV_OPT_TEST_STALL
    bool whole;         // tiles are not cut: their blocks are few
};

// The blocks of one tile that a CTA takes.
struct Part {
    int b, hk, row0, rows;    // rows of the sequence's (token, head) pairs
    int start, base;          // the sequence's first token row; position of its first new token
    int lo, hi;               // positions that some row attends to
    int all_lo, all_hi;       // positions that every row attends to
    int blk0, n;              // blocks
    int index, busy, gi;      // parts, parts with blocks, and blocks of this CTA before
    bool first, last;         // blocks of the tile are among them
    bool none;                // the tile has no blocks at all
};

// Walks a CTA's parts: by the warp that copies keys, for all roles.
template <class C>
struct Walk {
    const int *start, *len;   // shared memory
    Div G;
    int Hk, window, b, i, hk, off, index, busy, gi;
    bool whole;               // a unit is a tile, not a block
    long long left;

    __device__ __forceinline__ static int blocks_of(int lo, int hi) { return hi > lo ? (hi + kBlk - 1) / kBlk - lo / kBlk : 0; }
    __device__ __forceinline__ static int first_seen(int pos, int window) { return window > 0 && pos >= window ? pos - window + 1 : 0; }

    __device__ __forceinline__ bool next(Part& q) {
        if (left <= 0) return false;
        const int n = start[b + 1] - start[b], R = n * G.d;
        q.b = b;
        q.hk = hk;
        q.row0 = i * C::ROWS;
        q.rows = min(R - q.row0, C::ROWS);
        q.start = start[b];
        q.base = len[b] - n;
        const int p0 = q.base + G.of(q.row0), p1 = q.base + G.of(q.row0 + q.rows - 1);
        q.lo = first_seen(p0, window);
        q.hi = p1 + 1;
        q.all_lo = first_seen(p1, window);
        q.all_hi = p0 + 1;
        const int c = blocks_of(q.lo, q.hi), units = c + kTileCost;
        const int take = whole ? units : (int)min((long long)(units - off), left);
        const int b0 = max(off - kTileCost, 0), b1 = max(off + take - kTileCost, 0);
        q.blk0 = q.lo / kBlk + b0;
        q.n = b1 - b0;
        q.first = b0 == 0;
        q.last = b1 == c;
        q.none = c == 0;
        q.index = index++;
        q.busy = busy;
        busy += q.n > 0;
        q.gi = gi;
        gi += q.n;
        left -= whole ? 1 : take;
        off += take;
        if (off == units) {
            off = 0;
            if (++hk == Hk) {
                hk = 0;
                if (++i > (R - 1) / C::ROWS) {
                    i = 0;
                    if (left > 0)
                        do ++b;
                        while (start[b + 1] == start[b]);
                }
            }
        }
        return true;
    }
};

template <class T>
__device__ __forceinline__ T scan_up(T v) {   // inclusive, over a warp
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(~0u, v, o);
        if ((int)(threadIdx.x % 32) >= o) v += u;
    }
    return v;
}
// Sum of v over the threads before this one, and over all of them.
template <class T, int WARPS>
__device__ __forceinline__ T scan_cta(T v, T* sums, T& total) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const T incl = scan_up(v);
    __syncthreads();
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    const T w = scan_up(lane < WARPS ? sums[lane] : T(0));
    total = __shfl_sync(~0u, w, WARPS - 1);
    const T before = __shfl_sync(~0u, w, max(warp - 1, 0));
    return incl - v + (warp ? before : T(0));
}

// The registers of a thread from here on, for the warps of a group of four together.
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// the same of two numbers by one, in place
__device__ __forceinline__ void put2(float& a, float& b, float2 v) { a = v.x, b = v.y; }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ void fma_in(float& a, float& b, float y, float z) { put2(a, b, fma2(make_float2(a, b), both(y), both(z))); }
__device__ __forceinline__ void add_in(float& a, float& b, float y, float z) { put2(a, b, add2(make_float2(a, b), make_float2(y, z))); }
// cap tanh(k x) of two scores, as tanh_of has it, on both sides and without a branch: scores lie
// on either.
__device__ __forceinline__ void tanh_cap(float& x0, float& x1, float k, float cap) {
    const float2 x = mul2(make_float2(x0, x1), both(k)), u = mul2(x, x);
    float2 n = fma2(fma2(fma2(fma2(both(kTanh9), u, both(kTanh7)), u, both(kTanh5)), u, both(kTanh3)), u, both(1.f));
    n = mul2(n, x);
    float2 e = mul2(x, both(2.f * kLog2e));
    e = add2(make_float2(ex2(e.x), ex2(e.y)), both(1.f));
    e = fma2(make_float2(rcp(e.x), rcp(e.y)), both(-2.f), both(1.f));
    put2(x0, x1, mul2(make_float2(fabsf(x.x) > 0.5f ? e.x : n.x, fabsf(x.y) > 0.5f ? e.y : n.y), both(cap)));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        return pack_bf16(lo, hi);
    }
}
// Two weights, neither negative, as two bf16 numbers each: their upper 16 bits, and what those
// leave, rounded (2^-8 of 2^-7 of the weight). 2^-20 of the weight is added to that, so that it is
// not zero where the weight is not: an infinite value times either has the same sign.
__device__ __forceinline__ void split2(float a, float b, uint32_t& upper, uint32_t& rest) {
    upper = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    auto minus = [](float x) { return __uint_as_float((__float_as_uint(x) & 0xffff0000u) | 0x80000000u); };   // its upper bits
    const float2 left = fma2(make_float2(a, b), both(1.f + 0x1p-20f), make_float2(minus(a), minus(b)));
    rest = pack_bf16(left.x, left.y);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint4 ld_shared(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// The upper bit of every byte that is an e4m3 NaN (0x7f, 0xff): the sum carries into it.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t x) { return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ bool all_lanes(bool x) { return __all_sync(~0u, x) != 0; }

// v[c] of the row of this lane becomes v[r]: vector lane % 4 of the r-th row of its four lanes.
__device__ __forceinline__ void turn4(uint4 (&v)[4], int lane) {
    auto swap = [&](uint4& keep0, uint4& keep1, int by) {   // what the other lane gave comes back
        uint32_t* const x = reinterpret_cast<uint32_t*>(&keep0);
        uint32_t* const y = reinterpret_cast<uint32_t*>(&keep1);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t got = __shfl_xor_sync(~0u, lane & by ? x[e] : y[e], by);
            if (lane & by) x[e] = got;
            else y[e] = got;
        }
    };
    swap(v[0], v[2], 2);
    swap(v[1], v[3], 2);
    swap(v[0], v[1], 1);
    swap(v[2], v[3], 1);
}

__device__ __forceinline__ float max32(const float* x, float top) {
    float m[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 32; i += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = fmaxf(m[k], fmaxf(x[i + 2 * k], x[i + 2 * k + 1]));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// Stages in the order of their use. A 16-bit cache has a ring for keys and one for values, each
// filled by a warp of its own (on one ring a warp could take a stage's phase for the one two
// before); an 8-bit cache has one of each kind, filled in order by one warp.
template <bool SPLIT, int N>
struct Turn {
    uint32_t n[2] = {0, 0}, stage, use;   // use: how often the stage was in use before
    __device__ __forceinline__ void take(bool values) {
        const int r = SPLIT && values;
        constexpr int EACH = SPLIT ? N / 2 : N;
        stage = r * EACH + n[r] % EACH;
        use = n[r]++ / EACH;
    }
};

// The stages of a part in the order in which the products take them: f(values?, block).
template <class C, class F>
__device__ __forceinline__ void each_block(int n, F f) {
#pragma unroll 1
    for (int i = 0; i < 2 * n; ++i) {
        if (C::NS == 2) {
            f((i & 1) != 0, i >> 1);
        } else {   // keys are a block ahead
            const int t = i >> 1;
            const bool values = i & 1 ? t + 1 == n : i > 0;
            f(values, i & 1 ? (values ? t : t + 1) : max(t - 1, 0));
        }
    }
}

template <class C>
struct Shared {
    uint64_t full[C::FP8 ? C::NRAW : C::NST], raw_free[4], ready[C::NST], empty[C::NST];
    uint64_t q_full[2], s_full[2], p_full[2], o_done[2], o_last[2], o_free[2], drain;
    uint64_t part_full[kParts], part_free[kParts], pair[4], order[2];
    Part part[kParts + 1];            // as the keys' copies go ahead; one of -1 blocks is the last, as is the one past them
    long long sums[C::WARPS];
    long long rem;                    // where this CTA's first tile starts, in units
    struct {
        long long left;
        int b, i, hk, off;
    } share;                          // where this CTA's walk begins
    uint32_t tmem;
    int abort, bad_start, first;
    int lost;                         // some page was not in the pool
    uint8_t pages[kRing][2];          // per block and part: groups of 16 tokens whose page is in the pool
    uint8_t odd[8][4];                // per part and warp: values that are not finite were set aside
    float row_max[2][2][C::NS == 1 ? 128 : 1], row_sum[2][C::NS == 1 ? 128 : 1];
    int start[1025], len[1024];
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    k_kv_chunk(const ChunkArgs p, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
    constexpr int D = C::D, NST = C::NST, G16 = C::SR / 16;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(16) Shared<C> sm;
    const KvShape& s = p.s;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, B = p.a.B;
    const Div& G = p.G;
    const uint32_t base = (bw::saddr(smem_raw) + 1023) & ~1023u;
    const uint32_t q_at = base, stages = base + C::NS * C::QTILE, raws = stages + NST * C::STAGE;
    const uint32_t full = bw::saddr(sm.full), raw_free = bw::saddr(sm.raw_free), ready = bw::saddr(sm.ready),
                   empty = bw::saddr(sm.empty), q_full = bw::saddr(sm.q_full), s_full = bw::saddr(sm.s_full),
                   p_full = bw::saddr(sm.p_full), o_done = bw::saddr(sm.o_done), o_last = bw::saddr(sm.o_last), o_free = bw::saddr(sm.o_free),
                   drain = bw::saddr(&sm.drain), part_full = bw::saddr(sm.part_full), part_free = bw::saddr(sm.part_free),
                   pair = bw::saddr(sm.pair), order = bw::saddr(sm.order);
    uint32_t bits = 0;

    if (threadIdx.x == 0) {
#pragma unroll 1
        for (int i = 0; i < NST; ++i) {
            if (!C::FP8) bw::mbar_init(full + 8 * i, 1);
            bw::mbar_init(ready + 8 * i, C::READY);
            bw::mbar_init(empty + 8 * i, C::NS);
        }
#pragma unroll 1
        for (int i = 0; i < C::NRAW; ++i) {
            bw::mbar_init(full + 8 * i, 1);
            bw::mbar_init(raw_free + 8 * i, 4);
        }
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            bw::mbar_init(q_full + 8 * i, C::NS == 2 ? 4 : 8);
            bw::mbar_init(s_full + 8 * i, 1);
            bw::mbar_init(p_full + 8 * i, C::NS == 2 ? 4 : 8);
            bw::mbar_init(o_done + 8 * i, 1);
            bw::mbar_init(o_last + 8 * i, 1);
            bw::mbar_init(o_free + 8 * i, C::NS == 2 ? 4 : 8);
        }
        bw::mbar_init(drain, C::NS);
        bw::mbar_init(order, 1);
        bw::mbar_init(order + 8, 1);
#pragma unroll 1
        for (int i = 0; i < kParts; ++i) {
            bw::mbar_init(part_full + 8 * i, 1);
            bw::mbar_init(part_free + 8 * i, 8 + C::NS + C::READY + (C::FP8 ? 0 : 1));
            bw::mbar_init(pair + 8 * i, 2);
        }
        sm.part[kParts].n = -1;
        sm.abort = sm.bad_start = sm.lost = 0;
        bw::mbar_fence_init();
        bw::tma_prefetch_desc(&tm_k);
        bw::tma_prefetch_desc(&tm_v);
    }
    if (warp == 8) bw::tmem_alloc(bw::saddr(&sm.tmem), 512);
    bw::tc_fence_before();
    __syncthreads();
    bw::tc_fence_after();
    const uint32_t tmem = *const_cast<volatile uint32_t*>(&sm.tmem);
    pdl_wait();      // nothing of the caller's is read before the preceding kernel is done
    pdl_trigger();

    // ---- tiles of every sequence, blocks of every tile, this CTA's share of them ---------------
    Walk<C> walk{nullptr, nullptr, p.G};
    {
        int* const pre = reinterpret_cast<int*>(smem_raw + (base - bw::saddr(smem_raw)));   // tiles before a sequence
        const int most = p.a.max_pages * s.page_size;
        const int per = (B + C::THREADS - 1) / C::THREADS, b0 = threadIdx.x * per, b1 = min(B, b0 + per);
        int mine = 0;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const int s0 = p.a.starts[b], s1 = p.a.starts[b + 1];
            int len = max(p.a.lens[b], 0);
            if (len > most) {
                len = most;
                bits |= MOE_KV_BAD_LENGTH;
            }
            if (s0 < 0 || s1 < s0 || s1 > p.a.T) sm.bad_start = 1;
            sm.start[b] = s0;
            if (b == B - 1) sm.start[B] = s1;
            sm.len[b] = len;
            mine += s1 > s0 ? ((s1 - s0) * G.d - 1) / C::ROWS + 1 : 0;
        }
        long long tiles;
        long long run = scan_cta<long long, C::WARPS>(mine, sm.sums, tiles);
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            pre[b] = (int)run;
            const int n = sm.start[b + 1] - sm.start[b];
            run += n > 0 ? (n * G.d - 1) / C::ROWS + 1 : 0;
        }
        if (threadIdx.x == 0) pre[B] = (int)tiles;
        __syncthreads();
        // units of tile r: its blocks, and what goes before and after them
        auto find = [&](int r) {
            int lo = 0, hi = B;   // the last b with pre[b] <= r that has tiles
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (pre[mid] <= r) lo = mid;
                else hi = mid;
            }
            return lo;
        };
        auto per_head = [&](int r) {
            const int b = find(r), n = sm.start[b + 1] - sm.start[b], row0 = (r - pre[b]) * C::ROWS;
            const int p0 = sm.len[b] - n + G.of(row0), p1 = sm.len[b] - n + G.of(min(row0 + C::ROWS, n * G.d) - 1);
            return p.whole ? 1 : Walk<C>::blocks_of(Walk<C>::first_seen(p0, p.a.window), p1 + 1) + kTileCost;
        };
        walk.left = 0;
        if (!sm.bad_start) {
            const int rt = (int)tiles;
            long long total = 0, sum = 0, chunk = 0, at = 0;
#pragma unroll 1
            for (int r = threadIdx.x; r < rt; r += C::THREADS) sum += (long long)per_head(r) * s.n_kv_heads;
            at = scan_cta<long long, C::WARPS>(sum, sm.sums, total);   // (of use where a thread has one tile)
            const long long ctas = min((long long)gridDim.x, total), c = blockIdx.x;
            // an even share, the first `more` CTAs one unit more (one 64-bit division)
            const long long each = ctas ? total / ctas : 0, more = total - each * ctas;
            const long long from = c < ctas ? each * c + min(c, more) : total, to = c < ctas ? from + each + (c < more) : total;
            walk.left = to - from;
            long long before = 0;
#pragma unroll 1
            for (int r0 = 0; walk.left > 0 && r0 < rt && before <= from; r0 += C::THREADS) {
                const int r = r0 + threadIdx.x;
                long long u = sum;
                if (rt > C::THREADS) {
                    u = r < rt ? (long long)per_head(r) * s.n_kv_heads : 0;
                    at = before + scan_cta<long long, C::WARPS>(u, sm.sums, chunk);
                    before += chunk;
                }
                if (at <= from && from < at + u) {
                    sm.first = r;
                    sm.rem = from - at;
                }
            }
            __syncthreads();
            if (walk.left > 0) {
                const int r = sm.first, b = find(r), u = per_head(r);
                walk.b = b;
                walk.i = r - pre[b];
                walk.hk = 0;
#pragma unroll 1
                for (long long left = sm.rem; left >= u || (walk.off = (int)left, false); left -= u) ++walk.hk;
            }
        } else if (threadIdx.x == 0) {
            bits |= MOE_KV_BAD_START;
        }
        walk.start = sm.start;
        walk.len = sm.len;
        walk.Hk = s.n_kv_heads;
        walk.window = p.a.window;
        walk.whole = p.whole;
        walk.index = walk.busy = walk.gi = 0;
        if (threadIdx.x == 0) sm.share = {walk.left, walk.b, walk.i, walk.hk, walk.off};
        bw::fence_async_smem();   // `pre` lies where copies will land
        __syncthreads();
    }
    auto wait = [&](uint32_t bar, uint32_t parity) {
        return all_lanes(bw::mbar_wait_short(bar, parity & 1, &sm.abort));
    };

    // A wait that runs out sets sm.abort, which ends all others: a role then leaves, arrives nowhere
    // any more (a barrier may have no arrivals left in its phase) and writes nothing shared; the
    // softmax warps fill the CTA's rows with NaN at their end.
    // The parts in their order: n is the reader's own count, and what it took it gives back.
    auto take = [&](uint32_t n) -> const volatile Part& {
        return sm.part[wait(part_full + 8 * (n % kParts), n / kParts) ? n % kParts : kParts];
    };
    auto give = [&](uint32_t n) {
        __syncwarp();
        if (lane == 0) bw::mbar_arrive(part_free + 8 * (n % kParts));
    };

    if (warp >= 8) regs_down<C::REGS>();
    if (warp == 9 || (!C::FP8 && warp == 10)) {
        // ---- copies: of keys by one warp, of values by another. A lane looks up a box's page a
        // block ahead, one lane starts the copies ------------------------------------------------------
        constexpr int RING = C::FP8 ? C::NRAW : NST, BYTES = C::FP8 ? C::RAW : C::STAGE;
        const bool keys = warp == 9, vals = C::FP8 || warp == 10;   // whose copies this warp starts
        const uint32_t at = C::FP8 ? raws : stages, gone = C::FP8 ? raw_free : empty;
        const int boxes = C::SR / p.box_rows;
        const uint64_t pol = bw::l2_evict_normal();
        // lane: box `lane` of the block's keys (or values), all of whose channels it stands for
        struct Box {
            int page, slot;   // as the table has it; -1 where no row is attended to
            bool need;
        };
        struct Piece {
            int b, hk, lo, hi, blk0, n, gi;
        };
        auto look_up = [&](const Piece& q, int j) {
            const int pos = (q.blk0 + j) * kBlk + lane * p.box_rows;
            Box x;
            x.need = lane < boxes * C::PARTS && pos < q.hi && pos + p.box_rows > q.lo;
            const int i = p.page.of(pos);
            x.slot = pos - i * s.page_size;
            x.page = x.need ? p.a.block_table[(int64_t)q.b * p.a.max_pages + i] : -1;
            return x;
        };
        uint32_t parts = 0;
        bool ok = true;
        // the next part with blocks; the keys' warp finds it for all, and writes the rows of tiles
        // that have no blocks at all
        auto advance = [&](Piece& q) {
            if (keys) {
                Part x;
#pragma unroll 1
                for (;;) {
                    if (!walk.next(x)) {
                        x.n = -1;
                        break;
                    }
                    if (x.n) break;
                    if (!x.none) continue;
#pragma unroll 1
                    for (int r = lane; r < x.rows; r += 32) {
                        const int64_t o = (int64_t)(x.start + G.of(x.row0 + r)) * s.n_heads + x.hk * G.d + G.rest(x.row0 + r);
                        uint4* const to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.out) + o * D);
#pragma unroll 1
                        for (int i = 0; i < D / 8; ++i) to[i] = make_uint4(0, 0, 0, 0);
                        if (p.a.lse) p.a.lse[o] = -INFINITY;
                    }
                }
                ok = wait(part_free + 8 * (parts % kParts), parts / kParts + 1) && ok;
                if (!ok) return false;
                if (lane == 0) {
                    sm.part[parts % kParts] = x;
                    bw::mbar_arrive(part_full + 8 * (parts % kParts));
                }
                // its queries on their way to the second-level cache while the part before it runs
                if (parts && x.n > 0) {
                    const int last = G.of(x.row0 + x.rows - 1);
#pragma unroll 1
                    for (int t = G.of(x.row0) + lane; t <= last; t += 32)
                        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                                         static_cast<const __nv_bfloat16*>(p.a.q) + (x.start + t) * p.a.q_stride + x.hk * G.d * D),
                                     "r"(G.d * D * 2)
                                     : "memory");
                }
                q = Piece{x.b, x.hk, x.lo, x.hi, x.blk0, x.n, x.gi};
            } else {
                const volatile Part& x = take(parts);
                q = Piece{x.b, x.hk, x.lo, x.hi, x.blk0, x.n, x.gi};
                if (q.n < 0) return false;
                give(parts);
            }
            ++parts;
            return q.n > 0;
        };
        Turn<!C::FP8, RING> turn;
        uint32_t filled = 0, phases = 0;   // stages with a copy of this warp's, and the parity of its phase
        Piece q, nq;
        bool have = advance(q);
        Box ahead{}, seen[2] = {};   // of the next block; of keys that came, for their values
        if (have) ahead = look_up(q, 0);
#pragma unroll 1
        while (have) {
            const bool more = advance(nq);
            each_block<C>(q.n, [&](bool values, int j) {
                if (!(values ? vals : keys) || !ok) return;
                Box x = ahead;
                if (values && keys) {
                    x = j & 1 ? seen[1] : seen[0];
                } else {
                    if (j & 1) seen[1] = x;
                    else seen[0] = x;
                    if (j + 1 < q.n) ahead = look_up(q, j + 1);
                    else if (more) ahead = look_up(nq, 0);
                }
                const int page = x.need ? kv_page(s, x.page, bits) : -1;
                const uint32_t lost = __ballot_sync(~0u, x.need && page < 0), come = __ballot_sync(~0u, page >= 0);
                if (!values && lane < C::PARTS) {
                    uint32_t groups = (1u << G16) - 1;
#pragma unroll 1
                    for (int g = 0; lost && g < G16; ++g)
                        if (lost >> (lane * boxes + g * 16 / p.box_rows) & 1) groups &= ~(1u << g);
                    sm.pages[(q.gi + j) % kRing][lane] = (uint8_t)groups;
                    if (lost) *const_cast<volatile int*>(&sm.lost) = 1;
                }
                __syncwarp();
#pragma unroll
                for (int part = 0; part < C::PARTS; ++part) {
                    turn.take(values);
                    const uint32_t bar = full + 8 * turn.stage, to = at + turn.stage * BYTES;
                    ok = wait(gone + 8 * turn.stage, turn.use + 1) && ok;
                    if (!ok) return;
                    const bool stalled = q.b == p.stall;
                    if (!stalled) filled |= 1u << turn.stage;
                    phases = (phases & ~(1u << turn.stage)) | (turn.use & 1) << turn.stage;
                    // boxes of this stage, and their panels
                    const int b0 = values ? part * boxes : 0, b1 = values ? b0 + boxes : C::PARTS * boxes;
                    const int x0 = values ? 0 : part * C::KD, width = values ? D : C::KD;
                    const uint32_t box_bytes = p.box_rows * (C::FP8 ? width : 128);
                    if (bw::elect_one())
                        bw::mbar_arrive_tx(bar, __popc(come >> b0 & ((1u << (b1 - b0)) - 1)) * p.box_rows * width * (C::FP8 ? 1 : 2));
#pragma unroll 1
                    for (int box = b0; box < b1; ++box) {
                        const int from = __shfl_sync(~0u, page, box), slot = __shfl_sync(~0u, x.slot, box);
                        if (from >= 0 && !stalled && bw::elect_one())
#pragma unroll
                            for (int c = 0; c < (C::FP8 ? 1 : D / 64); ++c)
                                if (C::FP8 || c * 64 < width)
                                    bw::tma_load_4d(to + c * (values ? C::PANEL : C::KPANEL) + (box - b0) * box_bytes,
                                                    values ? &tm_v : &tm_k, x0 + 64 * c, slot, q.hk, from, bar, pol);
                    }
                    __syncwarp();
                }
            });
            q = nq;
            have = more && ok;
        }
        // no copy is in flight at the end, after a wait that ran out either
        int none = 0;
#pragma unroll 1
        for (int i = 0; i < RING; ++i)
            if (filled >> i & 1) bw::mbar_wait_short(full + 8 * i, phases >> i & 1, &none);
    } else if (warp == 8 || (C::NS == 2 && warp == 11)) {
        // ---- products ------------------------------------------------------------------------------
        constexpr uint32_t id_qk = bw::idesc_16_f32(128, kBlk, !C::FP8), id_pv = bw::idesc_16_f32(128, D, !C::FP8, true);
        Turn<!C::FP8, NST> turn;
        uint32_t parts = 0, uses = 0, steps = 0;   // of this tile: parts, blocks, turns with the other
        const int slot = warp == 8 ? 0 : 1;
        bool ok = true;
        // one lane issues; descriptors differ from step to step in their address alone
        auto scores = [&](int slot, uint32_t stage, uint32_t to, int part) {
            if (ok && bw::elect_one()) {
                const uint64_t a = bw::desc_sw128(q_at + slot * C::QTILE + part * (C::KD / 64) * C::QPANEL), b = bw::desc_sw128(stages + stage * C::STAGE);
#pragma unroll
                for (int k = 0; k < C::KD / 16; ++k)
                    bw::mma_f16(to, a + ((k / 4) * C::QPANEL + (k % 4) * 32) / 16, b + ((k / 4) * C::KPANEL + (k % 4) * 32) / 16, id_qk,
                                part > 0 || k > 0);
            }
            __syncwarp();
        };
        auto outputs = [&](uint32_t weights, uint32_t stage, uint32_t to, bool more) {
            if (ok && bw::elect_one()) {
                const uint64_t b = bw::desc_sw128_mn(stages + stage * C::STAGE, C::PANEL);
#pragma unroll
                for (int k = 0; k < C::SR / 16; ++k) bw::mma_f16_ta(to, weights + 8 * k, b + k * (2048 / 16), id_pv, more || k > 0);
                if constexpr (C::FINE)
#pragma unroll
                    for (int k = 0; k < C::SR / 16; ++k) bw::mma_f16_ta(to, weights + C::COLS / 2 + 8 * k, b + k * (2048 / 16), id_pv, true);
            }
            __syncwarp();
        };
        auto commit = [&](uint32_t bar) {
            if (ok && bw::elect_one()) bw::mma_commit(bar);
            __syncwarp();
        };
        auto stage_in = [&](bool values) {
            turn.take(values);
            ok = wait(ready + 8 * turn.stage, turn.use) && ok;
            bw::tc_fence_after();
            return turn.stage;
        };
        struct {
            int n, rows;
        } q;
#pragma unroll 1
        for (uint32_t part = 0;; ++part) {
            const volatile Part& x = take(part);
            q = {x.n, x.rows};
            if (q.n < 0 || !ok) break;
            give(part);
            // Block j's weights by its values, then block j + 1's queries by keys, so that one
            // tile's products run while the other's scores become weights. Each tile has an issuing
            // warp: a wait behind issued products ends only when those have left the queue, and
            // one warp for both left gaps of 400 and 680 cycles in a block's 3000.
            if constexpr (C::NS == 2) {
                const bool two = q.rows > 128;
                if (slot && !two) {   // not there: pass the stages on, one by one, so as not to lose count
                    each_block<C>(q.n, [&](bool values, int) {
                        const uint32_t st = stage_in(values);
                        if (ok && bw::elect_one()) bw::mbar_arrive(empty + 8 * st);
                        __syncwarp();
                    });
                    continue;
                }
#pragma unroll 1
                for (int j = -1; j < q.n && ok; ++j) {   // (-1: scores alone)
                    if (j < 0) {
                        ok = wait(q_full + 8 * slot, parts) && ok;
                    } else {
                        const uint32_t v = stage_in(true);
                        if (j == 0) ok = wait(o_free + 8 * slot, parts++ + 1) && ok;
                        // in turns, the first tile first: left alone, both tiles' products mix and
                        // both softmaxes wait for them at the same time (4900 cycles a block)
                        if (two) ok = wait(order + 8 * slot, slot ? steps : steps + 1) && ok;
                        steps += two;
                        ok = wait(p_full + 8 * slot, uses++) && ok;
                        bw::tc_fence_after();
                        outputs(tmem + slot * 128, v, tmem + C::O_AT + slot * D, j > 0);
                        commit(o_done + 8 * slot);
                        commit(empty + 8 * v);
                        if (j + 1 == q.n) commit(o_last + 8 * slot);
                    }
                    if (j + 1 < q.n) {
                        const uint32_t k = stage_in(false);
                        scores(slot, k, tmem + slot * 128, 0);
                        commit(s_full + 8 * slot);
                        commit(empty + 8 * k);
                    }
                    if (two && j >= 0) {
                        if (ok && bw::elect_one()) bw::mbar_arrive(order + 8 * (slot ^ 1));
                        __syncwarp();
                    }
                }
            } else {
                // the next block's scores go before this one's outputs: they have a buffer of their own
#pragma unroll 1
                for (int j = -1; j < q.n && ok; ++j) {
                    const uint32_t use = uses + (j < 0 ? 0 : 1);   // of the scores
                    if (j < 0) ok = wait(q_full, parts) && ok;
                    if (j + 1 < q.n) {
#pragma unroll 1
                        for (int part = 0; part < C::PARTS; ++part) {
                            const uint32_t k = stage_in(false);
                            scores(0, k, tmem + (use & 1) * 128, part);
                            commit(empty + 8 * k);
                        }
                        commit(s_full + 8 * (use & 1));
                    }
                    if (j < 0) continue;
                    const uint32_t now = uses++;
                    ok = wait(p_full + 8 * (now & 1), now >> 1) && ok;
                    if (j == 0) ok = wait(o_free, parts++ + 1) && ok;
#pragma unroll 1
                    for (int part = 0; part < C::PARTS; ++part) {
                        const uint32_t v = stage_in(true);
                        outputs(tmem + (now & 1) * 128 + part * C::SR, v, tmem + C::O_AT, j > 0 || part > 0);
                        commit(empty + 8 * v);
                    }
                    commit(o_done);
                    if (j + 1 == q.n) commit(o_last);
                }
            }
        }
        // no product is running at the end
        if (bw::elect_one()) bw::mma_commit(drain);
        __syncwarp();
        int none = 0;
        bw::mbar_wait_short(drain, 0, &none);
    } else if (warp >= 12) {
        // ---- between the copies and the products: 8-bit values become fp16; of values that not
        // every row attends to, rows that none does become zero, and what is not finite too (a
        // weight of zero would not hide it): its sign to the rows that see it is settled at their end
        constexpr int RING = C::FP8 ? C::NRAW : NST, FIRST = 12, TEAM = 32 * C::READY;
        const int me = threadIdx.x - 32 * FIRST;
        bool ok = true;
        Turn<!C::FP8, RING> in;
        Turn<!C::FP8, NST> turn;
        struct {
            int n, blk0, lo, hi, all_lo, all_hi, gi;
        } q;
#pragma unroll 1
        for (uint32_t at = 0;; ++at) {
            const volatile Part& x = take(at);
            q = {x.n, x.blk0, x.lo, x.hi, x.all_lo, x.all_hi, x.gi};
            volatile uint8_t* const odd = &sm.odd[x.busy % 8][warp - FIRST];
            if (q.n < 0 || !ok) break;
            give(at);
            if (lane == 0) *odd = 0;
            __syncwarp();
            each_block<C>(q.n, [&](bool values, int j) {
                if (!ok) return;
                const int pos = (q.blk0 + j) * kBlk;
                const bool part_seen = pos < q.all_lo || pos + kBlk > q.all_hi;
#pragma unroll 1
                for (int part = 0; part < C::PARTS; ++part) {
                    const int p0 = pos + part * C::SR;
                    in.take(values);
                    turn.take(values);
                    ok = wait(full + 8 * in.stage, in.use) && ok;
                    if (!ok) return;
                    const uint32_t pages = *const_cast<volatile uint8_t*>(&sm.pages[(q.gi + j) % kRing][part]);
                    const bool look = values && (part_seen || pages != (1u << G16) - 1);
                    auto live = [&](int row) { return p0 + row >= q.lo && p0 + row < q.hi && (pages >> (row / 16) & 1); };
                    const uint32_t stage = stages + turn.stage * C::STAGE;
                    if constexpr (C::FP8) {
                        ok = wait(empty + 8 * turn.stage, turn.use + 1) && ok;
                        if (!ok) return;
                        const uint32_t raw = raws + in.stage * C::RAW;
                        // units of 16 channels in a row, a power of two
                        constexpr int KU = C::KD / 16, KLOG = KU == 4 ? 2 : 3;
                        const int log = C::PARTS == 1 || !values ? KLOG : KLOG + 1;
                        // in place and apart: few stages need it, and the loop below stays short
                        if (__builtin_expect(look, 0)) {
                            const int rows = TEAM >> log;   // of a step
#pragma unroll 1
                            for (int r0 = 0; r0 < C::SR; r0 += rows) {
                                if (p0 + r0 >= q.all_lo && p0 + r0 + rows <= q.all_hi && pages == (1u << G16) - 1) continue;
                                const uint32_t at = raw + (r0 << log) * 16 + me * 16;
                                uint4 w = ld_shared(at);
                                const bool on = live(r0 + (me >> log));
                                const bool nan = part_seen && (nan_bytes(w.x) | nan_bytes(w.y) | nan_bytes(w.z) | nan_bytes(w.w));
                                if (!on) {
                                    st_shared(at, make_uint4(0, 0, 0, 0));
                                } else if (nan) {
                                    w.x &= ~((nan_bytes(w.x) >> 7) * 0xffu);
                                    w.y &= ~((nan_bytes(w.y) >> 7) * 0xffu);
                                    w.z &= ~((nan_bytes(w.z) >> 7) * 0xffu);
                                    w.w &= ~((nan_bytes(w.w) >> 7) * 0xffu);
                                    st_shared(at, w);
                                    *odd = 1;
                                }
                            }
                        }
                        // four vectors' reads are on their way before the first is converted
                        constexpr int MOST = D == 256 ? 4 : 8, EACH = C::RAW / 16 / TEAM < MOST ? C::RAW / 16 / TEAM : MOST;
#pragma unroll 1
                        for (int i0 = me; i0 < C::RAW / 16; i0 += EACH * TEAM) {
                            uint4 w[EACH];
#pragma unroll
                            for (int k = 0; k < EACH; ++k) w[k] = ld_shared(raw + (i0 + k * TEAM) * 16);
#pragma unroll
                            for (int k = 0; k < EACH; ++k) {
                                const int i = i0 + k * TEAM, row = i >> log, u = i & ((1 << log) - 1), panel = u / 4, unit = 2 * (u % 4);
                                const uint4 h0 = make_uint4(e4m3_lo(w[k].x), e4m3_hi(w[k].x), e4m3_lo(w[k].y), e4m3_hi(w[k].y)),
                                            h1 = make_uint4(e4m3_lo(w[k].z), e4m3_hi(w[k].z), e4m3_lo(w[k].w), e4m3_hi(w[k].w));
                                // odd panels store their second half first, so that a row's eight lanes
                                // meet eight banks' groups
                                const uint32_t to = stage + panel * (values ? C::PANEL : C::KPANEL) + row * 128;
                                const int f = panel & 1;
                                st_shared(to + (((unit + f) ^ (row & 7)) << 4), f ? h1 : h0);
                                st_shared(to + (((unit + 1 - f) ^ (row & 7)) << 4), f ? h0 : h1);
                            }
                        }
                        bw::fence_async_smem();
                        __syncwarp();
                        if (lane == 0) bw::mbar_arrive(raw_free + 8 * in.stage);
                    } else if (look) {
                        // sixteen rows at a time: those that all rows attend to need no look, and those
                        // that none does no read (one vector after the other a stage takes 7700 cycles)
#pragma unroll 1
                        for (int g = 0; g < G16; ++g) {
                            const int first = p0 + 16 * g, at = first + me / 8;
                            const bool here = pages >> g & 1;
                            if (here && first >= q.all_lo && first + 16 <= q.all_hi) continue;
                            const bool on = here && at >= q.lo && at < q.hi;
                            uint4 w[D / 64];
#pragma unroll
                            for (int k = 0; k < D / 64; ++k) w[k] = ld_shared(stage + k * C::PANEL + g * 2048 + me * 16);
#pragma unroll
                            for (int k = 0; k < D / 64; ++k) {
                                const uint32_t to = stage + k * C::PANEL + g * 2048 + me * 16;
                                // exponents of ones carry into the sign's place
                                auto high = [](uint32_t x) { return (x & 0x7f807f80u) + 0x00800080u; };
                                const uint32_t bad = (high(w[k].x) | high(w[k].y) | high(w[k].z) | high(w[k].w)) & 0x80008000u;
                                if (!on) {
                                    st_shared(to, make_uint4(0, 0, 0, 0));
                                } else if (bad && part_seen) {
                                    uint32_t* const x = reinterpret_cast<uint32_t*>(&w[k]);
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        if ((x[e] & 0x7f80u) == 0x7f80u) x[e] &= 0xffff0000u;
                                        if ((x[e] & 0x7f800000u) == 0x7f800000u) x[e] &= 0xffffu;
                                    }
                                    st_shared(to, w[k]);
                                    *odd = 1;
                                }
                            }
                        }
                        bw::fence_async_smem();
                        __syncwarp();
                    }
                    if (lane == 0) bw::mbar_arrive(ready + 8 * turn.stage);
                }
            });
        }
    } else if (warp < 8) {
        // ---- softmax: a thread per row (heads of 256: two, by columns) -----------------------------
        regs_up<C::SOFTMAX_REGS>();
        const int wg = warp / 4, slot = C::NS == 2 ? wg : 0, row = threadIdx.x % 128;
        const uint32_t lanes = tmem + ((uint32_t)(warp % 4 * 32) << 16);
        const uint32_t o_at = lanes + C::O_AT + (C::NS == 2 ? slot * D : wg * (D / 2));
        constexpr int OC = C::NS == 2 ? D : D / 2;       // output channels of a thread
        const int ch0 = C::NS == 2 ? 0 : wg * OC;
        const int64_t token_heads = s.n_heads;
        uint32_t uses = 0, ended = 0, written = 0;       // blocks and parts of this slot; cut sides recorded
        bool ok = true;
        const float scale = fabsf(p.a.scale);
        const uint32_t flip = p.a.scale < 0.f ? 0x80008000u : 0u;
        float c_next = 0.f;

        auto out_row = [&](const volatile Part& q, int r) {       // row of out and lse
            return (int64_t)(q.start + G.of(q.row0 + r)) * token_heads + q.hk * G.d + G.rest(q.row0 + r);
        };
        // The queries of this warp's 32 rows, to shared memory: neighbouring lanes read neighbouring
        // vectors, UR to a row (a lane per row meets 32 lines with every read, 4000 cycles for a
        // tile). An 8-bit cache's are scaled by a power of two, so that a row's largest lies in
        // [2^14, 2^15).
        auto load_q = [&](const volatile Part& q) {
            constexpr int UR = OC / 8, RI = 32 / UR;   // vectors of a row, rows of a read
            const int r = slot * 128 + row;
            const int t = q.start + G.of(q.row0 + r), head = q.hk * G.d + G.rest(q.row0 + r);
            // (rows past the last read the last one's place, and become zero)
            const int64_t at = r < q.rows ? (int64_t)t * p.a.q_stride + (int64_t)head * D : -1;
            float c = scale * p.k_scale[q.hk];
            // (four reads at a time where they are scaled: the instructions of sixteen do not stay cached)
            constexpr int BATCH = C::FP8 ? 4 : UR;
#pragma unroll 1
            for (int i0 = 0; i0 < UR; i0 += BATCH) {
            uint4 v[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int64_t from = __shfl_sync(~0u, at, RI * (i0 + i) + lane / UR);
                v[i] = from < 0 ? make_uint4(0, 0, 0, 0)
                                : *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.a.q) + from + ch0 + lane % UR * 8);
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                uint32_t x[4] = {v[i].x ^ flip, v[i].y ^ flip, v[i].z ^ flip, v[i].w ^ flip};
                const int rr = warp % 4 * 32 + RI * (i0 + i) + lane / UR, unit = ch0 / 8 + lane % UR;
                if constexpr (C::FP8) {
                    uint32_t big = 0;
                    auto look = [&](uint32_t w) { big = max(big, max(w & 0x7fffu, w >> 16 & 0x7fffu)); };
#pragma unroll
                    for (int k = 0; k < 4; ++k) look(x[k]);
                    if constexpr (C::NS == 1) {   // and the other half of the channels
                        const int64_t from = __shfl_sync(~0u, at, RI * (i0 + i) + lane / UR);
                        if (from >= 0) {
                            const uint4 o = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.a.q) + from + (ch0 ^ OC) +
                                                                            lane % UR * 8);
                            look(o.x), look(o.y), look(o.z), look(o.w);
                        }
                    }
#pragma unroll
                    for (int o = 1; o < UR; o <<= 1) big = max(big, __shfl_xor_sync(~0u, big, o));
                    // exponent field e: the largest is below 2^(e - 126); a factor within fp32's range
                    const int e = big >> 7, by = big == 0 || e == 255 ? 0 : max(-126, min(126, 141 - e));
                    const float up = exp2i(by);
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] = pack2<true>(bf16_lo(x[k]) * up, bf16_hi(x[k]) * up);
                    // to the lane whose row it is
                    const int got = __shfl_sync(~0u, by, lane % RI * UR);
                    if (lane / RI == i0 + i) c *= exp2i(-got);
                }
                st_shared(q_at + slot * C::QTILE + unit / 8 * C::QPANEL + rr * 128 + ((unit % 8 ^ (rr & 7)) << 4),
                          make_uint4(x[0], x[1], x[2], x[3]));
            }
            }
            bw::fence_async_smem();
            __syncwarp();
            if (lane == 0) bw::mbar_arrive(q_full + 8 * slot);
            // (no score of fp32's range sees the smallest number, and -inf times it stays -inf)
            c_next = fmaxf(c, 0x1p-149f);
        };
        // the two warps of a row's columns meet (heads of 256)
        uint32_t met = 0;
        auto pair_meets = [&] {
            __syncwarp();
            if (lane == 0) bw::mbar_arrive(pair + 8 * (warp % 4));
            ok = wait(pair + 8 * (warp % 4), met++) && ok;
        };

        float m = -INFINITY, m_raw = 0.f, l[4] = {};   // maximum (scaled, base two; as it came), sums
        uint32_t at_part = 0, parts = 0;
        bool have = false;
#pragma unroll 1
        for (;;) {
            // the next part's queries go ahead of this one's end; a second tile is not there for
            // every part (and the end does not wait until it is: the part has to be given back)
            if (!ok) break;
            const volatile Part& v = take(parts);
            const int blocks = v.n;
            if (*const_cast<volatile int*>(&sm.abort)) break;
            const bool mine = blocks > 0 && (C::NS == 1 || slot == 0 || v.rows > 128);
            if (mine) load_q(v);
            if (have) {
                const volatile Part& q = sm.part[at_part % kParts];
                float sum = (l[0] + l[2]) + (l[1] + l[3]);
                if constexpr (C::NS == 1) {
                    sm.row_sum[wg][row] = sum;
                    pair_meets();
                    sum = sm.row_sum[0][row] + sm.row_sum[1][row];
                }
                const float of_values = p.v_scale[q.hk];
                const int r = slot * 128 + row, pos = q.base + G.of(q.row0 + r);
                const int64_t o_row = r < q.rows ? out_row(q, r) : -1;
                ok = wait(o_last + 8 * slot, ended++) && ok;
                if (!ok) break;
                bw::tc_fence_after();
                const int see0 = Walk<C>::first_seen(pos, p.a.window), see1 = pos + 1;
                const bool cut = !(q.first && q.last), on = r < q.rows;
                const int side = q.index ? 1 : 0, rec = blockIdx.x * 2 + side;
                const volatile uint8_t* f = sm.odd[q.busy % 8];
                bool odd = false;
    #pragma unroll 1
                for (int i = 0; i < C::READY; ++i) odd |= f[i] != 0;
                if (cut && threadIdx.x == 0) {
                    written |= 1u << side;
                    p.recs[rec] = Rec{REC_CUT | (q.first ? REC_FIRST : 0) | (q.last ? REC_LAST : 0), q.rows, q.row0, q.start, q.hk, {}};
                }
                if (cut && on && ch0 == 0) p.part_ml[(int64_t)rec * C::ROWS + r] = make_float2(m, sum);
                const float inv = sum == 0.f ? 0.f : of_values / sum;
    #pragma unroll 1
                for (int i = 0; i < OC; i += 32) {
                    uint32_t o[32];
                    __syncwarp();   // lanes walk over rows and positions of their own
                    bw::tmem_ld32(o_at + i, o);
                    bw::tmem_wait_ld32(o);
                    if (odd && on) {
                        // what is not finite among the values set aside goes to the rows that see it
    #pragma unroll 1
                        for (int j = 0; j < q.n; ++j) {
                            const int p0 = (q.blk0 + j) * kBlk;
                            if (p0 >= q.all_lo && p0 + kBlk <= q.all_hi) continue;
    #pragma unroll 1
                            for (int at = max(p0, see0); at < min(p0 + kBlk, see1); ++at) {
                                const int page = p.a.block_table[(int64_t)q.b * p.a.max_pages + p.page.of(at)];
                                if (page < 0 || page >= s.n_pages) continue;
                                const int64_t from = kv_offset(s, page, q.hk, p.page.rest(at)) + ch0 + i;
    #pragma unroll
                                for (int k = 0; k < 32; ++k) {
                                    float v;
                                    if constexpr (C::FP8)
                                        v = (static_cast<const uint8_t*>(p.v_pages)[from + k] & 0x7f) == 0x7f ? NAN : 0.f;
                                    else v = __bfloat162float(static_cast<const __nv_bfloat16*>(p.v_pages)[from + k]);
                                    if (!isfinite(v)) o[k] = __float_as_uint(__uint_as_float(o[k]) + v);
                                }
                            }
                        }
                    }
                    if (cut) {
                        if (on) {
                            float4* to = p.part_o + ((int64_t)rec * (D / 4) + (ch0 + i) / 4) * C::ROWS + r;
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                to[k * C::ROWS] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                                              __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
                        }
                    } else {
                        // four lanes write 64 bytes of one row together: a lane per row is a line per
                        // lane and store, 4100 cycles for a tile
                        uint4 h[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = pack2<false>(__uint_as_float(o[8 * k + 2 * e]) * inv, __uint_as_float(o[8 * k + 2 * e + 1]) * inv);
                            h[k] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        turn4(h, lane);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int64_t to = __shfl_sync(~0u, o_row, (lane & ~3) + k);
                            if (to >= 0)
                                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.out) + to * D + ch0 + i + lane % 4 * 8) = h[k];
                        }
                    }
                }
                bw::tc_fence_before();
                __syncwarp();
                if (lane == 0) bw::mbar_arrive(o_free + 8 * slot);
                if (!cut && on && p.a.lse && ch0 == 0) p.a.lse[o_row] = sum == 0.f ? -INFINITY : m * kLn2 + logf(sum * C::DOWN);
                give(at_part);
            }
            if (blocks < 0) break;
            have = mine;
            if (!mine) {
                give(parts++);
                continue;
            }
            at_part = parts++;
            const float c = C::CAP ? 1.f : c_next * kLog2e;
            // (no quotient past fp32's range, which would make NaN of a score of zero; one near its end
            // has few bits: an 8-bit cache's sums are below 2^32, and tanh z is z by far)
            float to_cap = C::CAP ? fminf(c_next / p.a.softcap, 0x1.fffffep127f) : 0.f, cap = p.a.softcap * kLog2e;
            if (C::CAP && C::FP8 && to_cap < 0x1p-100f) {
                to_cap = 0x1p-100f;
                cap = c_next * 0x1p100f * kLog2e;
            }
            const int pos = v.base + G.of(v.row0 + slot * 128 + row);
            const int see0 = Walk<C>::first_seen(pos, p.a.window), see1 = pos + 1;
            const int n = v.n, blk0 = v.blk0, all_lo = v.all_lo, all_hi = v.all_hi;
            m = -INFINITY;
            m_raw = l[0] = l[1] = l[2] = l[3] = 0.f;
#pragma unroll 1
            for (int j = 0; j < n; ++j, ++uses) {
                const int buf = C::NS == 2 ? slot : uses & 1, phase = C::NS == 2 ? uses : uses >> 1;
                const int at = (blk0 + j) * kBlk + (C::NS == 2 ? 0 : wg * C::COLS);
                const uint32_t s_at = lanes + buf * 128 + (C::NS == 2 ? 0 : wg * C::COLS);
                ok = wait(s_full + 8 * buf, phase) && ok;
                if (!ok) break;
                bw::tc_fence_after();
                const bool edge = at < all_lo || at + C::COLS > all_hi || *const_cast<volatile int*>(&sm.lost);
                if (C::CAP || __builtin_expect(edge, 0)) {
                    const volatile uint8_t* pages = sm.pages[(v.gi + j) % kRing];
                    const uint32_t in = C::NS == 2 ? pages[0] : pages[wg];
                    // scores are capped, and what this row does not attend to goes out, in place
#pragma unroll 1
                    for (int c0 = 0; c0 < C::COLS; c0 += 32) {
                        const bool some = edge && (at + c0 < all_lo || at + c0 + 32 > all_hi || *const_cast<volatile int*>(&sm.lost));
                        if (!C::CAP && !some) continue;
                        uint32_t u[32];
                        float* const x = reinterpret_cast<float*>(u);
                        bw::tmem_ld32(s_at + c0, u);
                        bw::tmem_wait_ld32(u);
                        if constexpr (C::CAP) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) tanh_cap(x[2 * i], x[2 * i + 1], to_cap, cap);
                        }
                        if (some) {
                            const int a = see0 - at - c0, b = see1 - at - c0;
                            const uint32_t two = in >> (c0 / 16);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i < a || i >= b || !(two >> (i / 16) & 1)) x[i] = -INFINITY;
                        }
                        bw::tmem_st32(s_at + c0, u);
                    }
                    bw::tmem_wait_st();
                }
                // the row in registers from here on: read again for the exponentials it takes 1340
                // cycles instead of 905
                uint32_t u[C::COLS / 32][32];
#pragma unroll
                for (int i = 0; i < C::COLS / 32; ++i) bw::tmem_ld32(s_at + 32 * i, u[i]);
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < C::COLS / 32; ++i) {
                    bw::tmem_wait_ld32(u[i]);
                    top = max32(reinterpret_cast<float*>(u[i]), top);
                }
                if constexpr (C::NS == 1) {
                    sm.row_max[uses & 1][wg][row] = top;
                    pair_meets();
                    top = fmaxf(top, sm.row_max[uses & 1][wg ^ 1][row]);
                }
                const float cand = top * c;
                const bool raise = cand > m + 8.f;
                if (__builtin_expect(__any_sync(~0u, raise), 0)) {
                    const float f = !raise ? 1.f : m == -INFINITY ? 0.f : ex2(m - cand);
                    if (raise) {
                        m = cand;
                        m_raw = top;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) l[i] *= f;
                    if (j > 0) {
                        // (a parity tells a phase from its neighbours: the products up to the last
                        // but one ended before these scores, and the next has not begun)
                        ok = wait(o_done + 8 * slot, uses - 1) && ok;
                        bw::tc_fence_after();
#pragma unroll 1
                        for (int i = 0; i < OC; i += 32) {
                            uint32_t o[32];
                            bw::tmem_ld32(o_at + i, o);
                            bw::tmem_wait_ld32(o);
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            bw::tmem_st32(o_at + i, o);
                        }
                    }
                }
                // exp2(x c - m): one rounding, and a maximum that is itself rounded shifts all
                // weights of a row alike; past 2^20 that shift would be seen, and the
                // difference is taken first
                const float mu = m == -INFINITY ? 0.f : m, minus = C::UP - mu;
                const float raw = m == -INFINITY ? 0.f : m_raw;
                const bool far = __any_sync(~0u, fabsf(mu) > 0x1p20f);
                float times = c, plus = minus;
                if (__builtin_expect(far, 0)) {
#pragma unroll
                    for (int i = 0; i < C::COLS; ++i) {
                        float* const x = reinterpret_cast<float*>(u[i / 32]);
                        x[i % 32] = (x[i % 32] - raw) * c;
                    }
                    times = 1.f;
                    plus = C::UP;
                }
#pragma unroll
                for (int c0 = 0; c0 < C::COLS; c0 += 32) {
                    float* const x = reinterpret_cast<float*>(u[c0 / 32]);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) fma_in(x[i], x[i + 1], times, plus);
                    uint32_t w[16], rest[C::FINE ? 16 : 1];
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[i + k] = ex2(x[i + k]);
                        add_in(l[0], l[1], x[i], x[i + 1]);
                        add_in(l[2], l[3], x[i + 2], x[i + 3]);
                        if constexpr (C::FINE) {
                            split2(x[i], x[i + 1], w[i / 2], rest[i / 2]);
                            split2(x[i + 2], x[i + 3], w[i / 2 + 1], rest[i / 2 + 1]);
                        } else {
                            w[i / 2] = pack2<C::FP8>(x[i], x[i + 1]);
                            w[i / 2 + 1] = pack2<C::FP8>(x[i + 2], x[i + 3]);
                        }
                    }
                    bw::tmem_st16(s_at + c0 / 2, w);   // over scores that have been read
                    if constexpr (C::FINE) bw::tmem_st16(s_at + C::COLS / 2 + c0 / 2, rest);
                }
                bw::tmem_wait_st();
                bw::tc_fence_before();
                __syncwarp();
                if (!ok) break;
                if (lane == 0) bw::mbar_arrive(p_full + 8 * buf);
            }
        }
        // After a wait that ran out the rows of all of this CTA's parts become NaN, by way of their
        // sums where the tile is cut (some of them may be whole: which is not told).
        __syncwarp();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (*const_cast<volatile int*>(&sm.abort)) {
            Walk<C> again{sm.start, sm.len, p.G};
            again.left = sm.share.left;
            again.b = sm.share.b, again.i = sm.share.i, again.hk = sm.share.hk, again.off = sm.share.off;
            again.Hk = s.n_kv_heads;
            again.window = p.a.window;
            again.whole = p.whole;
            again.index = again.busy = again.gi = 0;
            Part q;
#pragma unroll 1
            while (again.next(q)) {
                if (!q.n && !q.none) continue;
                const bool cut = !(q.first && q.last);
                const int side = q.index ? 1 : 0, rec = blockIdx.x * 2 + side;
                const uint32_t fill = q.none ? 0 : 0x7fff7fffu;
                if (cut && threadIdx.x == 0) {
                    written |= 1u << side;
                    p.recs[rec] = Rec{REC_CUT | (q.first ? REC_FIRST : 0) | (q.last ? REC_LAST : 0), q.rows, q.row0, q.start, q.hk, {}};
                }
#pragma unroll 1
                for (int r = threadIdx.x; r < q.rows; r += 256) {
                    if (cut) {
                        p.part_ml[(int64_t)rec * C::ROWS + r] = make_float2(0.f, NAN);
                        continue;
                    }
                    const int64_t o = out_row(q, r);
                    uint4* const to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.out) + o * D);
#pragma unroll 1
                    for (int i = 0; i < D / 8; ++i) to[i] = make_uint4(fill, fill, fill, fill);
                    if (p.a.lse) p.a.lse[o] = q.none ? -INFINITY : NAN;
                }
            }
        }
        if (threadIdx.x == 0)
#pragma unroll 1
            for (int side = 0; side < 2; ++side)
                if (!(written >> side & 1)) p.recs[blockIdx.x * 2 + side].flags = 0;
    }
    bw::tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && sm.abort) bits |= MOE_KV_TIMEOUT;
    if (bits) atomicOr(p.health, bits);
    __syncwarp();
    if (warp == 8) {
        bw::tc_fence_after();
        bw::tmem_dealloc(tmem, 512);
    }
}

// Joins the parts of the tiles that were cut between CTAs, in order: a CTA per CTA that began
// such a tile and 32 of its rows, a lane per row, four channels at a time. A record is followed only
// to rows that the call has: one that another call, on the same workspace at the same time, wrote
// over it names rows of its own.
template <class C>
__global__ void __launch_bounds__(256) k_kv_chunk_join(const ChunkArgs p, int ctas) {
    constexpr int D = C::D, V = D / 32;   // vectors of four channels of a thread
    __shared__ int sm_last;
    __shared__ Rec sm_rec;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, c0 = blockIdx.x, r = blockIdx.y * 32 + lane;
    pdl_wait();
    pdl_trigger();
    for (int side = 0; side < 2; ++side) {
        __syncthreads();
        if (threadIdx.x == 0) {
            sm_rec = p.recs[c0 * 2 + side];
            sm_last = ctas - 1;
        }
        __syncthreads();
        const Rec rec = sm_rec;
        if ((rec.flags & (REC_CUT | REC_FIRST)) != (REC_CUT | REC_FIRST) || (int)blockIdx.y * 32 >= rec.rows) continue;
        if (rec.rows > C::ROWS || (unsigned)rec.hk >= (unsigned)p.s.n_kv_heads || rec.start < 0 || rec.row0 < 0 ||
            rec.row0 > INT32_MAX - C::ROWS || rec.start >= p.a.T - p.G.of(rec.row0 + rec.rows - 1))
            continue;
        for (int k = c0 + 1 + threadIdx.x; k < ctas; k += 256)
            if ((p.recs[k * 2].flags & (REC_CUT | REC_FIRST | REC_LAST)) == (REC_CUT | REC_LAST)) {
                atomicMin(&sm_last, k);
                break;
            }
        __syncthreads();
        const int n = sm_last - c0 + 1;
        if (r >= rec.rows) continue;
        auto part = [&](int i) { return (int64_t)((c0 + i) * 2 + (i ? 0 : side)); };
        float M = -INFINITY, L = 0.f;
#pragma unroll 8
        for (int i = 0; i < n; ++i) M = fmaxf(M, p.part_ml[part(i) * C::ROWS + r].x);
        const float mb = M == -INFINITY ? 0.f : M;
        float4 o[V] = {};
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const float2 ml = p.part_ml[part(i) * C::ROWS + r];
            const float f = ex2(ml.x - mb);
            L += f * ml.y;
            const float4* from = p.part_o + (part(i) * (D / 4) + warp) * C::ROWS + r;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float4 x = from[k * 8 * C::ROWS];
                o[k].x += f * x.x;
                o[k].y += f * x.y;
                o[k].z += f * x.z;
                o[k].w += f * x.w;
            }
        }
        const float inv = L == 0.f ? 0.f : p.v_scale[rec.hk] / L;
        const int64_t row = (int64_t)(rec.start + p.G.of(rec.row0 + r)) * p.s.n_heads + rec.hk * p.G.d + p.G.rest(rec.row0 + r);
        uint2* to = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.a.out) + row * D) + warp;
#pragma unroll
        for (int k = 0; k < V; ++k)
            to[k * 8] = make_uint2(pack2<false>(o[k].x * inv, o[k].y * inv), pack2<false>(o[k].z * inv, o[k].w * inv));
        if (warp == 0 && p.a.lse) p.a.lse[row] = L == 0.f ? -INFINITY : mb * kLn2 + logf(L * C::DOWN);
    }
}

// The kernel of a cache, of capped or plain scores, and of weights as one number or two.
template <class F>
auto pick(const KvShape& s, bool cap, bool fine, F f) {
    if (s.e4m3) {
        if (s.head_dim == 64) return cap ? f(Cfg<64, true, true>{}) : f(Cfg<64, true, false>{});
        if (s.head_dim == 128) return cap ? f(Cfg<128, true, true>{}) : f(Cfg<128, true, false>{});
        return cap ? f(Cfg<256, true, true>{}) : f(Cfg<256, true, false>{});
    }
    if (fine) {
        if (s.head_dim == 64) return cap ? f(Cfg<64, false, true, true>{}) : f(Cfg<64, false, false, true>{});
        if (s.head_dim == 128) return cap ? f(Cfg<128, false, true, true>{}) : f(Cfg<128, false, false, true>{});
        return cap ? f(Cfg<256, false, true, true>{}) : f(Cfg<256, false, false, true>{});
    }
    if (s.head_dim == 64) return cap ? f(Cfg<64, false, true>{}) : f(Cfg<64, false, false>{});
    if (s.head_dim == 128) return cap ? f(Cfg<128, false, true>{}) : f(Cfg<128, false, false>{});
    return cap ? f(Cfg<256, false, true>{}) : f(Cfg<256, false, false>{});
}

struct Space {
    size_t recs, ml, o;   // bytes, each a multiple of 256
};
Space space_of(const Kv& K) {
    const int rows = pick(K.s, false, false, [](auto c) { return decltype(c)::ROWS; });
    const size_t n = (size_t)K.num_sms * 2;
    return {(n * sizeof(Rec) + 255) / 256 * 256, n * rows * sizeof(float2), n * rows * K.s.head_dim * 4};
}

}  // namespace

size_t kv_chunk_workspace(const Kv& K) {
    const Space w = space_of(K);
    return w.recs + w.ml + w.o;
}

cudaError_t kv_chunk_setup(Kv& K) {
    const int sr = pick(K.s, false, false, [](auto c) { return decltype(c)::SR; });
    K.chunk_box = 16;
    while (K.chunk_box * 2 <= sr && K.s.page_size % (K.chunk_box * 2) == 0) K.chunk_box *= 2;
    const auto encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const size_t es = K.s.e4m3 ? 1 : 2;
    const cuuint64_t dims[4] = {(cuuint64_t)K.s.head_dim, (cuuint64_t)K.s.page_size, (cuuint64_t)K.s.n_kv_heads,
                                (cuuint64_t)K.s.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)K.s.token_stride * es, (cuuint64_t)K.s.head_stride * es,
                                   (cuuint64_t)K.s.page_stride * es};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    const int key_width = pick(K.s, false, false, [](auto c) { return decltype(c)::KD; });
    for (int i = 0; i < 2; ++i) {
        const cuuint32_t box[4] = {(cuuint32_t)(!K.s.e4m3 ? 64 : i ? K.s.head_dim : key_width), (cuuint32_t)K.chunk_box, 1, 1};
        if (encode(i ? &K.tm_chunk_v : &K.tm_chunk_k, K.s.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                   4, i ? K.v_pages : K.k_pages, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   K.s.e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    for (const int i : {0, 1, 2, 3}) {
        const cudaError_t e = pick(K.s, i & 1, i & 2, [](auto c) {
            using C = decltype(c);
            return cudaFuncSetAttribute(k_kv_chunk<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::smem);
        });
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

moe_status kv_chunk_launch(Kv& K, const moe_kv_chunk_args& a, cudaStream_t stream) {
    const Space w = space_of(K);
    uint8_t* const at = static_cast<uint8_t*>(a.workspace);
    ChunkArgs p{a, K.s, K.v_pages, K.k_scale, K.v_scale, K.health, reinterpret_cast<Rec*>(at),
                reinterpret_cast<float2*>(at + w.recs), reinterpret_cast<float4*>(at + w.recs + w.ml),
                Div(K.s.n_heads / K.s.n_kv_heads), Div(K.s.page_size), K.chunk_box, K.stall, false};
    // a window that holds every position is none
    if (p.a.window >= a.max_pages * K.s.page_size) p.a.window = 0;
    // Up to four blocks of a sequence, a CTA does a tile in less time than the second launch takes.
    p.whole = a.max_pages * K.s.page_size <= 4 * kBlk;
    // A cap of 2^80 changes no score below 2^68, one of 2^126 times the scale none of products
    // below 2^114; a score's share of it would lose bits, or all.
    const bool cap = a.softcap > 0.f && a.softcap < 0x1p80f && a.softcap * 0x1p-126 < std::fabs((double)a.scale);
    const cudaError_t e = pick(K.s, cap, K.chunk_fine, [&](auto c) {
        using C = decltype(c);
        const cudaError_t e = launch_pdl(k_kv_chunk<C>, dim3(K.num_sms), dim3(C::THREADS), C::smem, stream, true, p,
                                         K.tm_chunk_k, K.tm_chunk_v);
        if (e != cudaSuccess || p.whole) return e;
        return launch_pdl(k_kv_chunk_join<C>, dim3(K.num_sms, C::ROWS / 32), dim3(256), 0, stream, true, p, K.num_sms);
    });
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "attend chunk launch");
}

}  // namespace moe
