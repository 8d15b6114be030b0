// y = act(x W^T + bias) + residual over token rows, on the 5th-generation tensor cores.
//
// The weights' channels are the 128 rows of a tile, whatever T is, and the tokens its
// 16 to 256 columns: one token pads 15 columns and no rows, and the epilogue's lanes hold
// neighbouring channels of one token, so that bias, residual and output go by whole
// 64-byte (bf16) or 128-byte (fp32) runs without passing through shared memory.
//
// Few tokens: the kernel is a stream over W, and its tiles are cut along K into the CTAs
// of a cluster, so that most SMs stream; their sums meet in shared memory and are added in
// order. Many tokens: one CTA per SM takes tile after tile, the epilogue of one under the
// products of the next (two accumulators in tensor memory).
//
// Measured (GB300; floors at 6.80 TB/s and 1897 TFLOP/s): one token 6144 x 8192 17.1 us (87% of
// the copy rate), 6144 x 6144 15.4 us (72%), 512 x 768 3.4 us; 128 tokens 6144 x 6144 onto a fp32
// residual 24.9 us (49%: 48 tiles, two CTAs each, and 16 KB of weights per 372 cycles of products
// and 130 of waiting; clusters of three do not all fit; in bf16 21 us), 300 54 us (25%); 8191 tokens
// 2816 x 8192 with gelu 254 us, 1.49 PFLOP/s (78%: 48 KB of operands for 512 cycles of products come
// from the second-level cache at 60 bytes a cycle and SM; a pair of CTAs on one tile would need two
// thirds); 4096 tokens 6144 x 6144 232 us (70%), onto a fp32 residual 520 us (31%: tiles of 128).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "common.cuh"
#include "moe_internal.h"
#include "overlap.h"
#include "per_device.h"
#include "sm100_more.cuh"

namespace moe {

namespace {

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

moe_status check_linear(const moe_linear_desc* d, const void* x, const void* w, const float* bias, const void* residual,
                        const void* y, int T) {
    if (!d) return fail(MOE_E_INVALID, "desc is NULL");
    if (d->abi_version != MOE_ABI_VERSION) return fail(MOE_E_INVALID, "abi_version mismatch");
    if (d->in_features < 1 || d->in_features % 8 || d->out_features < 1 || d->out_features % 8)
        return fail(MOE_E_INVALID, "in_features and out_features must be positive multiples of 8");
    if (d->in_features > 1 << 20 || d->out_features > 1 << 20)
        return fail(MOE_E_UNSUPPORTED, "in_features and out_features are limited to 2^20");
    if (d->out_dtype != MOE_F32 && d->out_dtype != MOE_BF16) return fail(MOE_E_INVALID, "out_dtype must be MOE_F32 or MOE_BF16");
    if (d->activation < MOE_ACT_NONE || d->activation > MOE_ACT_SIGMOID) return fail(MOE_E_INVALID, "unknown activation");
    if (T < 0) return fail(MOE_E_INVALID, "T must not be negative");
    if (T > 1 << 24) return fail(MOE_E_UNSUPPORTED, "T is limited to 2^24");
    if (T == 0) return MOE_OK;
    if (!x || !w || !y) return fail(MOE_E_INVALID, "x, w or y is NULL");
    for (const void* p : {x, w, static_cast<const void*>(bias), residual, y})
        if (!aligned16(p)) return fail(MOE_E_INVALID, "pointers must be 16-byte aligned");
    const int out_step = d->out_dtype == MOE_F32 ? 4 : 8;
    const struct { const void* p; int64_t st; int n, step; const char* name; } rows[] = {
        {x, d->x_stride, d->in_features, 8, "x_stride"}, {w, d->w_stride, d->in_features, 8, "w_stride"},
        {y, d->y_stride, d->out_features, out_step, "y_stride"},
        {residual, d->residual_stride, d->out_features, out_step, "residual_stride"}};
    for (const auto& r : rows)
        if (r.p && (r.st % r.step || r.st < r.n || r.st > (int64_t)1 << 38))
            return fail(MOE_E_INVALID, std::string(r.name) + " must be a multiple of 16 bytes, cover a row, and be at most 2^38");
    if (residual == y && residual && d->residual_stride != d->y_stride)
        return fail(MOE_E_INVALID, "residual may be y only with y's stride");
    return MOE_OK;
}

// Other CTAs still read what a tile's outputs would overwrite.
bool overwrites(const moe_linear_desc& d, const void* x, const void* w, const float* bias, const void* residual, const void* y,
                int64_t T) {
    const int64_t K = d.in_features, N = d.out_features, es = d.out_dtype == MOE_F32 ? 4 : 2;
    const Span out{y, T, N * es, d.y_stride * es};
    return overlap(out, {x, T, K * 2, d.x_stride * 2}) || overlap(out, {w, N, K * 2, d.w_stride * 2}) ||
           overlap(out, {bias, 1, N * 4, N * 4}) || (residual != y && overlap(out, {residual, T, N * es, d.residual_stride * es}));
}

// 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u)), so that every activation is z times a logistic, or
// one. The hardware's exponential and reciprocal are off by 2^-22 each, and the exponent's
// product by 2^-24 of |u|, where the result is small by then.
__device__ __forceinline__ float logistic(float u) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * u));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
template <int N>
__device__ __forceinline__ void activate(float (&z)[N], int act) {
    if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] *= logistic(z[i]);
    } else if (act == MOE_ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] *= logistic(1.5957691216057308f * (z[i] + 0.044715f * z[i] * z[i] * z[i]));
    } else if (act == MOE_ACT_SIGMOID) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = logistic(z[i]);
    }
}

constexpr int kRows = 128, kChunk = 64;             // channels of a tile; K of a panel, 128 bytes
constexpr int kRing = 196608;                       // bytes of stages, and of a split tile's sums
constexpr int kMaxSplits = 8;                       // a portable cluster
constexpr int kThreads = 192;                       // four epilogue warps, the copies', the products'
// Panels of a stage. The products wait once per stage, and a wait behind issued products takes
// 130 cycles more than theirs (89 each up to 128 tokens): two panels where the ring holds them.
// (A fine tile's sums, 512 bytes per token, stand behind the stages; see k_linear.)
constexpr int panels_of(int BN, bool fine) { return BN <= (fine ? 64 : 128) ? 2 : 1; }
constexpr uint32_t stage_bytes(int BN, bool fine) { return (kRows + BN) * kChunk * 2 * panels_of(BN, fine); }
constexpr int ring_bytes(int BN, bool fine) { return kRing - (fine ? BN * kRows * 4 : 0); }
constexpr int stages_of(int BN, bool fine) { return ring_bytes(BN, fine) / stage_bytes(BN, fine); }

struct LinearArgs {
    const float* bias;
    const void* residual;
    void* y;
    int64_t y_stride, residual_stride;
    int T, K, N, out_f32, act;
    int row_tiles, tiles, splits;   // tiles: all of them, channels fastest; splits: CTAs of a cluster
    int stall;                      // MOE_LINEAR_OPT_TEST_STALL
};

__device__ __forceinline__ void prefetch_2d(const CUtensorMap* tm, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(tm), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile("{.reg .b32 a; mapa.shared::cluster.u32 a, %4, %5; ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];}"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}
// Channel n of tokens t.. t + 15, as far as `count` goes: the lanes of a warp hold
// neighbouring channels. The residual's reads are all on their way before any is used.
__device__ __forceinline__ void finish16(const LinearArgs& p, int t, int count, int n, float (&v)[16], float bias) {
    const int64_t at = (int64_t)t * p.y_stride + n, rt = (int64_t)t * p.residual_stride + n;
    float r[16];
    if (p.residual)
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (j < count)
                r[j] = p.out_f32 ? static_cast<const float*>(p.residual)[rt + j * p.residual_stride]
                                 : __bfloat162float(static_cast<const __nv_bfloat16*>(p.residual)[rt + j * p.residual_stride]);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] += bias;
    activate(v, p.act);
    if (p.residual)
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] += r[j];
    if (p.out_f32) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (j < count) static_cast<float*>(p.y)[at + j * p.y_stride] = v[j];
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (j < count) static_cast<__nv_bfloat16*>(p.y)[at + j * p.y_stride] = __float2bfloat16(v[j]);
    }
}

// A tile whose sums lie in shared memory, of as many CTAs as `splits` says: the columns
// `split`, `split` + `splits`, ..., a warp one at a time, four channels a lane.
__device__ __forceinline__ void finish_shared(const LinearArgs& p, int tile, int BN, uint32_t sums_at, int split, int splits,
                                              int warps) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int n = tile % p.row_tiles * kRows + 4 * lane, t0 = tile / p.row_tiles * BN, cols = min(BN, p.T - t0);
    if (n < p.N) {
        const float4 bias = p.bias ? *reinterpret_cast<const float4*>(p.bias + n) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int c = warp * splits + split; c < cols; c += warps * splits) {
            const int64_t at = (int64_t)(t0 + c) * p.y_stride + n, rt = (int64_t)(t0 + c) * p.residual_stride + n;
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f), part[kMaxSplits];
            if (p.residual) {
                if (p.out_f32) {
                    r = *reinterpret_cast<const float4*>(static_cast<const float*>(p.residual) + rt);
                } else {
                    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.residual) + rt);
                    r = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                                    __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
                }
            }
#pragma unroll
            for (int s = 0; s < kMaxSplits; ++s)
                if (s < splits) part[s] = ld_cluster4(sums_at + (c * kRows + 4 * lane) * 4, s);
            float z[4] = {};
#pragma unroll
            for (int s = 0; s < kMaxSplits; ++s)
                if (s < splits) {
                    z[0] += part[s].x;
                    z[1] += part[s].y;
                    z[2] += part[s].z;
                    z[3] += part[s].w;
                }
            z[0] += bias.x;
            z[1] += bias.y;
            z[2] += bias.z;
            z[3] += bias.w;
            activate(z, p.act);
            const float4 o = make_float4(z[0] + r.x, z[1] + r.y, z[2] + r.z, z[3] + r.w);
            if (p.out_f32) {
                *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = o;
            } else {
                const __nv_bfloat162 a = __floats2bfloat162_rn(o.x, o.y), b = __floats2bfloat162_rn(o.z, o.w);
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.y) + at) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
            }
        }
    }
}

// FINE (fp32 outputs): the tensor cores cut bits off at every step of a sum of 16 products,
// 1.8e-8 of the result and always towards zero: 1.5e-6 of the norm over 6144 products of both
// signs. So their sums end after 512 and are added by the epilogue's threads, which round:
// 2.1e-7. It caps the tokens of a tile at 128, whose sums a thread can hold. The rounding of bf16
// outputs, 1.7e-3, hides all that.
template <int BN, bool FINE>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear(const LinearArgs p, const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x) {
    constexpr int S = stages_of(BN, FINE), PN = panels_of(BN, FINE);
    constexpr uint32_t W_PANEL = kRows * kChunk * 2, X_PANEL = BN * kChunk * 2, SB = stage_bytes(BN, FINE), COLS = 2 * BN < 32 ? 32 : 2 * BN;
    constexpr int RUN = FINE ? 512 / (PN * kChunk) : 1 << 30;   // stages of one sum
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_full[S], s_empty[S], s_done[2], s_free[2], s_drain;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t ring = (bw::saddr(smem_raw) + 1023) & ~1023u;
    const uint32_t sums_at = ring + (FINE ? ring_bytes(BN, true) : 0);
    const uint32_t full = bw::saddr(s_full), empty = bw::saddr(s_empty), done = bw::saddr(s_done), free_ = bw::saddr(s_free);
    // this CTA's share of every tile's K, in chunks
    const int split = p.splits > 1 ? (int)cluster_rank() : 0, chunks = (p.K + PN * kChunk - 1) / (PN * kChunk);
    const int k0 = (int)((int64_t)chunks * split / p.splits), k1 = (int)((int64_t)chunks * (split + 1) / p.splits);
    const int first = blockIdx.x / p.splits, step = gridDim.x / p.splits;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            bw::mbar_init(full + 8 * i, 1);
            bw::mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            bw::mbar_init(done + 8 * i, 1);
            bw::mbar_init(free_ + 8 * i, 4);
        }
        bw::mbar_init(bw::saddr(&s_drain), 1);
        s_abort = 0;
        bw::mbar_fence_init();
        bw::tma_prefetch_desc(&tm_w);
        bw::tma_prefetch_desc(&tm_x);
    }
    if (warp == 5) bw::tmem_alloc(bw::saddr(&s_tmem), COLS);
    bw::tc_fence_before();
    __syncthreads();
    bw::tc_fence_after();
    const uint32_t tmem = *const_cast<volatile uint32_t*>(&s_tmem);
    // the first tile's weights come into the second-level cache while the preceding kernel ends (a
    // hint: what it may still write there is what the copies find)
    if (warp == 4 && lane == 0 && first < p.tiles)
        for (int k = k0; k < min(k1, k0 + S); ++k)
            for (int q = 0; q < PN; ++q) prefetch_2d(&tm_w, (k * PN + q) * kChunk, first % p.row_tiles * kRows);
    pdl_wait();      // nothing of the caller's is read before the preceding kernel is done
    pdl_trigger();
    // a wait that runs out (2^18 tries) sets s_abort, which ends the others: the CTA's outputs are NaN
    auto all = [](bool x) { return __all_sync(~0u, x) != 0; };
    auto wait = [&](uint32_t bar, uint32_t parity) { return bw::mbar_wait_short(bar, parity, &s_abort); };

    if (warp == 4) {
        // copies: each stage a box of W and one of x
        if (lane == 0) {
            const uint64_t stream = bw::l2_evict_first(), keep = bw::l2_evict_last();
            const uint64_t pol_w = p.tiles > p.row_tiles ? keep : stream;
            uint32_t it = 0, copied = 0;
            bool ok = true;
            for (int tile = first; tile < p.tiles && ok; tile += step) {
                const int n0 = tile % p.row_tiles * kRows, t0 = tile / p.row_tiles * BN;
                for (int k = k0; k < k1; ++k, ++it) {
                    const uint32_t s = it % S, at = ring + s * SB;
                    if (!(ok = wait(empty + 8 * s, ((it / S) & 1) ^ 1))) break;
                    bw::mbar_arrive_tx(full + 8 * s, SB);
                    if (tile == p.stall) continue;
                    copied = it + 1;
#pragma unroll
                    for (int q = 0; q < PN; ++q) {
                        bw::tma_load_2d(at + q * W_PANEL, &tm_w, (k * PN + q) * kChunk, n0, full + 8 * s, pol_w);
                        bw::tma_load_2d(at + PN * W_PANEL + q * X_PANEL, &tm_x, (k * PN + q) * kChunk, t0, full + 8 * s, keep);
                    }
                }
            }
            // no copy is in flight at the end, after a wait that ran out either
            int none = 0;
            for (uint32_t q = it > (uint32_t)S ? it - S : 0; q < copied; ++q)
                bw::mbar_wait_short(full + 8 * (q % S), (q / S) & 1, &none);
        }
        // after a wait that ran out a copy may have landed on a split tile's sums
        __syncwarp();
        if (p.splits > 1 && *const_cast<volatile int*>(&s_abort))
            for (int i = lane; i < BN * kRows; i += 32) reinterpret_cast<float*>(smem_raw + (sums_at - bw::saddr(smem_raw)))[i] = NAN;
    } else if (warp == 5) {
        uint32_t it = 0, acc = 0;
        bool ok = true;
        for (int tile = first; tile < p.tiles && ok; tile += step)
            for (int k = k0; k < k1 && ok; ++k, ++it) {
                const bool begins = FINE ? (k - k0) % RUN == 0 : k == k0;
                const bool ends = k == k1 - 1 || (FINE && (k - k0) % RUN == RUN - 1);
                if (begins) {
                    if (!(ok = all(wait(free_ + 8 * (acc & 1), ((acc >> 1) & 1) ^ 1)))) break;
                    bw::tc_fence_after();
                }
                const uint32_t d = tmem + (acc & 1) * BN, s = it % S, at = ring + s * SB;
                if (!(ok = all(wait(full + 8 * s, (it / S) & 1)))) break;
                bw::tc_fence_after();
                if (bw::elect_one()) {
#pragma unroll
                    for (int j = 0; j < PN * kChunk / 16; ++j)
                        bw::mma_f16(d, bw::desc_sw128(at + j / 4 * W_PANEL + 32 * (j % 4)),
                                    bw::desc_sw128(at + PN * W_PANEL + j / 4 * X_PANEL + 32 * (j % 4)),
                                    bw::idesc_16_f32(kRows, BN, true), !begins || j > 0);
                    bw::mma_commit(empty + 8 * s);
                    if (ends) bw::mma_commit(done + 8 * (acc & 1));
                }
                __syncwarp();
                acc += ends;
            }
        if (!ok) {   // no product is running at the end
            if (bw::elect_one()) bw::mma_commit(bw::saddr(&s_drain));
            __syncwarp();
            int none = 0;
            bw::mbar_wait_short(bw::saddr(&s_drain), 0, &none);
        }
    } else {
        const int row = warp * 32 + lane;
        float* const sums = reinterpret_cast<float*>(smem_raw + (sums_at - bw::saddr(smem_raw)));
        uint32_t acc = 0;
        for (int tile = first; tile < p.tiles; tile += step) {
            const int n = tile % p.row_tiles * kRows + row, t0 = tile / p.row_tiles * BN, cols = min(BN, p.T - t0);
            const float bias = p.bias && n < p.N ? p.bias[n] : 0.f;
            float sum[FINE ? BN / 16 : 1][16];
            bool ok = true;
            if constexpr (FINE)
#pragma unroll
                for (int c = 0; c < BN; ++c) sum[c / 16][c % 16] = 0.f;
            for (int k = k0; k < k1; k += min(RUN, k1 - k), ++acc) {
                const bool last = k1 - k <= RUN;
                ok = all(wait(done + 8 * (acc & 1), (acc >> 1) & 1) && !*const_cast<volatile int*>(&s_abort)) && ok;
                bw::tc_fence_after();
                const uint32_t from = tmem + ((uint32_t)(warp * 32) << 16) + (acc & 1) * BN;
                // out of here, or to shared memory: a fine tile's sums behind the ring, a split tile's
                // into it (its copies and products are done)
                if constexpr (FINE) {
#pragma unroll
                    for (int i = 0; i < BN / 16; ++i)
                        if (16 * i < cols) {
                            float v[16];
                            bw::tmem_ld16(from + 16 * i, v);
#pragma unroll
                            for (int j = 0; j < 16; ++j) sum[i][j] += v[j];
                            if (last)
#pragma unroll
                                for (int j = 0; j < 16; ++j) sums[(16 * i + j) * kRows + row] = ok ? sum[i][j] : NAN;
                        }
                } else if (p.splits > 1) {
                    for (int c = 0; c < cols; c += 16) {
                        float v[16];
                        bw::tmem_ld16(from + c, v);
#pragma unroll
                        for (int j = 0; j < 16; ++j) sums[(c + j) * kRows + row] = ok ? v[j] : NAN;
                    }
                } else {
                    for (int c = 0; c < cols; c += 16) {
                        float v[16];
                        bw::tmem_ld16(from + c, v);
                        if (n < p.N) finish16(p, t0 + c, cols - c, n, v, ok ? bias : NAN);
                        __syncwarp();   // the next read of tensor memory is all lanes'
                    }
                }
                bw::tc_fence_before();
                __syncwarp();
                if (lane == 0) bw::mbar_arrive(free_ + 8 * (acc & 1));
            }
            if (FINE && p.splits == 1) {
                asm volatile("bar.sync 1, 128;" ::: "memory");
                finish_shared(p, tile, BN, sums_at, 0, 1, 4);
                __syncwarp();
                asm volatile("bar.sync 1, 128;" ::: "memory");
            }
        }
    }
    __syncwarp();
    if (p.splits > 1) {
        cluster_meet();
        finish_shared(p, first, BN, sums_at, split, p.splits, kThreads / 32);
        __syncwarp();
        cluster_meet();   // no CTA leaves while its sums are read
    }
    bw::tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        bw::tc_fence_after();
        bw::tmem_dealloc(tmem, COLS);
    }
}

using LinearKernel = void (*)(const LinearArgs, const CUtensorMap, const CUtensorMap);
struct Shape {
    int BN;
    LinearKernel kernel;
};
const Shape kShapes[] = {{16, k_linear<16, false>}, {32, k_linear<32, false>}, {64, k_linear<64, false>},
                         {128, k_linear<128, false>}, {256, k_linear<256, false>},
                         {16, k_linear<16, true>}, {32, k_linear<32, true>}, {64, k_linear<64, true>},
                         {128, k_linear<128, true>}};
constexpr int kFine = 5;   // the first of the fine ones

int set_up(int device) {
    int sms = 0;
    if (!tensor_map_encoder()) return 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return 0;
    for (const Shape& s : kShapes)
        if (cudaFuncSetAttribute(s.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing + 1024) != cudaSuccess) return 0;
    return sms;
}
thread_local int t_stall = -1;
PerDevice g_sms, g_clusters[kMaxSplits + 1];

// Clusters of n CTAs that the current device runs at once (every shape takes a whole SM per CTA).
int resident_clusters(int n) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kRing + 1024;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = n;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int active = 0;
    return cudaOccupancyMaxActiveClusters(&active, kShapes[0].kernel, &cfg) == cudaSuccess ? active : 0;
}

bool map_rows(CUtensorMap* tm, const void* base, int K, int rows, int64_t stride, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {kChunk, (cuuint32_t)box_rows}, ones[2] = {1, 1};
    return tensor_map_encoder()(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, ones,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch(const moe_linear_desc& d, const void* x, const void* w, const float* bias, const void* residual, void* y,
                   int T, int device, cudaStream_t stream) {
    const int sms = g_sms.get(device, [&] { return set_up(device); });
    if (!sms) {
        const cudaError_t e = cudaGetLastError();
        return e == cudaSuccess ? cudaErrorNotSupported : e;
    }
    const bool fine = d.out_dtype == MOE_F32;
    const Shape* s = kShapes + (fine ? kFine : 0);
    while (s->BN < T && s->BN < (fine ? 128 : 256)) ++s;
    LinearArgs p{bias, residual, y, d.y_stride, d.residual_stride, T, d.in_features, d.out_features,
                 d.out_dtype == MOE_F32, d.activation, 0, 0, 1, t_stall};
    p.row_tiles = (p.N + kRows - 1) / kRows;
    const int64_t tiles = (int64_t)p.row_tiles * ((T + s->BN - 1) / s->BN);
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    p.tiles = (int)tiles;
    // As many CTAs to a tile as leave all clusters resident at once: the SMs lie in groups, and
    // 48 tiles of 3 CTAs, of which 46 fit, take 25.3 us (one token, 6144 x 6144) where 2 take
    // 16.9; 6 tiles of 8 chunks (512 x 768) 3.2 us by 8 CTAs each, 3.9 by 2.
    const int stage_k = kChunk * panels_of(s->BN, fine), chunks = (p.K + stage_k - 1) / stage_k;
    for (int n = std::min({sms / p.tiles, kMaxSplits, chunks}); n > 1; --n)
        if (g_clusters[n].get(device, [&] { return resident_clusters(n); }) >= p.tiles) {
            p.splits = n;
            break;
        }
    CUtensorMap tm_w, tm_x;
    if (!map_rows(&tm_w, w, p.K, p.N, d.w_stride, kRows) || !map_rows(&tm_x, x, p.K, T, d.x_stride, s->BN))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.splits > 1 ? p.tiles * p.splits : std::min(p.tiles, sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kRing + 1024;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, s->kernel, p, tm_w, tm_x);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_linear_check(const moe_linear_desc* desc, const void* x, const void* w, const float* bias,
                            const void* residual, const void* y, int32_t T) {
    return check_linear(desc, x, w, bias, residual, y, T);
}

moe_status moe_linear_set_option(int32_t option, int64_t value) {
    if (option != MOE_LINEAR_OPT_TEST_STALL) return fail(MOE_E_INVALID, "unknown option");
    if (value < -1 || value > INT32_MAX) return fail(MOE_E_INVALID, "a tile, or -1 for none");
    t_stall = (int)value;
    return MOE_OK;
}

moe_status moe_linear(const moe_linear_desc* desc, const void* x, const void* w, const float* bias,
                      const void* residual, void* y, int32_t T, int32_t device, void* stream) {
    const moe_status st = check_linear(desc, x, w, bias, residual, y, T);
    if (st != MOE_OK || T == 0) return st;
    if (overwrites(*desc, x, w, bias, residual, y, T))
        return fail(MOE_E_INVALID, "y overlaps an input (residual may be y itself, with y's stride)");
    DeviceGuard g(device);
    if (!g.ok) return cuda_fail(g.err, "cudaSetDevice");
    const cudaError_t e = launch(*desc, x, w, bias, residual, y, T, device, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "linear launch");
}

}  // extern "C"
