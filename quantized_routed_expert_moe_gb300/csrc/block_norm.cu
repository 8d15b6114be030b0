// The step between two blocks of a decoder layer: the norm after a block, its
// gate and residual scale, the residual sum, and the norm before the next block.
#include <cuda_bf16.h>

#include <cmath>
#include <string>

#include "common.cuh"
#include "moe_internal.h"
#include "per_device.h"

namespace moe {

namespace {

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

bool is_act(int t) { return t == MOE_F32 || t == MOE_BF16; }

moe_status check_norm(const moe_block_norm_desc* d, const void* x, const void* o, const void* gate,
                      const float* w_post, const float* w_pre, const void* r, const void* h, int T) {
    if (!d) return fail(MOE_E_INVALID, "desc is NULL");
    if (d->abi_version != MOE_ABI_VERSION) return fail(MOE_E_INVALID, "abi_version mismatch");
    if (d->hidden <= 0 || d->hidden % 64) return fail(MOE_E_INVALID, "hidden must be a positive multiple of 64");
    if (d->hidden > 16384) return fail(MOE_E_UNSUPPORTED, "hidden is limited to 16384");
    if (!is_act(d->res_dtype) || !is_act(d->block_dtype) || !is_act(d->out_dtype))
        return fail(MOE_E_INVALID, "res_dtype, block_dtype and out_dtype must be MOE_F32 or MOE_BF16");
    if (!std::isfinite(d->eps) || d->eps < 0) return fail(MOE_E_INVALID, "eps must be finite and >= 0");
    if (!std::isfinite(d->res_scale) || !std::isfinite(d->weight_offset))
        return fail(MOE_E_INVALID, "res_scale and weight_offset must be finite");
    if (T < 0) return fail(MOE_E_INVALID, "T must not be negative");
    if (T == 0) return MOE_OK;
    if (!x) return fail(MOE_E_INVALID, "x is NULL");
    if (!r && !h) return fail(MOE_E_INVALID, "r and h are both NULL");
    if (!o && (gate || w_post)) return fail(MOE_E_INVALID, "gate and w_post need o");
    if ((h != nullptr) != (w_pre != nullptr)) return fail(MOE_E_INVALID, "h and w_pre go together");
    for (const void* p : {x, o, gate, static_cast<const void*>(w_post), static_cast<const void*>(w_pre), r, h})
        if (!aligned16(p)) return fail(MOE_E_INVALID, "pointers must be 16-byte aligned");
    const struct { const void* p; int64_t st; const char* n; } rows[] = {
        {x, d->x_stride, "x_stride"}, {o, d->o_stride, "o_stride"}, {r, d->r_stride, "r_stride"}, {h, d->h_stride, "h_stride"}};
    for (const auto& w : rows)
        if (w.p && (w.st % 8 || w.st < d->hidden))
            return fail(MOE_E_INVALID, std::string(w.n) + " must be a multiple of 8, at least hidden");
    if (gate && d->gate_stride != 0 && (d->gate_stride % 8 || d->gate_stride < d->hidden))
        return fail(MOE_E_INVALID, "gate_stride must be 0, or a multiple of 8 of at least hidden");
    if (r == x && r && d->r_stride != d->x_stride) return fail(MOE_E_INVALID, "r may be x only with x's stride");
    return MOE_OK;
}

constexpr int kSlotBytes = 226 * 1024;   // shared memory of a CTA beside its sums

struct NormArgs {
    moe_block_norm_desc d;
    const void *x, *o, *gate;
    const float *w_post, *w_pre;
    void *r, *h;
    int T;
    bool near;   // the weights are in shared memory
    int device;
};

// A row is cut into tiles of 256 channels; a lane holds channels 4 lane.. and 128 +
// 4 lane.. of its tiles, so that fp32 and bf16 rows are both read in whole lines.
// Rows pass once, around L1. Not the read-only path, as r may be written over x.
template <typename T>
__device__ __forceinline__ float4 load4(const T* p) {
    if constexpr (sizeof(T) == 4) {
        float4 v;
        asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
        return v;
    } else {
        uint2 v;
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
        return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                           __uint_as_float(v.y & 0xffff0000u));
    }
}
// The same by way of shared memory, in the thread's own slot: nothing to wait for but
// the thread's own copies.
template <typename T>
__device__ __forceinline__ void copy4(uint32_t slot, const T* p) {
    if constexpr (sizeof(T) == 4) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot), "l"(p) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(slot), "l"(p) : "memory");
}
template <typename T>
__device__ __forceinline__ float4 slot4(uint32_t slot) {
    if constexpr (sizeof(T) == 4) {
        float4 v;
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(slot) : "memory");
        return v;
    } else {
        uint2 v;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(slot) : "memory");
        return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                           __uint_as_float(v.y & 0xffff0000u));
    }
}
template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = v;
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(p) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
}
__device__ __forceinline__ void put4(uint32_t slot, float4 v) {
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(slot), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ float4 times(float4 a, float4 b) {
    return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}
__device__ __forceinline__ float sq(float4 v) { return v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w; }

// A row's sum over its warps, in a fixed order. `sm` is used again only after the
// row's other sum, whose barrier every reader of this one has passed.
template <bool CTA>
__device__ __forceinline__ float row_sum(float v, float* sm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if constexpr (CTA) {
        const int lane = threadIdx.x % 32;
        if (lane == 0) sm[threadIdx.x / 32] = v;
        __syncthreads();
        v = lane < blockDim.x / 32 ? sm[lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    }
    return v;
}

// The rows are independent streams: read x, o and gate once, write r and h once,
// with two sums over the row between (of o, then of r). A row stays in the registers
// of one CTA (CTA) or of one warp, K tiles per warp. Where a CTA has many rows (AHEAD),
// a thread copies its channels of the next row into shared memory, so that they are on
// their way while this one waits for its sums (two rows ahead: from 13% faster, fp32 x of
// 5120, to 14% slower, bf16 of 2816; one is kept). Measured: 8191 rows of 6144 (fp32 x and
// r, bf16 o, gate and h) 108.5 us, 6.5 TB/s, 96% of the copy rate; 4000 rows of 2816 in
// bf16 18.2 us; 8191 rows of 1024 in bf16 15.6 us; one row of 6144 3.0 us, a chain of two
// sums. The wider a row, the more of its CTA's time the two meetings take, and above 8192
// channels an SM holds one CTA: 3001 rows of 12352 in bf16 with rows of gates 75.2 us, 73% of
// the copy rate, and r alone, without the norms, 88%.
template <typename R, typename B, typename O, int K, bool CTA, bool AHEAD, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k_block_norm(const NormArgs p) {
    __shared__ float sm[2][32];
    extern __shared__ __align__(16) uint8_t slots[];
    const moe_block_norm_desc& d = p.d;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int warps = CTA ? blockDim.x / 32 : 1;
    const int per = CTA ? 1 : blockDim.x / 32;   // rows of a CTA at a time
    const int c0 = (CTA ? warp * 256 : 0) + lane * 4, left = d.hidden - c0;
    const float inv_h = 1.f / d.hidden;
    // vector (k, i) is channels c0 + at(k, i) ..
    auto at = [&](int k, int i) { return k * warps * 256 + i * 128; };
    // slots of this thread: x's vectors of the next row, o's, and the gate's where it has rows;
    // then the weights, which every row takes
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(slots);
    const uint32_t dx = blockDim.x * 4 * sizeof(R), db = blockDim.x * 4 * sizeof(B);   // between vectors
    const uint32_t dw = (CTA ? blockDim.x : 32) * 16;   // warps with a row each share the weights
    const uint32_t sx = base + threadIdx.x * 4 * sizeof(R), so = base + 2 * K * dx + threadIdx.x * 4 * sizeof(B);
    const bool gate_rows = p.gate && d.gate_stride != 0, gate_row = p.gate && d.gate_stride == 0;
    const bool weighted = p.w_post || (AHEAD && gate_row);
    const uint32_t sg = so + 2 * K * db, stage = 2 * K * (dx + (gate_rows ? 2 : 1) * db);
    const uint32_t sw = base + stage + (CTA ? threadIdx.x : lane) * 16, sn = sw + (weighted ? 2 * K * dw : 0);
    const int t0 = blockIdx.x * per + (CTA ? 0 : warp), step = gridDim.x * per;
    pdl_wait();      // nothing of the caller's is read before the preceding kernel is done
    pdl_trigger();
    if (t0 >= p.T) return;   // a whole CTA, or a warp that meets no other
    const R* x = static_cast<const R*>(p.x) + t0 * d.x_stride + c0;
    const B* o = static_cast<const B*>(p.o) + t0 * d.o_stride + c0;
    const B* gate = static_cast<const B*>(p.gate) + t0 * d.gate_stride + c0;
    R* ro = static_cast<R*>(p.r) + t0 * d.r_stride + c0;
    O* ho = static_cast<O*>(p.h) + t0 * d.h_stride + c0;
    auto next_row = [&] {
        x += step * d.x_stride;
        o += step * d.o_stride;
        gate += step * d.gate_stride;
    };
    auto fetch = [&] {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (at(k, i) < left) {
                    copy4(sx + (2 * k + i) * dx, x + at(k, i));
                    if (p.o) copy4(so + (2 * k + i) * db, o + at(k, i));
                    if (gate_rows) copy4(sg + (2 * k + i) * db, gate + at(k, i));
                }
        next_row();
    };
    auto weight = [&](const float* w, int k, int i) {
        const float4 v = *reinterpret_cast<const float4*>(w + c0 + at(k, i));
        return make_float4(v.x + d.weight_offset, v.y + d.weight_offset, v.z + d.weight_offset, v.w + d.weight_offset);
    };
    // o's factor that every row takes
    auto factor = [&](int k, int i) {
        float4 w = p.w_post ? weight(p.w_post, k, i) : make_float4(1.f, 1.f, 1.f, 1.f);
        if (gate_row) w = times(w, load4(static_cast<const B*>(p.gate) + c0 + at(k, i)));
        return w;
    };
    // only rows above 8192 channels can have their weights elsewhere: up to there a row and its
    // weights take at most 160 KB
    const bool near = AHEAD && (K * MAXT <= 1024 || p.near);
    if constexpr (AHEAD) {
        fetch();
        // a gate of one row is a weight too (where warps share the weights, each writes them all:
        // the same values, and it reads what it wrote)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (near && at(k, i) < left) {
                    if (weighted) put4(sw + (2 * k + i) * dw, factor(k, i));
                    if (p.h) put4(sn + (2 * k + i) * dw, weight(p.w_pre, k, i));
                }
    }

    for (int64_t t = t0; t < p.T; t += step) {
        float4 r[K][2], a[K][2];
        if constexpr (AHEAD) asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool on = at(k, i) < left;
                r[k][i] = a[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (on) r[k][i] = AHEAD ? slot4<R>(sx + (2 * k + i) * dx) : load4(x + at(k, i));
                if (on && p.o) a[k][i] = AHEAD ? slot4<B>(so + (2 * k + i) * db) : load4(o + at(k, i));
            }
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) ss += sq(a[k][i]);
        if (AHEAD ? gate_rows : p.gate != nullptr) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (at(k, i) < left)
                        a[k][i] = times(a[k][i], AHEAD ? slot4<B>(sg + (2 * k + i) * db) : load4(gate + at(k, i)));
        }
        if constexpr (AHEAD) {
            if (t + step < p.T) fetch();
        } else {
            next_row();
        }
        float f = d.res_scale;
        if (p.w_post) f *= rsqrtf(row_sum<CTA>(ss, sm[0]) * inv_h + d.eps);
        if (weighted) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (at(k, i) < left)
                        a[k][i] = times(a[k][i], near    ? slot4<float>(sw + (2 * k + i) * dw)
                                                 : AHEAD ? factor(k, i)
                                                         : weight(p.w_post, k, i));
        }
        ss = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                r[k][i] = make_float4(r[k][i].x + f * a[k][i].x, r[k][i].y + f * a[k][i].y, r[k][i].z + f * a[k][i].z,
                                      r[k][i].w + f * a[k][i].w);
                ss += sq(r[k][i]);
                if (p.r && at(k, i) < left) store4(ro + at(k, i), r[k][i]);
            }
        ro += step * d.r_stride;
        if (p.h) {
            const float inv = rsqrtf(row_sum<CTA>(ss, sm[1]) * inv_h + d.eps);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (at(k, i) < left) {
                        const float4 w = near ? slot4<float>(sn + (2 * k + i) * dw) : weight(p.w_pre, k, i), v = r[k][i];
                        store4(ho + at(k, i), times(make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv), w));
                    }
        }
        ho += step * d.h_stride;
        // a row with one sum only: its readers meet before the next row's sum
        if (CTA && !(p.w_post && p.h)) __syncthreads();
    }
}

// CTAs of a kernel that the device holds at a time, 0 with `e` set on failure. `held` keeps it;
// the attribute counts for the current device alone.
int resident(const void* kernel, int threads, size_t smem, int device, PerDevice& held, cudaError_t& e) {
    e = cudaSuccess;
    return held.get(device, [&] {
        int sms = 0, n = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
        if (e == cudaSuccess && smem)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSlotBytes);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
        return e == cudaSuccess ? sms * (n > 0 ? n : 1) : 0;
    });
}

// Few rows: each has a CTA or a warp of its own. Returns whether the device holds them all.
template <typename R, typename B, typename O, int K, bool CTA, int MAXT, int MINB>
bool launch_few(const NormArgs& p, int threads, cudaStream_t s, cudaError_t& e) {
    const auto kernel = k_block_norm<R, B, O, K, CTA, false, MAXT, MINB>;
    const int per = CTA ? 1 : threads / 32, need = (p.T - 1) / per + 1;
    static PerDevice kept[33];       // by warps of a CTA
    const int held = resident(reinterpret_cast<const void*>(kernel), threads, 0, p.device, kept[threads / 32], e);
    if (!held) return true;
    if (need > held) return false;
    e = launch_pdl(kernel, dim3(need), dim3(threads), 0, s, true, p);
    return true;
}

// Many rows: resident CTAs that copy a row ahead. A row above some 11000 channels may leave
// no room for its weights beside it (128 KB for 16384): they are then read for every row.
template <typename R, typename B, typename O, int K, bool CTA, int MAXT, int MINB>
cudaError_t launch_many(NormArgs p, int threads, cudaStream_t s) {
    const auto kernel = k_block_norm<R, B, O, K, CTA, true, MAXT, MINB>;
    const int per = CTA ? 1 : threads / 32, need = (p.T - 1) / per + 1;
    const bool gate_rows = p.gate && p.d.gate_stride != 0;
    const int inputs = gate_rows ? 2 : 1, kept = (p.w_post || (p.gate && !gate_rows)) + (p.h != nullptr);
    const size_t stage = (size_t)threads * 2 * K * 4 * (sizeof(R) + inputs * sizeof(B));
    const size_t weights = (size_t)(CTA ? threads : 32) * 2 * K * 16 * kept;
    p.near = stage + weights <= kSlotBytes;
    const size_t smem = stage + (p.near ? weights : 0);
    static PerDevice kinds[33][2][3];   // the same warps, inputs and weights take the same shared memory
    cudaError_t e;
    const int held = resident(reinterpret_cast<const void*>(kernel), threads, smem, p.device,
                              kinds[threads / 32][inputs - 1][kept], e);
    if (!held) return e;
    return launch_pdl(kernel, dim3(need < held ? need : held), dim3(threads), smem, s, true, p);
}

// By the row's tiles of 256 channels: a warp for one, above that a CTA with a warp per
// tile (a warp with two to four tiles took 5 to 35% longer over 1024 to 6144 channels,
// and a warp per row as much over 512 to 1024), above 32 a warp per two. Many rows of up
// to 18 tiles hold two CTAs per SM or more, with 56 registers; of 16-bit rows of 19 to 24
// tiles, half as many warps with two tiles each do (57.6 against 68.6 us at 5120).
template <typename R, typename B, typename O>
cudaError_t launch_row(const NormArgs& p, cudaStream_t s) {
    const int n = (p.d.hidden + 255) / 256;
    cudaError_t e;
    if (n == 1)
        return launch_few<R, B, O, 1, false, 256, 4>(p, 256, s, e) ? e : launch_many<R, B, O, 1, false, 256, 4>(p, 256, s);
    if (n <= 32) {
        if (launch_few<R, B, O, 1, true, 1024, 1>(p, n * 32, s, e)) return e;
        if (n <= 18) return launch_many<R, B, O, 1, true, 576, 2>(p, n * 32, s);
        if constexpr (sizeof(R) + sizeof(B) + sizeof(O) == 6)
            if (n <= 24) return launch_many<R, B, O, 2, true, 384, 2>(p, (n + 1) / 2 * 32, s);
        return launch_many<R, B, O, 1, true, 1024, 1>(p, n * 32, s);
    }
    const int threads = (n + 1) / 2 * 32;
    return launch_few<R, B, O, 2, true, 1024, 1>(p, threads, s, e) ? e : launch_many<R, B, O, 2, true, 1024, 1>(p, threads, s);
}

template <typename R, typename B>
cudaError_t launch_out(const NormArgs& p, cudaStream_t s) {
    return p.d.out_dtype == MOE_F32 ? launch_row<R, B, float>(p, s) : launch_row<R, B, __nv_bfloat16>(p, s);
}

template <typename R>
cudaError_t launch_block(const NormArgs& p, cudaStream_t s) {
    return p.d.block_dtype == MOE_F32 ? launch_out<R, float>(p, s) : launch_out<R, __nv_bfloat16>(p, s);
}

cudaError_t launch(const NormArgs& p, cudaStream_t s) {
    return p.d.res_dtype == MOE_F32 ? launch_block<float>(p, s) : launch_block<__nv_bfloat16>(p, s);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_block_norm_check(const moe_block_norm_desc* desc, const void* x, const void* o, const void* gate,
                                const float* w_post, const float* w_pre, const void* r, const void* h, int32_t T) {
    return check_norm(desc, x, o, gate, w_post, w_pre, r, h, T);
}

moe_status moe_block_norm(const moe_block_norm_desc* desc, const void* x, const void* o, const void* gate,
                          const float* w_post, const float* w_pre, void* r, void* h, int32_t T,
                          int32_t device, void* stream) {
    const moe_status st = check_norm(desc, x, o, gate, w_post, w_pre, r, h, T);
    if (st != MOE_OK || T == 0) return st;
    DeviceGuard g(device);
    if (!g.ok) return cuda_fail(g.err, "cudaSetDevice");
    const NormArgs p{*desc, x, o, gate, w_post, w_pre, r, h, T, true, device};
    const cudaError_t e = launch(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "block norm launch");
}

}  // extern "C"
