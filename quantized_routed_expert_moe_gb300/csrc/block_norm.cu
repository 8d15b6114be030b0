// The step between two blocks of a decoder layer: the norm after a block, its
// gate and residual scale, the residual sum, and the norm before the next block.
#include <cuda_bf16.h>

#include <cmath>
#include <string>

#include "moe_internal.h"

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

struct NormArgs {
    moe_block_norm_desc d;
    const void *x, *o, *gate;
    const float *w_post, *w_pre;
    void *r, *h;
    int T;
};

__device__ __forceinline__ float load_as(const void* p, int t, int64_t i) {
    return t == MOE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store_as(void* p, int t, int64_t i, float v) {
    if (t == MOE_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<float*>(p)[i] = v;
}

constexpr int kThreads = 256;

__device__ float block_sum(float v, float* sm) {
    for (int i = 16; i; i >>= 1) v += __shfl_xor_sync(~0u, v, i);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sm[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < kThreads / 32; ++i) v += sm[i];
    return v;
}

// One CTA per row; the row of r in shared memory, in fp32.
__global__ void __launch_bounds__(kThreads) k_block_norm_rows(const NormArgs p) {
    extern __shared__ float row[];
    __shared__ float sm[kThreads / 32];
    const moe_block_norm_desc& d = p.d;
    const int H = d.hidden;
    for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
        float inv = 1.f;
        if (p.w_post) {
            float ss = 0.f;
            for (int i = threadIdx.x; i < H; i += kThreads) {
                const float v = load_as(p.o, d.block_dtype, t * d.o_stride + i);
                ss += v * v;
            }
            inv = 1.f / sqrtf(block_sum(ss, sm) / H + d.eps);
        }
        float ss = 0.f;
        for (int i = threadIdx.x; i < H; i += kThreads) {
            float v = load_as(p.x, d.res_dtype, t * d.x_stride + i);
            if (p.o) {
                float a = load_as(p.o, d.block_dtype, t * d.o_stride + i) * inv;
                if (p.w_post) a *= p.w_post[i] + d.weight_offset;
                if (p.gate) a *= load_as(p.gate, d.block_dtype, t * d.gate_stride + i);
                v += d.res_scale * a;
            }
            row[i] = v;
            ss += v * v;
            if (p.r) store_as(p.r, d.res_dtype, t * d.r_stride + i, v);
        }
        if (!p.h) continue;
        inv = 1.f / sqrtf(block_sum(ss, sm) / H + d.eps);
        for (int i = threadIdx.x; i < H; i += kThreads)
            store_as(p.h, d.out_dtype, t * d.h_stride + i, row[i] * inv * (p.w_pre[i] + d.weight_offset));
    }
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
    const NormArgs p{*desc, x, o, gate, w_post, w_pre, r, h, T};
    const size_t smem = (size_t)desc->hidden * 4;
    cudaError_t e = cudaFuncSetAttribute(k_block_norm_rows, cudaFuncAttributeMaxDynamicSharedMemorySize, 65536);
    if (e == cudaSuccess) {
        k_block_norm_rows<<<T < 4096 ? T : 4096, kThreads, smem, static_cast<cudaStream_t>(stream)>>>(p);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "block norm launch");
}

}  // extern "C"
