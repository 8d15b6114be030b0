// y = act(x W^T + bias) + residual over token rows: tiles of 64 x 64 on the CUDA cores.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "common.cuh"
#include "moe_internal.h"

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

__device__ __forceinline__ float activate(float z, int act) {
    if (act == MOE_ACT_SILU) return z / (1.f + expf(-z));
    if (act == MOE_ACT_GELU_TANH) return 0.5f * z * (1.f + tanhf(0.7978845608028654f * (z + 0.044715f * z * z * z)));
    if (act == MOE_ACT_SIGMOID) return 1.f / (1.f + expf(-z));
    return z;
}

struct LinearArgs {
    moe_linear_desc d;
    const __nv_bfloat16 *x, *w;
    const float* bias;
    const void* residual;
    void* y;
    int T;
};

__global__ void __launch_bounds__(256) k_linear(const LinearArgs p) {
    __shared__ float xs[64][17], ws[64][17];
    const int K = p.d.in_features, N = p.d.out_features, n0 = blockIdx.x * 64, t0 = blockIdx.y * 64;
    pdl_wait();
    pdl_trigger();
    float c[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += 16) {
        for (int i = threadIdx.x; i < 64 * 16; i += 256) {
            const int r = i / 16, k = k0 + i % 16;
            xs[r][i % 16] = t0 + r < p.T && k < K ? __bfloat162float(p.x[(t0 + r) * p.d.x_stride + k]) : 0.f;
            ws[r][i % 16] = n0 + r < N && k < K ? __bfloat162float(p.w[(n0 + r) * p.d.w_stride + k]) : 0.f;
        }
        __syncthreads();
        for (int k = 0; k < 16; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) c[i][j] += xs[threadIdx.x / 16 + 16 * i][k] * ws[threadIdx.x % 16 + 16 * j][k];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int t = t0 + threadIdx.x / 16 + 16 * i, n = n0 + threadIdx.x % 16 + 16 * j;
            if (t >= p.T || n >= N) continue;
            float z = activate(c[i][j] + (p.bias ? p.bias[n] : 0.f), p.d.activation);
            const int64_t at = t * p.d.y_stride + n, rt = t * p.d.residual_stride + n;
            if (p.d.out_dtype == MOE_F32) {
                if (p.residual) z += static_cast<const float*>(p.residual)[rt];
                static_cast<float*>(p.y)[at] = z;
            } else {
                if (p.residual) z += __bfloat162float(static_cast<const __nv_bfloat16*>(p.residual)[rt]);
                static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16(z);
            }
        }
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_linear_check(const moe_linear_desc* desc, const void* x, const void* w, const float* bias,
                            const void* residual, const void* y, int32_t T) {
    return check_linear(desc, x, w, bias, residual, y, T);
}

moe_status moe_linear(const moe_linear_desc* desc, const void* x, const void* w, const float* bias,
                      const void* residual, void* y, int32_t T, int32_t device, void* stream) {
    const moe_status st = check_linear(desc, x, w, bias, residual, y, T);
    if (st != MOE_OK || T == 0) return st;
    DeviceGuard g(device);
    if (!g.ok) return cuda_fail(g.err, "cudaSetDevice");
    const LinearArgs p{*desc, static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(w), bias, residual, y, T};
    const dim3 grid((desc->out_features + 63) / 64, (T + 63) / 64);
    const cudaError_t e = launch_pdl(k_linear, grid, dim3(256), 0, static_cast<cudaStream_t>(stream), true, p);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "linear launch");
}

}  // extern "C"
