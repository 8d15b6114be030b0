// Attention of one new token per sequence over a paged key-value cache.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "kv_cache.h"
#include "moe_internal.h"

namespace moe {

namespace {

struct AttendArgs {
    moe_kv_attend_args a;
    KvShape s;
    const void *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    unsigned* health;
};

constexpr int kWarps = 4;

__device__ __forceinline__ float load_cached(const void* pool, int e4m3, int64_t at) {
    if (!e4m3) return __bfloat162float(static_cast<const __nv_bfloat16*>(pool)[at]);
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(pool)[at], __NV_E4M3);
    return __half2float(__half(h));
}

// One CTA per (query head, sequence): the warps take positions in turn, a lane
// holds D / 32 channels, the softmax runs with a running maximum and sum, and
// the warps' results are joined in shared memory.
template <int D>
__global__ void __launch_bounds__(32 * kWarps) k_kv_attend_rows(const AttendArgs p) {
    constexpr int C = D / 32;
    __shared__ float sm_o[kWarps][D], sm_m[kWarps], sm_l[kWarps];
    const KvShape& s = p.s;
    const int head = blockIdx.x, b = blockIdx.y, hk = head / (s.n_heads / s.n_kv_heads);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    uint32_t bits = 0;
    int len = max(p.a.lens[b], 0);
    if (len > p.a.max_pages * s.page_size) {
        len = p.a.max_pages * s.page_size;
        bits |= MOE_KV_BAD_LENGTH;
    }
    const int first = p.a.window > 0 ? max(0, len - p.a.window) : 0;
    const float ks = p.k_scale[hk], vs = p.v_scale[hk];
    float q[C], o[C], m = -INFINITY, l = 0.f;
    for (int c = 0; c < C; ++c) {
        q[c] = __bfloat162float(static_cast<const __nv_bfloat16*>(
            p.a.q)[(int64_t)b * p.a.q_stride + (int64_t)head * D + lane + 32 * c]);
        o[c] = 0.f;
    }
    for (int j = first + warp; j < len; j += kWarps) {
        const int page = kv_page(s, p.a.block_table, p.a.B, p.a.max_pages, b, j, bits);
        if (page < 0) continue;
        const int64_t at = kv_offset(s, page, hk, j % s.page_size) + lane;
        float x = 0.f;
        for (int c = 0; c < C; ++c) x += q[c] * load_cached(p.k_pages, s.e4m3, at + 32 * c);
        for (int i = 16; i; i >>= 1) x += __shfl_xor_sync(~0u, x, i);
        x *= p.a.scale * ks;
        if (p.a.softcap > 0.f) x = p.a.softcap * tanhf(x / p.a.softcap);
        const float mn = fmaxf(m, x), w = expf(x - mn), f = m == -INFINITY ? 0.f : expf(m - mn);
        l = l * f + w;
        for (int c = 0; c < C; ++c) o[c] = o[c] * f + w * load_cached(p.v_pages, s.e4m3, at + 32 * c);
        m = mn;
    }
    for (int c = 0; c < C; ++c) sm_o[warp][lane + 32 * c] = o[c];
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
        if (bits) atomicOr(p.health, bits);
    }
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w]);
    for (int w = 0; w < kWarps; ++w) L += sm_m[w] == -INFINITY ? 0.f : sm_l[w] * expf(sm_m[w] - M);
    for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
        float x = 0.f;
        for (int w = 0; w < kWarps; ++w) x += sm_m[w] == -INFINITY ? 0.f : sm_o[w][d] * expf(sm_m[w] - M);
        static_cast<__nv_bfloat16*>(p.a.out)[((int64_t)b * s.n_heads + head) * D + d] =
            __float2bfloat16_rn(L == 0.f ? 0.f : x * vs / L);
    }
    if (p.a.lse && threadIdx.x == 0)
        p.a.lse[(int64_t)b * s.n_heads + head] = L == 0.f ? -INFINITY : M + logf(L);
}

}  // namespace

moe_status kv_attend_launch(Kv& K, const moe_kv_attend_args& a, cudaStream_t stream) {
    const AttendArgs p{a, K.s, K.k_pages, K.v_pages, K.k_scale, K.v_scale, K.health};
    const dim3 grid(K.s.n_heads, a.B);
    if (K.s.head_dim == 64) k_kv_attend_rows<64><<<grid, 32 * kWarps, 0, stream>>>(p);
    else if (K.s.head_dim == 128) k_kv_attend_rows<128><<<grid, 32 * kWarps, 0, stream>>>(p);
    else k_kv_attend_rows<256><<<grid, 32 * kWarps, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "attend launch");
}

}  // namespace moe
