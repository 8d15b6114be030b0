// Attention of a chunk of new tokens per sequence over a paged key-value cache: a warp
// per token and query head, its cached positions one after the other.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"
#include "kv_cache.h"
#include "moe_internal.h"

namespace moe {

namespace {

struct ChunkArgs {
    moe_kv_chunk_args a;
    KvShape s;
    const void *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    unsigned* health;
};

__device__ __forceinline__ float cached(const void* pool, int64_t at, int e4m3) {
    return e4m3 ? (float)static_cast<const __nv_fp8_e4m3*>(pool)[at]
                : __bfloat162float(static_cast<const __nv_bfloat16*>(pool)[at]);
}

template <int D>
__global__ void __launch_bounds__(256) k_kv_chunk(const ChunkArgs p) {
    constexpr int C = D / 32;
    const KvShape& s = p.s;
    const int lane = threadIdx.x % 32, heads = s.n_heads;
    pdl_wait();
    pdl_trigger();
    uint32_t bits = 0;
    bool bad = p.a.starts[0] < 0 || p.a.starts[p.a.B] > p.a.T;
    for (int b = 0; b < p.a.B; ++b) bad |= p.a.starts[b] > p.a.starts[b + 1];
    if (bad) {
        if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(p.health, MOE_KV_BAD_START);
        return;
    }
    const int first = p.a.starts[0], rows = p.a.starts[p.a.B] - first;
    for (int64_t w = blockIdx.x * 8 + threadIdx.x / 32; w < (int64_t)rows * heads; w += gridDim.x * 8) {
        const int t = first + (int)(w / heads), head = (int)(w % heads), hk = head / (heads / s.n_kv_heads);
        int b = 0;
        while (p.a.starts[b + 1] <= t) ++b;
        const int most = p.a.max_pages * s.page_size;
        int len = p.a.lens[b];
        if (len > most) {
            bits |= MOE_KV_BAD_LENGTH;
            len = most;
        }
        const int pos = len - (p.a.starts[b + 1] - t);
        float q[C], o[C] = {}, m = -INFINITY, l = 0.f;
        for (int c = 0; c < C; ++c)
            q[c] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.a.q)[t * p.a.q_stride + head * D + 32 * c + lane]);
        const float ks = p.k_scale[hk], vs = p.v_scale[hk];
        for (int j = p.a.window > 0 ? max(0, pos - p.a.window + 1) : 0; j <= pos; ++j) {
            const int page = kv_page(s, p.a.block_table[(int64_t)b * p.a.max_pages + j / s.page_size], bits);
            if (page < 0) continue;
            const int64_t at = kv_offset(s, page, hk, j % s.page_size) + lane;
            float z = 0.f;
            for (int c = 0; c < C; ++c) z += q[c] * cached(p.k_pages, at + 32 * c, s.e4m3);
            z = warp_sum(z) * ks * p.a.scale;
            if (p.a.softcap > 0) z = p.a.softcap * tanhf(z / p.a.softcap);
            const float mn = fmaxf(m, z), base = mn == -INFINITY ? 0.f : mn, f = expf(m - base), e = expf(z - base);
            l = l * f + e;
            for (int c = 0; c < C; ++c) o[c] = o[c] * f + e * cached(p.v_pages, at + 32 * c, s.e4m3);
            m = mn;
        }
        const float r = l == 0.f ? 0.f : vs / l;
        for (int c = 0; c < C; ++c)
            static_cast<__nv_bfloat16*>(p.a.out)[((int64_t)t * heads + head) * D + 32 * c + lane] = __float2bfloat16(o[c] * r);
        if (lane == 0 && p.a.lse) p.a.lse[(int64_t)t * heads + head] = l == 0.f ? -INFINITY : m + logf(l);
    }
    if (bits) atomicOr(p.health, bits);
}

}  // namespace

size_t kv_chunk_workspace(const Kv&) { return 256; }
cudaError_t kv_chunk_setup(Kv&) { return cudaSuccess; }

moe_status kv_chunk_launch(Kv& K, const moe_kv_chunk_args& a, cudaStream_t stream) {
    const ChunkArgs p{a, K.s, K.k_pages, K.v_pages, K.k_scale, K.v_scale, K.health};
    const auto kernel = K.s.head_dim == 64 ? k_kv_chunk<64> : K.s.head_dim == 128 ? k_kv_chunk<128> : k_kv_chunk<256>;
    const unsigned grid = (unsigned)std::min<int64_t>(((int64_t)a.T * K.s.n_heads + 7) / 8, (int64_t)K.num_sms * 8);
    const cudaError_t e = launch_pdl(kernel, dim3(grid), dim3(256), 0, stream, true, p);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "attend chunk launch");
}

}  // namespace moe
