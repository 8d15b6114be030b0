// The paged key-value cache: what its translation units share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "moe.h"

namespace moe {

// Shape and strides of a cache as the kernels see them.
struct KvShape {
    int n_heads, n_kv_heads, head_dim, page_size, n_pages, rotary_dim, rotary_adjacent, e4m3;
    int64_t page_stride, head_stride, token_stride;  // elements
};

// Index of (seq, position)'s entry in the block table, or -1 with a health bit.
__host__ __device__ inline int64_t kv_entry(const KvShape& s, int n_seqs, int max_pages, int seq, int position,
                                            uint32_t& bits) {
    if (seq < 0 || seq >= n_seqs) {
        bits |= MOE_KV_BAD_SEQ;
        return -1;
    }
    const int at = position / s.page_size;
    if (position < 0 || at >= max_pages) {
        bits |= MOE_KV_BAD_LENGTH;
        return -1;
    }
    return (int64_t)seq * max_pages + at;
}

// A page read from the block table, or -1 with a health bit.
__host__ __device__ inline int kv_page(const KvShape& s, int page, uint32_t& bits) {
    if (page >= 0 && page < s.n_pages) return page;
    bits |= MOE_KV_BAD_PAGE;
    return -1;
}

// Element offset of a row of a pool; 64-bit throughout.
__host__ __device__ inline int64_t kv_offset(const KvShape& s, int page, int head, int slot) {
    return (int64_t)page * s.page_stride + (int64_t)head * s.head_stride + (int64_t)slot * s.token_stride;
}

struct Kv {
    moe_kv_desc d{};
    KvShape s{};
    int device = 0, num_sms = 0;
    void *k_pages = nullptr, *v_pages = nullptr;
    uint64_t* turns = nullptr;   // [rotary_dim / 2] turns per position, as a fraction of 2^64
    float *k_scale = nullptr, *v_scale = nullptr;  // [n_kv_heads], ones for a bf16 cache
    float2* scales = nullptr;    // [2][n_kv_heads], as append takes them: scale and its rounded reciprocal
    unsigned* health = nullptr;
    // attention: the page pools as tensor maps, the parts of segments that are cut between
    // CTAs, and how many of a segment's CTAs have arrived
    CUtensorMap tm_k{}, tm_v{};
    int box_rows = 16;
    int stall = -1;              // MOE_KV_OPT_TEST_STALL
    float4 *part_o = nullptr, *part_ml = nullptr;
    int* arrived = nullptr;
    void* block = nullptr;       // the allocation that holds all of the above
    size_t device_bytes = 0;
};

// Bytes of part_o, part_ml and arrived; needs K.d, K.s and K.num_sms.
size_t kv_attend_workspace(const Kv& K, size_t out[3]);
cudaError_t kv_attend_setup(Kv& K);
// Whether the kernel's 32 bits count the chunks of B full rows of a block table.
bool kv_attend_countable(const KvShape& s, int B, int max_pages);
moe_status kv_attend_launch(Kv& kv, const moe_kv_attend_args& a, cudaStream_t s);

}  // namespace moe

struct moe_kv {
    moe::Kv K;
};
