// Paged key-value cache: handle, argument checks, and the append with the
// position rotation on the way.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <iterator>
#include <new>
#include <string>

#include "common.cuh"
#include "kv_cache.h"
#include "moe_internal.h"

namespace moe {

namespace {

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

moe_status check_desc(const moe_kv_desc* d) {
    if (!d) return fail(MOE_E_INVALID, "desc is NULL");
    if (d->abi_version != MOE_ABI_VERSION) return fail(MOE_E_INVALID, "abi_version mismatch");
    if (d->n_kv_heads < 1 || d->n_kv_heads > 256) return fail(MOE_E_INVALID, "n_kv_heads must be in 1..256");
    if (d->n_heads < 1 || d->n_heads > 4096 || d->n_heads % d->n_kv_heads)
        return fail(MOE_E_INVALID, "n_heads must be a positive multiple of n_kv_heads, at most 4096");
    if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256)
        return fail(MOE_E_UNSUPPORTED, "head_dim must be 64, 128 or 256");
    if (d->page_size < 16 || d->page_size > 4096 || d->page_size % 16)
        return fail(MOE_E_UNSUPPORTED, "page_size must be a multiple of 16 in 16..4096");
    if (d->n_pages < 1) return fail(MOE_E_INVALID, "n_pages must be positive");
    if (d->cache_dtype != MOE_BF16 && d->cache_dtype != MOE_E4M3)
        return fail(MOE_E_UNSUPPORTED, "cache_dtype must be MOE_BF16 or MOE_E4M3");
    if (d->rotary_dim < 0 || d->rotary_dim % 16 || d->rotary_dim > d->head_dim)
        return fail(MOE_E_INVALID, "rotary_dim must be 0 or a multiple of 16, at most head_dim");
    if (d->rotary_adjacent != 0 && d->rotary_adjacent != 1) return fail(MOE_E_INVALID, "rotary_adjacent must be 0 or 1");
    if (d->max_batch < 1 || d->max_batch > 1024) return fail(MOE_E_INVALID, "max_batch must be in 1..1024");
    // The rows of a pool in any order of its three dimensions, without overlap: from the smallest
    // stride up, each steps over all that the ones below it span. One row needs no step.
    const int64_t step = d->cache_dtype == MOE_E4M3 ? 16 : 8;
    struct { int64_t n, st; } dims[] = {{d->n_pages, d->page_stride}, {d->n_kv_heads, d->head_stride}, {d->page_size, d->token_stride}};
    std::sort(std::begin(dims), std::end(dims), [](const auto& a, const auto& b) { return a.st < b.st; });
    int64_t span = d->head_dim;
    for (const auto& m : dims) {
        if (m.n == 1) continue;
        if (m.st % step || m.st > ((int64_t)1 << 38))
            return fail(MOE_E_INVALID, "strides must be multiples of 16 bytes, and at most 2^38");
        if (m.st < span) return fail(MOE_E_INVALID, "rows of a pool overlap");
        span = m.st * m.n;
    }
    return MOE_OK;
}

KvShape shape_of(const moe_kv_desc& d) {
    KvShape s{};
    s.n_heads = d.n_heads;
    s.n_kv_heads = d.n_kv_heads;
    s.head_dim = d.head_dim;
    s.page_size = d.page_size;
    s.n_pages = d.n_pages;
    s.rotary_dim = d.rotary_dim;
    s.rotary_adjacent = d.rotary_adjacent;
    s.e4m3 = d.cache_dtype == MOE_E4M3;
    // (the step over a dimension of one row is never taken, but stands in the tensor maps)
    s.page_stride = d.n_pages > 1 ? d.page_stride : d.head_dim;
    s.head_stride = d.n_kv_heads > 1 ? d.head_stride : d.head_dim;
    s.token_stride = d.token_stride;
    return s;
}

moe_status check_table(const int32_t* table, int n_seqs, int max_pages, int page_size) {
    if (!table) return fail(MOE_E_INVALID, "block_table is NULL");
    if (n_seqs < 1) return fail(MOE_E_INVALID, "n_seqs must be positive");
    // room above every position for the kernels' 32-bit steps
    if (max_pages < 1 || (int64_t)max_pages * page_size > INT32_MAX - 4095)
        return fail(MOE_E_INVALID, "max_pages must be positive, and max_pages * page_size at most 2^31 - 4096");
    return MOE_OK;
}

moe_status check_append(const moe_kv_desc* d, const moe_kv_append_args* a) {
    moe_status st = check_desc(d);
    if (st != MOE_OK) return st;
    if (!a) return fail(MOE_E_INVALID, "args is NULL");
    if (a->T < 0) return fail(MOE_E_INVALID, "T must not be negative");
    if (a->T == 0) return MOE_OK;
    if (!a->k || !a->v || !a->positions) return fail(MOE_E_INVALID, "k, v or positions is NULL");
    if (!a->q != !a->q_out) return fail(MOE_E_INVALID, "q and q_out go together");
    st = check_table(a->block_table, a->n_seqs, a->max_pages, d->page_size);
    if (st != MOE_OK) return st;
    if (!a->seq && a->T > a->n_seqs) return fail(MOE_E_INVALID, "T exceeds n_seqs, and seq is NULL");
    for (const void* p : {a->q, a->k, a->v, static_cast<const void*>(a->q_out)})
        if (!aligned16(p)) return fail(MOE_E_INVALID, "q, k, v and q_out must be 16-byte aligned");
    const int64_t D = d->head_dim;
    if (a->k_stride % 8 || a->v_stride % 8 || a->k_stride < D * d->n_kv_heads || a->v_stride < D * d->n_kv_heads ||
        (a->q && (a->q_stride % 8 || a->q_stride < D * d->n_heads)))
        return fail(MOE_E_INVALID, "token strides must be multiples of 8 and cover a token's heads");
    if (a->q && a->q_out == a->q && a->q_stride != D * d->n_heads && a->T > 1)
        return fail(MOE_E_INVALID, "q_out may be q only where q is contiguous");
    return MOE_OK;
}

moe_status check_attend(const moe_kv_desc* d, const moe_kv_attend_args* a) {
    moe_status st = check_desc(d);
    if (st != MOE_OK) return st;
    if (!a) return fail(MOE_E_INVALID, "args is NULL");
    if (a->B < 0 || a->B > d->max_batch) return fail(MOE_E_INVALID, "B must be in 0..max_batch");
    if (!std::isfinite(a->scale)) return fail(MOE_E_INVALID, "scale must be finite");
    if (!std::isfinite(a->softcap) || a->softcap < 0) return fail(MOE_E_INVALID, "softcap must be finite and >= 0");
    if (a->window < 0) return fail(MOE_E_INVALID, "window must be >= 0");
    if (a->B == 0) return MOE_OK;
    if (!a->q || !a->lens || !a->out) return fail(MOE_E_INVALID, "q, lens or out is NULL");
    st = check_table(a->block_table, a->B, a->max_pages, d->page_size);
    if (st != MOE_OK) return st;
    if (!aligned16(a->q) || !aligned16(a->out)) return fail(MOE_E_INVALID, "q and out must be 16-byte aligned");
    if (a->q_stride % 8 || a->q_stride < (int64_t)d->head_dim * d->n_heads)
        return fail(MOE_E_INVALID, "q_stride must be a multiple of 8 and cover the heads");
    if (!kv_attend_countable(shape_of(*d), a->B, a->max_pages))
        return fail(MOE_E_UNSUPPORTED, "the block table spans 2^31 chunks or more");
    return MOE_OK;
}

// ---- append ---------------------------------------------------------------------
//
// A head is D / 16 groups of 16 channels, two 16-byte vectors each, so laid that
// neighbouring lanes read and write neighbouring vectors: channels 8g.. and D / 2 + 8g..
// of a value or of adjacent pairs; of pairs half the rotary channels apart, the 8 pairs
// 8g.. and rotary_dim / 2 + 8g.., and past rotary_dim the two halves of the rest. One
// lane moves a whole group and reads both vectors before it writes, so q may be rotated
// in place.
//
// The angle p * inv_freq is kept as a 64-bit fraction of a turn: turns =
// frac(inv_freq / 2 pi) * 2^64, and p * turns mod 2^64 is the exact phase of
// any position, where a 32-bit product loses the phase from 10^5 or so. The
// upper 32 bits (2^-32 of a turn) go to sincospif.

__device__ __forceinline__ float2 unpack2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(float2 v) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// x * y + z of both halves
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    float2 d;
    asm("{.reg .b64 a, b, c; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7};"
        " fma.rn.f32x2 a, a, b, c; mov.b64 {%0, %1}, a;}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
    return d;
}
// e4m3 of two values / scale, saturating, NaN stays NaN; inv = 1 / scale, rounded. The
// product with inv is off by 2^-23, which takes the wrong neighbour where the quotient is
// half way between two (one value in 10^6); with the remainder's share added it is the
// rounded quotient (P. Markstein, IBM J. Res. Dev. 34, 1990). Past 448 any product saturates,
// so that it may stop at 1024: an infinite one would have no remainder. 7040 tokens of 64 +
// 16 + 16 heads of 64: 29.0 us, without the remainder 28.2, by the division 33.4.
__device__ __forceinline__ uint32_t quant2(float2 v, float scale, float inv) {
    const float2 i2 = make_float2(inv, inv), product = fma2(v, i2, make_float2(0.f, 0.f));
    const float2 p = make_float2(fminf(fmaxf(product.x, -1024.f), 1024.f), fminf(fmaxf(product.y, -1024.f), 1024.f));
    return __nv_cvt_float2_to_fp8x2(fma2(fma2(p, make_float2(-scale, -scale), v), i2, p), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ void phase(uint64_t turns, int position, float& c, float& s) {
    const uint64_t ph = turns * (uint64_t)position;
    sincospif((float)(int32_t)(ph >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
}

struct AppendArgs {
    moe_kv_append_args a;
    KvShape s;
    void *k_pages, *v_pages;
    const uint64_t* turns;
    const float2* scales;   // of the keys, then of the values: scale and its rounded reciprocal
    unsigned* health;
    int parts, rounds;   // units and rounds of a token
};

// A round is 32 / (D / 16) heads of a token, one warp's copy of 1 KB; a unit is
// every `parts`-th round of a token. A warp streams the rounds of its units through
// its own ring of shared memory, each lane its own vectors (so it waits for nothing
// but its own copies), kAhead of them on their way, and looks up the next unit's page
// meanwhile. The lanes share the sines and cosines of a unit's angles. The kernel
// reads and writes every value once: bound by memory for many tokens, by latency for
// few, where a warp has one round. Measured (48 + 8 + 8 heads of 128 in bf16): 8192
// tokens 42.4 us, 6.3 TB/s, 94% of the copy rate; one token 2.3 us.
constexpr int kAhead = 4;
constexpr int kAppendRing = 8 * kAhead * 1024;   // of a CTA's warps

template <bool ADJACENT, bool E4M3>
__global__ void __launch_bounds__(256, 3) k_kv_append(const AppendArgs p) {
    extern __shared__ __align__(16) uint4 ring[];
    __shared__ __align__(16) float sm_c[8][128], sm_s[8][128];
    const KvShape& s = p.s;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int groups = s.head_dim / 16, g = lane % groups, side = 32 / groups, half = s.rotary_dim / 2;
    const int q_heads = p.a.q ? s.n_heads : 0, k_heads = q_heads + s.n_kv_heads, heads = k_heads + s.n_kv_heads;
    // the group's two vectors of a query or key, and of a value
    const bool pairs = !ADJACENT && 16 * g < s.rotary_dim, past = !ADJACENT && !pairs;
    const int v0 = 8 * g, v1 = v0 + s.head_dim / 2;
    const int c0 = v0 + (past ? half : 0), c1 = pairs ? c0 + half : v1;
    const bool turn0 = ADJACENT ? c0 < s.rotary_dim : pairs, turn1 = ADJACENT ? c1 < s.rotary_dim : pairs;
    const int a0 = ADJACENT ? c0 / 2 : c0, a1 = ADJACENT ? c1 / 2 : c0 + 4;   // their angles, four each
    const int stride = gridDim.x * 8, dt = stride / p.parts, dp = stride - dt * p.parts;   // to a warp's next unit
    uint4* const slots = ring + warp * (kAhead * 64) + lane;
    uint32_t bits = 0;
    auto advance = [&](int& t, int& part) {
        t += dt;
        part += dp;
        if (part >= p.parts) {
            part -= p.parts;
            ++t;
        }
    };
    uint64_t turns[4];   // of the angles lane, lane + 32, ...
#pragma unroll
    for (int i = 0; i < 4; ++i) turns[i] = lane + 32 * i < half ? p.turns[lane + 32 * i] : 0;
    pdl_wait();      // nothing of the caller's is read before the preceding kernel is done
    pdl_trigger();
    const int first = blockIdx.x * 8 + warp;
    int t = first / p.parts, part = first - t * p.parts;
    if (t >= p.a.T) return;

    // the copies: round fr of unit (ft, fp) next, into slot `put`
    int ft = t, fp = part, fr = part, put = 0;
    auto fetch = [&] {
        const int head = fr * side + lane / groups;
        if (ft < p.a.T && head < heads) {
            const bool turned = head < k_heads;
            const __nv_bfloat16* src =
                head < q_heads ? static_cast<const __nv_bfloat16*>(p.a.q) + ft * p.a.q_stride + head * s.head_dim
                : turned       ? static_cast<const __nv_bfloat16*>(p.a.k) + ft * p.a.k_stride + (head - q_heads) * s.head_dim
                               : static_cast<const __nv_bfloat16*>(p.a.v) + ft * p.a.v_stride + (head - k_heads) * s.head_dim;
            const uint32_t to = (uint32_t)__cvta_generic_to_shared(slots + put * 64);
            const __nv_bfloat16 *src0 = src + (turned ? c0 : v0), *src1 = src + (turned ? c1 : v1);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src0) : "memory");
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 512), "l"(src1) : "memory");
        }
        if ((fr += p.parts) >= p.rounds) {
            advance(ft, fp);
            fr = fp;
        }
        put = (put + 1) % kAhead;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    // position and page of a unit, read one unit ahead
    int pos = p.a.positions[t], seq = p.a.seq ? p.a.seq[t] : t;
#pragma unroll 1
    for (int i = 0; i < kAhead; ++i) fetch();
    auto look_up = [&](int pos, int seq, bool& read) {
        const int64_t at = pos >= 0 ? kv_entry(s, p.a.n_seqs, p.a.max_pages, seq, pos, bits) : -1;
        read = at >= 0;
        return read ? p.a.block_table[at] : -1;
    };
    bool read;
    int page = look_up(pos, seq, read);
    for (int take = 0; t < p.a.T;) {
        int nt = t, np = part;
        advance(nt, np);
        int next_pos = -1, next_seq = 0;
        if (nt < p.a.T) {
            next_pos = p.a.positions[nt];
            next_seq = p.a.seq ? p.a.seq[nt] : nt;
        }
        if (pos >= 0)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (lane + 32 * i < half) phase(turns[i], pos, sm_c[warp][lane + 32 * i], sm_s[warp][lane + 32 * i]);
        if (read) page = kv_page(s, page, bits);
        const int64_t row = page >= 0 ? kv_offset(s, page, 0, pos % s.page_size) : 0;
        bool next_read = false;
        int next_page = -1;
        __syncwarp();
        for (int r = part; r < p.rounds; r += p.parts) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
            const uint4 u0 = slots[take * 64], u1 = slots[take * 64 + 32];
            take = (take + 1) % kAhead;
            if (r == part) next_page = look_up(next_pos, next_seq, next_read);
            const int head = r * side + lane / groups;
            const bool is_q = head < q_heads, is_v = head >= k_heads;
            if (head < heads && (is_q || page >= 0)) {
                const int hk = head - (is_v ? k_heads : q_heads);
                const int at0 = is_v ? v0 : c0, at1 = is_v ? v1 : c1;
                const float2 scale = E4M3 && !is_q ? p.scales[(is_v ? s.n_kv_heads : 0) + hk] : make_float2(1.f, 1.f);
                uint32_t w[2][4] = {{u0.x, u0.y, u0.z, u0.w}, {u1.x, u1.y, u1.z, u1.w}};
                uint32_t e[2][2] = {};
                float c[8], sn[8];
                const bool t0 = turn0 && !is_v, t1 = ADJACENT ? turn1 && !is_v : t0;
                if (t0) {
                    *reinterpret_cast<float4*>(c) = *reinterpret_cast<const float4*>(&sm_c[warp][a0]);
                    *reinterpret_cast<float4*>(sn) = *reinterpret_cast<const float4*>(&sm_s[warp][a0]);
                }
                if (t1) {
                    *reinterpret_cast<float4*>(c + 4) = *reinterpret_cast<const float4*>(&sm_c[warp][a1]);
                    *reinterpret_cast<float4*>(sn + 4) = *reinterpret_cast<const float4*>(&sm_s[warp][a1]);
                }
                // two channels of either vector at a time
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    float2 a = unpack2(w[0][x]), b = unpack2(w[1][x]);
                    if constexpr (ADJACENT) {
                        if (t0) a = make_float2(a.x * c[x] - a.y * sn[x], a.y * c[x] + a.x * sn[x]);
                        if (t1) b = make_float2(b.x * c[4 + x] - b.y * sn[4 + x], b.y * c[4 + x] + b.x * sn[4 + x]);
                    } else if (t0) {
                        const float2 u = a;
                        a = make_float2(a.x * c[2 * x] - b.x * sn[2 * x], a.y * c[2 * x + 1] - b.y * sn[2 * x + 1]);
                        b = make_float2(b.x * c[2 * x] + u.x * sn[2 * x], b.y * c[2 * x + 1] + u.y * sn[2 * x + 1]);
                    }
                    if (E4M3 && !is_q) {
                        e[0][x / 2] |= quant2(a, scale.x, scale.y) << 16 * (x % 2);
                        e[1][x / 2] |= quant2(b, scale.x, scale.y) << 16 * (x % 2);
                    } else {
                        if (t0) w[0][x] = pack2(a);
                        if (t1) w[1][x] = pack2(b);
                    }
                    if (is_q && pos < 0) w[0][x] = w[1][x] = 0;
                }
                const int64_t off = row + hk * s.head_stride;
                if (E4M3 && !is_q) {
                    uint8_t* to = static_cast<uint8_t*>(is_v ? p.v_pages : p.k_pages) + off;
                    *reinterpret_cast<uint2*>(to + at0) = make_uint2(e[0][0], e[0][1]);
                    *reinterpret_cast<uint2*>(to + at1) = make_uint2(e[1][0], e[1][1]);
                } else {
                    __nv_bfloat16* dst = is_q ? static_cast<__nv_bfloat16*>(p.a.q_out) + ((int64_t)t * s.n_heads + head) * s.head_dim
                                              : static_cast<__nv_bfloat16*>(is_v ? p.v_pages : p.k_pages) + off;
                    *reinterpret_cast<uint4*>(dst + at0) = make_uint4(w[0][0], w[0][1], w[0][2], w[0][3]);
                    *reinterpret_cast<uint4*>(dst + at1) = make_uint4(w[1][0], w[1][1], w[1][2], w[1][3]);
                }
            }
            fetch();
        }
        t = nt;
        part = np;
        pos = next_pos;
        page = next_page;
        read = next_read;
        __syncwarp();   // every lane is done with the sines
    }
    if (bits) atomicOr(p.health, bits);
}

using AppendKernel = void (*)(const AppendArgs);

AppendKernel append_kernel(const KvShape& s) {
    return s.rotary_adjacent ? (s.e4m3 ? k_kv_append<true, true> : k_kv_append<true, false>)
                             : (s.e4m3 ? k_kv_append<false, true> : k_kv_append<false, false>);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_kv_append_check(const moe_kv_desc* desc, const moe_kv_append_args* args) {
    return check_append(desc, args);
}

moe_status moe_kv_attend_check(const moe_kv_desc* desc, const moe_kv_attend_args* args) {
    return check_attend(desc, args);
}

moe_status moe_kv_locate(const moe_kv_desc* desc, const int32_t* block_table, int32_t n_seqs, int32_t max_pages,
                         int32_t seq, int32_t position, int32_t head, int64_t* offset, uint32_t* bits) {
    moe_status st = check_desc(desc);
    if (st != MOE_OK) return st;
    st = check_table(block_table, n_seqs, max_pages, desc->page_size);
    if (st != MOE_OK) return st;
    if (!offset) return fail(MOE_E_INVALID, "offset is NULL");
    if (head < 0 || head >= desc->n_kv_heads) return fail(MOE_E_INVALID, "head outside 0..n_kv_heads-1");
    const KvShape s = shape_of(*desc);
    uint32_t b = 0;
    const int64_t at = kv_entry(s, n_seqs, max_pages, seq, position, b);
    const int page = at >= 0 ? kv_page(s, block_table[at], b) : -1;
    if (bits) *bits = b;
    if (page < 0) return fail(MOE_E_STATE, "the position has no slot (health bits " + std::to_string(b) + ")");
    *offset = kv_offset(s, page, head, position % s.page_size);
    return MOE_OK;
}

moe_status moe_kv_create(const moe_kv_desc* desc, void* k_pages, void* v_pages, const double* inv_freq,
                         const float* k_scale, const float* v_scale, int32_t device, moe_kv** out) {
    if (!out) return fail(MOE_E_INVALID, "out is NULL");
    *out = nullptr;
    moe_status st = check_desc(desc);
    if (st != MOE_OK) return st;
    if (!k_pages || !v_pages || !aligned16(k_pages) || !aligned16(v_pages))
        return fail(MOE_E_INVALID, "k_pages and v_pages must be non-NULL and 16-byte aligned");
    const int half = desc->rotary_dim / 2, Hk = desc->n_kv_heads;
    if (half && !inv_freq) return fail(MOE_E_INVALID, "inv_freq is required where rotary_dim > 0");
    for (int i = 0; i < half; ++i)
        if (!std::isfinite(inv_freq[i])) return fail(MOE_E_INVALID, "inv_freq must be finite");
    const bool e4m3 = desc->cache_dtype == MOE_E4M3;
    if (e4m3 != (k_scale != nullptr) || e4m3 != (v_scale != nullptr))
        return fail(MOE_E_INVALID, "k_scale and v_scale go with an e4m3 cache, and only with it");
    for (int h = 0; e4m3 && h < Hk; ++h)
        if (!(std::isnormal(k_scale[h]) && k_scale[h] > 0 && std::isnormal(v_scale[h]) && v_scale[h] > 0))
            return fail(MOE_E_INVALID, "k_scale and v_scale must be positive normal numbers");   // and their reciprocals finite

    DeviceGuard g(device);
    if (!g.ok) return cuda_fail(g.err, "cudaSetDevice");
    moe_kv* kv = new (std::nothrow) moe_kv();
    if (!kv) return fail(MOE_E_NOMEM, "host memory");
    Kv& K = kv->K;
    K.d = *desc;
    K.s = shape_of(*desc);
    K.device = device;
    K.k_pages = k_pages;
    K.v_pages = v_pages;
    auto bail = [&](moe_status s) {
        std::string m = moe_last_error();
        moe_kv_destroy(kv);
        return fail(s, m);
    };
    cudaError_t e = cudaDeviceGetAttribute(&K.num_sms, cudaDevAttrMultiProcessorCount, device);
    if (e != cudaSuccess) return bail(cuda_fail(e, "cudaDeviceGetAttribute"));

    size_t need = 0;
    auto add = [&](size_t b) {
        const size_t off = need;
        need += (b + 255) / 256 * 256;
        return off;
    };
    const size_t o_turns = add((size_t)std::max(half, 1) * 8), o_ks = add((size_t)Hk * 4), o_vs = add((size_t)Hk * 4),
                 o_scales = add((size_t)Hk * 16), o_health = add(4);
    size_t ws[3];
    kv_attend_workspace(K, ws);
    const size_t o_po = add(ws[0]), o_pml = add(ws[1]), o_arr = add(ws[2]);
    size_t free_b = 0, total_b = 0;
    e = cudaMemGetInfo(&free_b, &total_b);
    if (e != cudaSuccess) return bail(cuda_fail(e, "cudaMemGetInfo"));
    if (need > free_b) return bail(fail(MOE_E_NOMEM, "the workspace does not fit in free device memory"));
    e = cudaMalloc(&K.block, need);
    if (e != cudaSuccess) return bail(cuda_fail(e, "cudaMalloc"));
    K.device_bytes = need;
    uint8_t* base = static_cast<uint8_t*>(K.block);
    K.turns = reinterpret_cast<uint64_t*>(base + o_turns);
    K.k_scale = reinterpret_cast<float*>(base + o_ks);
    K.v_scale = reinterpret_cast<float*>(base + o_vs);
    K.scales = reinterpret_cast<float2*>(base + o_scales);
    K.health = reinterpret_cast<unsigned*>(base + o_health);
    K.part_o = reinterpret_cast<float4*>(base + o_po);
    K.part_ml = reinterpret_cast<float4*>(base + o_pml);
    K.arrived = reinterpret_cast<int*>(base + o_arr);

    // inv_freq / 2 pi in double keeps 2^-53 of a turn per position; its fraction
    // times 2^64 is rounded to an integer
    uint64_t turns[128] = {};   // rotary_dim <= 256
    for (int i = 0; i < half; ++i) {
        const double t = inv_freq[i] / 6.283185307179586476925287;
        const double f = t - std::floor(t);
        turns[i] = f >= 1.0 ? 0 : (uint64_t)std::ldexp(f, 64);
    }
    float ks[256], vs[256];     // n_kv_heads <= 256
    float2 scales[512];
    for (int h = 0; h < Hk; ++h) {
        ks[h] = e4m3 ? k_scale[h] : 1.0f;
        vs[h] = e4m3 ? v_scale[h] : 1.0f;
        scales[h] = make_float2(ks[h], 1.0f / ks[h]);
        scales[Hk + h] = make_float2(vs[h], 1.0f / vs[h]);
    }
    e = cudaMemset(K.block, 0, need);
    if (e == cudaSuccess) e = cudaMemcpy(K.turns, turns, (size_t)half * 8, cudaMemcpyHostToDevice);
    if (e == cudaSuccess) e = cudaMemcpy(K.k_scale, ks, (size_t)Hk * 4, cudaMemcpyHostToDevice);
    if (e == cudaSuccess) e = cudaMemcpy(K.v_scale, vs, (size_t)Hk * 4, cudaMemcpyHostToDevice);
    if (e == cudaSuccess) e = cudaMemcpy(K.scales, scales, (size_t)Hk * 16, cudaMemcpyHostToDevice);
    if (e == cudaSuccess) e = kv_attend_setup(K);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(append_kernel(K.s), cudaFuncAttributeMaxDynamicSharedMemorySize, kAppendRing);
    // the set-up ran on the legacy stream: finish it before any other stream may run a call
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return bail(cuda_fail(e, "moe_kv_create set-up"));
    *out = kv;
    return MOE_OK;
}

void moe_kv_destroy(moe_kv* kv) {
    if (!kv) return;
    DeviceGuard g(kv->K.device);
    if (kv->K.block) {
        cudaDeviceSynchronize();
        cudaFree(kv->K.block);
    }
    delete kv;
}

size_t moe_kv_device_bytes(const moe_kv* kv) { return kv ? kv->K.device_bytes : 0; }

moe_status moe_kv_append(moe_kv* kv, const moe_kv_append_args* args, void* stream) {
    if (!kv) return fail(MOE_E_INVALID, "NULL handle");
    Kv& K = kv->K;
    moe_status st = check_append(&K.d, args);
    if (st != MOE_OK) return st;
    if (args->T == 0) return MOE_OK;
    DeviceGuard g(K.device);
    if (!g.ok) return cuda_fail(g.err, "cudaSetDevice");
    AppendArgs p{*args, K.s, K.k_pages, K.v_pages, K.turns, K.scales, K.health, 1, 1};
    const int heads = (args->q ? K.s.n_heads : 0) + 2 * K.s.n_kv_heads, side = 32 / (K.s.head_dim / 16);
    p.rounds = (heads + side - 1) / side;
    // Units per token: a warp takes ceil(T n / warps) units, each of rounds / n rounds (the most
    // of them, where its next unit is always the same part) and about 0.9 of a round for its
    // angles and page; n with the least of that. 8192 tokens of 16 rounds: n = 4, 42.4 us, with
    // 3 or 2 47 and 50; 7040 of 12 in 8 bits: n = 1, 29.1, with 2 or 4 31.3 and 34.7.
    const int64_t warps = (int64_t)K.num_sms * 3 * 8;
    if ((int64_t)args->T * p.rounds <= warps) {
        p.parts = p.rounds;
    } else {
        double least = 0;
        for (int n = 1; n <= p.rounds; ++n) {
            const double each = warps % n ? (double)p.rounds / n : (p.rounds + n - 1) / n;
            const double cost = (double)(((int64_t)args->T * n + warps - 1) / warps) * (each + 0.9);
            if (n == 1 || cost < least) {
                least = cost;
                p.parts = n;
            }
        }
    }
    const unsigned grid = (unsigned)std::min<int64_t>(((int64_t)args->T * p.parts + 7) / 8, (int64_t)K.num_sms * 3);
    const cudaError_t e =
        launch_pdl(append_kernel(K.s), dim3(grid), dim3(256), kAppendRing, static_cast<cudaStream_t>(stream), true, p);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "append launch");
}

moe_status moe_kv_attend(moe_kv* kv, const moe_kv_attend_args* args, void* stream) {
    if (!kv) return fail(MOE_E_INVALID, "NULL handle");
    Kv& K = kv->K;
    moe_status st = check_attend(&K.d, args);
    if (st != MOE_OK) return st;
    if (args->B == 0) return MOE_OK;
    DeviceGuard g(K.device);
    if (!g.ok) return cuda_fail(g.err, "cudaSetDevice");
    return kv_attend_launch(K, *args, static_cast<cudaStream_t>(stream));
}

moe_status moe_kv_set_option(moe_kv* kv, int32_t option, int64_t value) {
    if (!kv) return fail(MOE_E_INVALID, "NULL handle");
    if (option != MOE_KV_OPT_TEST_STALL) return fail(MOE_E_INVALID, "unknown option");
    if (value < -1 || value >= kv->K.d.max_batch) return fail(MOE_E_INVALID, "a sequence, or -1 for none");
    kv->K.stall = (int)value;
    return MOE_OK;
}

moe_status moe_kv_health(moe_kv* kv, uint32_t* bits) {
    if (!kv) return fail(MOE_E_INVALID, "NULL handle");
    DeviceGuard g(kv->K.device);
    if (!g.ok) return cuda_fail(g.err, "cudaSetDevice");
    MOE_CUDA_TRY(cudaDeviceSynchronize());
    uint32_t v = 0;
    MOE_CUDA_TRY(cudaMemcpy(&v, kv->K.health, 4, cudaMemcpyDeviceToHost));
    if (bits) *bits = v;
    if (!v) return MOE_OK;
    MOE_CUDA_TRY(cudaMemset(kv->K.health, 0, 4));
    MOE_CUDA_TRY(cudaDeviceSynchronize());   // before any stream's next call may set a bit
    if (v & MOE_KV_TIMEOUT) return fail(MOE_E_TIMEOUT, "a bounded device-side wait gave up (health bits " + std::to_string(v) + ")");
    return fail(MOE_E_STATE, "kernels refused part of their work (health bits " + std::to_string(v) + ")");
}

}  // extern "C"
