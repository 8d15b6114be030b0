// More of the same primitives, for the kernels of a prompt's chunk: short waits, copies of four
// dimensions, operands whose rows are their K, 32 columns of tensor memory at a time.
#pragma once

#include "sm100.cuh"

namespace moe {
namespace bw {

// mbar_wait in a few instructions: a try that does not succeed suspends the warp, for 1.3 us as
// measured (unless the phase completes: 106 cycles from the arrival), so that warps that wait
// leave the issue slots and the instruction cache to those that work. The limit is a count, 2^18
// tries, and no time: 0.35 s at 1.3 us, which is the machine's choice. (A look at the global timer
// in this loop takes registers and instructions of every role: a batch of short chunks in 8 bits
// 214 -> 223 us, windows with heads of 256 64 -> 66.) The longest wait of a call that gets on is that
// of the tile of a pair that is not there, as long as the other's blocks: 1 ms for 100 000 tokens.
__device__ __forceinline__ bool mbar_wait_short(uint32_t bar, uint32_t parity, volatile int* abort) {
#pragma unroll 1
    for (uint32_t n = 0; !mbar_try(bar, parity); ++n) {
        if (n >> 18) *abort = 1;
        if (*abort) return false;
    }
    return true;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, int w,
                                            uint32_t bar, uint64_t pol) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
        "l"(tm), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "l"(pol)
        : "memory");
}

// desc_sw128 for an operand whose rows are its K and whose 64-element panels lie `panel` bytes
// apart: groups of 8 rows 1024 bytes apart, 128-byte swizzle. `addr`: the first row of the step.
__device__ __forceinline__ uint64_t desc_sw128_mn(uint32_t addr, uint32_t panel) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(panel >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

// Instruction descriptor of kind::f16 with fp16 or bf16 A and B (K-major, B also the other
// way) and an fp32 accumulator, shape M x N.
__host__ __device__ constexpr uint32_t idesc_16_f32(int M, int N, bool bf16 = false, bool b_mn = false) {
    return (1u << 4)                       // accumulator format: f32
           | (bf16 ? (1u << 7) | (1u << 10) : 0u)   // A, B format: f16 or bf16
           | (b_mn ? 1u << 16 : 0u)        // B's rows are its K
           | ((uint32_t)(N >> 3) << 17)    // N / 8
           | ((uint32_t)(M >> 4) << 24);   // M / 16
}

// 32 consecutive 32-bit columns of this thread's tensor-memory lane (warp-wide), as bits; they
// have arrived after tmem_wait_ld32().
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// Wait for this warp's loads. The registers pass through it, so that nothing that reads them
// comes before it.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

}  // namespace bw
}  // namespace moe
