// int8 helpers for the quantised K/V cache: codes widened to exact 16-bit
// floats with byte permutes and one packed subtraction per pair (no
// conversion instructions, whose rate is a quarter of these), and small
// shared-memory loads.
#pragma once

#include <cstdint>

#include "fp8.cuh"

namespace kvp {

// Four codes (bytes 0-3 of w) -> two bf16x2 (lo: bytes 0-1, hi: bytes 2-3). Under 0x43 the code's byte makes a bf16 of 7
// mantissa bits: its low 7 bits x give 128 + x, and its sign bit lands on the
// lowest exponent bit, so the byte's upper part alone is 128 (code >= 0) or
// 256 (code < 0, where code = x - 128). The difference is the code, exactly.
__device__ __forceinline__ void s8x4_to_bf16x2x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t a = byte_perm(w, 0x43434343u, 0x4140u), b = byte_perm(w, 0x43434343u, 0x4342u);
    asm("sub.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(a & 0xff7fff7fu), "r"(a & 0xff80ff80u));
    asm("sub.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(b & 0xff7fff7fu), "r"(b & 0xff80ff80u));
}

// D = A (16x32, row) * B (32x8, col) + D in integers: four codes to a register, exact sums.
__device__ __forceinline__ void mma_16832_s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float lds_float(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

}  // namespace kvp
