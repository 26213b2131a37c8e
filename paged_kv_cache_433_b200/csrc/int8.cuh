// int8 helpers for the quantised K/V cache: codes widened to exact 16-bit
// floats with byte permutes and one packed subtraction per pair (no
// conversion instructions, whose rate is a quarter of these), and small
// shared-memory loads.
#pragma once

#include <cstdint>

#include "fp8.cuh"

namespace kvp {

// Four codes (bytes 0-3 of w) -> two f16x2 (lo: bytes 0-1, hi: bytes 2-3).
// With u = code + 128 in the low byte under 0x64, the half is 1024 + u
// (its last place is 1 there); subtracting 1152 leaves the code.
__device__ __forceinline__ void s8x4_to_f16x2x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = byte_perm(u, 0x64646464u, 0x4140u), b = byte_perm(u, 0x64646464u, 0x4342u);
    asm("sub.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

// Four codes -> two bf16x2. Under 0x43 the code's byte makes a bf16 of 7
// mantissa bits: its low 7 bits x give 128 + x, and its sign bit lands on the
// lowest exponent bit, so the byte's upper part alone is 128 (code >= 0) or
// 256 (code < 0, where code = x - 128). The difference is the code, exactly.
__device__ __forceinline__ void s8x4_to_bf16x2x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t a = byte_perm(w, 0x43434343u, 0x4140u), b = byte_perm(w, 0x43434343u, 0x4342u);
    asm("sub.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(a & 0xff7fff7fu), "r"(a & 0xff80ff80u));
    asm("sub.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(b & 0xff7fff7fu), "r"(b & 0xff80ff80u));
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
