// Modified attention scores and masks, shared by the decode and prefill
// kernels: for query row i at position pos and key t,
//   s = scale * (q . k);  s = c * tanh(s / c) (if a cap c is set);
//   s -= slope_h * |pos - t| (if slopes are given),
// and the row sees the keys t in [lo, hi):
//   lo = max(0, key_start[i], pos - window + 1), hi = max(pos + 1, prefix_b),
// prefix_b = min(prefix_lens[b], seq_lens[b]). A row with lo >= hi sees none.
// Scores come out in log2 units (times log2 e).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "decode_kernel.cuh"
#include "plan_layout.cuh"

namespace kvp {

// First key that the query in row `row` (of key_start) at position pos may see.
__device__ __forceinline__ int first_key(const DecodeParams& p, int row, int pos) {
    return first_visible_key(pos, p.window, p.key_start, row);
}

// The grids of the chunked prefill with modified scores: sequence b has the tile slots from q_start[b] / q_tile + b on, as
// many as its rows can need, n_rows / q_tile + B in all whatever the chunks' lengths are. (A slot per sequence and tile of
// the longest chunk, with one chunk of 4096 among 256: 262144 tiles, 1.8 ms for nothing.) Slots past a chunk's end have
// no rows. The grids run through the KV heads of a slot first and through the slots from the last one down: a prompt's
// last tiles see the most keys, and a launch that ends with its small ones ends evenly (capped prefill, two prompts in
// windowed documents: 251 us, 300 with a head's slots in ascending order behind one another).
struct ChunkTile {
    int b, qs0, n_q, t0, nt;  // sequence, its first row, its rows; the tile's first row of them, and its rows (<= 0: none)
};
__device__ __forceinline__ int first_slot(const DecodeParams& p, int b) { return p.q_start[b] / p.q_tile + b; }
__device__ __forceinline__ ChunkTile tile_of(const DecodeParams& p, int b, int slot) {
    ChunkTile t;
    t.b = b;
    t.qs0 = p.q_start[b];
    t.n_q = p.q_start[b + 1] - t.qs0;
    t.t0 = (slot - first_slot(p, b)) * p.q_tile;
    if (t.t0 < 0 || t.qs0 < 0) t.n_q = t.t0 = t.qs0 = 0;  // (a first row other than 0)
    // no row past max_q_len, and none past q and out whatever q_start says
    t.nt = min(min(p.q_tile, min(t.n_q, p.max_q_len) - t.t0), p.n_rows - t.qs0 - t.t0);
    return t;
}
// The tile in `slot`; called by whole warps: the last sequence whose slots begin no later, 32 candidates a step.
__device__ __forceinline__ ChunkTile chunk_tile(const DecodeParams& p, int slot, int lane) {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, c = lo + lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, lane == 0 || (c < hi && first_slot(p, c) <= slot));
        lo += (31 - __clz(m)) * step;
        hi = min(hi, lo + step);
    }
    return tile_of(p, lo, slot);
}

// Keys of a tile of nt query rows (chunk tokens) at positions pos0 ..: some row sees keys in [begin, end) only;
// every row sees all keys in [all0, all1). Called by whole warps.
struct TileKeys {
    int begin, end, all0, all1;
};
__device__ __forceinline__ TileKeys tile_keys(const DecodeParams& p, int row0, int pos0, int nt, int prefix, int lane) {
    TileKeys k;
    k.end = max(pos0 + nt, prefix);
    k.all1 = max(pos0 + 1, prefix);
    int lo_min = first_visible_key(pos0, p.window, nullptr, 0);
    int lo_max = first_visible_key(pos0 + nt - 1, p.window, nullptr, 0);
    if (p.key_start != nullptr) {
        lo_min = 0x7fffffff;
        lo_max = 0;
        for (int t = lane; t < nt; t += 32) {
            const int lo = first_key(p, row0 + t, pos0 + t);
            lo_min = min(lo_min, lo);
            lo_max = max(lo_max, lo);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            lo_min = min(lo_min, __shfl_xor_sync(0xffffffffu, lo_min, o));
            lo_max = max(lo_max, __shfl_xor_sync(0xffffffffu, lo_max, o));
        }
    }
    k.begin = lo_min;
    k.all0 = lo_max;
    return k;
}

// Where |u| <= kTanhSmall: tanh(u) = u * P(u^2), P of degree 5 fitted to tanh(u) / u by least squares reweighted
// towards equal relative errors (2.9e-8). No special-function unit, and relative instead of absolute accuracy:
// scores that are small beside the cap, the usual case, keep all their bits. With u = x * scale / c for a product
// x = q . k, the capped score in log2 units is x times a polynomial in x^2 whose coefficients the host scales by
// the powers of (scale / c)^2 (p.cap_coef), valid for |x| <= p.cap_small.
constexpr int kCapTerms = 6;
// max(|a|, |b|, |c|) in one instruction (three-input form, sm_100)
__device__ __forceinline__ float fmax3_abs(float a, float b, float c) {
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
constexpr double kTanhSmall = 0.75;
constexpr double kTanhPoly[kCapTerms] = {0.999999971, -0.333329589, 0.13325406, -0.0533444284, 0.0195829047, -0.00471625478};
// And for |u| <= kTanhTiny degree 2 (1.1e-7): three operations fewer a pair, which the chunked prefill feels.
constexpr int kCapTinyTerms = 3;
constexpr double kTanhTiny = 0.2;
constexpr double kTanhTinyPoly[kCapTinyTerms] = {0.999999895, -0.333285909, 0.130154075};
// tanh(u) = 1 - 2 / (1 + e^2u): an error of 1e-7 of 1 (+-inf give +-1), for what the polynomials do not serve. Beside a small
// u that is much, so the host keeps such u away: p.cap_small covers all up to kTanhSmall, under caps above about 500 (whose
// coefficients leave fp32's range one after another) all up to 0.3, 0.17, 0.09 or 0.02, and a cap far above that is none.
__device__ __forceinline__ float tanh_large(float u) {
    return 1.f - 2.f * __frcp_rn(1.f + exp2f(u * 2.885390081777927f));
}
// Chunked prefill: the largest cap (log2 units; 50 in natural ones) with one softmax reference for all rows, and the
// largest power of two that its probabilities then reach: they lie in 2^-96 .. 2^50, a residual of 16-bit splitting 2^9
// lower, so that sums with values from 1e-6 to 1e17 stay inside the normal range.
constexpr float kFixedRefMax = 73.f, kFixedTop = 50.f;
// The coefficients as packed pairs in registers: loaded once through volatile moves, or the compiler fetches both
// halves of each again for every pair of scores (the packed operations take no constant-bank operand).
struct CapCoef {
    float2 c[kCapTerms];
};
__device__ __forceinline__ CapCoef cap_coefs(const DecodeParams& p) {
    CapCoef k;
#pragma unroll
    for (int i = 0; i < kCapTerms; ++i)
        asm volatile("{\n\tmov.b32 %0, %2;\n\tmov.b32 %1, %2;\n\t}" : "=f"(k.c[i].x), "=f"(k.c[i].y) : "f"(p.cap_coef[i]));
    return k;
}
__device__ __forceinline__ float2 cap_small2(const CapCoef& k, float2 x) {
    const float2 z = fmul2(x, x);
    float2 r = k.c[kCapTerms - 1];
#pragma unroll
    for (int i = kCapTerms - 2; i >= 0; --i) r = ffma2(z, r, k.c[i]);
    return fmul2(x, r);
}

// x[0 .. 1] of every pair: products -> capped (or only scaled) scores in log2 units. Called by whole warps.
template <int N>
__device__ __forceinline__ void cap_scores(const DecodeParams& p, const CapCoef& k, float (&x)[N]) {
    if (p.cap_out != 0.f) {
        float big = fmaxf(fabsf(x[0]), fabsf(x[1]));
#pragma unroll
        for (int c = 2; c < N; c += 2) big = fmax3_abs(big, x[c], x[c + 1]);
        if (__any_sync(0xffffffffu, big > p.cap_small)) {
            // which form a score takes goes by itself alone: no other key or row has an effect on it
#pragma unroll
            for (int c = 0; c < N; c += 2) {
                const float2 t = cap_small2(k, make_float2(x[c], x[c + 1]));
                x[c] = fabsf(x[c]) <= p.cap_small ? t.x : tanh_large(x[c] * p.cap_in) * p.cap_out;
                x[c + 1] = fabsf(x[c + 1]) <= p.cap_small ? t.y : tanh_large(x[c + 1] * p.cap_in) * p.cap_out;
            }
        } else {
#pragma unroll
            for (int c = 0; c < N; c += 2) {
                const float2 t = cap_small2(k, make_float2(x[c], x[c + 1]));
                x[c] = t.x;
                x[c + 1] = t.y;
            }
        }
    } else {
        const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
#pragma unroll
        for (int c = 0; c < N; c += 2) {
            const float2 t = fmul2(make_float2(x[c], x[c + 1]), sl2);
            x[c] = t.x;
            x[c + 1] = t.y;
        }
    }
}

// Products of one warp's MMA tiles, query rows as MMA rows: sc[n][e] is row e / 2, token n * 8 + (e & 1) of the stage
// counted from the lane's first; dist0 / dist1: position minus that first token for rows 0 / 1.
template <int NT>
__device__ __forceinline__ void modify_rows(const DecodeParams& p, const CapCoef& k, float (&sc)[NT][4],
                                            const float (&slope)[2], int dist0, int dist1) {
    cap_scores(p, k, reinterpret_cast<float(&)[NT * 4]>(sc));
    if (p.alibi_slopes != nullptr) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sc[n][e] -= slope[e >> 1] * fabsf(static_cast<float>((e >= 2 ? dist1 : dist0) - (n * 8 + (e & 1))));
    }
}

// The same with heads as MMA columns: sc[nt][mt][e] is head column e & 1 of tile nt, token mt * 16 + 8 (e / 2) counted
// from the lane's first; dist: the query's position minus that first token.
template <int NT, int MT>
__device__ __forceinline__ void modify_cols(const DecodeParams& p, const CapCoef& k, float (&sc)[NT][MT][4],
                                            const float (&slope)[NT][2], int dist) {
    cap_scores(p, k, reinterpret_cast<float(&)[NT * MT * 4]>(sc));
    if (p.alibi_slopes != nullptr) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float d = fabsf(static_cast<float>(dist - (mt * 16 + 8 * (e >> 1))));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) sc[nt][mt][e] -= slope[nt][e & 1] * d;
            }
    }
}

// The same for one thread's run of N consecutive keys of one row: dist0 = position minus the first key. FIXED (capped
// chunked prefill: a cap is set and no bias): minus p.fixed_ref.
struct CapRowCoef {
    float2 tiny[kCapTinyTerms], neg_ref;
};
__device__ __forceinline__ CapRowCoef cap_row_coefs(const DecodeParams& p) {
    CapRowCoef k;
    auto pair = [](float x) {
        float2 v;
        asm volatile("{\n\tmov.b32 %0, %2;\n\tmov.b32 %1, %2;\n\t}" : "=f"(v.x), "=f"(v.y) : "f"(x));
        return v;
    };
#pragma unroll
    for (int i = 0; i < kCapTinyTerms; ++i) k.tiny[i] = pair(p.cap_coef_tiny[i]);
    k.neg_ref = pair(-p.fixed_ref);
    return k;
}
// Largest magnitude of s, for the choices below.
template <int N>
__device__ __forceinline__ float largest(const float (&s)[N]) {
    float big = fmaxf(fabsf(s[0]), fabsf(s[1]));
#pragma unroll
    for (int c = 2; c < N; c += 2) big = fmax3_abs(big, s[c], s[c + 1]);
    return big;
}
// A pair where both |s| <= p.cap_tiny.
template <bool FIXED>
__device__ __forceinline__ float2 cap_tiny2(const CapRowCoef& k, float2 x) {
    const float2 z = fmul2(x, x);
    const float2 r = ffma2(z, ffma2(z, k.tiny[2], k.tiny[1]), k.tiny[0]);
    return FIXED ? ffma2(x, r, k.neg_ref) : fmul2(x, r);
}
// Any scores; large: one is above p.cap_small. Which form a score takes goes by itself alone: no other key or row has an
// effect on it. (Scalar forms: their coefficients come from the constant bank.)
template <bool FIXED, int N>
__device__ __forceinline__ void cap_row_any(const DecodeParams& p, const CapRowCoef& k, float (&s)[N], bool large) {
    auto other = [&](float x) {
        const float z = x * x;
        float r = p.cap_coef[kCapTerms - 1];
#pragma unroll
        for (int i = kCapTerms - 2; i >= 0; --i) r = fmaf(z, r, p.cap_coef[i]);
        const float y = FIXED ? fmaf(x, r, k.neg_ref.x) : x * r;
        return !large || fabsf(x) <= p.cap_small ? y : tanh_large(x * p.cap_in) * p.cap_out - (FIXED ? p.fixed_ref : 0.f);
    };
#pragma unroll
    for (int c = 0; c < N; c += 2) {
        const float2 t = cap_tiny2<FIXED>(k, make_float2(s[c], s[c + 1]));
        s[c] = fabsf(s[c]) <= p.cap_tiny ? t.x : other(s[c]);
        s[c + 1] = fabsf(s[c + 1]) <= p.cap_tiny ? t.y : other(s[c + 1]);
    }
}
template <int N>
__device__ __forceinline__ void modify_row(const DecodeParams& p, const CapRowCoef& k, float (&s)[N], float slope, int dist0) {
    if (p.cap_out != 0.f) {
        const float big = largest(s);
        if (!__any_sync(0xffffffffu, big > p.cap_tiny)) {
#pragma unroll
            for (int c = 0; c < N; c += 2) {
                const float2 t = cap_tiny2<false>(k, make_float2(s[c], s[c + 1]));
                s[c] = t.x;
                s[c + 1] = t.y;
            }
        } else {
            cap_row_any<false>(p, k, s, __any_sync(0xffffffffu, big > p.cap_small));
        }
    } else {
        const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
#pragma unroll
        for (int c = 0; c < N; c += 2) {
            const float2 t = fmul2(make_float2(s[c], s[c + 1]), sl2);
            s[c] = t.x;
            s[c + 1] = t.y;
        }
    }
    if (p.alibi_slopes != nullptr) {
        const float d = static_cast<float>(dist0);
#pragma unroll
        for (int c = 0; c < N; ++c) s[c] -= slope * fabsf(d - static_cast<float>(c));
    }
}

// The tensor core rounds each sum of 16 products and the accumulator towards zero. Over n keys an accumulator loses
// about n 2^-29 of the result for values around zero (8.4e-6 at 4224 keys, 6.5e-5 at 32K, measured with warp MMA and
// tcgen05 alike), and up to n / 8 times 2^-23 for values of one sign (1.0e-5 at 2048). The multi-token kernels
// therefore move their output accumulators into fp32 sums after every kFlushKeys keys, in registers (tcgen05) or in the
// output rows that the same threads write at the end (warp MMA). More often costs more than it gives: 8 chunks of 512
// tokens over 4096, capped, 435 us at 2048 keys and 5.3e-6 off; 464 us at 1024; 520 us at 512
// (the rest is the 16-bit splitting of the probabilities).
constexpr int kFlushKeys = 2048;

// ---- 16-bit values with an all-ones exponent (NaN, +-inf) -----------------
// The halves of w that are not finite, with 0 in the place of finite ones.
template <bool IS_BF16>
__device__ __forceinline__ uint32_t nonfinite16(uint32_t w) {
    constexpr uint32_t m = IS_BF16 ? 0x7f807f80u : 0x7c007c00u;
    return w & __vcmpeq2(w & m, m);
}
template <bool IS_BF16>
__device__ __forceinline__ bool has_nonfinite16(const uint4& v) {
    return (nonfinite16<IS_BF16>(v.x) | nonfinite16<IS_BF16>(v.y) | nonfinite16<IS_BF16>(v.z) |
            nonfinite16<IS_BF16>(v.w)) != 0;
}
template <bool IS_BF16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
    if constexpr (IS_BF16)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else
        return make_float2(__half2float(__ushort_as_half(static_cast<unsigned short>(w & 0xffffu))),
                           __half2float(__ushort_as_half(static_cast<unsigned short>(w >> 16))));
}

// x[i] = sum of the NaN and infinite elements of dim d0 + i of V over the keys lo .. hi - 1 that this lane's row of
// sequence b sees (lo >= hi: none), pages outside the pool left out: what an attention sum over those keys is once it holds
// one; 0 where there is none. Called by whole warps, which stand between other warps and their next stage: the lanes
// search different keys, four each with their loads in flight together, and only keys that hold such an element are then
// gone through by all of them. (A thread on its own, dim by dim and key by key, needs seconds for a context of 100,000
// keys, and the waits for its warp end after one.)
template <bool IS_BF16>
__device__ __noinline__ void sum_nonfinite16(const DecodeParams& p, int b, int kvh, int P, int DH, int d0, int lo, int hi,
                                             float (&x)[16]) {
    constexpr int kBatch = 4;
    const uint32_t lane = threadIdx.x & 31;
    const int lg = P == 16 ? 4 : 5;
    const uint32_t first = __reduce_min_sync(0xffffffffu, lo < hi ? static_cast<uint32_t>(lo) : 0xffffffffu);
    const uint32_t end = __reduce_max_sync(0xffffffffu, lo < hi ? static_cast<uint32_t>(hi) : 0u);
    const int32_t* table = p.block_tables + (int64_t)b * p.max_blocks;
    auto row = [&](uint32_t t) -> const uint4* {  // the sixteen elements of key t
        const int pg = table[t >> lg];
        if (pg < 0 || pg >= p.num_pages) return nullptr;
        return reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.v_pages) +
                                              ((((int64_t)pg * p.H_kv + kvh) << lg) + (t & (P - 1))) * DH + d0);
    };
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
    for (uint32_t t0 = first; t0 < end; t0 += 32 * kBatch) {
        uint4 v[kBatch][2];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const uint32_t t = t0 + 32 * k + lane;
            const uint4* src = t < end ? row(t) : nullptr;
            v[k][0] = v[k][1] = make_uint4(0u, 0u, 0u, 0u);
            if (src != nullptr) v[k][0] = src[0], v[k][1] = src[1];
        }
#pragma unroll 1
        for (int k = 0; k < kBatch; ++k) {
            bool found = false;
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (j == k) found = has_nonfinite16<IS_BF16>(v[j][0]) || has_nonfinite16<IS_BF16>(v[j][1]);
            for (unsigned m = __ballot_sync(0xffffffffu, found); m != 0; m &= m - 1) {
                const uint32_t t = t0 + 32 * k + __ffs(m) - 1;
                if (t < static_cast<uint32_t>(lo) || t >= static_cast<uint32_t>(hi) || lo >= hi) continue;
                const uint4* src = row(t);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 u = src[h];
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 e = unpack16<IS_BF16>(nonfinite16<IS_BF16>(w[i]));
                        x[8 * h + 2 * i] += e.x;
                        x[8 * h + 2 * i + 1] += e.y;
                    }
                }
            }
        }
    }
}

// The same for dims d0 .. d1 - 1 (a multiple of sixteen) of this lane's output row, at dst from dim d0 on: a NaN there is an
// infinity times a residual of 0, anything else lacks what was zeroed for the product. Sums of 0 (nothing found, or finite
// values whose weighted sum left fp32) change nothing. inv: 1 / the row's sum of weights.
template <bool IS_BF16>
__device__ __noinline__ void add_nonfinite(const DecodeParams& p, int b, int kvh, int P, int DH, int d0, int d1, int lo,
                                           int hi, float inv, float* dst) {
    for (int d = d0; d < d1; d += 16) {
        float x[16];
        sum_nonfinite16<IS_BF16>(p, b, kvh, P, DH, d, lo, hi, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (x[i] == 0.f) continue;
            float& y = dst[d - d0 + i];
            y = y != y ? x[i] * inv : y + x[i] * inv;
        }
    }
}

}  // namespace kvp
