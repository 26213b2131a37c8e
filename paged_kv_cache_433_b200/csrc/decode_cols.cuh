// Paged decode attention with the heads as MMA columns (sm_100a): the kernel
// of paged_decode_attention_int8 (int8 K/V with a scale per token and head)
// and of paged_decode_attention_mod (16-bit K/V, modified scores and masks).
//
// Same contract and the same online (m, l, u) merge as decode_mma.cuh
// ("07｜KV Cache、FlashAttention与PagedAttention的内部过程", Q027), with the two
// contractions of a stage of TP = 32 tokens transposed:
//   S^T[TP x 8 NT]  = K[TP x Dh] . Q^T[Dh x 8 NT]     (m16n8k16, k over dims)
//   O^T[Dh x 8 NT] += V^T[Dh x TP] . P^T[TP x 8 NT]   (m16n8k16, k over tokens)
// A GQA group of up to 8 heads fills an MMA's 8 columns, where it would fill
// half of the 16 rows: half the MMAs, and half the registers of Q and of the
// output, so that three CTAs of four consumer warps run on an SM. That
// matters most for int8: a stage costs about 900 instructions there (the codes
// are widened with integer operations), far from what one warp scheduler
// issues but with few warps bound by their latencies (8B-shaped layer, B = 64:
// rows as heads 81 us, 8 consumer warps an SM, 0.45 instructions a cycle and
// scheduler).
//
// Probabilities go into the second product as a 16-bit value plus its rounded
// residual. Their fragment (token rows, head columns) becomes the second
// product's B operand by movmatrix, 8 x 8 at a time. With at most 4 heads
// (DUP), columns 4..7 repeat the queries of columns 0..3: their lanes compute
// the same probabilities and hand over the residuals, so one MMA does both.
// The row maximum is only voted on (any score above the reference by more than
// 2^8?); the lanes of a head meet in shuffles when it has to move.
//
// Data movement as in decode_mma.cuh: one producer warp, 2-D TMA boxes of a
// page's rows x 128 bytes with 128-byte swizzle (64 for int8 rows of 64
// bytes), a ring of stages; int8 scales are one bulk copy per (page, head).
// Pages outside the pool are skipped one by one (KV_DEV_ERR_PAGE_RANGE).
// Bound by HBM where the batch fills the machine.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "decode_launch.cuh"
#include "int8.cuh"
#include "score_mod.cuh"

namespace kvp {

template <int KT, int DH, int P, int NT>
struct ColsCfg {
    static constexpr bool kI8 = KT == KV_DTYPE_INT8;
    static constexpr int kEB = kI8 ? 1 : 2;
    static constexpr int kTP = 32;                               // tokens per stage
    static constexpr int kPPS = kTP / P;                         // pages per stage
    static constexpr int kRowB = DH * kEB;                       // bytes per token row
    static constexpr int kBoxInner = kRowB < 128 ? kRowB : 128;  // bytes per box row
    static constexpr int kBoxes = kRowB / kBoxInner;             // boxes per token row
    static constexpr int kBoxElems = kBoxInner / kEB;
    static constexpr int kPageB = P * kBoxInner;                 // one page's rows of one box column
    static constexpr int kBoxB = kTP * kBoxInner;                // one box column of a stage
    static constexpr int kChunk = kTP * kRowB;                   // K (or V) of one stage
    static constexpr int kStage = 2 * kChunk;
    static constexpr int kScaleB = kI8 ? P * 8 : 0;              // scales of one (page, head): K's P, then V's
    static constexpr int kNC = 4;                                // consumer warps
    static constexpr int kCtas = NT == 1 ? 3 : 2;                // CTAs per SM
    static constexpr int kBudget = (NT == 1 ? 64 : 96) * 1024;   // ring bytes
    static constexpr int kNS0 = kBudget / kStage / kNC * kNC;
    static constexpr int kNS = kNS0 > 16 ? 16 : kNS0;            // stages: a multiple of the consumer warps
    static constexpr int kMergeB = kNC * NT * 8 * (DH + 2) * 4;  // per-warp (O, m, l) rows, aliased on the ring
    static constexpr int kRing = kNS * kStage;
    static constexpr int kOffBars = kRing > kMergeB ? kRing : kMergeB;
    static constexpr int kOffPages = kOffBars + 16 * kNS;        // bit j of word s: page j of stage s was loaded
    static constexpr int kOffScales = (kOffPages + 4 * kNS + 127) / 128 * 128;
    static constexpr int kSmem = 1024 + kOffScales + kNS * kPPS * kScaleB;  // + slack to align the ring to 1024 bytes
    static constexpr int kThreads = 32 * (kNC + 1);
    static_assert(kTP % P == 0 && (kBoxInner == 128 || kBoxInner == 64), "shape");
    static_assert(kNS >= kNC && kNS % kNC == 0, "every stage goes to the same warp each time");
    static_assert(kSmem * kCtas <= 227 * 1024, "shared memory");
};

// Transpose of an 8 x 8 matrix of 16-bit values held two to a lane (row lane / 4, columns 2 (lane % 4), + 1).
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

template <int KT, int QT, int DH, int P, int NT, bool DUP, bool MOD>
__global__ void __launch_bounds__(160, (ColsCfg<KT, DH, P, NT>::kCtas))
    paged_decode_cols_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ CUtensorMap tmap_k,
                             const __grid_constant__ CUtensorMap tmap_v) {
    using C = ColsCfg<KT, DH, P, NT>;
    constexpr bool kI8 = C::kI8;
    constexpr bool kQBF16 = !kI8 && KT == KV_DTYPE_BF16;  // QK operands: bf16, else f16 (int8 codes are exact in both)
    constexpr bool kPBF16 = kI8 || KT == KV_DTYPE_BF16;   // PV operands (int8: bf16, whose range holds any V scale)
    constexpr int kTP = C::kTP, kKS = DH / 16, kMT = kTP / 16, kOM = DH / 16, kPPS = C::kPPS;
    static_assert(!DUP || NT == 1, "doubled columns");
    extern __shared__ __align__(1024) unsigned char smem_raw[];

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
    }
    grid_dependency_wait();  // inputs (and a plan) may come from the previous kernel in the stream
    if (threadIdx.x == 0) grid_launch_dependents();

    // ---- work of this CTA: (split, kvh, b) from the grid, or a planned chunk
    int split, kvh, b, item = 0, chunk_pages;
    if (p.items != nullptr) {
        const int4 it = p.items[blockIdx.x];
        if (it.x < 0) return;
        b = it.x;
        kvh = it.y;
        split = it.z;
        item = it.w;
        chunk_pages = p.plan[0];
    } else {
        split = blockIdx.x;
        kvh = blockIdx.y;
        b = blockIdx.z;
        chunk_pages = p.pages_per_split;
    }
    const bool chunked = p.items != nullptr || p.num_splits > 1;
    int len = p.seq_lens[b];
    if (len < 0 || len > p.max_blocks * P) {
        if (threadIdx.x == 0 && split == 0 && p.items == nullptr) raise_err(p.err, KV_DEV_ERR_SEQ_LEN);
        len = 0;
    }
    // the row's pages are counted from its first visible key
    const int key_begin = MOD ? first_key(p, b, len - 1) : 0;
    const int n_pages = (len + P - 1) / P;
    const int first0 = min(key_begin, len) / P;
    const int first = first0 + (chunked ? split * chunk_pages : 0);
    const int n_local = chunked ? min(chunk_pages, n_pages - first) : n_pages - first;
    const bool split_mode = p.items != nullptr ? n_pages - first0 > chunk_pages : p.num_splits > 1;
    if (n_local <= 0) {
        if (!split_mode)
            for (int e = threadIdx.x; e < p.g * DH; e += blockDim.x)
                p.out[((int64_t)b * p.H_q + (int64_t)kvh * p.g) * DH + e] = 0.f;
        return;
    }
    const int n_st = (n_local + kPPS - 1) / kPPS;

    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    unsigned char* smem = smem_raw + (sbase - raw);
    const uint32_t full_bar = sbase + C::kOffBars;
    const uint32_t empty_bar = full_bar + 8 * C::kNS;
    volatile int* stage_pages = reinterpret_cast<volatile int*>(smem + C::kOffPages);
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kNS; ++s) {
            mbar_init(full_bar + 8 * s, 1);
            mbar_init(empty_bar + 8 * s, p.HS);
        }
        fence_barrier_init();
    }
    __syncthreads();

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        // kGrp stages per step: lane l < kGrp claims stage base + l (bounded wait on its empty barrier, expect_tx for
        // its good pages), then every lane issues one TMA box and, for int8, the first lanes one copy of scales each
        constexpr int kBPS = kPPS * 2 * C::kBoxes;           // boxes per stage
        constexpr int kGrp = C::kNS >= 16 ? 4 : C::kNS >= 8 ? 2 : 1;  // a group waits for all its stages: at most a quarter of the ring
        static_assert(kGrp * kBPS <= 32, "one TMA box per lane");
        static_assert(32 % (kGrp * kPPS) == 0, "page groups must tile the 32-entry table window");
        const int32_t* row = p.block_tables + (int64_t)b * p.max_blocks + first;
        bool ok = true;
        int issued = 0;
        int tab = 0;  // block-table entry of page (first page of the group & ~31) + lane
        for (int base = 0; base < n_st; base += kGrp) {
            const int pbase = base * kPPS;
            if ((pbase & 31) == 0) tab = pbase + lane < n_local ? row[pbase + lane] : -1;
            const int cnt = min(kGrp, n_st - base);
            int good = 0;
#pragma unroll
            for (int j = 0; j < kPPS; ++j) {
                const int pg = __shfl_sync(0xffffffffu, tab, ((base + lane) * kPPS + j) & 31);
                const bool here = lane < cnt && (base + lane) * kPPS + j < n_local;
                const bool in = pg >= 0 && pg < p.num_pages;
                if (here && !in) raise_err(p.err, KV_DEV_ERR_PAGE_RANGE);
                good |= here && in ? 1 << j : 0;
            }
            if (lane < cnt) {
                const int i = base + lane, s = i % C::kNS;
                if (i >= C::kNS && !mbar_wait_bounded(empty_bar + 8 * s, ((i / C::kNS) - 1) & 1, kWaitLimitNs)) {
                    raise_err(p.err, KV_DEV_ERR_TIMEOUT);
                    ok = false;
                } else {
                    stage_pages[s] = good;
                    if (good)
                        mbar_arrive_expect_tx(full_bar + 8 * s, __popc(good) * (2 * C::kBoxes * C::kPageB + C::kScaleB));
                    else
                        mbar_arrive(full_bar + 8 * s);
                }
            }
            if (!__all_sync(0xffffffffu, ok)) break;
            if constexpr (kI8) {
                const int st = lane / kPPS, j = lane % kPPS;
                const int g_st = __shfl_sync(0xffffffffu, good, st & 31);
                const int pg = __shfl_sync(0xffffffffu, tab, ((base + st) * kPPS + j) & 31);
                if (st < cnt && ((g_st >> j) & 1)) {
                    const int s = (base + st) % C::kNS;
                    bulk_g2s(sbase + C::kOffScales + (s * kPPS + j) * C::kScaleB,
                             p.kv_scales + ((int64_t)pg * p.H_kv + kvh) * (2 * P), C::kScaleB, full_bar + 8 * s);
                }
            }
            const int st = lane / kBPS, bx = lane % kBPS;
            const int j = bx / (2 * C::kBoxes);             // page of the stage
            const bool is_v = ((bx / C::kBoxes) & 1) != 0;
            const int bb = bx % C::kBoxes;                  // box of the token row
            const int g_st = __shfl_sync(0xffffffffu, good, st & 31);
            const int pg = __shfl_sync(0xffffffffu, tab, ((base + st) * kPPS + j) & 31);
            if (st < cnt && ((g_st >> j) & 1)) {
                const int s = (base + st) % C::kNS;
                const uint32_t dst = sbase + s * C::kStage + (is_v ? C::kChunk : 0) + bb * C::kBoxB + j * C::kPageB;
                tma_load_2d(dst, is_v ? static_cast<const void*>(&tmap_v) : static_cast<const void*>(&tmap_k),
                            bb * C::kBoxElems, (pg * p.H_kv + kvh) * P, full_bar + 8 * s);
            }
            issued = base + cnt;
        }
        if (lane == 0)  // every copy has landed before the CTA exits
            for (int i = max(0, issued - C::kNS); i < issued; ++i)
                if (!mbar_wait_bounded(full_bar + 8 * (i % C::kNS), (i / C::kNS) & 1, kWaitLimitNs))
                    raise_err(p.err, KV_DEV_ERR_TIMEOUT);
        return;
    }

    // -------------------------------------------------------------- consumers
    const int cw = warp - 1;
    const int hs = cw % p.HS;   // slice of 8 NT heads
    const int wp = cw / p.HS;   // page-warp: stages wp, wp + WP, ...
    const int r0 = lane >> 2, quad = lane & 3;
    const int heads = min(NT * 8, p.g - hs * NT * 8);  // heads of this slice
    const int head0 = kvh * p.g + hs * NT * 8;

    // Q^T as the B operand: column lane / 4 of column tile nt is head nt * 8 + lane / 4 (DUP: 4 heads twice). 16-bit
    // K/V: k-step kk covers dims kk*16 .. +15; int8: the lane's K words hold dims quad*Dh/4 + 4*kk .. +3.
    uint32_t qb[NT][kKS][2];
    float q_pow[NT][2];  // int8, bf16 q: what a row was divided by, for the lane's score columns
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int n = nt * 8 + r0;
        const int h = DUP ? n & 3 : n;
        const uint32_t* q32 = static_cast<const uint32_t*>(p.q) + (((int64_t)b * p.H_q + head0 + h) * DH >> 1);
        float pow = 1.f;
#pragma unroll
        for (int kk = 0; kk < kKS; ++kk)
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) {
                const int d = kI8 ? quad * (DH / 4) + 4 * kk + 2 * ch : kk * 16 + ch * 8 + 2 * quad;
                qb[nt][kk][ch] = h < heads ? q32[d >> 1] : 0u;
            }
        if constexpr (kI8 && QT == KV_DTYPE_BF16) {
            // the products with codes run in f16: a bf16 row is divided by a power of two that brings its largest
            // magnitude to 2^14 (exact but for elements 2^-28 below it and smaller, whose rounding is at most 2^-39
            // of the largest) and its scores are multiplied back: the whole bf16 range works
            uint32_t top = 0;
#pragma unroll
            for (int kk = 0; kk < kKS; ++kk)
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    const uint32_t v = qb[nt][kk][ch];
                    top = max(top, max((v << 16) & 0x7fffffffu, v & 0x7fff0000u));
                }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = max(static_cast<int>(top >> 23) - 127, -100);  // floor(log2(largest)); 128: inf or NaN
            const float down = __int_as_float((14 - ex + 127) << 23);
            pow = __int_as_float((ex - 14 + 127) << 23);
#pragma unroll
            for (int kk = 0; kk < kKS; ++kk)
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    const float2 v = unpack16<true>(qb[nt][kk][ch]);
                    qb[nt][kk][ch] = pack2<false>(v.x * down, v.y * down);
                }
        }
        // score columns of this lane: 2 quad, 2 quad + 1 (rows of lanes 8 quad, 8 quad + 4 above)
        q_pow[nt][0] = __shfl_sync(0xffffffffu, pow, 8 * quad) * p.scale_log2;
        q_pow[nt][1] = __shfl_sync(0xffffffffu, pow, 8 * quad + 4) * p.scale_log2;
    }
    float slope[NT][2] = {};
    if constexpr (MOD) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = nt * 8 + 2 * quad + e, h = DUP ? n & 3 : n;
                slope[nt][e] = p.alibi_slopes != nullptr && h < heads ? p.alibi_slopes[head0 + h] * kLog2e : 0.f;
            }
    }

    // O^T: rows r0 / r0 + 8 of dim tile m, columns 2 quad, + 1
    float o[NT][kOM][4];
    float m_ref[NT][2], l_part[NT][2];  // reference maximum (log2 units) and this lane's sums, per column
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int m = 0; m < kOM; ++m) o[nt][m][0] = o[nt][m][1] = o[nt][m][2] = o[nt][m][3] = 0.f;
        m_ref[nt][0] = m_ref[nt][1] = -INFINITY;
        l_part[nt][0] = l_part[nt][1] = 0.f;
    }

    bool ok = true;
    if (wp < p.WP) {
        const int mi = lane >> 3, r8 = lane & 7;  // ldmatrix: matrix and row this lane addresses
        for (int i = wp; i < n_st; i += p.WP) {
            const int s = i % C::kNS;
            if (!mbar_wait_bounded(full_bar + 8 * s, (i / C::kNS) & 1, kWaitLimitNs)) {
                raise_err(p.err, KV_DEV_ERR_TIMEOUT);
                ok = false;
            }
            if (!__all_sync(0xffffffffu, ok)) break;
            const int pages = stage_pages[s];
            const uint32_t sK = sbase + s * C::kStage, sV = sK + C::kChunk;
            const uint32_t sS = sbase + C::kOffScales + s * (kPPS * C::kScaleB);
            const int kbase = (first + i * kPPS) * P;
            // visible tokens of the stage: [tlo, thi), on pages that were loaded (the same for every head)
            const int thi = min(min(kPPS, n_local - i * kPPS) * P, len - kbase);
            const int tlo = MOD ? key_begin - kbase : 0;
            const bool whole = tlo <= 0 && thi >= kTP && pages == (1 << kPPS) - 1;

            // ---- S^T = K Q^T: rows r0 / r0 + 8 of token tile mt, columns 2 quad, + 1
            float sc[NT][kMT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt) sc[nt][mt][0] = sc[nt][mt][1] = sc[nt][mt][2] = sc[nt][mt][3] = 0.f;
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) {
                if constexpr (kI8) {
                    uint32_t w[2][DH / 16];  // tokens r0, r0 + 8: this lane's Dh/4 codes
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int c = 0; c < DH / 64; ++c) {
                            const uint4 x = lds128(sK + swz<C::kBoxInner>(mt * 16 + r0 + 8 * h, quad * (DH / 64) + c));
                            w[h][4 * c] = x.x, w[h][4 * c + 1] = x.y, w[h][4 * c + 2] = x.z, w[h][4 * c + 3] = x.w;
                        }
#pragma unroll
                    for (int kk = 0; kk < kKS; ++kk) {
                        uint32_t a[4];
                        s8x4_to_f16x2x2(w[0][kk], a[0], a[2]);
                        s8x4_to_f16x2x2(w[1][kk], a[1], a[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_16816<false>(sc[nt][mt], a, qb[nt][kk][0], qb[nt][kk][1]);
                    }
                } else {
#pragma unroll
                    for (int kk = 0; kk < kKS; ++kk) {
                        const int c = kk * 2 + (mi >> 1), t = mt * 16 + (mi & 1) * 8 + r8;
                        uint32_t a[4];
                        ldsm_x4(sK + (c >> 3) * C::kBoxB + swz<128>(t, c), a[0], a[1], a[2], a[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_16816<kQBF16>(sc[nt][mt], a, qb[nt][kk][0], qb[nt][kk][1]);
                    }
                }
            }

            // ---- scores in log2 units, masked; has any moved above the reference by more than 2^8?
            float vs[kMT][2];  // int8: V scales of tokens r0, r0 + 8
            bool grow = false;
            if constexpr (MOD) modify_cols<NT, kMT>(p, sc, slope, len - 1 - kbase - r0);
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int t = mt * 16 + h * 8 + r0;
                    float ks = 1.f;
                    if constexpr (kI8) {
                        const uint32_t at = sS + (mt * 16 / P) * C::kScaleB + (mt * 16 % P + h * 8 + r0) * 4;
                        ks = lds_float(at);
                        vs[mt][h] = lds_float(at + P * 4);
                    }
                    const bool seen = whole || (t >= tlo && t < thi && ((pages >> (mt * 16 / P)) & 1));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float& x = sc[nt][mt][2 * h + e];
                            if constexpr (kI8) x *= ks * q_pow[nt][e];
                            if (!seen) x = -INFINITY;
                            grow |= x > m_ref[nt][e] + 8.f;
                        }
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = -INFINITY;
#pragma unroll
                        for (int mt = 0; mt < kMT; ++mt) mx = fmaxf(mx, fmaxf(sc[nt][mt][e], sc[nt][mt][2 + e]));
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                        const float mn = fmaxf(m_ref[nt][e], mx);
                        const float al = mn == m_ref[nt][e] ? 1.f : exp2f(m_ref[nt][e] - mn);
                        m_ref[nt][e] = mn;
                        l_part[nt][e] *= al;
#pragma unroll
                        for (int m = 0; m < kOM; ++m) o[nt][m][e] *= al, o[nt][m][2 + e] *= al;
                    }
            }

            // ---- probabilities, transposed into the B operand (tokens 2 quad, + 1 of each block of 8; head lane / 4)
            uint32_t ph[NT][kMT][2], pl[NT][kMT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float pv[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float x = sc[nt][mt][2 * h + e];
                            pv[e] = x == -INFINITY ? 0.f : exp2f(x - m_ref[nt][e]);
                            l_part[nt][e] += pv[e];
                            // a masked token's scale may be anything: its weight is 0
                            if constexpr (kI8) pv[e] = x == -INFINITY ? 0.f : pv[e] * vs[mt][h];
                        }
                        uint32_t hi, lo;
                        pack2_split<kPBF16>(pv[0], pv[1], hi, lo);
                        if constexpr (DUP) {
                            ph[nt][mt][h] = movmatrix_trans(quad < 2 ? hi : lo);
                        } else {
                            ph[nt][mt][h] = movmatrix_trans(hi);
                            pl[nt][mt][h] = movmatrix_trans(lo);
                        }
                    }

            // ---- V rows that no head sees may hold NaN (int8 codes cannot): zero them
            if constexpr (!kI8) {
                if (!whole) {
                    constexpr int kCPR = 8;  // 16-byte chunks per box row
                    for (int idx = lane; idx < kTP * C::kBoxes * kCPR; idx += 32) {
                        const int t = idx / (C::kBoxes * kCPR), rem = idx % (C::kBoxes * kCPR);
                        if (t < tlo || t >= thi || !((pages >> (t / P)) & 1))
                            sts128_zero(sV + (rem / kCPR) * C::kBoxB + t * 128 + ((rem % kCPR) << 4));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
            }

            // ---- O^T += V^T P^T
#pragma unroll
            for (int ks = 0; ks < kMT; ++ks) {
                if constexpr (kI8) {
                    // dim tile m, row r0 (+8) is dim r0 * Dh/8 + 2 m (+1): the lane reads its Dh/8 codes of tokens
                    // 2 quad, + 1, + 8, + 9 and pairs the two tokens' bytes per dim
                    constexpr int kW = DH / 32;  // words per token row per lane
                    uint32_t wv[4][kW];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = ks * 16 + 2 * quad + (e & 1) + 8 * (e >> 1);
                        if constexpr (DH == 128) {
                            const uint4 x = lds128(sV + swz<C::kBoxInner>(t, r0));
                            wv[e][0] = x.x, wv[e][1] = x.y, wv[e][2] = x.z, wv[e][3] = x.w;
                        } else {
                            const uint2 x = lds64(sV + swz<C::kBoxInner>(t, r0 >> 1) + (r0 & 1) * 8);
                            wv[e][0] = x.x, wv[e][1] = x.y;
                        }
                    }
#pragma unroll
                    for (int m = 0; m < kW; ++m)
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {  // bytes 0-1 or 2-3 of word m: dim tile 2m + hh
                            const uint32_t sel = hh ? 0x7362u : 0x5140u;
                            uint32_t a[4];
                            s8x4_to_bf16x2x2(byte_perm(wv[0][m], wv[1][m], sel), a[0], a[1]);
                            s8x4_to_bf16x2x2(byte_perm(wv[2][m], wv[3][m], sel), a[2], a[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma_16816<true>(o[nt][2 * m + hh], a, ph[nt][ks][0], ph[nt][ks][1]);
                                if constexpr (!DUP) mma_16816<true>(o[nt][2 * m + hh], a, pl[nt][ks][0], pl[nt][ks][1]);
                            }
                        }
                } else {
#pragma unroll
                    for (int m = 0; m < kOM; ++m) {
                        const int c = m * 2 + (mi & 1), t = ks * 16 + (mi >> 1) * 8 + r8;
                        uint32_t a[4];
                        ldsm_x4_trans(sV + (c >> 3) * C::kBoxB + swz<128>(t, c), a[0], a[1], a[2], a[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_16816<kPBF16>(o[nt][m], a, ph[nt][ks][0], ph[nt][ks][1]);
                            if constexpr (!DUP) mma_16816<kPBF16>(o[nt][m], a, pl[nt][ks][0], pl[nt][ks][1]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty_bar + 8 * s);
        }
    }

    // ---- finalize: column sums over the lanes of a head, then merge the page-warps in shared memory
    named_bar_sync(1, 32 * C::kNC);  // every consumer is done with the stages (the merge rows alias them)
    float* merge = reinterpret_cast<float*>(smem);  // [kNC][8 NT][DH + 2]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float l = l_part[nt][e];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
            // a NaN sum keeps its place in the merge whatever the column's maximum is
            const float mr = l != l && m_ref[nt][e] == -INFINITY ? 0.f : m_ref[nt][e];
            const int n = nt * 8 + 2 * quad + e;
            float* dst = merge + (cw * NT * 8 + n) * (DH + 2);
#pragma unroll
            for (int m = 0; m < kOM; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x = o[nt][m][2 * h + e];
                    if constexpr (DUP) x += __shfl_xor_sync(0xffffffffu, x, 2);  // values and residuals of a head
                    const int d = kI8 ? r0 * (DH / 8) + 2 * m + h : m * 16 + h * 8 + r0;
                    if (n < heads && wp < p.WP) dst[d] = x;
                }
            if (r0 == 0 && n < heads && wp < p.WP) dst[DH] = mr, dst[DH + 1] = l;
        }
    named_bar_sync(1, 32 * C::kNC);

    for (int e = threadIdx.x - 32; e < p.g * DH; e += 32 * C::kNC) {
        const int hh = e / DH, d = e % DH;
        const int slice = hh / (NT * 8), n = hh % (NT * 8);
        float mstar = -INFINITY;
        for (int w = 0; w < p.WP; ++w) mstar = fmaxf(mstar, merge[((w * p.HS + slice) * NT * 8 + n) * (DH + 2) + DH]);
        float L = 0.f, U = 0.f;
        if (mstar != -INFINITY) {
            for (int w = 0; w < p.WP; ++w) {
                const float* src = merge + ((w * p.HS + slice) * NT * 8 + n) * (DH + 2);
                if (src[DH] == -INFINITY) continue;
                const float sw = exp2f(src[DH] - mstar);
                L += sw * src[DH + 1];
                U += sw * src[d];
            }
        }
        // An infinity among the visible values meets a probability's residual, which may be 0 or negative: a NaN.
        // Where a sum is NaN and the weights are not (rare), the values say what it is.
        if constexpr (MOD)
            if (U != U && L == L)
                U = sum_nonfinite<kPBF16>(p, b, kvh, P, DH, d, max(key_begin, first * P), min(len, (first + n_local) * P));
        const int64_t hq = (int64_t)b * p.H_q + (int64_t)kvh * p.g + hh;
        if (!split_mode) {
            p.out[hq * DH + d] = L != 0.f ? U / L : 0.f;
        } else {
            const int64_t ps = p.items != nullptr ? (int64_t)item * p.g + hh : hq * p.num_splits + split;
            p.part_u[ps * DH + d] = U;
            if (d == 0) p.part_ml[ps] = make_float2(mstar, L);
        }
    }
}

// ---- dispatch ---------------------------------------------------------------
template <int KT, int QT, int DH, int P, int NT, bool DUP, bool MOD>
cudaError_t launch_cols_inst(DecodeParams p, const CUtensorMap& tk, const CUtensorMap& tv, dim3 grid, cudaStream_t st) {
    using C = ColsCfg<KT, DH, P, NT>;
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    auto* kern = paged_decode_cols_kernel<KT, QT, DH, P, NT, DUP, MOD>;
    if (!(configured.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    p.HS = (p.g + NT * 8 - 1) / (NT * 8);
    p.WP = C::kNC / p.HS;
    return launch_pdl(kern, grid, dim3(C::kThreads), C::kSmem, st, p, tk, tv);
}

// Groups of at most 4 heads: doubled columns; at most 8: one column tile; larger ones (up to 64): slices of 16 heads.
template <int KT, int QT, int DH, int P, bool MOD>
cudaError_t launch_cols_group(const DecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, dim3 grid,
                              cudaStream_t st) {
    if (p.g <= 4) return launch_cols_inst<KT, QT, DH, P, 1, true, MOD>(p, tk, tv, grid, st);
    if (p.g <= 8) return launch_cols_inst<KT, QT, DH, P, 1, false, MOD>(p, tk, tv, grid, st);
    return launch_cols_inst<KT, QT, DH, P, 2, false, MOD>(p, tk, tv, grid, st);
}

template <int KT, int QT, bool MOD>
cudaError_t launch_cols_dt(const DecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int DH, int P, dim3 grid,
                           cudaStream_t st) {
    if (DH == 128)
        return P == 16 ? launch_cols_group<KT, QT, 128, 16, MOD>(p, tk, tv, grid, st)
                       : launch_cols_group<KT, QT, 128, 32, MOD>(p, tk, tv, grid, st);
    return P == 16 ? launch_cols_group<KT, QT, 64, 16, MOD>(p, tk, tv, grid, st)
                   : launch_cols_group<KT, QT, 64, 32, MOD>(p, tk, tv, grid, st);
}

}  // namespace kvp
