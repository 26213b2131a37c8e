// Paged decode attention with the heads as MMA columns (sm_100a): the kernel
// of paged_decode_attention_int8 (int8 K/V with a scale per token and head)
// and of paged_decode_attention_mod (16-bit K/V, modified scores and masks).
//
// Same contract and the same online (m, l, u) merge as decode_mma.cuh
// ("07｜KV Cache、FlashAttention与PagedAttention的内部过程", Q027), with the two
// contractions of a stage of TP tokens (16; int8: 32) transposed:
//   S^T[TP x 8 NT]  = K[TP x Dh] . Q^T[Dh x 8 NT]     (k over dims)
//   O^T[Dh x 8 NT] += V^T[Dh x TP] . P^T[TP x 8 NT]   (m16n8k16, k over tokens)
// A GQA group of up to 8 heads fills an MMA's 8 columns, where it would fill
// half of the 16 rows: half the MMAs, and half the registers of Q and of the
// output, so that three CTAs of four consumer warps run on an SM. That
// matters most for int8, whose warps are bound by latencies: 64 sequences of
// 512..4096 tokens of an 8B-shaped layer (32 heads on 8, Dh = 128) took 81 us
// with heads as rows and 8 consumer warps an SM, and take 62 us.
//
// int8: the K codes are the first product's operand as they are (m16n8k32 of
// signed bytes, 32-bit sums, exact); a query row, behind a power of two, is an
// integer of 23 bits split into three signed bytes, an MMA each. The V codes
// are widened to bf16, which holds them exactly, and their scales multiply the
// probabilities.
//
// Probabilities go into the second product as a 16-bit value plus its rounded
// residual (bf16 K/V: and that one's). Their fragment (token rows, head columns) becomes the second
// product's B operand by movmatrix, 8 x 8 at a time. With at most 4 heads
// (DUP), columns 4..7 repeat the queries of columns 0..3: their lanes compute
// the same probabilities and hand over the residuals, so one MMA does both.
// The row maximum is only voted on (any score above the reference by more than
// 2^8?); the lanes of a head meet in shuffles when it has to move.
//
// Work: pieces of (sequence, KV head) rows. With explicit splits a CTA has one
// piece, given by the grid. Otherwise the launch is balanced: every CTA reads
// the lengths, lays the rows end to end -- each counted with a few pages more
// for its fixed cost -- and takes an equal range of that line (the plan of
// plan_kernel.cuh's stream form, computed by every CTA for itself: no launch
// before this one; B up to kColsMaxB). The CTAs are as many as fit the machine
// and walk their range piece by piece, the producer running ahead of the
// consumers into the next piece. A row cut between CTAs leaves partials in two
// slots per CTA, which paged_combine_cols_kernel merges.
//
// Data movement as in decode_mma.cuh: one producer warp, 2-D TMA boxes of a
// page's rows x 128 bytes with 128-byte swizzle (64 for int8 rows of 64
// bytes; at most 16 rows for 16-bit pages), a ring of stages; int8 scales are
// one bulk copy per (page, head). Pages outside the pool are skipped one by
// one (KV_DEV_ERR_PAGE_RANGE).
//
// Measured (8B-shaped layer, time of the whole call on the GPU, of the measured
// copy rate): 16-bit, capped, 64 sequences of 512..4096 tokens 69 us, 5.76 TB/s
// (0.88); 256 of 16..8192 with document masks and a distance bias 65 us (0.78,
// the lengths' spread and the merge); int8, those 64: 62 us, 4.18 TB/s (0.64:
// its loads alone take 47 us; scales, integer products and widening share the
// issue slots); int8, one sequence of 32768: 26 us (0.41: 444 CTAs' start and
// the merge of one row's 55 pieces). Groups above 8 heads spill at Dh = 128:
// int8, 128 heads on 8, 125 us for the 64 sequences.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "decode_launch.cuh"
#include "int8.cuh"
#include "score_mod.cuh"

namespace kvp {

constexpr int kColsMaxB = 1024;      // sequences of a balanced launch
// Groups of at most 8 heads: consumer warps per CTA, CTAs per SM (8B-shaped layer, int8, 64 sequences of 512..4096
// tokens: 68 us when 2 CTAs of 7 warps took 77, 2 of 6 72, 4 of 3 74.5, one of 15 97).
constexpr int kColsWarps1 = 4, kColsCtas1 = 3;
constexpr int kColsItemTokens = 128; // a row's fixed cost in tokens (its queries, its merge)
constexpr int kColsMinTokens = 128;  // at least one stage per consumer warp and CTA

template <int KT, int DH, int P, int NT, bool DUP>
struct ColsCfg {
    static constexpr bool kI8 = KT == KV_DTYPE_INT8;
    static constexpr int kEB = kI8 ? 1 : 2;
    static constexpr int kTP = kI8 ? 32 : 16;                    // tokens per stage
    static constexpr int kU = P < kTP ? P : kTP;                 // rows of a TMA box: a page, or half a page of 32
    static constexpr int kUPS = kTP / kU;                        // boxes of rows per stage
    static constexpr int kUPP = P / kU;                          // and per page
    static constexpr int kRowB = DH * kEB;                       // bytes per token row
    static constexpr int kBoxInner = kRowB < 128 ? kRowB : 128;  // bytes per box row
    static constexpr int kBoxes = kRowB / kBoxInner;             // boxes per token row
    static constexpr int kBoxElems = kBoxInner / kEB;
    static constexpr int kUnitB = kU * kBoxInner;                // one box
    static constexpr int kBoxB = kTP * kBoxInner;                // one box column of a stage
    static constexpr int kChunk = kTP * kRowB;                   // K (or V) of one stage
    static constexpr int kStage = 2 * kChunk;
    static constexpr int kScaleB = kI8 ? P * 8 : 0;              // scales of one (page, head): K's P, then V's
    static constexpr int kNC = NT == 1 ? kColsWarps1 : 4;        // consumer warps
    static constexpr int kCtas = NT == 1 ? kColsCtas1 : 2;       // CTAs per SM
    // a warp's (O, m, l) fragments on their way to the warp that merges: [registers][lanes]
    static constexpr int kRegs = NT * (DH / 16) * 4 + 4 * NT;
    static constexpr int kMergeWarp = kRegs * (DUP ? 16 : 32) * 4;
    static constexpr int kMergeB = (kNC - 1) * kMergeWarp;
    static constexpr int kFixed = 1024 /* alignment */ + 1024 /* reserved */ + kMergeB + 4 * (kColsMaxB + 1) + 256;
    static constexpr int kNS0 = (227 * 1024 / kCtas - kFixed) / (kStage + kUPS * kScaleB + 20);
    static constexpr int kNS = kNS0 > 16 ? 16 : kNS0;            // stages
    static constexpr int kOffMerge = kNS * kStage;
    static constexpr int kOffScales = (kOffMerge + kMergeB + 127) / 128 * 128;
    static constexpr int kOffBars = kOffScales + kNS * kUPS * kScaleB;
    static constexpr int kOffPages = kOffBars + 16 * kNS;        // bit j of word s: unit j of stage s was loaded
    static constexpr int kOffPre = kOffPages + 4 * kNS;          // balanced launch: prefix of the rows' spans
    static constexpr int kSmem = 1024 + kOffPre + 4 * (kColsMaxB + 1) + 4 * 16;
    static constexpr int kThreads = 32 * (kNC + 1);
    static_assert(P % kU == 0 && (kBoxInner == 128 || kBoxInner == 64), "shape");
    static_assert(kNS >= kNC, "a stage per consumer warp");
    static_assert((kSmem + 1024) * kCtas <= 227 * 1024, "shared memory");
};

// Transpose of an 8 x 8 matrix of 16-bit values held two to a lane (row lane / 4, columns 2 (lane % 4), + 1).
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// One piece of a row: pages [page0, page0 + n) of (b, kvh); slot < 0: the whole row (its output is written), else the
// partial slot it leaves.
struct ColsPiece {
    int b, kvh, page0, n, len, key_begin, slot;
    __device__ __forceinline__ int tokens(int P) const { return n > 0 ? min(len - page0 * P, n * P) : 0; }
};

// Walks a CTA's pieces; every warp of the CTA runs one in step (all values are uniform over the warp).
template <int P, bool MOD>
struct ColsWalk {
    const DecodeParams& p;
    const int* pre;  // shared: exclusive prefix over b of the row spans D_b (B + 1 entries); nullptr: one grid piece
    int pos, end;   // line positions (the host keeps the line below 2^31)
    int start = 0;  // the first one
    int b, v;
    bool grid_done = false;

    __device__ __forceinline__ int length(int bb) const {
        const int len = p.seq_lens[bb];
        return len < 0 || len > p.max_blocks * P ? 0 : len;
    }
    __device__ __forceinline__ int begin_key(int bb, int len) const { return MOD ? min(first_key(p, bb, len - 1), len) : 0; }

    __device__ __forceinline__ bool next(ColsPiece& o) {
        if (pre == nullptr) {  // (split, kvh, b) of the grid; its slot is set by the caller's row order
            if (grid_done) return false;
            grid_done = true;
            o.b = blockIdx.z;
            o.kvh = blockIdx.y;
            o.len = length(o.b);
            o.key_begin = begin_key(o.b, o.len);
            const int first0 = o.key_begin / P, n_pages = (o.len + P - 1) / P - first0;
            const int skip = blockIdx.x * p.pages_per_split;
            o.page0 = first0 + skip;
            o.n = p.num_splits > 1 ? min(p.pages_per_split, n_pages - skip) : n_pages;
            o.slot = p.num_splits > 1 ? 0 : -1;
            return true;
        }
        while (pos < end) {
            while (pre[b + 1] * p.H_kv <= pos) ++b;
            const int D = pre[b + 1] - pre[b], local = pos - pre[b] * p.H_kv;
            const int kvh = local / D, off = local - kvh * D, row_end = pos - off + D;
            const int take = min(end, row_end) - pos;
            pos += take;
            const int p0 = max(off - v, 0), p1 = off + take - v;  // real pages of the row, its span less v
            if (p1 <= p0) continue;                               // only the fixed cost's part of the span
            o.b = b;
            o.kvh = kvh;
            o.len = length(b);
            o.key_begin = begin_key(b, o.len);
            o.page0 = o.key_begin / P + p0;
            o.n = p1 - p0;
            const bool whole = p0 == 0 && pos == row_end;
            o.slot = whole ? -1 : 2 * static_cast<int>(blockIdx.x) + (p0 == 0 ? 1 : 0);
            return true;
        }
        return false;
    }
};

template <int KT, int QT, int DH, int P, int NT, bool DUP, bool MOD>
__global__ void __launch_bounds__((ColsCfg<KT, DH, P, NT, DUP>::kThreads), (ColsCfg<KT, DH, P, NT, DUP>::kCtas))
    paged_decode_cols_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ CUtensorMap tmap_k,
                             const __grid_constant__ CUtensorMap tmap_v) {
    using C = ColsCfg<KT, DH, P, NT, DUP>;
    constexpr bool kI8 = C::kI8;
    constexpr bool kQBF16 = KT == KV_DTYPE_BF16;         // QK operands of 16-bit K/V: bf16, else f16
    constexpr bool kPBF16 = kI8 || KT == KV_DTYPE_BF16;   // PV operands (int8: bf16, whose range holds any V scale)
    constexpr int kTP = C::kTP, kKS = DH / 16, kMT = kTP / 16, kOM = DH / 16, kUPS = C::kUPS;
    // 16-bit bf16 K/V: a third term of the probabilities, so that they keep 24 bits (2.3e-7 of the result off; 2.4e-6 with
    // two, in the same 69 us: the product waits for memory). int8, bound by its instructions, keeps two (61.5 us; 65.3 with
    // three): its values are rounded to 8 bits anyway. fp16 has 22 bits with two.
    constexpr bool kThird = MOD && kPBF16;
    static_assert(!DUP || NT == 1, "doubled columns");
    extern __shared__ __align__(1024) unsigned char smem_raw[];

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
    }
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    unsigned char* smem = smem_raw + (sbase - raw);
    const uint32_t full_bar = sbase + C::kOffBars;
    const uint32_t empty_bar = full_bar + 8 * C::kNS;
    volatile int* stage_pages = reinterpret_cast<volatile int*>(smem + C::kOffPages);
    int* pre = reinterpret_cast<int*>(smem + C::kOffPre);
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kNS; ++s) {
            mbar_init(full_bar + 8 * s, 1);
            mbar_init(empty_bar + 8 * s, p.HS);
        }
        fence_barrier_init();
    }
    grid_dependency_wait();  // the inputs may come from the previous kernel in the stream
    // Persistent CTAs fill the machine: kernels launched behind them early would take their places (their combine's
    // CTAs, waiting on SMs that the next launch of this kernel then finds too full: 90 against 70 us a step).
    if (threadIdx.x == 0 && p.stream_plan == 0) grid_launch_dependents();

    // ---- this CTA's pieces
    const bool balanced = p.stream_plan != 0;
    constexpr int v = kColsItemTokens / P;
    int T = 0, G = 0;
    ColsWalk<P, MOD> walk{p, balanced ? pre : nullptr, 0, 0, 0, 0, v};
    if (balanced) {
        // spans D_b = pages from the first visible key on, plus v (0 without pages), and their prefix: thread t takes
        // rows t * per .. + per - 1
        int* warp_sum = pre + kColsMaxB + 1;
        const int per = (p.B + C::kThreads - 1) / C::kThreads, b0 = threadIdx.x * per;
        int sum = 0;
        for (int k = 0; k < per; ++k) {
            const int bb = b0 + k;
            if (bb >= p.B) break;
            const int raw_len = p.seq_lens[bb], len = walk.length(bb);
            if (raw_len != len && blockIdx.x == 0) raise_err(p.err, KV_DEV_ERR_SEQ_LEN);
            const int n = (len + P - 1) / P - walk.begin_key(bb, len) / P;
            if (n > 0) sum += n + v;
            pre[bb + 1] = sum;
        }
        int x = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        if (lane == 31) warp_sum[warp] = x;
        __syncthreads();
        int before = x - sum;
        for (int w = 0; w < warp; ++w) before += warp_sum[w];
        for (int k = 0; k < per && b0 + k < p.B; ++k) pre[b0 + k + 1] += before;
        if (threadIdx.x == 0) pre[0] = 0;
        __syncthreads();
        for (int bb = blockIdx.x; bb < p.B; bb += gridDim.x)  // rows without a visible page: no piece writes them
            if (pre[bb + 1] == pre[bb]) {
                for (int e = threadIdx.x; e < p.H_q * DH; e += C::kThreads) p.out[(int64_t)bb * p.H_q * DH + e] = 0.f;
                if (p.cuts_by_row && threadIdx.x < p.H_kv) p.cuts[bb * p.H_kv + threadIdx.x] = make_int4(-1, 0, 0, 0);
            }
        T = pre[p.B] * p.H_kv;
        constexpr int kMin = kColsMinTokens / P;
        G = min(static_cast<int>(gridDim.x), (T + kMin - 1) / kMin);
        const int c = blockIdx.x;
        if (c >= G) {
            if (threadIdx.x == 0 && !p.cuts_by_row) p.cuts[c] = make_int4(-1, 0, 0, 0);
            return;
        }
        // positions floor(c T / G) .. floor((c + 1) T / G) (without 64-bit divisions: G^2 fits an int)
        const int whole = T / G, rest = T - whole * G;
        walk.pos = walk.start = whole * c + rest * c / G;
        walk.end = whole * (c + 1) + rest * (c + 1) / G;
        int hi = p.B;  // largest b with H_kv * pre[b] <= pos
        while (hi - walk.b > 1) {
            const int mid = (walk.b + hi) >> 1;
            if (pre[mid] * p.H_kv <= walk.pos) walk.b = mid;
            else hi = mid;
        }
    } else {
        __syncthreads();
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && walk.length(blockIdx.z) != p.seq_lens[blockIdx.z])
            raise_err(p.err, KV_DEV_ERR_SEQ_LEN);
    }

    ColsPiece pc;
    int gs = 0;  // stages of the pieces before this one
    if (warp == 0) {
        // ------------------------------------------------------------ producer
        // kGrp stages per step: lane l < kGrp claims stage base + l (bounded wait on its empty barrier, expect_tx for
        // its good pages), then every lane issues one TMA box and, for int8, the first lanes one copy of scales each
        constexpr int kBPS = kUPS * 2 * C::kBoxes;  // boxes per stage
        constexpr int kGrp = C::kNS >= 16 ? 4 : C::kNS >= 6 ? 2 : 1;  // a group waits for all its stages
        constexpr int kPPG = kGrp * kUPS / C::kUPP > 0 ? kGrp * kUPS / C::kUPP : 1;  // pages per group (1: or half)
        static_assert(kGrp * kBPS <= 32, "one TMA box per lane");
        static_assert(32 % kPPG == 0, "page groups must tile the 32-entry table window");
        bool ok = true;
        int issued = 0;
        while (walk.next(pc)) {
            if (p.cuts_by_row && lane == 0 && (pc.slot & 1)) {  // the row starts here: whole (-1) or cut (2c + 1)
                const int64_t after = pre[pc.b] * p.H_kv + static_cast<int64_t>(pc.kvh + 1) * (pre[pc.b + 1] - pre[pc.b]);
                const int c = blockIdx.x, pieces = static_cast<int>((after * G - 1) / T) - c + 1;
                p.cuts[pc.b * p.H_kv + pc.kvh] = make_int4(pc.slot < 0 ? -1 : pc.b, pc.kvh, pieces, c);
            }
            if (!ok) continue;  // a wait ran out: no load any more, but the merge finds every row's entry
            const int n_units = (pc.tokens(P) + C::kU - 1) / C::kU, n_st = (n_units + kUPS - 1) / kUPS;
            const int32_t* row = p.block_tables + (int64_t)pc.b * p.max_blocks + pc.page0;
            int tab = 0;  // block-table entry of page (first page of the group & ~31) + lane
            for (int base = 0; base < n_st; base += kGrp) {
                const int pbase = base * kUPS / C::kUPP;
                if ((pbase & 31) == 0 && base * kUPS % C::kUPP == 0) tab = pbase + lane < pc.n ? row[pbase + lane] : -1;
                const int cnt = min(kGrp, n_st - base);
                int good = 0;
#pragma unroll
                for (int j = 0; j < kUPS; ++j) {
                    const int u = (base + lane) * kUPS + j;
                    const int pg = __shfl_sync(0xffffffffu, tab, (u / C::kUPP) & 31);
                    const bool here = lane < cnt && u < n_units;
                    const bool in = pg >= 0 && pg < p.num_pages;
                    if (here && !in) raise_err(p.err, KV_DEV_ERR_PAGE_RANGE);
                    good |= here && in ? 1 << j : 0;
                }
                if (lane < cnt) {
                    const int i = gs + base + lane, s = i % C::kNS;
                    if (i >= C::kNS && !mbar_wait_bounded(empty_bar + 8 * s, ((i / C::kNS) - 1) & 1, kWaitLimitNs)) {
                        raise_err(p.err, KV_DEV_ERR_TIMEOUT);
                        ok = false;
                    } else {
                        stage_pages[s] = good;
                        if (good)
                            mbar_arrive_expect_tx(full_bar + 8 * s,
                                                  __popc(good) * (2 * C::kBoxes * C::kUnitB + C::kScaleB));
                        else
                            mbar_arrive(full_bar + 8 * s);
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if constexpr (kI8) {  // one page per unit
                    const int st = lane / kUPS, j = lane % kUPS;
                    const int g_st = __shfl_sync(0xffffffffu, good, st & 31);
                    const int pg = __shfl_sync(0xffffffffu, tab, ((base + st) * kUPS + j) & 31);
                    if (st < cnt && ((g_st >> j) & 1)) {
                        const int s = (gs + base + st) % C::kNS;
                        bulk_g2s(sbase + C::kOffScales + (s * kUPS + j) * C::kScaleB,
                                 p.kv_scales + ((int64_t)pg * p.H_kv + pc.kvh) * (2 * P), C::kScaleB, full_bar + 8 * s);
                    }
                }
                const int st = lane / kBPS, bx = lane % kBPS;
                const int j = bx / (2 * C::kBoxes);  // unit of the stage
                const bool is_v = ((bx / C::kBoxes) & 1) != 0;
                const int bb = bx % C::kBoxes;       // box of the token row
                const int u = (base + st) * kUPS + j;
                const int g_st = __shfl_sync(0xffffffffu, good, st & 31);
                const int pg = __shfl_sync(0xffffffffu, tab, (u / C::kUPP) & 31);
                if (st < cnt && ((g_st >> j) & 1)) {
                    const int s = (gs + base + st) % C::kNS;
                    const uint32_t dst = sbase + s * C::kStage + (is_v ? C::kChunk : 0) + bb * C::kBoxB + j * C::kUnitB;
                    tma_load_2d(dst, is_v ? static_cast<const void*>(&tmap_v) : static_cast<const void*>(&tmap_k),
                                bb * C::kBoxElems, (pg * p.H_kv + pc.kvh) * P + u % C::kUPP * C::kU, full_bar + 8 * s);
                }
                issued = gs + base + cnt;
            }
            gs += n_st;
        }
        if (balanced && !p.cuts_by_row && lane == 0) {
            // the row that holds this CTA's last position: does it start here (its first real page, that is) and run on?
            int4 cut = make_int4(-1, 0, 0, 0);
            const int pos0 = walk.start, last = walk.end - 1;
            int b = walk.b;  // the walk ended in or before that row's sequence
            while (pre[b + 1] * p.H_kv <= last) ++b;
            const int D = pre[b + 1] - pre[b], kvh = (last - pre[b] * p.H_kv) / D, start = pre[b] * p.H_kv + kvh * D;
            if (walk.end < start + D && walk.end > start + v && pos0 <= start + v) {
                const int64_t after = static_cast<int64_t>(start) + D;  // the CTA of position after - 1 has the last piece
                cut = make_int4(b, kvh, static_cast<int>((after * G - 1) / T) - static_cast<int>(blockIdx.x) + 1,
                                blockIdx.x);
            }
            p.cuts[blockIdx.x] = cut;
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
    const int wp = cw / p.HS;   // page-warp: every WP-th stage
    if (wp >= p.WP) return;     // three slices: one warp has no part
    const int r0 = lane >> 2, quad = lane & 3;
    const int heads = min(NT * 8, p.g - hs * NT * 8);  // heads of this slice
    const uint32_t bar_written = 1 + 2 * hs, bar_free = 2 + 2 * hs;  // named barriers of the slice's warps
    // fragments of page-warps 1 .. WP - 1 of this slice: [warp][register][lane]
    constexpr int kLanes = DUP ? 16 : 32;
    float* merge = reinterpret_cast<float*>(smem + C::kOffMerge) + hs * (p.WP - 1) * (C::kMergeWarp / 4);
    const int mlane = DUP ? r0 * 2 + (quad & 1) : lane;
    bool ok = true;
    for (int piece = 0; walk.next(pc); ++piece) {
    if (piece > 0 && wp == 0 && p.WP > 1) named_bar_arrive(bar_free, 32 * p.WP);  // the last piece's fragments are read
    const int n_st = (pc.tokens(P) + kTP - 1) / kTP;
    const int b = pc.b, kvh = pc.kvh, len = pc.len;
    const int head0 = kvh * p.g + hs * NT * 8;
    const int tok0 = pc.page0 * P;  // first token of the piece
    // Q^T as the B operand: column lane / 4 of column tile nt is head nt * 8 + lane / 4 (DUP: 4 heads twice).
    constexpr int kQR = kI8 ? DH / 32 * 2 * 3 : kKS * 2;  // registers of a column tile
    uint32_t qb[NT][kQR];
    float q_pow[NT][2];  // int8: what a row was scaled by, for the lane's score columns, times the softmax scale
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int n = nt * 8 + r0;
        const int h = DUP ? n & 3 : n;
        const uint32_t* q32 = static_cast<const uint32_t*>(p.q) + (((int64_t)b * p.H_q + head0 + h) * DH >> 1);
        if constexpr (kI8) {
            // The products with codes are exact integers: a row is scaled by a power of two that brings its largest
            // magnitude to [2^21, 2^22), rounded to an integer (2^-23 of the largest at most) and split into three signed
            // bytes, one MMA operand each. The lane holds dims quad*Dh/4 + 8*kk .. +7 of k-step kk, as its K words do.
            float x[DH / 4];
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < DH / 8; ++i) {
                const float2 v = unpack16<QT == KV_DTYPE_BF16>(h < heads ? q32[(quad * (DH / 4) >> 1) + i] : 0u);
                x[2 * i] = v.x, x[2 * i + 1] = v.y;
                top = max(top, max(__float_as_uint(v.x) & 0x7fffffffu, __float_as_uint(v.y) & 0x7fffffffu));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = max(static_cast<int>(top >> 23) - 127, -100);  // floor(log2(largest)); 128: inf or NaN
            const float up = __int_as_float((21 - ex + 127) << 23);
            const float pow = ex == 128 ? __int_as_float(0x7fc00000) : __int_as_float((ex - 21 + 127) << 23);
#pragma unroll
            for (int i = 0; i < DH / 16; ++i) {
                uint32_t d[3] = {0u, 0u, 0u};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int q = __float2int_rn(x[4 * i + j] * up);
                    const int lo = static_cast<int8_t>(q), q1 = (q - lo) >> 8;
                    const int mid = static_cast<int8_t>(q1), hi = (q1 - mid) >> 8;
                    d[0] |= static_cast<uint32_t>(hi & 0xff) << (8 * j);
                    d[1] |= static_cast<uint32_t>(mid & 0xff) << (8 * j);
                    d[2] |= static_cast<uint32_t>(lo & 0xff) << (8 * j);
                }
#pragma unroll
                for (int k = 0; k < 3; ++k) qb[nt][k * (DH / 16) + i] = d[k];
            }
            // score columns of this lane: 2 quad, 2 quad + 1 (rows of lanes 8 quad, 8 quad + 4 above)
            q_pow[nt][0] = __shfl_sync(0xffffffffu, pow, 8 * quad) * p.scale_log2;
            q_pow[nt][1] = __shfl_sync(0xffffffffu, pow, 8 * quad + 4) * p.scale_log2;
        } else {
            // k-step kk covers dims kk*16 .. +15
#pragma unroll
            for (int kk = 0; kk < kKS; ++kk)
#pragma unroll
                for (int ch = 0; ch < 2; ++ch)
                    qb[nt][kk * 2 + ch] = h < heads ? q32[(kk * 16 + ch * 8 + 2 * quad) >> 1] : 0u;
        }
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

    {
        const int mi = lane >> 3, r8 = lane & 7;  // ldmatrix: matrix and row this lane addresses
        for (int i = (wp + p.WP - gs % p.WP) % p.WP; i < n_st; i += p.WP) {
            const int gi = gs + i, s = gi % C::kNS;
            // The ring is not a multiple of the page-warps, so another warp may have the stage's previous use and copies
            // may land out of order: that use is waited for first (its release), or the parity of the fill could
            // still be that of two uses ago. The use before it is long released: the producer issues in order and has
            // issued stage gi - WP of this warp, hence seen the release of gi - WP - kNS >= gi - 2 kNS.
            if (ok && ((gi >= C::kNS && !mbar_wait_bounded(empty_bar + 8 * s, (gi / C::kNS - 1) & 1, kWaitLimitNs)) ||
                       !mbar_wait_bounded(full_bar + 8 * s, (gi / C::kNS) & 1, kWaitLimitNs))) {
                raise_err(p.err, KV_DEV_ERR_TIMEOUT);
                ok = false;  // no stage of this or a later piece any more; the barriers between warps go on
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const int pages = stage_pages[s];
            const uint32_t sK = sbase + s * C::kStage, sV = sK + C::kChunk;
            const uint32_t sS = sbase + C::kOffScales + s * (kUPS * C::kScaleB);
            const int kbase = tok0 + i * kTP;
            // visible tokens of the stage: [tlo, thi), on pages that were loaded (the same for every head)
            const int thi = min(tok0 + pc.n * P, len) - kbase;
            const int tlo = MOD ? pc.key_begin - kbase : 0;
            const bool whole = tlo <= 0 && thi >= kTP && pages == (1 << kUPS) - 1;

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
                    for (int nt = 0; nt < NT; ++nt) {
                        int acc[3][4] = {};
#pragma unroll
                        for (int kk = 0; kk < DH / 32; ++kk) {
                            const uint32_t a[4] = {w[0][2 * kk], w[1][2 * kk], w[0][2 * kk + 1], w[1][2 * kk + 1]};
#pragma unroll
                            for (int k = 0; k < 3; ++k)
                                mma_16832_s8(acc[k], a, qb[nt][k * (DH / 16) + 2 * kk], qb[nt][k * (DH / 16) + 2 * kk + 1]);
                        }
                        // |hi|, |mid| sums are at most 2^21: 256 hi + mid is an exact int
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            sc[nt][mt][e] = fmaf(static_cast<float>(acc[0][e] * 256 + acc[1][e]), 256.f, static_cast<float>(acc[2][e]));
                    }
                } else {
#pragma unroll
                    for (int kk = 0; kk < kKS; ++kk) {
                        const int c = kk * 2 + (mi >> 1), t = mt * 16 + (mi & 1) * 8 + r8;
                        uint32_t a[4];
                        ldsm_x4(sK + (c >> 3) * C::kBoxB + swz<128>(t, c), a[0], a[1], a[2], a[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_16816<kQBF16>(sc[nt][mt], a, qb[nt][kk * 2], qb[nt][kk * 2 + 1]);
                    }
                }
            }

            // ---- scores in log2 units, masked; has any moved above the reference by more than 2^8?
            float vs[kMT][2];  // int8: V scales of tokens r0, r0 + 8
            bool grow = false;
            if constexpr (MOD) modify_cols<NT, kMT>(p, cap_coefs(p), sc, slope, len - 1 - kbase - r0);
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
                    const bool seen = whole || (t >= tlo && t < thi && ((pages >> (mt * 16 / C::kU)) & 1));
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
            uint32_t ph[NT][kMT][2], pl[NT][kMT][2], pr[NT][kMT][2];
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
                        if constexpr (kThird) {
                            const uint32_t rest = pack2<true>(pv[0] - __uint_as_float(hi << 16) - __uint_as_float(lo << 16),
                                                              pv[1] - __uint_as_float(hi & 0xffff0000u) -
                                                                  __uint_as_float(lo & 0xffff0000u));
                            pr[nt][mt][h] = movmatrix_trans(DUP && quad >= 2 ? 0u : rest);
                        }
                    }

            // ---- V rows that no head sees may hold NaN (int8 codes cannot): zero them
            if constexpr (!kI8) {
                if (!whole) {
                    constexpr int kCPR = 8;  // 16-byte chunks per box row
                    for (int idx = lane; idx < kTP * C::kBoxes * kCPR; idx += 32) {
                        const int t = idx / (C::kBoxes * kCPR), rem = idx % (C::kBoxes * kCPR);
                        if (t < tlo || t >= thi || !((pages >> (t / C::kU)) & 1))
                            sts128_zero(sV + (rem / kCPR) * C::kBoxB + t * 128 + ((rem % kCPR) << 4));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
            }

            // ---- O^T += V^T P^T: sixteen tokens a product, added to fp32 sums. (Sums kept in the MMA's accumulator,
            // which rounds towards zero, cost the same time and grow less exact with the length: score_mod.cuh.)
            auto add_pv = [&](float(&sum)[4], const uint32_t(&a)[4], const uint32_t(&hi)[2], const uint32_t(&lo)[2],
                              const uint32_t(&rest)[2]) {
                float d[4] = {};
                if constexpr (kThird) mma_16816<true>(d, a, rest[0], rest[1]);
                if constexpr (!DUP) mma_16816<kPBF16>(d, a, lo[0], lo[1]);
                mma_16816<kPBF16>(d, a, hi[0], hi[1]);
                const float2 x = fadd2(make_float2(sum[0], sum[1]), make_float2(d[0], d[1]));
                const float2 y = fadd2(make_float2(sum[2], sum[3]), make_float2(d[2], d[3]));
                sum[0] = x.x, sum[1] = x.y, sum[2] = y.x, sum[3] = y.y;
            };
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
                            for (int nt = 0; nt < NT; ++nt)
                                add_pv(o[nt][2 * m + hh], a, ph[nt][ks], pl[nt][ks], pr[nt][ks]);
                        }
                } else {
#pragma unroll
                    for (int m = 0; m < kOM; ++m) {
                        const int c = m * 2 + (mi & 1), t = ks * 16 + (mi >> 1) * 8 + r8;
                        uint32_t a[4];
                        ldsm_x4_trans(sV + (c >> 3) * C::kBoxB + swz<128>(t, c), a[0], a[1], a[2], a[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) add_pv(o[nt][m], a, ph[nt][ks], pl[nt][ks], pr[nt][ks]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty_bar + 8 * s);
        }
    }

    gs += n_st;

    // ---- column sums over the lanes of a head; the slice's page-warps meet in the first of them
    float m_col[NT][2], l_col[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float l = l_part[nt][e];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
            l_col[nt][e] = l;
            // a NaN sum keeps its place in the merge whatever the column's maximum is
            m_col[nt][e] = l != l && m_ref[nt][e] == -INFINITY ? 0.f : m_ref[nt][e];
            if constexpr (DUP) {  // values and residuals of a head
#pragma unroll
                for (int m = 0; m < kOM; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        o[nt][m][2 * h + e] += __shfl_xor_sync(0xffffffffu, o[nt][m][2 * h + e], 2);
            }
        }
    if (wp > 0) {
        if (piece > 0) named_bar_sync(bar_free, 32 * p.WP);
        float* dst = merge + (wp - 1) * (C::kMergeWarp / 4) + mlane;
        if (!DUP || quad < 2) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int m = 0; m < kOM; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) dst[((nt * kOM + m) * 4 + e) * kLanes] = o[nt][m][e];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    dst[(NT * kOM * 4 + nt * 4 + e) * kLanes] = m_col[nt][e];
                    dst[(NT * kOM * 4 + nt * 4 + 2 + e) * kLanes] = l_col[nt][e];
                }
            }
        }
        named_bar_arrive(bar_written, 32 * p.WP);
        continue;
    }
    if (p.WP > 1) named_bar_sync(bar_written, 32 * p.WP);
    for (int w = 0; w < p.WP - 1; ++w) {
        const float* src = merge + w * (C::kMergeWarp / 4) + mlane;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float mw = src[(NT * kOM * 4 + nt * 4 + e) * kLanes];
                const float lw = src[(NT * kOM * 4 + nt * 4 + 2 + e) * kLanes];
                if (mw == -INFINITY) continue;
                const float mn = fmaxf(m_col[nt][e], mw);
                const float sa = m_col[nt][e] == -INFINITY ? 0.f : exp2f(m_col[nt][e] - mn), sb = exp2f(mw - mn);
                m_col[nt][e] = mn;
                l_col[nt][e] = l_col[nt][e] * sa + lw * sb;
#pragma unroll
                for (int m = 0; m < kOM; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        o[nt][m][2 * h + e] = o[nt][m][2 * h + e] * sa + src[((nt * kOM + m) * 4 + 2 * h + e) * kLanes] * sb;
            }
    }
    bool nan = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int n = nt * 8 + 2 * quad + e;
            if (n >= heads) continue;
            const int64_t hq = (int64_t)b * p.H_q + head0 + n;
            const bool whole = pc.slot < 0;
            const int64_t ps = balanced ? (int64_t)pc.slot * p.g + hs * NT * 8 + n : hq * p.num_splits + blockIdx.x;
            float* dst = whole ? p.out + hq * DH : p.part_u + ps * DH;
            const float L = l_col[nt][e], scale = whole ? (L != 0.f ? 1.f / L : 0.f) : 1.f;
#pragma unroll
            for (int m = 0; m < kOM; ++m) {
                float x[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    x[h] = o[nt][m][2 * h + e];
                    if constexpr (MOD) nan |= x[h] != x[h];
                    x[h] = whole && L == 0.f ? 0.f : x[h] * scale;
                }
                if constexpr (kI8) {
                    *reinterpret_cast<float2*>(dst + r0 * (DH / 8) + 2 * m) = make_float2(x[0], x[1]);
                } else {
                    dst[m * 16 + r0] = x[0];
                    dst[m * 16 + 8 + r0] = x[1];
                }
            }
            if (!whole && r0 == 0) p.part_ml[ps] = make_float2(m_col[nt][e], L);
        }
    if constexpr (MOD) {
        // An infinity among the visible values meets a probability's residual, which may be 0 or negative: a NaN. Where a
        // sum is NaN and the weights are not (rare), the values say what it is. (After the stores, so that the sums need
        // no registers beside the search.)
        if (__any_sync(0xffffffffu, nan)) {
#pragma unroll 1
            for (int m = 0; m < kOM; ++m) {
                float x[16], f[2] = {0.f, 0.f};
                sum_nonfinite16<kPBF16>(p, b, kvh, P, DH, m * 16, max(pc.key_begin, tok0), min(len, tok0 + pc.n * P), x);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i == r0) f[0] = x[i], f[1] = x[8 + i];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int n = nt * 8 + 2 * quad + e;
                        const float L = l_col[nt][e];
                        if (n >= heads || !(L > 0.f)) continue;
                        const bool whole = pc.slot < 0;
                        const int64_t hq = (int64_t)b * p.H_q + head0 + n;
                        const int64_t ps = balanced ? (int64_t)pc.slot * p.g + hs * NT * 8 + n : hq * p.num_splits + blockIdx.x;
                        float* dst = whole ? p.out + hq * DH : p.part_u + ps * DH;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float& y = dst[m * 16 + h * 8 + r0];
                            if (y != y && f[h] != 0.f) y = whole ? f[h] / L : f[h];  // (0: finite values whose sum left fp32)
                        }
                    }
            }
        }
    }
    }
}

// Merges the rows that a balanced launch cut, one CTA per entry of `cuts` (sequence, KV head, pieces, first CTA c): a
// row's pieces are in slots 2c + 1, 2 (c + 1), 2 (c + 2), ... (No pointer is __restrict__: the decode kernel before may still
// be writing these buffers when this one starts, so they must be read by ordinary loads behind the wait.) Latency-bound: the
// warps share out the heads of the row's group and, with fewer heads than warps, a head's pieces (a long row of a small
// batch is cut into dozens); a lane sums Dh / 32 dims with the loads of a round of pieces issued before any is used,
// relative to its warp's own maximum, and the warps of a head meet in shared memory. The host gives it few warps where
// rows have few pieces (large CTAs are slow to start) and kCombineColsWarps where they have many.
constexpr int kCombineColsWarps = 16;
template <int DH>
__global__ void __launch_bounds__(32 * kCombineColsWarps) paged_combine_cols_kernel(
    float* out, const float* part_u, const float2* part_ml, const int4* cuts, int32_t H_q, int32_t g) {
    constexpr int kD = DH / 32, kRound = 8;
    __shared__ float red_u[kCombineColsWarps][DH], red_m[kCombineColsWarps], red_l[kCombineColsWarps];
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 cut = cuts[blockIdx.x];
    if (cut.x < 0) return;
    const int ns = cut.z, c = cut.w;
    const int warps = blockDim.x >> 5, wph = max(1, warps / g);  // warps per head
    auto slot = [&](int s) -> int64_t { return s == 0 ? 2LL * c + 1 : 2LL * (c + s); };
    for (int h0 = 0; h0 < g; h0 += warps) {  // one round unless the group has more heads than warps
        const int h = h0 + warp / wph, part = warp % wph;
        float m = -INFINITY, L = 0.f, acc[kD] = {};
        if (h < g) {
            for (int s0 = part; s0 < ns; s0 += wph * kRound) {
                float2 ml[kRound];
                float x[kRound][kD];
#pragma unroll
                for (int j = 0; j < kRound; ++j) {
                    ml[j] = make_float2(-INFINITY, 0.f);
                    if (s0 + j * wph >= ns) continue;
                    const int64_t ps = slot(s0 + j * wph) * g + h;
                    ml[j] = part_ml[ps];
                    const float* src = part_u + ps * DH + lane * kD;
                    if constexpr (kD == 4) {
                        const float4 t = *reinterpret_cast<const float4*>(src);
                        x[j][0] = t.x, x[j][1] = t.y, x[j][2] = t.z, x[j][3] = t.w;
                    } else {
                        const float2 t = *reinterpret_cast<const float2*>(src);
                        x[j][0] = t.x, x[j][1] = t.y;
                    }
                }
                float mr = m;
#pragma unroll
                for (int j = 0; j < kRound; ++j) mr = fmaxf(mr, ml[j].x);
                if (mr == -INFINITY) continue;
                const float a = m == -INFINITY ? 0.f : merge_weight(m - mr);
                m = mr;
                L *= a;
#pragma unroll
                for (int i = 0; i < kD; ++i) acc[i] *= a;
#pragma unroll
                for (int j = 0; j < kRound; ++j) {
                    if (ml[j].x == -INFINITY) continue;
                    const float w = merge_weight(ml[j].x - m);
                    L += w * ml[j].y;
#pragma unroll
                    for (int i = 0; i < kD; ++i) acc[i] += w * x[j][i];
                }
            }
        }
        if (wph > 1) {
#pragma unroll
            for (int i = 0; i < kD; ++i) red_u[warp][lane * kD + i] = acc[i];
            if (lane == 0) red_m[warp] = m, red_l[warp] = L;
            __syncthreads();
            if (h < g && part == 0) {
                float ms = m;
                for (int w = 1; w < wph; ++w) ms = fmaxf(ms, red_m[warp + w]);
                const float a = m == -INFINITY ? 0.f : merge_weight(m - ms);
                L *= a;
#pragma unroll
                for (int i = 0; i < kD; ++i) acc[i] *= a;
                for (int w = 1; w < wph; ++w) {
                    if (red_m[warp + w] == -INFINITY) continue;
                    const float sw = merge_weight(red_m[warp + w] - ms);
                    L += sw * red_l[warp + w];
#pragma unroll
                    for (int i = 0; i < kD; ++i) acc[i] += sw * red_u[warp + w][lane * kD + i];
                }
            }
        }
        if (h < g && part == 0) {
            const float inv = L != 0.f ? 1.f / L : 0.f;
            float* dst = out + ((int64_t)cut.x * H_q + (int64_t)cut.y * g + h) * DH + lane * kD;
#pragma unroll
            for (int i = 0; i < kD; ++i) dst[i] = L != 0.f ? acc[i] * inv : 0.f;
        }
    }
}

// ---- dispatch ---------------------------------------------------------------
template <int KT, int QT, int DH, int P, int NT, bool DUP, bool MOD>
cudaError_t launch_cols_inst(DecodeParams p, const CUtensorMap& tk, const CUtensorMap& tv, dim3 grid, cudaStream_t st) {
    using C = ColsCfg<KT, DH, P, NT, DUP>;
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
