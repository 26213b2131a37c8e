// Multi-token query (chunked prefill) with modified scores and masks over the
// paged cache on the fifth-generation tensor cores (tcgen05), sm_100a: the
// kernel of paged_prefill_attention_mod for Dh = 128.
//
// The function is score_mod.cuh's: row i of sequence b's chunk, at position
// p_i = seq_lens[b] - n_b + i, sees the keys [lo, hi) of its window, document and
// prefix, with scores capped by a tanh and biased by distance. Tile, staging
// and MMAs are those of prefill_tc.cuh (128 rows = 128 / g chunk tokens x g
// heads; stages of 128 keys, S triple-buffered and O in tensor memory, P
// written over its S columns as a 16-bit value plus residual, two threads per
// row), with these differences:
//   - The stages run from the one that holds the first key any row of the tile
//     sees to the last; stages before a window or document are never loaded.
//   - A thread writes P over the S columns that it read itself, so that the two
//     threads of a row meet only to move the row's reference maximum: they vote
//     in one barrier whether any row has to, and exchange maxima only then.
//     (prefill_cap_tc.cuh serves bf16 under a cap of at most 50 without a bias:
//     no reference to move there.)
//   - value and residual are rounded, not truncated (pack2_split_near), and O is moved into fp32
//     sums in registers every kFlushKeys keys: against 64 bits the error is 5e-6
//     of the result at any length (1.1e-5 at 4096 keys, 7.5e-5 at 32K without).
//   - A stage that some rows see only in part ("boundary") has its V rows
//     searched for NaN and infinity, which a probability of 0 would not keep
//     from the rows that do not see them: found elements are zeroed in shared
//     memory, and the epilogue of such a tile adds them, read again from the
//     pool, to the rows that do.
// Measured, 32 heads on 8, 8 chunks of 512 tokens over 4096, back to back: bf16
// without a cap 555 us (217 under a window of 1024), with slopes 657; fp16 under
// a cap of 50 629, and 1770 where many scores pass a fifth of it (scalar forms of
// the tanh). Bound by the chain of a stage, as prefill_cap_tc.cuh, and a tile's
// start and end.
// Every wait is bounded (KV_DEV_ERR_TIMEOUT); block-table entries outside
// [0, num_pages) are never loaded (their keys are masked,
// KV_DEV_ERR_PAGE_RANGE).
#pragma once

#include <cuda.h>

#include <atomic>

#include "decode_kernel.cuh"
#include "decode_launch.cuh"
#include "score_mod.cuh"
#include "tc05.cuh"

namespace kvp {

template <int DH, int P>
struct PfModCfg {
    static constexpr int kTP = 128;              // keys per stage
    static constexpr int kPPS = kTP / P;         // pages per stage
    static constexpr int kBoxCols = DH / 64;
    static constexpr int kBoxB = kTP * 128;      // one 128-byte box column of an entry
    static constexpr int kEntry = kBoxCols * kBoxB;
    // entries 0..2 hold K of stages j % 3, entries 3..4 V of stages j % 2: a K entry is refilled as soon
    // as its QK has run, independently of the P.V of older stages
    static constexpr int kKSlots = 3, kVSlots = 2;
    static constexpr int kRing = kKSlots + kVSlots;
    static constexpr int kQB = 128 * DH * 2;     // Q tile: 128 rows
    static constexpr int kOffQ = kRing * kEntry;
    static constexpr int kParts = 2;             // threads per row: each with half of a stage's keys and of the dims
    static constexpr int kOffX = kOffQ + kQB;    // row exchange: [2][kParts][128] floats + ints
    static constexpr int kOffBar = kOffX + 2 * kParts * 128 * 4 * 2;
    // full[R], empty[R], q_full, s_full[3], p_full[3], p_empty[3], o_full, done (QK), done (PV)
    static constexpr int kNumBars = 2 * kRing + 1 + 3 + 3 + 3 + 3;
    static constexpr int kOffTmem = kOffBar + 8 * kNumBars;
    static constexpr int kOffDirty = kOffTmem + 8;  // a boundary stage held a NaN or an infinity in V
    static constexpr int kSmem = 1024 + kOffTmem + 16;
    static constexpr int kThreads = 128 + 128 * kParts;
    static constexpr int kVWarp = 2;             // the V producer (warp 0 produces K)
    static constexpr int kPVWarp = 3;            // issues P.V (warp 1 issues QK)
    static constexpr int kFirstSoftmaxWarp = 4;
    // registers per thread after the split: warpgroup 0 (producers, issuers) and the two softmax warpgroups;
    // 128 x kRegsLow + 256 x kRegsHigh must not exceed the launch's 384 x (registers per thread), which the
    // host checks before the first launch
    static constexpr uint32_t kRegsLow = 64, kRegsHigh = 216;
    static constexpr int kSoftmaxWarps = 4 * kParts;
    static constexpr uint32_t kTmemCols = 512;   // S x 3 (384) + O (128)
    static_assert(DH == 128, "instance: Dh = 128");
    static_assert(kPPS * kBoxCols <= 32, "one TMA box per lane");
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

// Bits 0 .. n - 1 of 64 (none for n <= 0, all for n >= 64).
__device__ __forceinline__ uint64_t bits_below(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

template <int KT, int DH, int P>
__global__ void __launch_bounds__(384, 1)
    paged_prefill_mod_tc_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ CUtensorMap tmap_k,
                            const __grid_constant__ CUtensorMap tmap_v) {
    using C = PfModCfg<DH, P>;
    constexpr bool kBF16 = KT == KV_DTYPE_BF16;
    constexpr int kParts = C::kParts;
    constexpr uint32_t kIdescQK = idesc_f16(kBF16, 128, C::kTP, false, false);
    constexpr uint32_t kIdescPV = idesc_f16(kBF16, 128, DH, false, true);
    constexpr int kFlush = kFlushKeys / C::kTP;  // stages whose P.V share one accumulation
    extern __shared__ __align__(1024) unsigned char smem_raw[];

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
    }
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_launch_dependents();

    // ---- this CTA's tile: chunk tokens t0 .. t0 + nt - 1 of sequence b, KV head kvh
    const ChunkTile ct = chunk_tile(p, (gridDim.x - 1 - blockIdx.x) / p.H_kv, lane);
    const int kvh = blockIdx.x % p.H_kv, b = ct.b;
    const int g = p.g;
    const int qs0 = ct.qs0, n_q = ct.n_q, t0 = ct.t0;
    const int nt = ct.nt;
    if (nt <= 0) return;
    int len = p.seq_lens[b];
    auto zero_tile = [&]() {
        for (int e = threadIdx.x; e < nt * g * DH; e += blockDim.x) {
            const int rr = e / DH;
            p.out[((int64_t)(qs0 + t0 + rr / g) * p.H_q + (int64_t)kvh * g + rr % g) * DH + e % DH] = 0.f;
        }
    };
    if (len < 0 || len > p.max_blocks * P || n_q > len) {
        if (threadIdx.x == 0 && t0 == 0 && kvh == 0) raise_err(p.err, KV_DEV_ERR_SEQ_LEN);
        zero_tile();
        return;
    }
    const int pos0 = len - n_q + t0;          // position of the tile's first token
    // some row sees keys in [key_begin, key_end) only; all rows see every key of [key_all0, key_all1)
    const int prefix = p.prefix_lens != nullptr ? min(p.prefix_lens[b], len) : 0;
    const TileKeys tk = tile_keys(p, qs0 + t0, pos0, nt, prefix, lane);
    const int key_begin = tk.begin, key_end = tk.end, key_all0 = tk.all0, key_all1 = tk.all1;
    if (key_begin >= key_end) {  // no row sees any key
        zero_tile();
        return;
    }
    // stages, pages and keys are counted from the first stage with a visible key
    const int key_first = key_begin / C::kTP * C::kTP;
    const int page_first = key_first / P;
    const int n_pages = (key_end + P - 1) / P - page_first;
    const int n_st = (key_end - key_first + C::kTP - 1) / C::kTP;

    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    unsigned char* smem = smem_raw + (sbase - raw);
    const uint32_t bar0 = sbase + C::kOffBar;
    auto full = [&](int e) { return bar0 + 8u * e; };
    auto empty = [&](int e) { return bar0 + 8u * (C::kRing + e); };
    auto kslot = [](int j) { return j % C::kKSlots; };
    auto vslot = [](int j) { return C::kKSlots + j % C::kVSlots; };
    auto kphase = [](int j) { return static_cast<uint32_t>((j / C::kKSlots) & 1); };
    auto vphase = [](int j) { return static_cast<uint32_t>((j / C::kVSlots) & 1); };
    const uint32_t q_full = bar0 + 8u * (2 * C::kRing);
    auto s_full = [&](int i) { return q_full + 8u + 8u * i; };
    // P of stage j is announced on p_full(j % 3) by all eight softmax warps. The warps of different lane
    // quarters do not wait for one another, and none waits for V, so one may arrive for stage j + 2 while
    // another is still writing P(j): with two barriers that early arrival would complete stage j's phase.
    // Stage j + 3 needs S(j + 3), hence QK(j + 3), hence P.V(j) done, hence every stage-j arrival: three
    // barriers keep each phase's arrivals to its own stage.
    auto p_full = [&](int i) { return q_full + 32u + 8u * i; };
    // P.V(j) completion is announced on p_empty(j % 3), the barrier of the S columns it read
    auto p_empty = [&](int i) { return q_full + 56u + 8u * i; };
    const uint32_t o_full = q_full + 80;
    const uint32_t done_qk = q_full + 88;
    const uint32_t done_pv = q_full + 96;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::kOffTmem);

    if (threadIdx.x == 0) {
        for (int e = 0; e < C::kRing; ++e) {
            mbar_init(full(e), 1);
            mbar_init(empty(e), 1);
        }
        mbar_init(q_full, C::kSoftmaxWarps);
        for (int i = 0; i < 3; ++i) mbar_init(s_full(i), 1);
        for (int i = 0; i < 3; ++i) mbar_init(p_full(i), C::kSoftmaxWarps);
        for (int i = 0; i < 3; ++i) mbar_init(p_empty(i), 1);
        mbar_init(o_full, 1);
        mbar_init(done_qk, 1);
        mbar_init(done_pv, 1);
        *reinterpret_cast<volatile int*>(smem + C::kOffDirty) = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tO = tmem + 3 * C::kTP;
    const uint32_t ring = sbase;
    const uint32_t sQ = sbase + C::kOffQ;

    // the register split sits at the top of each warpgroup's branch, so every code path after it is
    // compiled for its own budget
    if (warp < C::kFirstSoftmaxWarp) {
    regs_dec<C::kRegsLow>();
    if (warp == 0 || warp == C::kVWarp) {
        // ------------------------------------------------------------ producers
        // warp 0 issues the K boxes of every stage, warp kVWarp the V boxes: two streams of TMA requests
        const int half = warp == 0 ? 0 : 1;
        bool ok = true;
        int kfills = 0, vfills = 0;  // stages whose K / V boxes were issued
        const int32_t* row = p.block_tables + (int64_t)b * p.max_blocks + page_first;
        int tab_cur = lane < n_pages ? row[lane] : -1, tab_nxt = -1;
        // pages of the first stage that lie before the first key any row sees: not loaded, whatever their entries are
        const int skip = key_begin / P - page_first;
        for (int j = 0; j < n_st && ok; ++j) {
            const int np = min(C::kPPS, n_pages - j * C::kPPS);
            // block-table entries come 32 at a time, one per lane, the next 32 fetched while these are used
            // (stages never straddle a group: 32 is a multiple of the pages per stage)
            if (((j * C::kPPS) & 31) == 0) {
                const int base = j * C::kPPS;
                tab_cur = base == 0 ? tab_cur : tab_nxt;
                tab_nxt = (base + 32 + lane < n_pages) ? row[base + 32 + lane] : -1;
            }
            const int pg_all = __shfl_sync(0xffffffffu, tab_cur, (j * C::kPPS + lane) & 31);
            const bool wanted = lane < np && j * C::kPPS + lane >= skip;
            const int pg = wanted ? pg_all : -1;
            const bool good = wanted && pg >= 0 && pg < p.num_pages;
            if (wanted && !good) raise_err(p.err, KV_DEV_ERR_PAGE_RANGE);
            const unsigned gmask = __ballot_sync(0xffffffffu, good);
            const int box_page = lane / C::kBoxCols, bb = lane % C::kBoxCols;
            const int pgl = __shfl_sync(0xffffffffu, pg, box_page & 31);
            {
                const int e = half ? vslot(j) : kslot(j);
                const int use = half ? j / C::kVSlots : j / C::kKSlots;  // earlier fills of this entry
                if (lane == 0) {
                    if (use > 0 && !mbar_wait_bounded(empty(e), (use - 1) & 1, kWaitLimitNs)) {
                        raise_err(p.err, KV_DEV_ERR_TIMEOUT);
                        ok = false;
                    } else {
                        mbar_arrive_expect_tx(full(e), __popc(gmask) * C::kBoxCols * P * 128);
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                if (box_page < np && ((gmask >> box_page) & 1u)) {
                    const uint32_t dst = ring + e * C::kEntry + bb * C::kBoxB + box_page * P * 128;
                    tma_load_2d(dst, half ? static_cast<const void*>(&tmap_v) : static_cast<const void*>(&tmap_k),
                                bb * 64, (pgl * p.H_kv + kvh) * P, full(e));
                }
                if (half) vfills = j + 1;
                else kfills = j + 1;
            }
        }
        if (lane == 0) {  // the last fill of every entry has landed before the CTA exits
            if (half == 0) {
                for (int j = max(0, kfills - C::kKSlots); j < kfills; ++j)
                    if (!mbar_wait_bounded(full(kslot(j)), kphase(j), kWaitLimitNs))
                        raise_err(p.err, KV_DEV_ERR_TIMEOUT);
            } else {
                for (int j = max(0, vfills - C::kVSlots); j < vfills; ++j)
                    if (!mbar_wait_bounded(full(vslot(j)), vphase(j), kWaitLimitNs))
                        raise_err(p.err, KV_DEV_ERR_TIMEOUT);
            }
        }
    } else {
        // ------------------------------------------------------------ MMA issue
        // Warp 1 issues QK(j) once K(j) has landed and P.V(j - 3) has released S columns j % 3; the P.V
        // warp issues P.V(j) once the softmax has written P(j). Neither waits on the other's barriers.
        const bool qk = warp == 1;
        if (lane == 0) {
            bool ok = true;
            auto wait = [&](uint32_t bar, uint32_t parity) {
                if (ok && !mbar_wait_bounded(bar, parity, kWaitLimitNs)) {
                    raise_err(p.err, KV_DEV_ERR_TIMEOUT);
                    ok = false;
                }
                return ok;
            };
            if (qk) {
                if (wait(q_full, 0)) {
                    for (int j = 0; j < n_st; ++j) {
                        const int e = kslot(j);
                        if (!wait(full(e), kphase(j))) break;
                        if (j >= 3 && !wait(p_empty(j % 3), ((j - 3) / 3) & 1)) break;
                        tc_fence_after();
                        const uint32_t sK = ring + e * C::kEntry;
                        const uint32_t tS = tmem + (j % 3) * C::kTP;
#pragma unroll
                        for (int kk = 0; kk < DH / 16; ++kk) {
                            const uint32_t off = (kk >> 2) * C::kBoxB + (kk & 3) * 32;
                            umma_ss(tS, smem_desc(sQ + off, 16, 1024, kSwz128), smem_desc(sK + off, 16, 1024, kSwz128),
                                    kIdescQK, kk > 0 ? 1u : 0u);
                        }
                        umma_commit(s_full(j % 3));
                        umma_commit(empty(e));
                    }
                }
            } else {
                for (int j = 0; j < n_st; ++j) {
                    const int e = vslot(j);
                    if (!wait(full(e), vphase(j))) break;
                    if (!wait(p_full(j % 3), (j / 3) & 1)) break;
                    tc_fence_after();
                    const uint32_t sV = ring + e * C::kEntry;
                    const uint32_t tP = tmem + (j % 3) * C::kTP;
                    // each run of 64 keys, as one thread writes it over its own S columns: the values, then their residuals
                    constexpr int kRun = 64;
                    auto p_col = [](int kk) { return kk * 16 / kRun * kRun + kk * 16 % kRun / 2; };
#pragma unroll
                    for (int kk = 0; kk < C::kTP / 16; ++kk)
                        umma_ts(tO, tP + p_col(kk), smem_desc(sV + kk * 16 * 128, C::kBoxB, 1024, kSwz128), kIdescPV,
                                (j % kFlush != 0 || kk > 0) ? 1u : 0u);
#pragma unroll
                    for (int kk = 0; kk < C::kTP / 16; ++kk)
                        umma_ts(tO, tP + p_col(kk) + kRun / 2, smem_desc(sV + kk * 16 * 128, C::kBoxB, 1024, kSwz128),
                                kIdescPV, 1u);
                    umma_commit(empty(e));
                    umma_commit(p_empty(j % 3));
                }
                if (ok) umma_commit(o_full);
            }
            const uint32_t done = qk ? done_qk : done_pv;
            umma_commit(done);
            if (!mbar_wait_bounded(done, 0, kWaitLimitNs)) raise_err(p.err, KV_DEV_ERR_TIMEOUT);
        }
        __syncwarp();
    }
    } else {
        regs_inc<C::kRegsHigh>();
        // ------------------------------------------------------------ Q tile, softmax, epilogue
        const int quarter = warp & 3;
        const int part = (warp - C::kFirstSoftmaxWarp) >> 2;  // key columns [kH part, + kH) of S, dims of O likewise
        const int r = quarter * 32 + lane;   // MMA row: chunk token t0 + r / g, head kvh * g + r % g
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t row_bar = 1 + quarter;  // named barrier of the warps that share row r
        const int tr = r / g;
        const bool row_valid = tr < nt;
        const int pos = pos0 + tr;
        // this row sees keys row_lo .. row_hi - 1
        int row_lo = 0, row_hi = 0;
        float slope = 0.f;
        if (row_valid) {
            row_lo = first_key(p, qs0 + t0 + tr, pos);
            row_hi = max(pos + 1, prefix);
            if (p.alibi_slopes != nullptr) slope = p.alibi_slopes[kvh * g + r % g] * kLog2e;
        }
        const int64_t qrow = ((int64_t)(qs0 + t0 + tr) * p.H_q + (int64_t)kvh * g + r % g);
        float* xm = reinterpret_cast<float*>(smem + C::kOffX);  // [buf][part][row] maxima / sums
        int* xok = reinterpret_cast<int*>(smem + C::kOffX) + 2 * kParts * 128;
        int xbuf = 0;
        // Q row r -> the swizzled K-major tile, its sixteen 16-byte chunks shared out over the parts
        {
            const uint4* src = static_cast<const uint4*>(p.q) + qrow * (DH / 8);
            for (int c = part; c < DH / 8; c += kParts) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (row_valid) v = src[c];
                const uint32_t dst = sQ + (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z),
                             "r"(v.w)
                             : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        bool ok = true;
        // warp-uniform outcome: the tensor-memory loads and stores after a wait are warp-collective
        auto wait = [&](bool& okl, uint32_t bar, uint32_t parity) {
            if (okl && !mbar_wait_bounded(bar, parity, kWaitLimitNs)) {
                raise_err(p.err, KV_DEV_ERR_TIMEOUT);
                okl = false;
            }
            okl = __all_sync(0xffffffffu, okl);
            return okl;
        };
        // the parts of row r meet: every part's value in v; `okl` becomes the AND of all
        auto meet = [&](float mine, float (&v)[kParts], bool& okl) {
            xm[(xbuf * kParts + part) * 128 + r] = mine;
            xok[(xbuf * kParts + part) * 128 + r] = okl ? 1 : 0;
            named_bar_sync(row_bar, 32 * kParts);
            bool all = true;
#pragma unroll
            for (int k = 0; k < kParts; ++k) {
                v[k] = xm[(xbuf * kParts + k) * 128 + r];
                all = all && xok[(xbuf * kParts + k) * 128 + r] != 0;
            }
            okl = __all_sync(0xffffffffu, all);
            xbuf ^= 1;
        };
        const CapRowCoef coef = cap_row_coefs(p);
        float m_ref = -INFINITY, l = 0.f;
        constexpr int kH = C::kTP / kParts;  // keys per stage and dims of O per thread
        const int od = part * kH;                          // first of them
        // earlier accumulations of this thread's part of O, in units of the current reference
        float2 acc[kH / 2];
#pragma unroll
        for (int i = 0; i < kH / 2; ++i) acc[i] = make_float2(0.f, 0.f);
        // lanes 0 .. kPPS-1: the page ids of stage j, read one stage ahead; the mask of pages the producers
        // skip (entries outside the pool) is then known without waiting for the V entry
        const int32_t* trow = p.block_tables + (int64_t)b * p.max_blocks + page_first;
        int pg_cur = lane < C::kPPS && lane < n_pages ? __ldg(trow + lane) : -1;
        // A key no row may see (past the tile, or on a page not loaded) may hold stale bytes: zero its V row (this thread:
        // `n` 16-byte chunks of V row r from `chunk` on) once the V entry has landed. In a stage that some rows see only in
        // part a NaN or an infinity in V must not reach the others as 0 times it: those elements are zeroed too, and
        // noted. Only warps with such a row wait for the entry (the P.V issuer waits for every entry).
        auto clean_v = [&](int j, int kbase, int np, int bad, int chunk, int n, bool& okl) {
            const int pgi = r / P;
            const bool stale = kbase + r >= key_end || kbase + r < key_begin || pgi >= np || ((bad >> pgi) & 1);
            const bool boundary = kbase < key_all0 || kbase + C::kTP > key_all1;
            if (!__any_sync(0xffffffffu, stale) && !boundary) return;
            // the entry's previous fill (stage j - kVSlots) must have been consumed first: its P.V done means that
            // fill landed, so the wait below cannot pass on that older phase's parity
            const int ev = vslot(j), jp = j - C::kVSlots;
            if (jp >= 0 && !wait(okl, p_empty(jp % 3), (jp / 3) & 1)) return;
            if (!wait(okl, full(ev), vphase(j))) return;
            for (int c = chunk; c < chunk + n; ++c) {
                const uint32_t at = ring + ev * C::kEntry + (c >> 3) * C::kBoxB + r * 128 + (c & 7) * 16;
                if (stale) {
                    sts128_zero(at);
                } else if (boundary) {
                    const uint4 v = lds128(at);
                    if (has_nonfinite16<kBF16>(v)) {
                        *reinterpret_cast<volatile int*>(smem + C::kOffDirty) = 1;
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x ^ nonfinite16<kBF16>(v.x)),
                                     "r"(v.y ^ nonfinite16<kBF16>(v.y)), "r"(v.z ^ nonfinite16<kBF16>(v.z)),
                                     "r"(v.w ^ nonfinite16<kBF16>(v.w))
                                     : "memory");
                    }
                }
            }
        };
        for (int j = 0; j < n_st; ++j) {
            bool okl = ok;
            const uint32_t tS = tmem + (j % 3) * C::kTP + lane_addr;
            const int nxt = (j + 1) * C::kPPS + lane;
            const int pg_nxt = lane < C::kPPS && nxt < n_pages ? __ldg(trow + nxt) : -1;
            float s[kH];
            if (wait(okl, s_full(j % 3), (j / 3) & 1)) {
                tc_fence_after();
                uint32_t a[kH / 32][32];
#pragma unroll
                for (int q = 0; q < kH / 32; ++q) tmem_ld32(tS + part * kH + q * 32, a[q]);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < kH; ++i) s[i] = __uint_as_float(a[i / 32][i % 32]);
            }
            // keys of this stage: kbase .. kbase + 127
            const int kbase = key_first + j * C::kTP;
            const int np = min(C::kPPS, n_pages - j * C::kPPS);
            const unsigned loaded = __ballot_sync(0xffffffffu, lane < np && pg_cur >= 0 && pg_cur < p.num_pages);
            const int bad = static_cast<int>(~loaded & ((1u << np) - 1u));
            pg_cur = pg_nxt;
            // this row sees keys [low, lim) of the stage; pages skipped or not loaded are masked
            const int lim = row_valid ? min(C::kTP, row_hi - kbase) : 0;
            const int low = row_lo - kbase;
            modify_row(p, coef, s, slope, pos - kbase - part * kH);
            if (!(lim == C::kTP && np == C::kPPS && bad == 0 && low <= 0 && okl)) {
                // this thread's visible columns as bits: from low to lim, on loaded pages
                constexpr int kPer = kH / P;  // pages among this thread's columns
                const int c0 = part * kH;
                uint64_t see = bits_below(lim - c0) & ~bits_below(low - c0);
#pragma unroll
                for (int k = 0; k < kPer; ++k)
                    if (part * kPer + k >= np || ((bad >> (part * kPer + k)) & 1))
                        see &= ~(((1ull << P) - 1) << (k * P));
                if (!okl) see = 0;
#pragma unroll
                for (int c = 0; c < kH; ++c)
                    if (!((static_cast<uint32_t>(see >> (c & 32)) >> (c & 31)) & 1u)) s[c] = -INFINITY;
            }
            float alpha = 1.f;
            bool need = false;
            {
                // reference maximum: moves only when the row's max exceeds it by more than 2^8. The two warps of a row
                // meet in one barrier that votes whether any of its rows may have to; only then are the maxima exchanged.
                float mx = fmaxf(s[0], s[1]);
#pragma unroll
                for (int c = 2; c < kH; c += 2) mx = fmax3(mx, s[c], s[c + 1]);
                if (named_bar_any(row_bar, 32 * kParts, mx > m_ref + 8.f || !okl)) {
                    float v[kParts];
                    meet(mx, v, okl);
                    if (!okl) {
                        ok = false;  // both parts of every row of this quarter stop here
                        break;
                    }
                    const float row_max = fmaxf(v[0], v[1]);
                    need = row_max > m_ref + 8.f;
                    if (need) {
                        alpha = exp2f(m_ref - row_max);  // 0 while m_ref is -inf
                        m_ref = row_max;
                        l *= alpha;
                    }
                }
            }
            const bool flush = j > 0 && j % kFlush == 0;
            if (flush || (j > 0 && __any_sync(0xffffffffu, need))) {
                // O holds P.V of the earlier stages: wait for the last one, then rescale or move this part of the rows
                if (!wait(okl, p_empty((j - 1) % 3), ((j - 1) / 3) & 1)) {
                    ok = false;  // the next vote stops the quarter
                    continue;
                }
                tc_fence_after();
                // (the scores stay live across this block: 32 columns at a time)
#pragma unroll
                for (int q = 0; q < kH / 32; ++q) {
                    const uint32_t tOq = tO + lane_addr + part * kH + q * 32;
                    uint32_t a[32];
                    tmem_ld32(tOq, a);
                    tmem_wait_ld();
                    if (flush) {  // P.V of this stage starts a new accumulation
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            acc[q * 16 + i] = fadd2(acc[q * 16 + i], make_float2(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1])));
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) a[i] = __float_as_uint(__uint_as_float(a[i]) * alpha);
                        tmem_st32(tOq, a);
                    }
                }
                tmem_wait_st();
            }
            if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                for (int i = 0; i < kH / 2; ++i) acc[i] = fmul2(acc[i], make_float2(alpha, alpha));
            }
            // probabilities -> P over this thread's own S columns: 32 columns of pairs, then 32 of residual pairs
            const float neg = (m_ref == -INFINITY) ? 0.f : -m_ref;
            const float2 negv = make_float2(neg, neg);
            float2 lsum = make_float2(0.f, 0.f);
#pragma unroll
            for (int q = 0; q < kH / 32; ++q) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    // two keys at a time: one packed add for the exponents, one for the sums
                    const float2 x = fadd2(make_float2(s[q * 32 + 2 * i], s[q * 32 + 2 * i + 1]), negv);
                    const float p0 = exp2f(x.x), p1 = exp2f(x.y);  // exp2(-inf) = 0 for masked keys
                    lsum = fadd2(lsum, make_float2(p0, p1));
                    pack2_split_near<kBF16>(p0, p1, hi[i], lo[i]);
                }
                tmem_st16(tS + part * kH + q * 16, hi);
                tmem_st16(tS + part * kH + kH / 2 + q * 16, lo);
            }
            l += lsum.x + lsum.y;
            tmem_wait_st();
            clean_v(j, kbase, np, bad, part * 8, 8, okl);
            if (!okl) {
                ok = false;  // the next vote stops the quarter
                continue;
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(j % 3));
        }
        // ---- epilogue: O row / l (this thread: dims kH part .. + kH - 1)
        bool okl = ok;
        if (wait(okl, o_full, 0)) tc_fence_after();
        float lv[kParts];
        meet(l, lv, okl);
        float l_all = 0.f;
#pragma unroll
        for (int k = 0; k < kParts; ++k) l_all += lv[k];
        named_bar_sync(5, 32 * C::kSoftmaxWarps);  // every softmax warp is done with its stages
        const bool dirty = *reinterpret_cast<volatile int*>(smem + C::kOffDirty) != 0;
        float* dst = p.out + qrow * DH + od;
        if (okl) {
            const float inv = l_all != 0.f ? 1.f / l_all : 0.f;
            bool nan = false;
#pragma unroll
            for (int q = 0; q < kH / 16; ++q) {
                uint32_t a[16];
                tmem_ld16(tO + lane_addr + od + q * 16, a);
                tmem_wait_ld();
                if (row_valid) {
                    float o[16];
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        o[i] = __uint_as_float(a[i]) + acc[q * 8 + i / 2].x;
                        o[i + 1] = __uint_as_float(a[i + 1]) + acc[q * 8 + i / 2].y;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) nan = nan || o[i] != o[i];
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *reinterpret_cast<float4*>(dst + q * 16 + i) =
                            make_float4(o[i] * inv, o[i + 1] * inv, o[i + 2] * inv, o[i + 3] * inv);
                }
                __syncwarp();  // the next load is warp-collective
            }
            // NaN and infinities among the values this row sees (rare): those of boundary stages were zeroed for the
            // product, and an infinity elsewhere times a residual of 0 gave a NaN. Either way the row's values, read
            // again, say what those sums are.
            const bool again = row_valid && (dirty || nan) && l_all == l_all && l_all != 0.f;
            if (__any_sync(0xffffffffu, again))
                add_nonfinite<kBF16>(p, b, kvh, P, DH, od, od + kH, again ? row_lo : 0, again ? row_hi : 0, inv, dst);
        } else if (row_valid) {
            for (int d = 0; d < kH; ++d) dst[d] = 0.f;
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

template <int KT, int P>
cudaError_t launch_prefill_mod_tc_inst(const DecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, dim3 grid,
                                       cudaStream_t st) {
    using C = PfModCfg<128, P>;
    auto* kern = paged_prefill_mod_tc_kernel<KT, 128, P>;
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load(std::memory_order_acquire) & bit)) {
        // the kernel moves registers between its warpgroups (setmaxnreg): the shares must fit in what a CTA
        // is launched with, or the warpgroup asking for more would wait for ever
        cudaFuncAttributes fa{};
        e = cudaFuncGetAttributes(&fa, kern);
        if (e != cudaSuccess) return e;
        const long long pool = static_cast<long long>(fa.numRegs) * C::kThreads;
        const long long need = 128LL * C::kRegsLow + 256LL * C::kRegsHigh;
        if (need > pool) return cudaErrorInvalidConfiguration;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    return launch_pdl(kern, grid, dim3(C::kThreads), C::kSmem, st, p, tk, tv);
}

}  // namespace kvp
