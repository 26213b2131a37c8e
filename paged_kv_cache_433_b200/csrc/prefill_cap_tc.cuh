// Multi-token query (chunked prefill) with capped scores over the paged cache on the fifth-generation tensor cores
// (tcgen05), sm_100a: the kernel of paged_prefill_attention_mod for bf16, Dh = 128, a tanh cap of at most 50 and no
// distance bias.
//
// The cap bounds every score, so one softmax reference serves all rows: no row maximum is taken, nothing is rescaled and
// the threads that share a row never meet before its end (prefill_mod_tc.cuh has the general form, and score_mod.cuh the
// functions). The reference is subtracted by the last multiply-add of the cap's polynomial.
//
// Tile: 128 rows = 128 / g chunk tokens x the g heads of a KV head. Stages of 128 keys: S = Q K^T (tcgen05, fp32 in
// tensor memory, three buffers), then P written over S's columns as a 16-bit value plus residual, then O += P V.
// Roles of a CTA's 16 warps: 0 loads K and 2 loads V (TMA boxes of pages), 1 loads the Q tile and issues Q K^T, 3 issues
// P V; three softmax warpgroups take every third stage, a thread a whole row in chunks of 32 keys, so that one computes
// while the others wait for their scores.
//
// The grid has a CTA per tile, but a CTA that is done with its tile takes the place of one that has not started
// (clusterlaunchcontrol) and goes on, so that in effect one CTA per SM walks through tiles (whose costs differ: handed out
// in a fixed order the windowed case below took 345 us instead of 310). Stages, barriers and ring entries are counted over
// all of its tiles. Warp 0 asks for the next tile and lays its description out for the other warps; loads and Q K^T run
// ahead into it, and a warpgroup computes its first stage of it before it reads out O of the last one, for which it has to
// wait for the slowest. A tile's start and end, about 10 us with a CTA each, are hidden that way -- windowed layers have few stages per tile.
//
// Measured, 32 heads on 8: 8 chunks of 512 tokens over 4096, cap 50: 450 us at 1965 MHz, 650 TFLOP/s counted once, 975 with
// the residuals' products; 489 us back to back, where the power cap holds the clock at 1700 MHz (a CTA per tile took a
// tenth more; without the cap, prefill_tc.cuh: 425-430). Two prompts of 4096 tokens in documents of 1500 under a window of
// 1024, cap 30: 252 us (a CTA per tile, ascending: a third more). That is for scores below a fifth of the cap; 1283 us
// where many are above it (deviation 5) and 1841 at deviation 15, by the short loop in the softmax below. Bound by the
// chain Q K^T -> softmax -> P V of a stage, about 10,400 cycles at three stages in flight: the matrix pipe is busy for
// 1,536 cycles a stage, the exponentials for 1,024, and tensor memory has no room for a fourth buffer of scores.
//
// O is moved into fp32 sums in registers every kFlushKeys keys (score_mod.cuh). V rows that no row of the tile sees are
// zeroed, and in a stage that some rows see only in part NaN and infinities too; the rows that do see them add them from
// the pool at the end. Every wait is bounded (KV_DEV_ERR_TIMEOUT); block-table entries outside [0, num_pages) are never
// loaded (their keys are masked, KV_DEV_ERR_PAGE_RANGE).
#pragma once

#include <cuda.h>

#include <atomic>

#include "decode_kernel.cuh"
#include "decode_launch.cuh"
#include "score_mod.cuh"
#include "tc05.cuh"

namespace kvp {

template <int P>
struct PfCapCfg {
    static constexpr int kDH = 128;
    static constexpr int kTP = 128;              // keys per stage
    static constexpr int kPPS = kTP / P;         // pages per stage
    static constexpr int kBoxCols = kDH / 64;
    static constexpr int kBoxB = kTP * 128;      // one 128-byte box column of an entry
    static constexpr int kEntry = kBoxCols * kBoxB;
    // entries 0..1: K of stages j % 2; 2..4: V of stages j % 3, so that V of a stage is on its way when its scores are there
    static constexpr int kKSlots = 2, kVSlots = 3;
    static constexpr int kMasks = 8;             // stages whose loaded pages are noted (more than are in flight)
    static constexpr int kRing = kKSlots + kVSlots;
    static constexpr int kQB = 128 * kDH * 2;    // Q tile
    static constexpr int kOffQ = kRing * kEntry;
    static constexpr int kGroups = 3;            // softmax warpgroups
    static constexpr int kDims = 48;             // dims of O a thread reads out (the last group 32)
    static constexpr int kTileSlots = 4;         // tiles that may be under way
    static constexpr int kOffX = kOffQ + kQB;    // sums of weights: [tile][first stage][row]
    static constexpr int kOffBar = kOffX + kTileSlots * kGroups * 128 * 4;
    // full[R], empty[R], s_full[3], p_full[2][3], p_empty[3], q_free, o_full, o_free, done (QK), done (PV), next,
    // tile_full[4], tile_empty[4], summed[4]
    static constexpr int kNumBars = 2 * kRing + 12 + 6 + 3 * kTileSlots;
    static constexpr int kOffTmem = kOffBar + 8 * kNumBars;
    // [tile slot]: number + 1 of the last tile (with stages) of which a stage seen in part held a NaN or an infinity in V
    static constexpr int kOffDirty = kOffTmem + 8;
    static constexpr int kOffMasks = kOffDirty + 4 * kTileSlots;
    static constexpr int kOffNext = (kOffMasks + 4 * kMasks + 15) / 16 * 16;  // answer to the request for a tile
    static constexpr int kTileWords = 32 + 128;  // a tile's description and the first keys of its up to 128 tokens
    static constexpr int kOffTiles = kOffNext + 16;
    static constexpr int kSmem = 1024 + kOffTiles + kTileSlots * kTileWords * 4;
    static constexpr int kThreads = 128 + 128 * kGroups;
    static constexpr int kSoftmaxWarps = 4 * kGroups;
    static constexpr uint32_t kTmemCols = 512;   // S x 3 (384) + O (128)
    static_assert(kPPS * kBoxCols <= 32, "one TMA box per lane");
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

// Tile `tile`: chunk tokens t0 .. t0 + nt - 1 (nt <= 0: none) of sequence b, KV head kvh; n_st stages of keys from
// key_first on (0: no row sees any key). Called by whole warps.
struct CapTile {
    int tile;  // -1: no more
    int b, kvh, qs0, t0, nt, pos0, prefix, n_st, page_first, n_pages, key_first, bad_len;
    TileKeys k;
};
static_assert(sizeof(CapTile) <= 32 * 4, "description of a tile");
template <int P>
__device__ __forceinline__ CapTile cap_tile(const DecodeParams& p, int tile, int n_tiles, int lane) {
    constexpr int kTP = PfCapCfg<P>::kTP;
    CapTile t;
    t.tile = tile;
    const ChunkTile ct = chunk_tile(p, (n_tiles - 1 - tile) / p.H_kv, lane);
    t.kvh = tile % p.H_kv;
    t.b = ct.b;
    t.qs0 = ct.qs0;
    const int n_q = ct.n_q, len = p.seq_lens[t.b];
    t.t0 = ct.t0;
    t.nt = ct.nt;
    t.bad_len = len < 0 || len > p.max_blocks * P || n_q > len;
    t.pos0 = len - n_q + t.t0;
    t.prefix = p.prefix_lens != nullptr ? min(p.prefix_lens[t.b], len) : 0;
    t.n_st = t.page_first = t.n_pages = t.key_first = 0;
    t.k = TileKeys{0, 0, 0, 0};
    if (t.nt > 0 && !t.bad_len) {
        t.k = tile_keys(p, t.qs0 + t.t0, t.pos0, t.nt, t.prefix, lane);
        if (t.k.begin < t.k.end) {
            t.key_first = t.k.begin / kTP * kTP;
            t.page_first = t.key_first / P;
            t.n_pages = (t.k.end + P - 1) / P - t.page_first;
            t.n_st = (t.k.end - t.key_first + kTP - 1) / kTP;
        }
    }
    return t;
}

// Asks for the work of a CTA of the grid that has not started; the answer's 16 bytes complete on `bar`.
__device__ __forceinline__ void request_tile(uint32_t answer, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
                 "r"(bar)
                 : "memory");
}
// blockIdx.x of that CTA, which then never starts; -1: all have.
__device__ __forceinline__ int requested_tile(uint32_t answer) {
    int x;
    asm volatile(
        "{\n\t.reg .pred got;\n\t.reg .b128 a;\n\t"
        "ld.shared.b128 a, [%1];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 got, a;\n\t"
        "mov.b32 %0, -1;\n\t"
        "@got clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, a;\n\t}"
        : "=r"(x)
        : "r"(answer)
        : "memory");
    return x;
}

// Bits 0 .. n - 1 of 32 (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t bits32_below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

template <int P>
__global__ void __launch_bounds__(512, 1)
    paged_prefill_cap_tc_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ CUtensorMap tmap_k,
                                const __grid_constant__ CUtensorMap tmap_v) {
    using C = PfCapCfg<P>;
    constexpr int DH = C::kDH, kTP = C::kTP, kG = C::kGroups;
    constexpr uint32_t kIdescQK = idesc_f16(true, 128, kTP, false, false);
    constexpr uint32_t kIdescPV = idesc_f16(true, 128, DH, false, true);
    constexpr int kFlush = kFlushKeys / kTP;  // stages whose P.V share one accumulation
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const int n_tiles = gridDim.x;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
    }
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    unsigned char* smem = smem_raw + (sbase - raw);
    const uint32_t bar0 = sbase + C::kOffBar;
    auto full = [&](int e) { return bar0 + 8u * e; };
    auto empty = [&](int e) { return bar0 + 8u * (C::kRing + e); };
    auto s_full = [&](int i) { return bar0 + 8u * (2 * C::kRing + i); };
    auto p_empty = [&](int i) { return bar0 + 8u * (2 * C::kRing + 3 + i); };  // P.V has read buffer i
    // by the four warps of group i: P of the stage's first / second 64 keys is written (and V is clean)
    auto p_full = [&](int i, int h) { return bar0 + 8u * (2 * C::kRing + 6 + 2 * i + h); };
    const uint32_t bars1 = bar0 + 8u * (2 * C::kRing + 12);
    const uint32_t q_free = bars1;        // every Q K^T of a tile is done
    const uint32_t o_full = bars1 + 8;    // every P.V of a tile is done
    const uint32_t o_free = bars1 + 16;   // every softmax warp has read an accumulation out of O
    const uint32_t done_qk = bars1 + 24, done_pv = bars1 + 32;
    const uint32_t next = bars1 + 40;     // the answer to the request for a tile is there
    auto tile_full = [&](int i) { return bars1 + 48 + 8u * i; };
    auto tile_empty = [&](int i) { return bars1 + 48 + 8u * (C::kTileSlots + i); };  // read by the other 15 warps
    auto summed = [&](int i) { return bars1 + 48 + 8u * (2 * C::kTileSlots + i); };  // by every softmax warp
    // stage numbers below count over the CTA's tiles
    auto kslot = [](int j) { return j % C::kKSlots; };
    auto vslot = [](int j) { return C::kKSlots + j % C::kVSlots; };
    auto kphase = [](int j) { return static_cast<uint32_t>((j / C::kKSlots) & 1); };
    auto vphase = [](int j) { return static_cast<uint32_t>((j / C::kVSlots) & 1); };
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::kOffTmem);
    volatile int* dirty = reinterpret_cast<volatile int*>(smem + C::kOffDirty);
    // [stage % kMasks]: its pages that were loaded, written before its K is announced
    volatile uint32_t* masks = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMasks);

    if (threadIdx.x == 0) {
        for (int e = 0; e < C::kRing; ++e) {
            mbar_init(full(e), 1);
            mbar_init(empty(e), 1);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(s_full(i), 1);
            mbar_init(p_full(i, 0), 4);
            mbar_init(p_full(i, 1), 4);
            mbar_init(p_empty(i), 1);
        }
        mbar_init(q_free, 1);
        mbar_init(o_full, 1);
        mbar_init(o_free, C::kSoftmaxWarps);
        mbar_init(done_qk, 1);
        mbar_init(done_pv, 1);
        mbar_init(next, 1);
        for (int i = 0; i < C::kTileSlots; ++i) {
            mbar_init(tile_full(i), 1);
            mbar_init(tile_empty(i), C::kThreads / 32 - 1);
            mbar_init(summed(i), C::kSoftmaxWarps);
        }
        for (int i = 0; i < C::kTileSlots; ++i) dirty[i] = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), C::kTmemCols);
        tmem_relinquish();
    }
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tO = tmem + 3 * kTP;
    const uint32_t ring = sbase;
    const uint32_t sQ = sbase + C::kOffQ;

    // The CTA's tile number `it`, and the first key that the row of token tr sees (0 behind the tile's rows); false where a
    // wait ran out. Called by whole warps, in order.
    auto read_tile = [&](int it, int tr, CapTile& t, int& lo) {
        const int slot = it % C::kTileSlots;
        const bool there = mbar_wait_bounded(tile_full(slot), (it / C::kTileSlots) & 1, kWaitLimitNs);
        if (!__all_sync(0xffffffffu, there)) {
            if (lane == 0) raise_err(p.err, KV_DEV_ERR_TIMEOUT);
            return false;
        }
        const int* d = reinterpret_cast<const int*>(smem + C::kOffTiles) + slot * C::kTileWords;
        t = *reinterpret_cast<const CapTile*>(d);
        lo = tr < t.nt ? d[32 + tr] : 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(tile_empty(slot));
        return true;
    };
    int unused;

    if (warp == 0 || warp == 2) {
        // ------------------------------------------------------------ producers: warp 0 K (and the tiles), warp 2 V
        const bool is_v = warp == 2;
        bool ok = true;
        int gs = 0, fills = 0;  // stages of the tiles before this one; stages whose boxes were issued
        int tile = blockIdx.x;
        for (int it = 0; ok; ++it) {
            CapTile t{};
            if (is_v) {
                if (!read_tile(it, 0, t, unused)) break;
            } else {
                const int slot = it % C::kTileSlots;
                if (lane == 0 && it >= C::kTileSlots &&
                    !mbar_wait_bounded(tile_empty(slot), (it / C::kTileSlots - 1) & 1, kWaitLimitNs)) {
                    raise_err(p.err, KV_DEV_ERR_TIMEOUT);
                    ok = false;
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                int* d = reinterpret_cast<int*>(smem + C::kOffTiles) + slot * C::kTileWords;
                if (tile >= 0) t = cap_tile<P>(p, tile, n_tiles, lane);
                t.tile = tile;
                if (lane == 0) *reinterpret_cast<CapTile*>(d) = t;
                for (int i = lane; tile >= 0 && !t.bad_len && i < t.nt; i += 32)
                    d[32 + i] = first_key(p, t.qs0 + t.t0 + i, t.pos0 + i);
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(tile_full(slot));
                    if (tile >= 0) {
                        mbar_arrive_expect_tx(next, 16);
                        request_tile(sbase + C::kOffNext, next);
                    }
                }
            }
            if (t.tile < 0) break;
            const int32_t* row = p.block_tables + (int64_t)t.b * p.max_blocks + t.page_first;
            int tab_cur = lane < t.n_pages ? row[lane] : -1, tab_nxt = -1;
            // pages of the first stage that lie before the first key any row sees: not loaded, whatever their entries are
            const int skip = t.k.begin / P - t.page_first;
            for (int j = 0; j < t.n_st; ++j) {
                const int np = min(C::kPPS, t.n_pages - j * C::kPPS);
                // block-table entries come 32 at a time, one per lane, the next 32 fetched while these are used
                // (stages never straddle a group: 32 is a multiple of the pages per stage)
                if (((j * C::kPPS) & 31) == 0) {
                    const int base = j * C::kPPS;
                    tab_cur = base == 0 ? tab_cur : tab_nxt;
                    tab_nxt = (base + 32 + lane < t.n_pages) ? row[base + 32 + lane] : -1;
                }
                const int pg_all = __shfl_sync(0xffffffffu, tab_cur, (j * C::kPPS + lane) & 31);
                const bool wanted = lane < np && j * C::kPPS + lane >= skip;
                const int pg = wanted ? pg_all : -1;
                const bool good = wanted && pg >= 0 && pg < p.num_pages;
                if (wanted && !good) raise_err(p.err, KV_DEV_ERR_PAGE_RANGE);
                const unsigned gmask = __ballot_sync(0xffffffffu, good);
                const int box_page = lane / C::kBoxCols, bb = lane % C::kBoxCols;
                const int pgl = __shfl_sync(0xffffffffu, pg, box_page & 31);
                const int J = gs + j;
                const int e = is_v ? vslot(J) : kslot(J);
                const int use = is_v ? J / C::kVSlots : J / C::kKSlots;  // earlier fills of this entry
                if (lane == 0) {
                    if (use > 0 && !mbar_wait_bounded(empty(e), (use - 1) & 1, kWaitLimitNs)) {
                        raise_err(p.err, KV_DEV_ERR_TIMEOUT);
                        ok = false;
                    } else {
                        if (!is_v) masks[J % C::kMasks] = gmask;
                        mbar_arrive_expect_tx(full(e), __popc(gmask) * C::kBoxCols * P * 128);
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                if (box_page < np && ((gmask >> box_page) & 1u)) {
                    const uint32_t dst = ring + e * C::kEntry + bb * C::kBoxB + box_page * P * 128;
                    tma_load_2d(dst, is_v ? static_cast<const void*>(&tmap_v) : static_cast<const void*>(&tmap_k), bb * 64,
                                (pgl * p.H_kv + t.kvh) * P, full(e));
                }
                fills = J + 1;
            }
            gs += t.n_st;
            if (!is_v) {  // (with a failure above too: the answer's copy has landed before the CTA exits)
                if (lane == 0) {
                    if (mbar_wait_bounded(next, it & 1, kWaitLimitNs)) {
                        tile = requested_tile(sbase + C::kOffNext);
                        fence_proxy_async_smem();
                    } else {
                        raise_err(p.err, KV_DEV_ERR_TIMEOUT);
                        ok = false;
                    }
                }
                tile = __shfl_sync(0xffffffffu, tile, 0);
                ok = __shfl_sync(0xffffffffu, ok, 0);
            }
        }
        if (lane == 0) {  // the last fill of every entry has landed before the CTA exits
            const int slots = is_v ? C::kVSlots : C::kKSlots;
            for (int j = max(0, fills - slots); j < fills; ++j)
                if (!mbar_wait_bounded(full(is_v ? vslot(j) : kslot(j)), is_v ? vphase(j) : kphase(j), kWaitLimitNs))
                    raise_err(p.err, KV_DEV_ERR_TIMEOUT);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ Q tile, Q K^T once K has landed and P.V(j - 3) has
        // released S columns j % 3
        bool ok = true;
        int gs = 0, with_stages = 0;
        CapTile t;
        for (int it = 0; ok && read_tile(it, 0, t, unused) && t.tile >= 0; ++it) {
            if (t.n_st == 0) continue;
            if (with_stages > 0) {
                if (lane == 0 && !mbar_wait_bounded(q_free, (with_stages - 1) & 1, kWaitLimitNs)) {
                    raise_err(p.err, KV_DEV_ERR_TIMEOUT);
                    ok = false;
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
            }
            ++with_stages;
            // Q row r (chunk token t0 + r / g, head kvh * g + r % g) -> the swizzled K-major tile, zeros behind the chunk
            const uint4* q = static_cast<const uint4*>(p.q) + ((int64_t)(t.qs0 + t.t0) * p.H_q + (int64_t)t.kvh * p.g) * (DH / 8);
            const int c = lane & 15;
#pragma unroll 8
            for (int r = lane >> 4; r < 128; r += 2) {
                const int tr = r / p.g;
                const bool valid = tr < t.nt;
                const uint4* src = q + (valid ? ((int64_t)tr * p.H_q + r - tr * p.g) * (DH / 8) + c : 0);
                const uint32_t dst = sQ + (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                             : "memory");
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                auto wait = [&](uint32_t bar, uint32_t parity) {
                    if (ok && !mbar_wait_bounded(bar, parity, kWaitLimitNs)) {
                        raise_err(p.err, KV_DEV_ERR_TIMEOUT);
                        ok = false;
                    }
                    return ok;
                };
                for (int j = 0; j < t.n_st; ++j) {
                    const int J = gs + j, e = kslot(J);
                    if (!wait(full(e), kphase(J))) break;
                    if (J >= 3 && !wait(p_empty(J % 3), ((J - 3) / 3) & 1)) break;
                    tc_fence_after();
                    const uint32_t sK = ring + e * C::kEntry;
                    const uint32_t tS = tmem + (J % 3) * kTP;
#pragma unroll
                    for (int kk = 0; kk < DH / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * C::kBoxB + (kk & 3) * 32;
                        umma_ss(tS, smem_desc(sQ + off, 16, 1024, kSwz128), smem_desc(sK + off, 16, 1024, kSwz128), kIdescQK,
                                kk > 0 ? 1u : 0u);
                    }
                    umma_commit(s_full(J % 3));
                    umma_commit(empty(e));
                }
                umma_commit(q_free);
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            gs += t.n_st;
        }
        if (lane == 0) {
            umma_commit(done_qk);
            if (!mbar_wait_bounded(done_qk, 0, kWaitLimitNs)) raise_err(p.err, KV_DEV_ERR_TIMEOUT);
        }
        __syncwarp();
    } else if (warp == 3) {
        // ------------------------------------------------------------ P V once the softmax has written P
        bool ok = true;
        int gs = 0, acc = 0;  // accumulations begun
        CapTile t;
        for (int it = 0; ok && read_tile(it, 0, t, unused) && t.tile >= 0; ++it) {
            if (t.n_st == 0) continue;
            if (lane == 0) {
                auto wait = [&](uint32_t bar, uint32_t parity) {
                    if (ok && !mbar_wait_bounded(bar, parity, kWaitLimitNs)) {
                        raise_err(p.err, KV_DEV_ERR_TIMEOUT);
                        ok = false;
                    }
                    return ok;
                };
                for (int j = 0; j < t.n_st; ++j) {
                    const int J = gs + j, e = vslot(J);
                    if (!wait(full(e), vphase(J))) break;
                    const uint32_t sV = ring + e * C::kEntry;
                    const uint32_t tP = tmem + (J % 3) * kTP;
                    // each run of 32 keys, as one thread writes it over its own S columns: the values, then their residuals
                    auto p_col = [](int kk) { return kk * 16 / 32 * 32 + kk * 16 % 32 / 2; };
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (!wait(p_full(J % 3, h), (J / 3) & 1)) break;
                        if (h == 0 && j % kFlush == 0) {  // O starts anew: the accumulation before has been read out
                            if (acc > 0 && !wait(o_free, (acc - 1) & 1)) break;
                            ++acc;
                        }
                        tc_fence_after();
#pragma unroll
                        for (int kk = h * kTP / 32; kk < (h + 1) * kTP / 32; ++kk)
                            umma_ts(tO, tP + p_col(kk), smem_desc(sV + kk * 16 * 128, C::kBoxB, 1024, kSwz128), kIdescPV,
                                    (j % kFlush != 0 || kk > 0) ? 1u : 0u);
#pragma unroll
                        for (int kk = h * kTP / 32; kk < (h + 1) * kTP / 32; ++kk)
                            umma_ts(tO, tP + p_col(kk) + 16, smem_desc(sV + kk * 16 * 128, C::kBoxB, 1024, kSwz128), kIdescPV,
                                    1u);
                    }
                    if (!ok) break;
                    umma_commit(empty(e));
                    umma_commit(p_empty(J % 3));
                }
                if (ok) umma_commit(o_full);
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            gs += t.n_st;
        }
        if (lane == 0) {
            umma_commit(done_pv);
            if (!mbar_wait_bounded(done_pv, 0, kWaitLimitNs)) raise_err(p.err, KV_DEV_ERR_TIMEOUT);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax, read-out
        const int quarter = warp & 3, group = (warp >> 2) - 1;
        const int r = quarter * 32 + lane;   // MMA row
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        const int tr = r / p.g;
        const int od = group * C::kDims;       // first dim this thread reads out
        float* xl = reinterpret_cast<float*>(smem + C::kOffX);
        const CapRowCoef coef = cap_row_coefs(p);
        bool ok = true;
        // warp-uniform outcome: the tensor-memory loads and stores after a wait are warp-collective
        auto wait = [&](uint32_t bar, uint32_t parity) {
            if (ok && !mbar_wait_bounded(bar, parity, kWaitLimitNs)) {
                raise_err(p.err, KV_DEV_ERR_TIMEOUT);
                ok = false;
            }
            ok = __all_sync(0xffffffffu, ok);
            return ok;
        };
        // earlier accumulations of this thread's part of O
        float2 acc[C::kDims / 2];
#pragma unroll
        for (int i = 0; i < C::kDims / 2; ++i) acc[i] = make_float2(0.f, 0.f);
        auto release_o = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
        };

        int gs = 0, read_out = 0;  // stages of the tiles before this one; tiles read out
        // the tile that waits for its read-out: its number (-1: none), this thread's row (-1: none)
        int last_tile = -1;
        int64_t last_row = -1;
        // ---- O row / l of the last tile (this thread: dims od .. od + 47)
        auto read_last = [&]() {
            const int slot = read_out % C::kTileSlots;
            if (wait(o_full, read_out & 1) && wait(summed(slot), (read_out / C::kTileSlots) & 1)) tc_fence_after();
            ++read_out;
            float l = 0.f;
#pragma unroll
            for (int k = 0; k < kG; ++k) l += xl[(slot * kG + k) * 128 + r];
            const bool search = dirty[slot] == read_out;  // (read_out is the tile's number + 1 by now)
            bool nan = false;
            float* dst = p.out + last_row * DH + od;
            const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
            for (int q = 0; q < C::kDims / 16; ++q) {
                if (od + q * 16 >= DH) break;
                float o[16];
                if (ok) {
                    uint32_t a[16];
                    tmem_ld16(tO + lane_addr + od + q * 16, a);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        o[i] = __uint_as_float(a[i]) + acc[q * 8 + i / 2].x;
                        o[i + 1] = __uint_as_float(a[i + 1]) + acc[q * 8 + i / 2].y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = 0.f;
                }
                if (last_row >= 0) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) nan = nan || o[i] != o[i];
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *reinterpret_cast<float4*>(dst + q * 16 + i) =
                            make_float4(o[i] * inv, o[i + 1] * inv, o[i + 2] * inv, o[i + 3] * inv);
                }
                __syncwarp();  // the next load is warp-collective
            }
            release_o();
#pragma unroll
            for (int i = 0; i < C::kDims / 2; ++i) acc[i] = make_float2(0.f, 0.f);
            // NaN and infinities among the values this row sees (rare): those of stages seen in part were zeroed for the
            // product, and an infinity elsewhere times a residual of 0 gave a NaN. Either way the row's values, read
            // again, say what those sums are. (O is released before: P.V of the next tile waits for it.)
            const bool again = last_row >= 0 && (search || nan) && l == l && l != 0.f && ok;
            if (__any_sync(0xffffffffu, again)) {
                const ChunkTile ct = chunk_tile(p, (n_tiles - 1 - last_tile) / p.H_kv, lane);
                const int i0 = ct.t0 + tr, len = p.seq_lens[ct.b], pos = len - ct.n_q + i0;
                int lo = 0, hi = 0;
                if (again) {
                    lo = first_key(p, ct.qs0 + i0, pos);
                    hi = max(pos + 1, p.prefix_lens != nullptr ? min(p.prefix_lens[ct.b], len) : 0);
                }
                add_nonfinite<true>(p, ct.b, last_tile % p.H_kv, P, DH, od, min(od + C::kDims, DH), lo, hi, inv, dst);
            }
            last_tile = -1;
        };

        CapTile t;
        int row_lo;
        for (int it = 0; read_tile(it, tr, t, row_lo) && t.tile >= 0; ++it) {
            const bool row_valid = tr < t.nt;
            const int64_t row = row_valid ? (int64_t)(t.qs0 + t.t0 + tr) * p.H_q + (int64_t)t.kvh * p.g + r % p.g : -1;
            if (t.nt > 0 && t.bad_len && t.t0 == 0 && t.kvh == 0 && threadIdx.x == 128) raise_err(p.err, KV_DEV_ERR_SEQ_LEN);
            if (t.n_st == 0) {  // no row sees any key
                if (row_valid)
                    for (int d = od; d < min(DH, od + C::kDims); ++d) p.out[row * DH + d] = 0.f;
                continue;
            }
            const int pos = t.pos0 + tr;
            const int row_hi = row_valid ? max(pos + 1, t.prefix) : 0;  // this row sees keys row_lo .. row_hi - 1
            float l = 0.f;
            int next_flush = kFlush;
            // before stage next_flush, whose P.V starts a new accumulation: this thread's part of O joins its sums
            auto move_o = [&]() {
                const int Jf = gs + next_flush, Jp = Jf - 1;
                next_flush += kFlush;
                // S(Jf) is there: P.V(Jf - 3) is done, hence P.V(Jp - 3), so that the second wait's parity is that of
                // P.V(Jp). (S(Jf - 3) is too: this warp has seen a stage behind it.)
                if (!wait(s_full(Jf % 3), (Jf / 3) & 1) || !wait(p_empty(Jp % 3), (Jp / 3) & 1)) return;
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < C::kDims / 16; ++q) {
                    if (od + q * 16 >= DH) break;
                    uint32_t a[16];
                    tmem_ld16(tO + lane_addr + od + q * 16, a);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        acc[q * 8 + i] = fadd2(acc[q * 8 + i], make_float2(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1])));
                }
                release_o();
            };
            const int j0 = (group + 3 - gs % 3) % 3;  // this group's stages: gs + j0, + 3, ...
            for (int j = j0; j < t.n_st && ok; j += 3) {
                const int J = gs + j;
                if (!wait(s_full(J % 3), (J / 3) & 1)) break;
                while (next_flush <= j && ok) move_o();
                if (!ok) break;
                tc_fence_after();
                const uint32_t tS = tmem + (J % 3) * kTP + lane_addr;
                // keys of this stage: kbase .. kbase + 127; this row sees [low, lim) of them, on pages that were loaded
                const int kbase = t.key_first + j * kTP;
                const int np = min(C::kPPS, t.n_pages - j * C::kPPS);
                const int bad = static_cast<int>(~masks[J % C::kMasks] & ((1u << np) - 1u));
                const int lim = row_valid ? row_hi - kbase : 0, low = row_lo - kbase;
                // Thread r: V row r of the stage. A key no row of the tile sees (past its end, or on a page not loaded) may
                // hold stale bytes: zeroed. In a stage that some rows see only in part a NaN or an infinity must not reach
                // the others as 0 times it: zeroed too, and noted. Only then is V waited for before P is announced.
                const bool stale = kbase + r >= t.k.end || kbase + r < t.k.begin || r / P >= np || ((bad >> (r / P)) & 1);
                const bool part = kbase < t.k.all0 || kbase + kTP > t.k.all1;
                const bool clean = __any_sync(0xffffffffu, stale) || part;
                auto announce = [&](int h) {
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full(J % 3, h));
                };
                const bool full_stage = lim >= kTP && np == C::kPPS && bad == 0 && low <= 0;
                float2 lsum = make_float2(0.f, 0.f);
                // (one copy of the chunk's code: unrolled four times it outgrows the instruction caches)
#pragma unroll 1
                for (int q = 0; q < kTP / 32; ++q) {
                    uint32_t a[32];
                    tmem_ld32(tS + q * 32, a);
                    tmem_wait_ld();
                    float s[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(a[i]);
                    const float big = largest(s);
                    if (!__any_sync(0xffffffffu, big > p.cap_tiny)) {
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 x = cap_tiny2<true>(coef, make_float2(s[i], s[i + 1]));
                            s[i] = x.x;
                            s[i + 1] = x.y;
                        }
                    } else {  // in place, by a short loop: inlined for all 32 it slows the other branch down, 452 us for 481
                        const bool large = __any_sync(0xffffffffu, big > p.cap_small);
#pragma unroll 1
                        for (int h = 0; h < 4; ++h) {
                            uint32_t b[8];
                            float x[8];
                            tmem_ld8(tS + q * 32 + h * 8, b);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(b[i]);
                            cap_row_any<true>(p, coef, x, large);
#pragma unroll
                            for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(x[i]);
                            tmem_st8(tS + q * 32 + h * 8, b);
                        }
                        tmem_wait_st();
                        tmem_ld32(tS + q * 32, a);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(a[i]);
                    }
                    if (!full_stage) {
                        uint32_t see = bits32_below(lim - q * 32) & ~bits32_below(low - q * 32);
#pragma unroll
                        for (int k = 0; k < 32 / P; ++k) {
                            const int pgi = q * (32 / P) + k;
                            if (pgi >= np || ((bad >> pgi) & 1)) see &= P == 32 ? 0u : ~(0xffffu << (k * 16));
                        }
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (!((see >> c) & 1u)) s[c] = -INFINITY;
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t hi[8], lo[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float p0 = exp2f(s[h * 16 + 2 * i]), p1 = exp2f(s[h * 16 + 2 * i + 1]);
                            lsum = fadd2(lsum, make_float2(p0, p1));
                            pack2_split_near<true>(p0, p1, hi[i], lo[i]);
                        }
                        tmem_st8(tS + q * 32 + h * 8, hi);
                        tmem_st8(tS + q * 32 + 16 + h * 8, lo);
                    }
                    if (q == 1 && !clean) announce(0);
                }
                l += lsum.x + lsum.y;
                if (clean) {
                    // S(J) is there, so P.V(J - 3) is done and read the entry's fill before: the parity is this fill's
                    if (!wait(full(vslot(J)), vphase(J))) break;
                    const uint32_t at0 = ring + vslot(J) * C::kEntry + r * 128;
#pragma unroll 1
                    for (int c = 0; c < DH / 8; ++c) {
                        const uint32_t at = at0 + (c >> 3) * C::kBoxB + (c & 7) * 16;
                        if (stale) {
                            sts128_zero(at);
                        } else if (part) {
                            const uint4 v = lds128(at);
                            if (has_nonfinite16<true>(v)) {
                                const int number = read_out + (last_tile >= 0 ? 1 : 0);
                                dirty[number % C::kTileSlots] = number + 1;
                                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at),
                                             "r"(v.x ^ nonfinite16<true>(v.x)), "r"(v.y ^ nonfinite16<true>(v.y)),
                                             "r"(v.z ^ nonfinite16<true>(v.z)), "r"(v.w ^ nonfinite16<true>(v.w))
                                             : "memory");
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    announce(0);
                }
                announce(1);
                if (last_tile >= 0) read_last();
            }
            if (last_tile >= 0) read_last();
            while (ok && next_flush < t.n_st) move_o();
            last_tile = t.tile;
            last_row = row;
            {
                // This group's sums of weights, in the order of the tile's stages: which group has the first one depends on the
                // tiles before, and the total must not. (The slot was read four tiles ago: a stage of this tile is there only after
                // P.V of the tile three before it, which waited for that read-out.)
                const int slot = read_out % C::kTileSlots;
                xl[(slot * kG + j0) * 128 + r] = l;
                __syncwarp();
                if (lane == 0) mbar_arrive(summed(slot));
            }
            gs += t.n_st;
        }
        if (last_tile >= 0) read_last();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

template <int P>
cudaError_t launch_prefill_cap_tc_inst(const DecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int n_tiles,
                                       cudaStream_t st) {
    using C = PfCapCfg<P>;
    auto* kern = paged_prefill_cap_tc_kernel<P>;
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    return launch_pdl(kern, dim3(static_cast<unsigned>(n_tiles)), dim3(C::kThreads), C::kSmem, st, p, tk, tv);
}

}  // namespace kvp
