// Attention of drafted token trees over a paged key/value cache (attn_fwd_tree), and with
// one token per sequence the decoding step over pages.
//
// Sequence s has L_s positions in the cache, kept in pages: position j lies in row j % page
// of page table[s][j / page].  Its last T_s positions are the tokens of a tree, whose
// queries are packed rows [cu[s], cu[s+1]).  Token t sees every position before the tree
// (j < L_s - T_s), its ancestors and itself:
//   O_t = sum_j softmax_j(scale q_t.k_j) v_j   over those j,
// with the online softmax of the page "从零开始写Qwen3" (deepseek.csdn.net/6a3201f8...,
// section "在线softmax") over the key tiles and, across CTAs, over the pieces of a split.
//
// What bounds it: HBM.  A 128-key tile of K and V (64 KB at D = 128) feeds 4 T G D flops
// per key, far below the tensor rate for T G <= 128 rows, so K and V must be read once and
// the reads must never pause:
//   * the G query heads of a kv head and the T tokens of a tree are the rows of one
//     128-row tile (row = token * G + head in the group), so each K/V tile is read once per
//     kv head and 128 / G tokens;
//   * the key tiles of all (sequence, kv head, row tile) units form one list, of which every
//     CTA takes an equal contiguous share, whatever the lengths are; a unit counts for two tiles
//     more than it has, about what its change costs.  A unit cut by a share's border leaves
//     at most two pieces per CTA (fp32 O and log-sum-exp), merged by a second, dependent
//     launch; the others write O themselves.  (Merging in the CTA that brings the last piece
//     saves the launch, but its round trips come one after another: when it was tried, one token
//     over 4000 positions took 22.8 us that way and about 16 in two launches, 16 tokens over 32760
//     positions 86 and 47; the two launches, captured, take 12.9 and 33.5 by now.);
//   * the load order runs on across the units of a share: the next unit's first K tile is
//     loaded, and its scores computed, before the last P V of the unit before, the page
//     indexes of the next unit and of the next 32 pages are fetched ahead, and O has two
//     buffers, so that a unit's O is stored after the next unit's first weights.
//
// Roles (256 threads): warp 0 MMA issuer, warp 1 value guard (and TMEM), warp 2 TMA producer
// of K and V (the lanes issue one page box each), warp 3 scheduler, which also loads Q, warps
// 4-7 softmax (one row per thread).  P stays in TMEM over its scores.  TMEM: S0 [0,128),
// S1 [128,256), O0 [256,256+D), O1 [384,384+D).
//
// Window (attn_fwd_tree_window).  A unit's tiles are those of the first keys and those from the first
// position of the window of the tree's first token on, numbered without a gap; the bits of a row are
// cut to the token's nearest ancestors and the positions of its window.  16 sequences of one token,
// window 1024: 26 us captured, of which 8.5 are bytes at the copy rate, 7 pass until the first scores
// and 5 in the merge; 8 trees of 1 to 60, window 4096: 40 us.  (Leaving out the page pieces of a
// tile that no token sees reads 10% less and takes 0.5 and 1 us more.)
//
// Pages.  A page is [Hkv, page, D]; a tile is min(page, 128)-row boxes.  A page index past
// the end of the sequence or out of range is replaced by one past the last page, whose box
// reads as zeros; the second also sets the device error word.  Rows of the last page past
// L_s may hold anything: the guard zeroes them in V's tile, the mask drops their scores.
#pragma once
#include <cuda.h>  // CUtensorMap

#include "attn_fwd_varlen.cuh"
#include "kernel_common.cuh"

namespace gqa {

constexpr int kTreeThreads = 256;
constexpr int kTreeSlots = 8;      // unit descriptors in flight (256 sequences of 1000: 189 us with 4, 177 with 8)
constexpr int kTreeMax = 128;      // tokens of one tree
constexpr int kTreeSeqs = 2048;    // most sequences of one launch (their lengths lie in shared memory)
// The merge takes a warp (and block) per output row up to kMergeRows of them, and then blocks of
// 4 warps over 8 rows of each CTA's slot 1.  The first finds its row's pieces before it has to
// wait, but is bound by the blocks that are resident, as most wait for loads; in the second most
// blocks may have no row.  us per call, first / second: 128 rows 10.6 / 11.7, 1024 rows of 20
// pieces 27.9 / 32.1, 2048 rows 39.6 / 41.0, 5120 rows 35.8 / 36.3, 8192 rows 57.9 / 55.0 and
// 182.5 / 178.7, 12288 rows 46.2 / 41.8, 16384 rows 28.3 / 15.6, 32768 rows 88.7 / 66.4.
constexpr int kMergeRows = 6144, kMergeCtaThreads = 128, kMergeCtaRows = 8;
constexpr int kTreeBadTiles = 2;   // the tree's positions lie in at most two key tiles
constexpr int kTreeBadTilesWin = 8;  // and a window's start in two, the end of the first keys in one

struct TreeParams : Params {
    const int *cu, *table, *lens, *seqs, *parents;
    const uint8_t *v_ptr;
    int n_seqs, total_q, Hq, Hkv, n_rows;  // n_seqs <= kTreeSeqs; n_rows: rows of the page table
    int seq0;                  // row of the first sequence where seqs is NULL
    int page, page_shift, n_pages, table_w;
    int rt;                    // tokens per row tile: 128 / group
    int min_share;             // least weight of a CTA's share
    int window, sinks;         // window kernels: position pos sees j <= pos with j > pos - window or j < sinks
    long long o_row, o_head;   // strides in bytes
    float *part_o;             // [2 * CTAs][128][D]
    float *part_lse;           // [2 * CTAs][128]
    int grid;                  // CTAs of the first kernel
    // for the merge, one of the two: of each CTA's slot 1 the first packed row, kv head << 8 | tokens
    // (0: unused), key tiles behind this CTA and share; or [0]: share, [1 + s]: weights before sequence s
    int4 *starts;
    int *plan;
};

struct TreeUnit {
    int valid;
    int q0;       // packed row of the row tile's first token
    int ntok;     // its tokens
    int t0;       // index of the first one in the tree
    int T, base, L;  // tokens of the tree, positions before it, positions
    int row;      // row of the page table
    int kvh;
    int k0, k1;   // key tiles
    int piece;    // -1: the whole unit; 0, 1: piece slot of this CTA
    int first;    // packed row of the tree's first token
    int bad;      // set by the guard: some bad_rows bit is set
    uint32_t bad_rows[kTreeBadTilesWin][4];
};

template <int D>
struct TreeLayout {
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kTileBytes = (D / 64) * kAtomBytes;
    static constexpr int kQ = 0;
    static constexpr int kKV = kQ + kTileBytes;
    static constexpr int kBar = kKV + kStages * kTileBytes;
    // q_full, kv_full[S], kv_empty[S], v_ok[S], s_full[2], p_full[2], o_done[2], o_empty[2],
    // mma_done, q_empty, unit_full[slots], unit_empty[slots]
    static constexpr int kNumBars = 1 + 3 * kStages + 8 + 2 + 2 * kTreeSlots;
    static constexpr int kTmemSlot = kBar + kNumBars * 8;
    static constexpr int kAbort = kTmemSlot + 4;
    static constexpr int kUnits = (kAbort + 4 + 15) & ~15;
    static constexpr int kPar = kUnits + kTreeSlots * static_cast<int>(sizeof(TreeUnit));
    static constexpr int kSeqs = (kPar + 4 * kTreeMax * 4 + 15) & ~15;
    static constexpr int kUsed = kSeqs + kTreeSeqs * 8;
    // more than half of an SM's shared memory: one CTA (all 512 TMEM columns) per SM
    static constexpr int kAlloc = (kUsed + 1024) > 118 * 1024 ? (kUsed + 1024) : 118 * 1024;
};
static_assert(TreeLayout<128>::kAlloc <= 227 * 1024 && TreeLayout<64>::kAlloc <= 227 * 1024, "shared memory of one CTA");

// Tokens and positions of sequence s, clamped to what the tensors hold.
struct TreeSeq {
    int q0, T, L, row;
    bool bad;
};
template <bool kAhead = false>
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams &p, int s) {
    const VlSpan q = vl_span<kAhead>(p.cu, s, p.total_q);
    const int row = p.seqs != nullptr ? ld_state<kAhead>(p.seqs + s) : p.seq0 + s;
    TreeSeq r{q.a, q.b - q.a, 0, row, q.bad};
    if (row < 0 || row >= p.n_rows) {
        r.row = -1;
        r.bad = true;
    } else {
        r.L = ld_state<kAhead>(p.lens + row);
    }
    const long long cap = static_cast<long long>(p.table_w) << p.page_shift;
    if (r.L < 0) r.L = 0, r.bad = true;
    if (r.L > cap) r.L = static_cast<int>(cap), r.bad = true;
    // (a tree that is too long is cut, so that no offsets make the sum of the weights pass 32 bits)
    if (r.T > kTreeMax) r.T = kTreeMax, r.bad = true;
    if (r.T > r.L) r.bad = true;
    return r;
}
__device__ __forceinline__ int tree_row_tiles(const TreeParams &p, int T) { return (T + p.rt - 1) / p.rt; }
// Key tiles of a unit: all of the sequence's, or with a window those of the first keys and of the
// window of the tree's first token (win_skip).
__device__ __forceinline__ int tree_base(int T, int L) { return L > T ? L - T : 0; }
template <bool kWindow>
__device__ __forceinline__ int tree_key_tiles(const TreeParams &p, int T, int L) {
    int n = L > 0 ? (L + kBN - 1) / kBN : 1;
    if constexpr (kWindow) n -= win_skip(tree_base(T, L), p.window, p.sinks);
    return n > 1 ? n : 1;
}
// Tiles that every token of a tree sees whole; the others pass the guard (window kernels).
__device__ __forceinline__ WinWhole tree_whole(const TreeParams &p, int T, int base) {
    return win_whole(base, base, base + T - 1, p.window, p.sinks, win_skip(base, p.window, p.sinks));
}

// 128 bits as two words.
struct Bits128 {
    unsigned long long lo, hi;
};
__device__ __forceinline__ Bits128 bits_below(int n) {  // bits 0 .. n-1
    if (n <= 0) return {0ull, 0ull};
    if (n >= 128) return {~0ull, ~0ull};
    if (n >= 64) return {~0ull, n == 64 ? 0ull : (~0ull >> (128 - n))};
    return {~0ull >> (64 - n), 0ull};
}
__device__ __forceinline__ Bits128 bits_shl(Bits128 b, int n) {  // 0 <= n
    if (n >= 128) return {0ull, 0ull};
    if (n >= 64) return {0ull, b.lo << (n - 64)};
    if (n == 0) return b;
    return {b.lo << n, (b.hi << n) | (b.lo >> (64 - n))};
}
__device__ __forceinline__ Bits128 bits_shr(Bits128 b, int n) {
    if (n >= 128) return {0ull, 0ull};
    if (n >= 64) return {b.hi >> (n - 64), 0ull};
    if (n == 0) return b;
    return {(b.lo >> n) | (b.hi << (64 - n)), b.hi >> n};
}

// Weights of a unit in the shares: its key tiles and two for its change (with none a batch of
// eight trees takes 71 us, with one 62.5, with two 61.7, with three 60.2; one tree over 131000
// positions 98.9, 96.2, 94.1 and 96.3).
__device__ __forceinline__ int tree_unit_weight(int key_tiles) { return key_tiles + 2; }

// Weight of sequence s in the list of units.
template <bool kWindow>
__device__ __forceinline__ int tree_seq_weight(const TreeParams &p, int T, int L) {
    return p.Hkv * tree_row_tiles(p, T) * tree_unit_weight(tree_key_tiles<kWindow>(p, T, L));
}
__device__ __forceinline__ int tree_share(const TreeParams &p, int total) {
    const int share = (total + p.grid - 1) / p.grid;
    return share < p.min_share ? p.min_share : share;
}

// Ancestors of token t of a tree, itself among them; parents that are no earlier token end
// the walk.  par(u): the parent of token u.
template <typename F>
__device__ __forceinline__ Bits128 tree_ancestors(int t, F par) {
    Bits128 anc{0ull, 0ull};
    while (t >= 0 && t < kTreeMax) {
        if (t < 64) anc.lo |= 1ull << t; else anc.hi |= 1ull << (t - 64);
        const int up = par(t);
        if (up >= t) break;
        t = up;
    }
    return anc;
}

// With a window: of those ancestors the token's nearest `window` (itself among them) and those
// whose position is one of the first keys.  `depth` gets the token's: its position is base + depth.
template <typename F>
__device__ __forceinline__ Bits128 tree_window(int t, int base, int window, int sinks, int &depth, F par) {
    depth = -1;
    for (int u = t; u >= 0 && u < kTreeMax; ++depth) {
        const int up = par(u);
        u = up < u ? up : -1;
    }
    Bits128 anc{0ull, 0ull};
    int d = depth;
    for (int u = t; u >= 0 && u < kTreeMax; --d) {
        if (depth - d < window || base + d < sinks) {
            if (u < 64) anc.lo |= 1ull << u; else anc.hi |= 1ull << (u - 64);
        }
        const int up = par(u);
        u = up < u ? up : -1;
    }
    return anc;
}

// kWindow: attn_fwd_tree_window.
// tmQ: 3-D tensor map (D, Hq, tokens), box 64 x G x (128 / G); tmK, tmV: 3-D maps
// (D, page, n_pages * Hkv), box 64 x min(page, 128) x 1; all with the 128-byte swizzle.
template <int D, bool kBF16, bool kWindow>
__global__ void __launch_bounds__(kTreeThreads, 1)
    attn_fwd_tree_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TreeParams p) {
    using L = TreeLayout<D>;
    constexpr int S = L::kStages;
    constexpr int kBad = kWindow ? kTreeBadTilesWin : kTreeBadTiles;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const uint32_t sQ = base + L::kQ, sKV = base + L::kKV;
    const uint32_t bar0 = base + L::kBar;
    const uint32_t q_full = bar0;
    auto kv_full = [&](int s) { return bar0 + 8u * (1 + s); };
    auto kv_empty = [&](int s) { return bar0 + 8u * (1 + S + s); };
    auto v_ok = [&](int s) { return bar0 + 8u * (1 + 2 * S + s); };  // the V tile in stage s has passed the guard
    auto s_full = [&](int b) { return bar0 + 8u * (1 + 3 * S + b); };
    auto p_full = [&](int b) { return bar0 + 8u * (3 + 3 * S + b); };
    auto o_done = [&](int b) { return bar0 + 8u * (5 + 3 * S + b); };
    auto o_empty = [&](int b) { return bar0 + 8u * (7 + 3 * S + b); };  // O buffer b has been read
    const uint32_t mma_done = bar0 + 8u * (9 + 3 * S), q_empty = bar0 + 8u * (10 + 3 * S);
    auto unit_full = [&](int s) { return bar0 + 8u * (11 + 3 * S + s); };
    auto unit_empty = [&](int s) { return bar0 + 8u * (11 + 3 * S + kTreeSlots + s); };
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + L::kTmemSlot);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kAbort);
    TreeUnit *units = reinterpret_cast<TreeUnit *>(smem + L::kUnits);
    int2 *seqs = reinterpret_cast<int2 *>(smem + L::kSeqs);  // (T, L)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 64) {
        tma_prefetch_map(&tmQ);
        tma_prefetch_map(&tmK);
        tma_prefetch_map(&tmV);
    }
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int s = 0; s < S; ++s) {
            mbar_init(kv_full(s), 1);
            mbar_init(kv_empty(s), 2);  // the issuer and the guard
            mbar_init(v_ok(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(s_full(b), 1);
            mbar_init(p_full(b), 4);  // one arrival per softmax warp
            mbar_init(o_done(b), 1);
            mbar_init(o_empty(b), 4);
        }
        mbar_init(mma_done, 1);
        for (int s = 0; s < kTreeSlots; ++s) {
            mbar_init(unit_full(s), 1);
            mbar_init(unit_empty(s), 7);  // producer, MMA issuer, guard, 4 softmax warps
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(base + L::kTmemSlot, 512);
        tmem_relinquish();
    }
    // The set-up above overlaps the kernel before this one; its results are read from here on.
    // The merge is let go only now, so that what it reads before its own wait (offsets,
    // lengths) was written before this kernel.
    grid_dependency_wait();
    grid_launch_dependents();
    for (int s = threadIdx.x; s < p.n_seqs; s += kTreeThreads) {
        const TreeSeq q = tree_seq(p, s);
        seqs[s] = make_int2(q.T, q.L);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 3) {
        // -------------------------------------------------------- scheduler, and Q
        auto weight_of = [&](int s) -> int { return s < p.n_seqs ? tree_seq_weight<kWindow>(p, seqs[s].x, seqs[s].y) : 0; };
        auto scan = [&](int x) {  // inclusive prefix sum over the lanes
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            return x;
        };
        int total = 0;
        for (int s0 = 0; s0 < p.n_seqs; s0 += 32) {
            const int w = weight_of(s0 + lane);
            if (p.plan != nullptr && blockIdx.x == 0) {
                const int incl = scan(w);
                if (s0 + lane < p.n_seqs) p.plan[1 + s0 + lane] = total + incl - w;
            }
            total += __reduce_add_sync(0xffffffffu, w);
        }
        const int share = tree_share(p, total);
        if (lane == 0) {
            if (p.plan == nullptr)
                p.starts[blockIdx.x] = make_int4(0, 0, 0, 0);
            else if (blockIdx.x == 0)
                p.plan[0] = share;
        }
        // 64-bit: the last CTAs' first tiles may lie past the end
        const long long first = static_cast<long long>(blockIdx.x) * share;
        int at = first < total ? static_cast<int>(first) : total;
        const int end = first + share < total ? static_cast<int>(first + share) : total;
        int slot = 0, q_loads = 0, q_slot = 0;
        uint32_t phase = 0, emitted = 0, q_done = 0;  // units handed out, and Q tiles of them asked for
        int s0 = 0, before = 0;                       // weights of the sequences before s0
        bool ok = true, more = true;
        while (ok && (more || q_done < emitted)) {
            // A Q tile that is owed is asked for as soon as the buffer is free (the last scores of
            // the unit before are computed); until then further units are handed out, as far as
            // slots are free: one that is not depends on that tile.
            const bool owed = q_done < emitted;
            const bool q_ready = owed && __all_sync(0xffffffffu, mbar_try_wait(q_empty, (q_done & 1u) ^ 1u));
            if (!q_ready && more && (!owed || __all_sync(0xffffffffu, mbar_try_wait(unit_empty(slot), phase ^ 1u)))) {
                int seq = 0, nt = 0, unit = 0, k0 = 0, k1 = 0;
                while (at < end && k0 == k1) {
                    int in_seq = 0;
                    for (;; s0 += 32) {
                        const int w = weight_of(s0 + lane), all = __reduce_add_sync(0xffffffffu, w);
                        if (at < before + all) {
                            const int incl = scan(w);
                            const int src = __ffs(__ballot_sync(0xffffffffu, before + incl > at)) - 1;
                            seq = s0 + src;
                            in_seq = at - before - __shfl_sync(0xffffffffu, incl - w, src);
                            break;
                        }
                        before += all;
                    }
                    nt = tree_key_tiles<kWindow>(p, seqs[seq].x, seqs[seq].y);
                    const int uw = tree_unit_weight(nt);
                    unit = in_seq / uw;  // kv head * row tiles + row tile
                    // weights [0, uw - nt) of a unit are its change, then come its tiles; a share that
                    // ends within the change holds none of them
                    const int w0 = in_seq - unit * uw, w1 = w0 + (end - at) < uw ? w0 + (end - at) : uw;
                    k0 = w0 > uw - nt ? w0 - (uw - nt) : 0;
                    k1 = w1 > uw - nt ? w1 - (uw - nt) : 0;
                    at += w1 - w0;
                }
                more = k0 < k1;
                if (!(ok = __all_sync(0xffffffffu, wait_bar(unit_empty(slot), phase ^ 1u, p, abort_flag)))) break;
                TreeUnit &u = units[slot];
                if (more) {
                    const TreeSeq q = tree_seq(p, seq);
                    const int mt = tree_row_tiles(p, q.T), t0 = (unit % mt) * p.rt;
                    if (lane < kBad * 4) u.bad_rows[lane >> 2][lane & 3] = 0;
                    if (lane == 0) {
                        u.valid = 1;
                        u.t0 = t0;
                        u.q0 = q.q0 + t0;
                        u.ntok = q.T - t0 < p.rt ? q.T - t0 : p.rt;
                        u.T = q.T;
                        u.L = q.L;
                        u.base = tree_base(q.T, q.L);
                        u.row = q.row;
                        u.kvh = unit / mt;
                        u.k0 = k0;
                        u.k1 = k1;
                        u.piece = (k0 == 0 && k1 == nt) ? -1 : (k0 > 0 ? 0 : 1);
                        u.first = q.q0;
                        u.bad = 0;
                        // a unit that begins here and goes on in the next CTAs is merged
                        if (u.piece > 0 && p.plan == nullptr)
                            p.starts[blockIdx.x] = make_int4(u.q0, u.kvh << 8 | u.ntok, nt - k1, share);
                    }
                    ++emitted;
                } else if (lane == 0) {
                    u.valid = 0;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(unit_full(slot));
                if (++slot == kTreeSlots) {
                    slot = 0;
                    phase ^= 1u;
                }
            } else {
                if (!(ok = __all_sync(0xffffffffu, wait_bar(q_empty, (q_done & 1u) ^ 1u, p, abort_flag)))) break;
                if (!p.inject_stall) {
                    if (lane == 0) {
                        const TreeUnit &u = units[q_slot];
                        mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(p.group * p.rt) * D * 2);
#pragma unroll
                        for (int a = 0; a < D / 64; ++a)
                            tma_load_3d(sQ + a * kAtomBytes, &tmQ, 64 * a, u.kvh * p.group, u.q0, q_full);
                    }
                    ++q_loads;
                }
                ++q_done;
                if (++q_slot == kTreeSlots) q_slot = 0;
            }
        }
        if (lane == 0 && q_loads > 0) drain_bar(q_full, (q_loads - 1) & 1, p);  // landed before the CTA exits
        __syncwarp();
        if (ok && blockIdx.x == 0) {
            bool bad = false;
            for (int s = lane; s < p.n_seqs; s += 32) bad |= tree_seq(p, s).bad;
            if (bad) atomicCAS(&g_error_code, 0, static_cast<int>(ATTN_ERR_SHAPE));
        }
    } else if (warp == 2) {
        // -------------------------------------------------------- TMA producer
        constexpr int kAtoms = D / 64;
        const int box_rows = p.page < kBN ? p.page : kBN;
        const int boxes = (kBN / box_rows) * kAtoms;  // per tile
        const int oob = p.n_pages * p.Hkv;            // a box there reads as zeros
        // Page indexes: two windows of 32 entries, one entry per lane, so that the next
        // window is on its way while this one is used.  A tile's pages (128 / page of them,
        // from a multiple of that) never cross a window.
        struct Cur {
            int valid, row, kvh, k0, k1, pages;
            int win;           // first entry of window a; b holds the 32 after it
            int ent_a, ent_b;
            int skip;
        };
        // With an attention window the entries are those of the unit's steps, 128 / page (at least 1) of
        // each: entry i is that of page step_page(skip, i).
        const int per_tile = kBN / box_rows, per_shift = p.page < kBN ? 7 - p.page_shift : 0;
        auto step_page = [&](int skip, int i) -> int {
            if constexpr (!kWindow) return i;
            return ((win_key_tile<kWindow>(i >> per_shift, p.sinks, skip) << 7) >> p.page_shift) + (i & (per_tile - 1));
        };
        int slot = 0;
        uint32_t uphase = 0;
        auto entry = [&](const Cur &c, int i) -> int {
            const int x = step_page(c.skip, i);
            return c.row >= 0 && x < c.pages ? p.table[static_cast<long long>(c.row) * p.table_w + x] : -1;
        };
        auto take = [&](Cur &c) {  // the descriptor in the slot has arrived
            const TreeUnit &u = units[slot];
            c.valid = u.valid;
            if (c.valid) {
                c.row = u.row;
                c.kvh = u.kvh;
                c.k0 = u.k0;
                c.k1 = u.k1;
                c.pages = (u.L + p.page - 1) >> p.page_shift;
                c.skip = kWindow ? win_skip(u.base, p.window, p.sinks) : 0;
                c.win = (kWindow ? c.k0 << per_shift : (c.k0 << 7) >> p.page_shift) & ~31;
                c.ent_a = entry(c, c.win + lane);
                c.ent_b = entry(c, c.win + 32 + lane);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(unit_empty(slot));
            if (++slot == kTreeSlots) {
                slot = 0;
                uphase ^= 1u;
            }
        };
        int stage = 0, loads = 0;
        uint32_t phase = 0;
        Cur cur{}, nxt{};
        bool ok = __all_sync(0xffffffffu, wait_bar(unit_full(slot), uphase, p, abort_flag));
        if (ok) take(cur);
        // The order of the issuer: the first K tile, then for each key tile the K tile after it
        // (the next unit's first one, behind the last) and its V tile.
        bool lead = true;
        while (ok && cur.valid) {
            for (int kt = cur.k0; ok && kt < cur.k1; ++kt) {
#pragma unroll 1
                for (int h = lead ? -1 : 0; h < 2 && ok; ++h) {
                    // h = -1: the very first K tile, 0: the next K tile, 1: V
                    lead = false;
                    bool of_next = false;
                    int t = h == 0 ? kt + 1 : kt;
                    if (h == 0 && t == cur.k1) {
                        if (!(ok = __all_sync(0xffffffffu, wait_bar(unit_full(slot), uphase, p, abort_flag)))) break;
                        take(nxt);
                        if (!nxt.valid) continue;
                        of_next = true;
                        t = nxt.k0;
                    }
                    const int first = kWindow ? t << per_shift : (t << 7) >> p.page_shift;
                    // V is the last to use a window: the one after the next is fetched when V leaves it
                    if (h == 1 && first >= cur.win + 32) {
                        cur.win += 32;
                        cur.ent_a = cur.ent_b;
                        cur.ent_b = entry(cur, cur.win + 32 + lane);
                    }
                    if (!(ok = __all_sync(0xffffffffu, wait_bar(kv_empty(stage), phase ^ 1u, p, abort_flag)))) break;
                    const uint32_t dst = sKV + stage * L::kTileBytes;
                    if (lane == 0) mbar_arrive_expect_tx(kv_full(stage), L::kTileBytes);
                    __syncwarp();
                    // lane b issues box b: atom b % kAtoms of page piece b / kAtoms
                    const int piece = lane / kAtoms, a = lane % kAtoms;
                    const int at = first - (of_next ? nxt.win : cur.win) + piece;  // in [0, 64)
                    const int ea = __shfl_sync(0xffffffffu, of_next ? nxt.ent_a : cur.ent_a, at & 31);
                    const int eb = __shfl_sync(0xffffffffu, of_next ? nxt.ent_b : cur.ent_b, at & 31);
                    int e = at < 32 ? ea : eb;
                    if (lane < boxes) {
                        if (e < 0 || e >= p.n_pages) {
                            if (step_page(of_next ? nxt.skip : cur.skip, first + piece) < (of_next ? nxt.pages : cur.pages))
                                atomicCAS(&g_error_code, 0, static_cast<int>(ATTN_ERR_PAGE));
                            e = -1;
                        }
                        tma_load_3d(dst + a * kAtomBytes + piece * box_rows * 128, h == 1 ? &tmV : &tmK, 64 * a,
                                    (win_key_tile<kWindow>(t, p.sinks, of_next ? nxt.skip : cur.skip) << 7) & (p.page - 1),
                                    e < 0 ? oob : e * p.Hkv + (of_next ? nxt.kvh : cur.kvh),
                                    kv_full(stage));
                    }
                    ++loads;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            cur = nxt;
        }
        if (lane == 0) {
            // every copy has landed before the CTA exits (also after a timeout)
#pragma unroll
            for (int st = 0; st < S; ++st)
                if (loads > st) drain_bar(kv_full(st), st < stage ? phase : phase ^ 1u, p);
        }
        __syncwarp();
    } else if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------------- MMA issuer
            const uint32_t dq = desc_lo(sQ, 16), dk0 = desc_lo(sKV, 16), dv0 = desc_lo(sKV, kAtomBytes);
            constexpr uint32_t kTile16 = L::kTileBytes >> 4;
            int stage = 0, slot = 0;
            uint32_t phase = 0, uphase = 0, jj = 0, pj = 0;  // scores issued, P V issued
            uint32_t qn = 0, un = 0, vph = 0;                // Q tiles, units, phases of v_ok
            struct Cur {
                int valid, k0, k1, guard;
                WinWhole w;  // with a window: all but these tiles pass the guard
            };
            auto fetch = [&](Cur &c) -> bool {
                if (!wait_bar(unit_full(slot), uphase, p, abort_flag)) return false;
                const TreeUnit &u = units[slot];
                c.valid = u.valid;
                if (c.valid) {
                    c.k0 = u.k0;
                    c.k1 = u.k1;
                    if constexpr (kWindow) c.w = tree_whole(p, u.T, u.base);
                    else c.guard = u.base / kBN;  // tiles from here on pass the guard
                }
                mbar_arrive(unit_empty(slot));
                if (++slot == kTreeSlots) {
                    slot = 0;
                    uphase ^= 1u;
                }
                return true;
            };
            // Per key tile: the scores of the tile after it (the next unit's first one, behind the
            // last), then its P V; before the first unit a step without P V.
            Cur cur{1, 0, 1, 0, {0, 0, 0}}, nxt{};
            bool ok = true, start = true;
            while (ok && cur.valid) {
                for (int kt = cur.k0; kt < cur.k1; ++kt) {
                    const bool last = kt + 1 == cur.k1;
                    if (last && !(ok = fetch(nxt))) break;
                    if (!last || nxt.valid) {
                        if (last && !(ok = wait_bar(q_full, qn++ & 1u, p, abort_flag))) break;
                        if (!(ok = wait_bar(kv_full(stage), phase, p, abort_flag))) break;
                        tc_fence_after();
                        const uint32_t b = jj++ & 1u;
                        mma_qk<D, kBF16>(tmem + 128u * b, dq, dk0 + stage * kTile16);
                        mma_commit(s_full(b));
                        mma_commit(kv_empty(stage));
                        // the unit's last scores: Q may be replaced
                        if (last ? nxt.k0 + 1 == nxt.k1 : kt + 2 == cur.k1) mma_commit(q_empty);
                        if (++stage == S) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (start) break;
                    // O (+)= P_b V: P from TMEM (first 64 columns of S_b), V MN-major; a unit's first
                    // one waits until the O of the unit before the last has been read
                    const uint32_t b = pj & 1u, ob = un & 1u;
                    if (!(ok = wait_bar(kv_full(stage), phase, p, abort_flag))) break;
                    if (kWindow ? !cur.w(kt) : kt >= cur.guard) {
                        if (!(ok = wait_bar(v_ok(stage), (vph >> stage) & 1u, p, abort_flag))) break;
                        vph ^= 1u << stage;
                    }
                    if (kt == cur.k0 && !(ok = wait_bar(o_empty(ob), ((un >> 1) & 1u) ^ 1u, p, abort_flag))) break;
                    if (!(ok = wait_bar(p_full(b), (pj >> 1) & 1u, p, abort_flag))) break;
                    tc_fence_after();
                    mma_pv<D, kBF16>(tmem + 256u + 128u * ob, tmem + 128u * b, dv0 + stage * kTile16, kt > cur.k0 ? 1u : 0u);
                    mma_commit(o_done(b));
                    mma_commit(kv_empty(stage));
                    ++pj;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!start) ++un;
                start = false;
                cur = nxt;
            }
            mma_commit(mma_done);
            drain_bar(mma_done, 0, p);
        }
        __syncwarp();
    } else if (warp == 1) {
        // -------------------------------------------------------- value guard
        // The guard sees every tile arrive, in the producer's order, and a stage is loaded again
        // only after the guard, too, has released it: it never misses a phase, and it looks at
        // V tiles several tiles before their product.
        int slot = 0, stage = 0;
        uint32_t uphase = 0, phase = 0;
        bool ok = true;
        auto fetch = [&](int &held) -> bool {
            if (!__all_sync(0xffffffffu, wait_bar(unit_full(slot), uphase, p, abort_flag))) return false;
            held = slot;
            if (++slot == kTreeSlots) {
                slot = 0;
                uphase ^= 1u;
            }
            return true;
        };
        // the next tile: waits for it, lets the guard work on a V tile (key tile kt, the g-th guarded one of
        // the unit), releases the stage
        auto pass = [&](TreeUnit *u, int kt, int g) -> bool {
            if (!__all_sync(0xffffffffu, wait_bar(kv_full(stage), phase, p, abort_flag))) return false;
            if (u != nullptr) {
                int left = u->L - kt * kBN;
                left = left < 0 ? 0 : (left < kBN ? left : kBN);
                // a token alone sees the keys outside [z0, z1) of a tile on the window's border, as all its heads do
                // (rows of the tile, whatever the window is: the guard multiplies them)
                int z0 = 0, z1 = 0;
                if (kWindow && u->T <= 1) {
                    z0 = p.sinks - kt * kBN;
                    z1 = u->base - p.window + 1 - kt * kBN;
                    z0 = z0 < 0 ? 0 : (z0 < kBN ? z0 : kBN);
                    z1 = z1 < 0 ? 0 : (z1 < kBN ? z1 : kBN);
                }
                const bool any = vl_guard_tile<D, kBF16>(smem + L::kKV + stage * L::kTileBytes, left, u->T > 1,
                                                         u->bad_rows[g & (kBad - 1)], lane, z0, z1);
                if (any && lane == 0) u->bad = 1;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(v_ok(stage));
            }
            if (lane == 0) mbar_arrive(kv_empty(stage));
            if (++stage == S) {
                stage = 0;
                phase ^= 1u;
            }
            return true;
        };
        int cur = 0, nxt = 0;
        ok = fetch(cur) && (!units[cur].valid || pass(nullptr, 0, 0));
        while (ok && units[cur].valid) {
            TreeUnit &u = units[cur];
            const int k1 = u.k1, guard = u.base / kBN, skip = kWindow ? win_skip(u.base, p.window, p.sinks) : 0;
            const WinWhole w = kWindow ? tree_whole(p, u.T, u.base) : WinWhole{};
            int g = 0;
#pragma unroll 1
            for (int kt = u.k0; ok && kt < k1; ++kt) {
                if (kt + 1 == k1) ok = fetch(nxt);
                if (ok && (kt + 1 < k1 || units[nxt].valid)) ok = pass(nullptr, 0, 0);
                if constexpr (kWindow) {
                    const bool look = !w(kt);
                    ok = ok && pass(look ? &u : nullptr, win_key_tile<kWindow>(kt, p.sinks, skip), g);
                    g += look ? 1 : 0;
                } else {
                    ok = ok && pass(kt >= guard ? &u : nullptr, kt, kt - guard);
                }
            }
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(unit_empty(cur));
            cur = nxt;
        }
    } else {
        // -------------------------------------------------------- softmax rows
        const int wq = warp & 3;
        const int r = wq * 32 + lane;  // row within the tile == TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        const float c = p.scale_log2;
        const int tok = r / p.group;  // token within the row tile
        int *par = reinterpret_cast<int *>(smem + L::kPar) + wq * kTreeMax;
        int slot = -1, done_slot = -1;  // the unit at work, and the one whose O is still to be stored
        uint32_t uphase = 1, jj = 0, un = 0;  // tiles and units so far
        int kt = 0, k0 = 0, k1 = 0, tree0 = 0;
        bool valid = false, active = false, more = true;  // this row is real; some row of this warp is
        Bits128 anc{0ull, 0ull};
        int pos = 0, skip = 0;  // with a window: this row's position, key tiles left out, tiles seen whole
        WinWhole seen_whole{};
        float mrow = -INFINITY, l = 0.f, done_m = 0.f, done_l = 0.f;
        while (true) {
            if (kt == k1) {
                // the next unit; the one before has its last weights handed over
                done_slot = slot;
                done_m = mrow;
                done_l = l;
                if (++slot == kTreeSlots) slot = 0;
                if (slot == 0) uphase ^= 1u;
                if (!__all_sync(0xffffffffu, wait_bar(unit_full(slot), uphase, p, abort_flag))) break;
                const TreeUnit &u = units[slot];
                more = u.valid != 0;
                k0 = k1 = kt = 0;
                if (more) {
                    k0 = kt = u.k0;
                    k1 = u.k1;
                    tree0 = u.base;
                    valid = tok < u.ntok && tok < p.rt;
                    active = wq * 32 < u.ntok * p.group;
                    anc.lo = 1ull;
                    anc.hi = 0ull;
                    if (u.T > 1) {
                        // the tree's parents (without: a chain), a copy for each warp
#pragma unroll 1
                        for (int t = lane; t < u.T && t < kTreeMax; t += 32)
                            par[t] = p.parents != nullptr ? p.parents[u.first + t] : t - 1;
                        __syncwarp();
                        if (!kWindow && valid) anc = tree_ancestors(u.t0 + tok, [&](int t) { return par[t]; });
                    }
                    if constexpr (kWindow) {
                        seen_whole = tree_whole(p, u.T, u.base);
                        skip = win_skip(u.base, p.window, p.sinks);
                        int depth = 0;
                        if (u.T > 1 && valid)
                            anc = tree_window(u.t0 + tok, u.base, p.window, p.sinks, depth, [&](int t) { return par[t]; });
                        pos = u.base + depth;
                    }
                    ++un;
                }
                mrow = -INFINITY;
                l = 0.f;
            }
            const uint32_t ob = (un - 1) & 1u;  // O buffer of the unit at work
            if (kt < k1) {
                const uint32_t b = jj & 1u;
                if (!__all_sync(0xffffffffu, wait_bar(s_full(b), (jj >> 1) & 1u, p, abort_flag))) break;
                if (active) {
                    tc_fence_after();
                    __syncwarp();
                    const uint32_t tS = tmem + 128u * b + lane_off, tO = tmem + 256u + 128u * ob + lane_off;
                    // 32 columns at a time, in two passes over TMEM (the row's max, then its
                    // weights): a quarter of the instructions of one pass over 128 columns in
                    // registers, which together with the epilogue's did not stay in the instruction
                    // cache (the first tile after an epilogue took 4700 cycles instead of 1200).
                    const bool whole = kWindow ? seen_whole(kt) : (kt + 1) * kBN <= tree0;  // every row sees every key
                    uint32_t w[4] = {~0u, ~0u, ~0u, ~0u};  // bit c: this row sees key c of the tile
                    if (!whole) {
                        const int key0 = win_key_tile<kWindow>(kt, p.sinks, skip) * kBN;
                        const int sh = key0 - tree0;
                        Bits128 see = sh >= 0 ? bits_shr(anc, sh) : bits_shl(anc, -sh);
                        Bits128 old = bits_below(-sh);
                        if constexpr (kWindow) {
                            const Bits128 gone = bits_below(pos - p.window + 1 - key0), sink = bits_below(p.sinks - key0);
                            old.lo &= ~gone.lo | sink.lo;
                            old.hi &= ~gone.hi | sink.hi;
                        }
                        see.lo |= old.lo;
                        see.hi |= old.hi;
                        w[0] = static_cast<uint32_t>(see.lo);
                        w[1] = static_cast<uint32_t>(see.lo >> 32);
                        w[2] = static_cast<uint32_t>(see.hi);
                        w[3] = static_cast<uint32_t>(see.hi >> 32);
                    }
                    float mt = -INFINITY;
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t s[32];
                        if (whole) {
                            float mq[1];
                            tmem_ld32_max(tS + 32 * q, s, mq[0]);
                            tmem_ld_wait(s, mq);
                            mt = fmaxf(mt, mq[0]);
                        } else {
                            tmem_ld32(tS + 32 * q, s);
                            tmem_ld_wait(s);
                            const uint32_t wq32 = q == 0 ? w[0] : q == 1 ? w[1] : q == 2 ? w[2] : w[3];
                            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                mx[e & 1] = fmaxf(mx[e & 1], (wq32 >> e) & 1u ? u2f(s[e]) : -INFINITY);
                            mt = fmax3(mt, mx[0], mx[1]);
                        }
                    }
                    // The weights are taken against a stale max (mrow) until the true one is 2^8 above
                    // it: a rescale waits for the P V before, and on fresh rows the max grows in most
                    // of the first tiles.  Rows without a token ask for none.
                    float alpha = 1.f;
                    bool rescale = false;
                    if (mrow == -INFINITY) {
                        mrow = mt;  // nothing seen so far: the accumulator holds zeros at most
                    } else if (valid && (mt - mrow) * c > kRescaleLog2) {
                        alpha = ex2_approx((mrow - mt) * c);
                        mrow = mt;
                        rescale = true;
                    }
                    // a row that has seen no key yet takes its weights, all 0, against 0
                    const float m_use = mrow == -INFINITY ? 0.f : mrow;
                    if (__any_sync(0xffffffffu, rescale)) {
                        // rescale O: the P V before must have finished writing it
                        if (!__all_sync(0xffffffffu,
                                        wait_bar(o_done((jj - 1) & 1u), ((jj - 1) >> 1) & 1u, p, abort_flag)))
                            break;
                        tc_fence_after();
                        __syncwarp();
#pragma unroll 1
                        for (int q = 0; q < D / 32; ++q) {
                            uint32_t o[32];
                            tmem_ld32(tO + 32 * q, o);
                            tmem_ld_wait(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(u2f(o[e]) * alpha);
                            tmem_st32(tO + 32 * q, o);
                        }
                    }
                    const float2 c2 = make_float2(c, c);
                    const float2 nmc2 = make_float2(-m_use * c, -m_use * c);
                    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    // P (16 columns of pairs) overwrites scores that have been read
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t s[32];
                        tmem_ld32(tS + 32 * q, s);
                        tmem_ld_wait(s);
                        if (!whole) {
                            const uint32_t wq32 = q == 0 ? w[0] : q == 1 ? w[1] : q == 2 ? w[2] : w[3];
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!((wq32 >> e) & 1u)) s[e] = __float_as_uint(-INFINITY);
                        }
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float2 x = ffma2(make_float2(u2f(s[2 * e]), u2f(s[2 * e + 1])), c2, nmc2);
                            x.x = ex2_approx(x.x);
                            x.y = ex2_approx(x.y);
                            acc[e & 1] = fadd2(acc[e & 1], x);
                            pk[e] = pack2<kBF16>(x.x, x.y);
                        }
                        tmem_st16(tS + 16 * q, pk);
                    }
                    const float2 sum2 = fadd2(acc[0], acc[1]);
                    l = l * alpha + (sum2.x + sum2.y);
                    tmem_st_wait();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(b));
                ++jj;
                ++kt;
            }
            if (done_slot >= 0) {
                // ------------------------------------------------ O of the unit before
                // Its last tile is the one before the unit at work has begun: one tile back, or
                // none where no unit is left.
                const uint32_t last = jj - 1 - (more ? 1u : 0u), db = more ? ob ^ 1u : ob;
                if (!__all_sync(0xffffffffu, wait_bar(o_done(last & 1u), (last >> 1) & 1u, p, abort_flag))) break;
                const TreeUnit &u = units[done_slot];
                if (wq * 32 < u.ntok * p.group) {
                    tc_fence_after();
                    __syncwarp();
                    const uint32_t tO = tmem + 256u + 128u * db + lane_off;
                    const bool real = tok < u.ntok && tok < p.rt;
                    const float inv_l = done_l == 0.f ? 0.f : 1.f / done_l;  // 0: the row saw no key
                    const float lse = done_l == 0.f ? -INFINITY : (done_m * c + log2f(done_l)) * 0.6931471805599453f;
                    const int head = u.kvh * p.group + (r - tok * p.group);
                    const long long tok_row = u.q0 + tok;
                    uint8_t *orow = static_cast<uint8_t *>(p.o) + tok_row * p.o_row + head * p.o_head;
                    const size_t prow = (static_cast<size_t>(blockIdx.x) * 2 + (u.piece > 0 ? 1 : 0)) * kBM + r;
                    float *part = p.part_o + prow * D;
                    const bool whole = u.piece < 0;
#pragma unroll 1
                    for (int q = 0; q < D / 32; ++q) {
                        uint32_t o[32];
                        tmem_ld32(tO + 32 * q, o);
                        tmem_ld_wait(o);
                        if (!real) continue;
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(u2f(o[e]) * inv_l);
                        if (!whole) {
#pragma unroll
                            for (int v = 0; v < 8; ++v)
                                st_global_v4(part + q * 32 + v * 4, o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
                        } else {
                            uint32_t w[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) w[e] = pack2<kBF16>(u2f(o[2 * e]), u2f(o[2 * e + 1]));
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                st_global_v4(orow + q * 64 + v * 16, w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
                        }
                    }
                    if (real) {
                        if (!whole)
                            p.part_lse[prow] = lse;
                        else if (p.lse != nullptr)
                            p.lse[static_cast<size_t>(head) * p.total_q + tok_row] = lse;
                        if (*reinterpret_cast<const volatile int *>(&u.bad) != 0) {
                            // non-finite values that the guard took out of V, for the rows that see them:
                            // added to the stored row, whose other values they do not change
                            auto up = [&](int t) -> int {
                                return p.parents != nullptr && t < u.T ? p.parents[u.first + t] : t - 1;
                            };
                            int depth = 0;
                            Bits128 seen{1ull, 0ull};
                            if (u.T > 1)
                                seen = kWindow ? tree_window(u.t0 + tok, u.base, p.window, p.sinks, depth, up)
                                               : tree_ancestors(u.t0 + tok, up);
                            const WinWhole w = kWindow ? tree_whole(p, u.T, u.base) : WinWhole{};
                            const int win_skipped = kWindow ? win_skip(u.base, p.window, p.sinks) : 0;
                            int step = u.k0 - 1, tile0 = 0;  // with a window: guarded tile g >> 2, its first key
#pragma unroll 1
                            for (int g = 0; g < kBad * 4; ++g) {
                                if (kWindow && (g & 3) == 0) {
                                    do ++step; while (w(step));
                                    tile0 = win_key_tile<kWindow>(step, p.sinks, win_skipped) * kBN;
                                }
#pragma unroll 1
                                for (uint32_t bits = u.bad_rows[g >> 2][g & 3]; bits != 0; bits &= bits - 1) {
                                    const int key = (kWindow ? tile0 + 32 * (g & 3) : u.base / kBN * kBN + 32 * g) +
                                                    __ffs(bits) - 1;
                                    const int node = key - u.base;
                                    if (kWindow && node < 0 && key <= u.base + depth - p.window && key >= p.sinks) continue;
                                    if (node >= 0 && !((node < 64 ? seen.lo >> node : seen.hi >> (node - 64)) & 1ull))
                                        continue;
                                    const int pg = p.table[static_cast<long long>(u.row) * p.table_w + (key >> p.page_shift)];
                                    const uint8_t *vr = p.v_ptr + ((static_cast<size_t>(pg) * p.Hkv + u.kvh) * p.page +
                                                                   (key & (p.page - 1))) * (D * 2);
                                    if (whole)
                                        add_nonfinite<D, kBF16>(orow, vr);
                                    else
                                        add_nonfinite_f32<D, kBF16>(part, vr);
                                }
                            }
                        }
                    }
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(o_empty(db));
                    mbar_arrive(unit_empty(done_slot));
                }
                done_slot = -1;
            }
            if (!more) break;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Merges the pieces of row prow of a unit that begins in slot 1 of CTA c0 and ends in slot 0 of
// CTA c1: lse = log sum_s exp(lse_s) and O = sum_s exp(lse_s - lse) O_s (the online-softmax update
// of page "从零开始写Qwen3", deepseek.csdn.net/6a3201f8..., section "在线softmax", across CTAs).
// One round trip brings the log-sum-exps (lane j: piece j) and the rows of 8 pieces.
template <int D, bool kBF16>
__device__ __forceinline__ void tree_merge_row(const TreeParams &p, int c0, int c1, int prow, int tok, int head, int lane) {
    constexpr int kPer = D / 32;
    // where the kernel before gave up on a wait, its pieces may be stale: NaN
    const bool gave_up = *reinterpret_cast<volatile unsigned int *>(&g_abort_seq) == p.seq;
    // CTA c0's piece begins at the unit's start (slot 1), the others in mid-unit (slot 0)
    auto row_of = [&](int c) { return (static_cast<size_t>(c) * 2 + (c == c0 ? 1 : 0)) * kBM + prow; };
    float acc[kPer];
#pragma unroll
    for (int d = 0; d < kPer; ++d) acc[d] = 0.f;
    float mx = -INFINITY, sum = 0.f;
#pragma unroll 1
    for (int s0 = c0; s0 <= c1; s0 += 8) {
        const float ls = lane < 8 && s0 + lane <= c1 ? p.part_lse[row_of(s0 + lane)] : -INFINITY;
        float v[8][kPer];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float *src = p.part_o + row_of(s0 + j <= c1 ? s0 + j : c1) * D + lane * kPer;
            if constexpr (kPer == 4)
                *reinterpret_cast<float4 *>(v[j]) = *reinterpret_cast<const float4 *>(src);
            else
                *reinterpret_cast<float2 *>(v[j]) = *reinterpret_cast<const float2 *>(src);
        }
        float bm = ls;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
        bm = __shfl_sync(0xffffffffu, bm, 0);
        const float m_new = fmaxf(mx, bm);
        const float old = mx == -INFINITY ? 0.f : expf(mx - m_new);
        const float wl = ls == -INFINITY ? 0.f : expf(ls - m_new);
        sum = sum * old + wl;  // of this lane's pieces
        mx = m_new;
        // A weight (and a rebasing factor) that underflows to 0 drops the finite values of its piece
        // only: an infinity or NaN there is one of a key that the row sees, and stays.
#pragma unroll
        for (int d = 0; d < kPer; ++d) acc[d] = old != 0.f || isfinite(acc[d]) ? acc[d] * old : acc[d];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float w = __shfl_sync(0xffffffffu, wl, j);
            if (s0 + j > c1) continue;
            if (w != 0.f) {
#pragma unroll
                for (int d = 0; d < kPer; ++d) acc[d] += w * v[j][d];
            } else {
#pragma unroll
                for (int d = 0; d < kPer; ++d)
                    if (!isfinite(v[j][d])) acc[d] += v[j][d];
            }
        }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    sum = __shfl_sync(0xffffffffu, sum, 0);
    const float inv = gave_up ? __int_as_float(0x7FC00000) : (sum == 0.f ? 0.f : 1.f / sum);  // 0: the row saw no key
    uint8_t *dst = static_cast<uint8_t *>(p.o) + tok * p.o_row + head * p.o_head + lane * kPer * 2;
    uint32_t w[kPer / 2];
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) w[i] = pack2<kBF16>(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    if constexpr (kPer == 4)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    else
        *reinterpret_cast<uint32_t *>(dst) = w[0];
    if (p.lse != nullptr && lane == 0)
        p.lse[static_cast<size_t>(head) * p.total_q + tok] =
            gave_up ? __int_as_float(0x7FC00000) : (sum == 0.f ? -INFINITY : mx + logf(sum));
}

// The cut units, a warp per output row: a row whose unit lay in one share has been written already.
// The row's sequence is looked for before the wait for the kernel before; after it comes the plan.
// (Adding the plan up here before the wait, too, saves 0.3 us of 11 with one sequence and nothing
// with 16.)
template <int D, bool kBF16, bool kWindow>
__global__ void __launch_bounds__(32) attn_tree_merge_kernel(const __grid_constant__ TreeParams p) {
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, R = static_cast<int>(blockIdx.x);
    const int tok = R / p.Hq, head = R - tok * p.Hq;
    // the sequence of this token: the last one that starts at or before it
    int lo = 0, hi = p.n_seqs;  // cu[lo] <= tok < cu[hi], where the offsets ascend
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (ld_ahead_of_wait(p.cu + mid) <= tok) lo = mid; else hi = mid;
    }
    const TreeSeq q = tree_seq<true>(p, lo);
    const int nt = tree_key_tiles<kWindow>(p, q.T, q.L), mt = tree_row_tiles(p, q.T), uw = tree_unit_weight(nt);
    const int t = tok - q.q0, m = t / p.rt;
    const int prow = (t - m * p.rt) * p.group + head % p.group;  // row within the tile
    grid_dependency_wait();
    if (t < 0 || t >= q.T) return;
    const int share = p.plan[0], before = p.plan[1 + lo];
    // the weight past the unit's last tile, and the CTAs of its first and last one
    const int end = before + ((head / p.group) * mt + m + 1) * uw;
    const int c0 = (end - nt) / share, c1 = (end - 1) / share;
    // (lengths that changed since the kernel before, against the rules, must not lead outside)
    if (c0 >= c1 || c0 < 0 || c1 >= p.grid) return;
    tree_merge_row<D, kBF16>(p, c0, c1, prow, tok, head, lane);
}

// The same by CTAs, of which each has left what its slot 1 holds; the blocks of one CTA go to
// different SMs.
template <int D, bool kBF16>
__global__ void __launch_bounds__(kMergeCtaThreads) attn_tree_merge_ctas_kernel(const __grid_constant__ TreeParams p) {
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = static_cast<int>(blockIdx.x) / p.grid, c0 = (static_cast<int>(blockIdx.x) + 37 * g) % p.grid;
    grid_dependency_wait();
    const int4 unit = p.starts[c0];
    const int row0 = g * kMergeCtaRows, rows = (unit.y & 255) * p.group, kvh = unit.y >> 8;
    if (row0 >= rows) return;
    const int c1 = c0 + 1 + (unit.z - 1) / unit.w;
#pragma unroll 1
    for (int r = row0 + warp; r < row0 + kMergeCtaRows && r < rows; r += kMergeCtaThreads / 32) {
        const int t = r / p.group;
        tree_merge_row<D, kBF16>(p, c0, c1, r, unit.x + t, kvh * p.group + (r - t * p.group), lane);
    }
}

}  // namespace gqa
