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
//     CTA takes an equal contiguous share, whatever the lengths are.  A unit cut by a share's
//     border leaves at most two pieces per CTA (fp32 O and log-sum-exp), merged by a second,
//     dependent launch; the others write O themselves;
//   * the load order runs on across the units of a share (the next unit's first K tile is
//     loaded, and its scores computed, before the last P V of the unit before).
//
// Roles (256 threads): warp 0 MMA issuer, warp 1 value guard (and TMEM), warp 2 TMA producer
// (the lanes issue one page box each), warp 3 scheduler, warps 4-7 softmax (one row per
// thread).  P stays in TMEM over its scores.  TMEM: S0 [0,128), S1 [128,256), O [256,256+D).
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
constexpr int kTreeSlots = 4;
constexpr int kTreeMax = 128;      // tokens of one tree
constexpr int kTreeSeqCache = 512; // sequences whose lengths are kept in shared memory
constexpr int kTreeBadTiles = 2;   // the tree's positions lie in at most two key tiles

struct TreeParams : Params {
    const int *cu, *table, *lens, *seqs, *parents;
    const uint8_t *v_ptr;
    int n_seqs, total_q, Hq, Hkv, n_rows;  // n_rows: rows of the page table
    int page, page_shift, n_pages, table_w;
    int rt;                    // tokens per row tile: 128 / group
    int min_share;             // least number of key tiles per CTA
    long long o_row, o_head;   // strides in bytes
    float *part_o;             // [2 * CTAs][128][D]
    float *part_lse;           // [2 * CTAs][128]
    int *plan;                 // [0]: share, [1 + s]: first tile of sequence s
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
    int bad;
    uint32_t bad_rows[kTreeBadTiles][4];
    int par[kTreeMax];  // parents (-1: child of the last position before the tree)
};

template <int D>
struct TreeLayout {
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kTileBytes = (D / 64) * kAtomBytes;
    static constexpr int kQ = 0;
    static constexpr int kKV = kQ + kTileBytes;
    static constexpr int kBar = kKV + kStages * kTileBytes;
    // q_full, q_empty, kv_full[S], kv_empty[S], s_full[2], p_full[2], o_done[2], mma_done, v_ask,
    // v_ok, unit_full[slots], unit_empty[slots]
    static constexpr int kNumBars = 2 + 2 * kStages + 2 + 2 + 2 + 3 + 2 * kTreeSlots;
    static constexpr int kTmemSlot = kBar + kNumBars * 8;
    static constexpr int kAbort = kTmemSlot + 4;
    static constexpr int kAsk = kAbort + 4;
    static constexpr int kUnits = (kAsk + 4 + 15) & ~15;
    static constexpr int kSeqs = (kUnits + kTreeSlots * static_cast<int>(sizeof(TreeUnit)) + 7) & ~7;
    static constexpr int kUsed = kSeqs + kTreeSeqCache * 8;
    // more than half of an SM's shared memory: one CTA (all 512 TMEM columns) per SM
    static constexpr int kAlloc = (kUsed + 1024) > 118 * 1024 ? (kUsed + 1024) : 118 * 1024;
};
static_assert(TreeLayout<128>::kAlloc <= 227 * 1024 && TreeLayout<64>::kAlloc <= 227 * 1024, "shared memory of one CTA");

// Tokens and positions of sequence s, clamped to what the tensors hold.
struct TreeSeq {
    int q0, T, L, row;
    bool bad;
};
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams &p, int s) {
    const VlSpan q = vl_span(p.cu, s, p.total_q);
    int row = p.seqs != nullptr ? __ldg(p.seqs + s) : s;
    TreeSeq r{q.a, q.b - q.a, 0, row, q.bad};
    if (row < 0 || row >= p.n_rows) {
        r.row = -1;
        r.bad = true;
    } else {
        r.L = __ldg(p.lens + row);
    }
    const long long cap = static_cast<long long>(p.table_w) << p.page_shift;
    if (r.L < 0) r.L = 0, r.bad = true;
    if (r.L > cap) r.L = static_cast<int>(cap), r.bad = true;
    if (r.T > kTreeMax || r.T > r.L) r.bad |= r.T > 0;
    return r;
}
__device__ __forceinline__ int tree_row_tiles(const TreeParams &p, int T) { return (T + p.rt - 1) / p.rt; }
__device__ __forceinline__ int tree_key_tiles(int L) { return L > 0 ? (L + kBN - 1) / kBN : 1; }

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

// tmQ: 3-D tensor map (D, Hq, tokens), box 64 x G x (128 / G); tmK, tmV: 3-D maps
// (D, page, n_pages * Hkv), box 64 x min(page, 128) x 1; all with the 128-byte swizzle.
template <int D, bool kBF16>
__global__ void __launch_bounds__(kTreeThreads, 1)
    attn_fwd_tree_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TreeParams p) {
    using L = TreeLayout<D>;
    constexpr int S = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const uint32_t sQ = base + L::kQ, sKV = base + L::kKV;
    const uint32_t bar0 = base + L::kBar;
    const uint32_t q_full = bar0, q_empty = bar0 + 8u;
    auto kv_full = [&](int s) { return bar0 + 8u * (2 + s); };
    auto kv_empty = [&](int s) { return bar0 + 8u * (2 + S + s); };
    auto s_full = [&](int b) { return bar0 + 8u * (2 + 2 * S + b); };
    auto p_full = [&](int b) { return bar0 + 8u * (4 + 2 * S + b); };
    auto o_done = [&](int b) { return bar0 + 8u * (6 + 2 * S + b); };
    const uint32_t mma_done = bar0 + 8u * (8 + 2 * S);
    const uint32_t v_ask = bar0 + 8u * (9 + 2 * S), v_ok = bar0 + 8u * (10 + 2 * S);
    auto unit_full = [&](int s) { return bar0 + 8u * (11 + 2 * S + s); };
    auto unit_empty = [&](int s) { return bar0 + 8u * (11 + 2 * S + kTreeSlots + s); };
    volatile int *ask = reinterpret_cast<volatile int *>(smem + L::kAsk);
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + L::kTmemSlot);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kAbort);
    TreeUnit *units = reinterpret_cast<TreeUnit *>(smem + L::kUnits);
    int2 *seqs = reinterpret_cast<int2 *>(smem + L::kSeqs);  // (T, L)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    grid_launch_dependents();
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
            mbar_init(kv_empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(s_full(b), 1);
            mbar_init(p_full(b), 4);
            mbar_init(o_done(b), 1);
        }
        mbar_init(mma_done, 1);
        mbar_init(v_ask, 1);
        mbar_init(v_ok, 1);
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
    // the set-up above overlaps the kernel before this one; its results are read from here on
    grid_dependency_wait();
    for (int s = threadIdx.x; s < p.n_seqs && s < kTreeSeqCache; s += kTreeThreads) {
        const TreeSeq q = tree_seq(p, s);
        seqs[s] = make_int2(q.T, q.L);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 3) {
        // -------------------------------------------------------- scheduler
        auto tiles_of = [&](int s) -> int {
            if (s >= p.n_seqs) return 0;
            int T, Ls;
            if (s < kTreeSeqCache) {
                T = seqs[s].x;
                Ls = seqs[s].y;
            } else {
                const TreeSeq q = tree_seq(p, s);
                T = q.T;
                Ls = q.L;
            }
            return p.Hkv * tree_row_tiles(p, T) * tree_key_tiles(Ls);
        };
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
            const int w = tiles_of(s0 + lane), incl = scan(w);
            if (blockIdx.x == 0 && s0 + lane < p.n_seqs) p.plan[1 + s0 + lane] = total + incl - w;
            total += __shfl_sync(0xffffffffu, incl, 31);
        }
        int share = (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
        if (share < p.min_share) share = p.min_share;
        if (blockIdx.x == 0 && lane == 0) p.plan[0] = share;
        // 64-bit: the last CTAs' first tiles may lie past the end
        const long long first = static_cast<long long>(blockIdx.x) * share;
        int at = first < total ? static_cast<int>(first) : total;
        const int end = first + share < total ? static_cast<int>(first + share) : total;
        int slot = 0;
        uint32_t phase = 0;
        int s0 = 0, before = 0;  // tiles of the sequences before s0
        bool ok = true;
        for (;;) {
            const bool more = at < end;
            int seq = 0, in_seq = 0;
            if (more) {
                for (;; s0 += 32) {
                    const int w = tiles_of(s0 + lane), incl = scan(w);
                    const int all = __shfl_sync(0xffffffffu, incl, 31);
                    if (at < before + all) {
                        const int src = __ffs(__ballot_sync(0xffffffffu, before + incl > at)) - 1;
                        seq = s0 + src;
                        in_seq = at - before - __shfl_sync(0xffffffffu, incl - w, src);
                        break;
                    }
                    before += all;
                }
            }
            if (!__all_sync(0xffffffffu, wait_bar(unit_empty(slot), phase ^ 1u, p, abort_flag))) {
                ok = false;
                break;
            }
            TreeUnit &u = units[slot];
            if (more) {
                const TreeSeq q = tree_seq(p, seq);
                const int nt = tree_key_tiles(q.L), mt = tree_row_tiles(p, q.T);
                const int unit = in_seq / nt, k0 = in_seq - unit * nt;  // unit = kv head * row tiles + row tile
                const int k1 = k0 + (end - at) < nt ? k0 + (end - at) : nt;
                const int m = unit % mt;
                const int T = q.T < kTreeMax ? q.T : kTreeMax;
                for (int t = lane; t < kTreeMax; t += 32) {
                    int par = t - 1;  // no parents: a chain
                    if (p.parents != nullptr && t < T) par = __ldg(p.parents + q.q0 + t);
                    u.par[t] = par;
                }
                if (lane < kTreeBadTiles * 4) u.bad_rows[lane >> 2][lane & 3] = 0;
                if (lane == 0) {
                    u.valid = 1;
                    u.t0 = m * p.rt;
                    u.q0 = q.q0 + u.t0;
                    u.ntok = q.T - u.t0 < p.rt ? q.T - u.t0 : p.rt;
                    u.T = q.T;
                    u.L = q.L;
                    u.base = q.L > q.T ? q.L - q.T : 0;
                    u.row = q.row;
                    u.kvh = unit / mt;
                    u.k0 = k0;
                    u.k1 = k1;
                    u.piece = (k0 == 0 && k1 == nt) ? -1 : (k0 > 0 ? 0 : 1);
                    u.bad = 0;
                }
                at += k1 - k0;
            } else if (lane == 0) {
                u.valid = 0;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(unit_full(slot));
            if (!more) break;
            if (++slot == kTreeSlots) {
                slot = 0;
                phase ^= 1u;
            }
        }
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
            int valid, q0, row, kvh, k0, k1, pages;
            int win;           // first entry of window a; b holds the 32 after it
            int ent_a, ent_b;
        };
        int slot = 0;
        uint32_t uphase = 0;
        auto entry = [&](const Cur &c, int i) -> int {
            return c.row >= 0 && i < c.pages ? __ldg(p.table + static_cast<long long>(c.row) * p.table_w + i) : -1;
        };
        auto fetch = [&](Cur &c) -> bool {
            if (!__all_sync(0xffffffffu, wait_bar(unit_full(slot), uphase, p, abort_flag))) return false;
            const TreeUnit &u = units[slot];
            c.valid = u.valid;
            if (c.valid) {
                c.q0 = u.q0;
                c.row = u.row;
                c.kvh = u.kvh;
                c.k0 = u.k0;
                c.k1 = u.k1;
                c.pages = (u.L + p.page - 1) >> p.page_shift;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(unit_empty(slot));
            if (++slot == kTreeSlots) {
                slot = 0;
                uphase ^= 1u;
            }
            if (c.valid) {
                c.win = ((c.k0 << 7) >> p.page_shift) & ~31;
                c.ent_a = entry(c, c.win + lane);
                c.ent_b = entry(c, c.win + 32 + lane);
            }
            return true;
        };
        int stage = 0, loads = 0, q_units = 0, q_loads = 0;
        uint32_t phase = 0;
        auto load_tile_boxes = [&](Cur &c, const CUtensorMap *tm, int kt) -> bool {
            const int first = (kt << 7) >> p.page_shift;
            // V is the last to use a window: the one after the next is fetched when V leaves it
            if (tm == &tmV && first >= c.win + 32) {
                c.win += 32;
                c.ent_a = c.ent_b;
                c.ent_b = entry(c, c.win + 32 + lane);
            }
            if (!__all_sync(0xffffffffu, wait_bar(kv_empty(stage), phase ^ 1u, p, abort_flag))) return false;
            const uint32_t dst = sKV + stage * L::kTileBytes;
            if (lane == 0) mbar_arrive_expect_tx(kv_full(stage), L::kTileBytes);
            __syncwarp();
            // lane b issues box b: atom b % kAtoms of page piece b / kAtoms
            const int piece = lane / kAtoms, a = lane % kAtoms;
            const int at = first - c.win + piece;  // in [0, 64)
            const int ea = __shfl_sync(0xffffffffu, c.ent_a, at & 31);
            const int eb = __shfl_sync(0xffffffffu, c.ent_b, at & 31);
            int e = at < 32 ? ea : eb;
            if (lane < boxes) {
                if (e < 0 || e >= p.n_pages) {
                    if (first + piece < c.pages) atomicCAS(&g_error_code, 0, static_cast<int>(ATTN_ERR_PAGE));
                    e = -1;
                }
                tma_load_3d(dst + a * kAtomBytes + piece * box_rows * 128, tm, 64 * a, (kt << 7) & (p.page - 1),
                            e < 0 ? oob : e * p.Hkv + c.kvh, kv_full(stage));
            }
            ++loads;
            if (++stage == S) {
                stage = 0;
                phase ^= 1u;
            }
            return true;
        };
        // the first K tile of a unit, then its Q
        auto start = [&](Cur &c) -> bool {
            if (!load_tile_boxes(c, &tmK, c.k0)) return false;
            if (!__all_sync(0xffffffffu, wait_bar(q_empty, (q_units & 1) ^ 1u, p, abort_flag))) return false;
            ++q_units;
            if (!p.inject_stall) {
                if (lane == 0) {
                    const uint32_t bytes = static_cast<uint32_t>(p.group * p.rt) * D * 2;
                    mbar_arrive_expect_tx(q_full, bytes);
                    for (int a = 0; a < kAtoms; ++a)
                        tma_load_3d(sQ + a * kAtomBytes, &tmQ, 64 * a, c.kvh * p.group, c.q0, q_full);
                }
                ++q_loads;
            }
            return true;
        };
        Cur cur{}, nxt{};
        bool ok = fetch(cur) && (!cur.valid || start(cur));
        while (ok && cur.valid) {
            for (int kt = cur.k0; ok && kt < cur.k1; ++kt) {
                if (kt + 1 < cur.k1)
                    ok = load_tile_boxes(cur, &tmK, kt + 1);
                else
                    ok = fetch(nxt) && (!nxt.valid || start(nxt));
                ok = ok && load_tile_boxes(cur, &tmV, kt);
            }
            cur = nxt;
        }
        if (lane == 0) {
            // every copy has landed before the CTA exits (also after a timeout)
#pragma unroll
            for (int st = 0; st < S; ++st)
                if (loads > st) drain_bar(kv_full(st), st < stage ? phase : phase ^ 1u, p);
            if (q_loads > 0) drain_bar(q_full, (q_loads - 1) & 1, p);
        }
        __syncwarp();
    } else if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------------- MMA issuer
            constexpr uint32_t idesc_qk = idesc_f16_f32acc(kBF16, kBM, kBN, false);
            constexpr uint32_t idesc_pv = idesc_f16_f32acc(kBF16, kBM, D, true);
            const uint32_t tO = tmem + 256u;
            int stage = 0, slot = 0;
            uint32_t phase = 0, uphase = 0, qn = 0, vn = 0, jj = 0, pj = 0;  // scores issued, P V issued
            struct Cur {
                int valid, k0, k1, guard;
            };
            auto fetch = [&](Cur &c) -> bool {
                if (!wait_bar(unit_full(slot), uphase, p, abort_flag)) return false;
                const TreeUnit &u = units[slot];
                c.valid = u.valid;
                if (c.valid) {
                    c.k0 = u.k0;
                    c.k1 = u.k1;
                    c.guard = u.base / kBN;  // tiles from here on pass the guard
                }
                mbar_arrive(unit_empty(slot));
                if (++slot == kTreeSlots) {
                    slot = 0;
                    uphase ^= 1u;
                }
                return true;
            };
            auto take = [&]() -> int {  // next ring stage
                const int st = stage;
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
                return st;
            };
            auto qk = [&](bool last) -> bool {
                if (!wait_bar(kv_full(stage), phase, p, abort_flag)) return false;
                tc_fence_after();
                const int ks = take();
                const uint32_t sK = sKV + ks * L::kTileBytes, b = jj++ & 1u;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t koff = (kk >> 2) * kAtomBytes + (kk & 3) * 32;
                    mma_f16_ss(tmem + 128u * b, sdesc_sw128(sQ + koff, 16, 1024),
                               sdesc_sw128(sK + koff, 16, 1024), idesc_qk, kk > 0);
                }
                mma_commit(s_full(b));
                mma_commit(kv_empty(ks));
                if (last) mma_commit(q_empty);  // the unit's last score product: Q may be replaced
                return true;
            };
            auto start = [&](const Cur &c) -> bool {
                if (!wait_bar(q_full, qn++ & 1u, p, abort_flag)) return false;
                tc_fence_after();
                return qk(c.k0 + 1 == c.k1);
            };
            Cur cur{}, nxt{};
            bool ok = fetch(cur) && (!cur.valid || start(cur));
            while (ok && cur.valid) {
                for (int kt = cur.k0; ok && kt < cur.k1; ++kt) {
                    if (kt + 1 < cur.k1)
                        ok = qk(kt + 2 == cur.k1);
                    else
                        ok = fetch(nxt) && (!nxt.valid || start(nxt));
                    if (!ok) break;
                    // O (+)= P_b V: P from TMEM (first 64 columns of S_b), V MN-major
                    const uint32_t b = pj & 1u;
                    if (!(ok = wait_bar(kv_full(stage), phase, p, abort_flag))) break;
                    if (kt >= cur.guard) {
                        // V lies in its stage: the guard looks at it while P is computed
                        *ask = stage;
                        mbar_arrive(v_ask);
                        if (!(ok = wait_bar(v_ok, vn++ & 1u, p, abort_flag))) break;
                    }
                    if (!(ok = wait_bar(p_full(b), (pj >> 1) & 1u, p, abort_flag))) break;
                    tc_fence_after();
                    const int vs = take();
                    const uint32_t sV = sKV + vs * L::kTileBytes;
#pragma unroll
                    for (int kk = 0; kk < kBN / 16; ++kk)
                        mma_f16_ts(tO, tmem + 128u * b + 8u * kk, sdesc_sw128(sV + kk * 2048, kAtomBytes, 1024),
                                   idesc_pv, (kt > cur.k0 || kk > 0) ? 1u : 0u);
                    mma_commit(o_done(b));
                    mma_commit(kv_empty(vs));
                    ++pj;
                }
                cur = nxt;
            }
            mma_commit(mma_done);
            drain_bar(mma_done, 0, p);
        }
        __syncwarp();
    } else if (warp == 1) {
        // -------------------------------------------------------- value guard
        // The issuer asks for each guarded tile once it has seen the tile arrive, and waits for
        // the answer.
        int slot = 0;
        uint32_t uphase = 0, asked = 0;
        bool ok = true;
        while (ok) {
            if (!__all_sync(0xffffffffu, wait_bar(unit_full(slot), uphase, p, abort_flag))) break;
            TreeUnit &u = units[slot];
            if (!u.valid) break;
            const int guard = u.base / kBN;
            for (int kt = u.k0 > guard ? u.k0 : guard; kt < u.k1; ++kt) {
                if (!(ok = __all_sync(0xffffffffu, wait_bar(v_ask, asked & 1u, p, abort_flag)))) break;
                ++asked;
                int left = u.L - kt * kBN;
                left = left < 0 ? 0 : (left < kBN ? left : kBN);
                const bool any = vl_guard_tile<D, kBF16>(smem + L::kKV + *ask * L::kTileBytes, left, u.T > 1,
                                                         u.bad_rows[(kt - guard) & (kTreeBadTiles - 1)], lane);
                if (any && lane == 0) u.bad = 1;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(v_ok);
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(unit_empty(slot));
            if (++slot == kTreeSlots) {
                slot = 0;
                uphase ^= 1u;
            }
        }
    } else {
        // -------------------------------------------------------- softmax rows
        const int wq = warp & 3;
        const int r = wq * 32 + lane;  // row within the tile == TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t tO = tmem + 256u + lane_off;
        const float c = p.scale_log2;
        int slot = 0;
        uint32_t uphase = 0, jj = 0;  // tiles so far
        bool ok = true;
        while (ok) {
            if (!__all_sync(0xffffffffu, wait_bar(unit_full(slot), uphase, p, abort_flag))) break;
            const TreeUnit &u = units[slot];
            if (!u.valid) break;
            const int k0 = u.k0, k1 = u.k1, tree0 = u.base;
            const int tok = r / p.group;  // token within the row tile
            const bool valid = tok < u.ntok && tok < p.rt;
            const bool active = wq * 32 < u.ntok * p.group;  // some row of this warp is real
            // ancestors of this row's token, itself among them
            Bits128 anc{0ull, 0ull};
            if (valid) {
                int t = u.t0 + tok;
                while (t >= 0 && t < kTreeMax) {
                    if (t < 64) anc.lo |= 1ull << t; else anc.hi |= 1ull << (t - 64);
                    const int par = u.par[t];
                    if (par >= t) break;  // not a tree: the walk ends here
                    t = par;
                }
            }
            float mrow = -INFINITY, l = 0.f;
            for (int kt = k0; kt < k1; ++kt, ++jj) {
                const uint32_t b = jj & 1u;
                if (!__all_sync(0xffffffffu, wait_bar(s_full(b), (jj >> 1) & 1u, p, abort_flag))) {
                    ok = false;
                    break;
                }
                if (active) {
                    tc_fence_after();
                    __syncwarp();
                    const uint32_t tS = tmem + 128u * b + lane_off;
                    uint32_t s[128];
                    float mt;
                    if ((kt + 1) * kBN <= tree0) {
                        float mq[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            tmem_ld32_max(tS + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * q]), mq[q]);
                        tmem_ld_wait(s, mq);
                        mt = fmax3(mq[0], mq[1], fmaxf(mq[2], mq[3]));
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            tmem_ld32(tS + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * q]));
                        tmem_ld_wait(s);
                        // bit c: this row sees key kt * 128 + c
                        const int sh = kt * kBN - tree0;
                        Bits128 see = sh >= 0 ? bits_shr(anc, sh) : bits_shl(anc, -sh);
                        const Bits128 old = bits_below(-sh);
                        see.lo |= old.lo;
                        see.hi |= old.hi;
                        const uint32_t w[4] = {static_cast<uint32_t>(see.lo), static_cast<uint32_t>(see.lo >> 32),
                                               static_cast<uint32_t>(see.hi), static_cast<uint32_t>(see.hi >> 32)};
#pragma unroll
                        for (int cc = 0; cc < 128; ++cc)
                            if (!((w[cc >> 5] >> (cc & 31)) & 1u)) s[cc] = __float_as_uint(-INFINITY);
                        float mx[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) mx[k] = fmaxf(u2f(s[2 * k]), u2f(s[2 * k + 1]));
#pragma unroll
                        for (int cc = 16; cc < 128; cc += 16)
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                mx[k] = fmax3(mx[k], u2f(s[cc + 2 * k]), u2f(s[cc + 2 * k + 1]));
                        mt = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
                    }
                    const float m_new = fmaxf(mrow, mt);
                    // a row that has seen no key yet takes its weights, all 0, against 0
                    const float m_use = m_new == -INFINITY ? 0.f : m_new;
                    const float alpha = ex2_approx((mrow - m_use) * c);
                    if (kt > k0 && __any_sync(0xffffffffu, m_new > mrow)) {
                        // rescale O: the P V before must have finished writing it
                        if (!__all_sync(0xffffffffu,
                                        wait_bar(o_done((jj - 1) & 1u), ((jj - 1) >> 1) & 1u, p, abort_flag))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        __syncwarp();
#pragma unroll
                        for (int q = 0; q < D / 32; ++q) {
                            uint32_t o[32];
                            tmem_ld32(tO + 32 * q, o);
                            tmem_ld_wait(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(u2f(o[e]) * alpha);
                            tmem_st32(tO + 32 * q, o);
                        }
                    }
                    mrow = m_new;
                    const float2 c2 = make_float2(c, c);
                    const float2 nmc2 = make_float2(-m_use * c, -m_use * c);
                    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int cc = 32 * q + 2 * e;
                            float2 x = ffma2(make_float2(u2f(s[cc]), u2f(s[cc + 1])), c2, nmc2);
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
            }
            if (!ok) break;
            // ---------------------------------------------------- epilogue
            const uint32_t last = jj - 1;
            if (!__all_sync(0xffffffffu, wait_bar(o_done(last & 1u), (last >> 1) & 1u, p, abort_flag))) break;
            if (active) {
                tc_fence_after();
                __syncwarp();
                const bool bad = *reinterpret_cast<const volatile int *>(&u.bad) != 0;
                const float inv_l = l == 0.f ? 0.f : 1.f / l;  // 0: the row saw no key
                const float lse = l == 0.f ? -INFINITY : (mrow * c + log2f(l)) * 0.6931471805599453f;
                const int head = u.kvh * p.group + r % p.group;
                const long long tok_row = u.q0 + tok;
                uint8_t *orow = static_cast<uint8_t *>(p.o) + tok_row * p.o_row + head * p.o_head;
                const size_t prow = (static_cast<size_t>(blockIdx.x) * 2 + (u.piece > 0 ? 1 : 0)) * kBM + r;
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t o[32];
                    tmem_ld32(tO + 32 * q, o);
                    tmem_ld_wait(o);
                    if (!valid) continue;
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(u2f(o[e]) * inv_l);
                    if (bad) {
                        // non-finite values that the guard took out of V, for the rows that see them
                        for (int g = 0; g < kTreeBadTiles; ++g)
                            for (int w = 0; w < 4; ++w)
                                for (uint32_t bits = u.bad_rows[g][w]; bits != 0; bits &= bits - 1) {
                                    const int key = (tree0 / kBN + g) * kBN + 32 * w + __ffs(bits) - 1;
                                    const int node = key - tree0;
                                    if (node >= 0 && !((node < 64 ? anc.lo >> node : anc.hi >> (node - 64)) & 1ull))
                                        continue;
                                    const int pg = __ldg(p.table + static_cast<long long>(u.row) * p.table_w +
                                                         (key >> p.page_shift));
                                    const uint32_t *vr = reinterpret_cast<const uint32_t *>(
                                        p.v_ptr + ((static_cast<size_t>(pg) * p.Hkv + u.kvh) * p.page +
                                                   (key & (p.page - 1))) * (D * 2) + q * 64);
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        const uint32_t x = __ldg(vr + e);
                                        const float2 f = unpack2<kBF16>(x);
                                        if (nonfinite16<kBF16>(x & 0xFFFFu)) o[2 * e] = __float_as_uint(u2f(o[2 * e]) + f.x);
                                        if (nonfinite16<kBF16>(x >> 16)) o[2 * e + 1] = __float_as_uint(u2f(o[2 * e + 1]) + f.y);
                                    }
                                }
                    }
                    if (u.piece >= 0) {
                        float *dst = p.part_o + prow * D + q * 32;
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            st_global_v4(dst + v * 4, o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
                    } else {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = pack2<kBF16>(u2f(o[2 * e]), u2f(o[2 * e + 1]));
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            st_global_v4(orow + q * 64 + v * 16, w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
                    }
                }
                if (valid) {
                    if (u.piece >= 0)
                        p.part_lse[prow] = lse;
                    else if (p.lse != nullptr)
                        p.lse[static_cast<size_t>(head) * p.total_q + tok_row] = lse;
                }
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(unit_empty(slot));
            if (++slot == kTreeSlots) {
                slot = 0;
                uphase ^= 1u;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Merges the pieces of the units that were cut: lse = log sum_s exp(lse_s) and
// O = sum_s exp(lse_s - lse) O_s (the online-softmax update of page "从零开始写Qwen3",
// deepseek.csdn.net/6a3201f8..., section "在线softmax", across CTAs).  One warp per output
// row; a row whose unit lay in one share has been written already.  The pieces of a row
// are consecutive CTAs' and are loaded 16 at a time.
template <int D, bool kBF16>
__global__ void __launch_bounds__(128) attn_tree_merge_kernel(const __grid_constant__ TreeParams p) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long R = static_cast<long long>(blockIdx.x) * 4 + warp;
    if (R >= static_cast<long long>(p.total_q) * p.Hq) return;
    const int tok = static_cast<int>(R / p.Hq), head = static_cast<int>(R % p.Hq);
    // the sequence of this token: the last one that starts at or before it
    int lo = 0, hi = p.n_seqs;  // cu[lo] <= tok < cu[hi], where the offsets ascend
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.cu + mid) <= tok) lo = mid; else hi = mid;
    }
    const TreeSeq q = tree_seq(p, lo);
    if (tok < q.q0 || tok >= q.q0 + q.T) return;
    constexpr int kPer = D / 32;
    uint8_t *dst = static_cast<uint8_t *>(p.o) + tok * p.o_row + head * p.o_head + lane * kPer * 2;
    auto store = [&](const uint32_t (&w)[kPer / 2]) {
        if constexpr (kPer == 4)
            *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t *>(dst) = w[0];
    };
    float *lse_out = p.lse == nullptr ? nullptr : p.lse + static_cast<size_t>(head) * p.total_q + tok;
    if (*reinterpret_cast<volatile unsigned int *>(&g_abort_seq) == p.seq) {
        // the kernel before gave up on a wait: its pieces may be stale
        uint32_t w[kPer / 2];
#pragma unroll
        for (int t = 0; t < kPer / 2; ++t) w[t] = kBF16 ? 0x7FC07FC0u : 0x7E007E00u;
        store(w);
        if (lse_out != nullptr && lane == 0) *lse_out = __int_as_float(0x7FC00000);
        return;
    }
    const int share = p.plan[0];
    const int nt = tree_key_tiles(q.L), mt = tree_row_tiles(p, q.T);
    const int t = tok - q.q0, m = t / p.rt;
    const int u0 = p.plan[1 + lo] + ((head / p.group) * mt + m) * nt;  // the unit's first tile
    const int c0 = u0 / share, c1 = (u0 + nt - 1) / share;
    if (c0 == c1) return;
    const int prow = (t - m * p.rt) * p.group + head % p.group;  // row within the tile
    // CTA c0's piece begins at the unit's start (slot 1), the others in mid-unit (slot 0)
    auto row_of = [&](int c) { return (static_cast<size_t>(c) * 2 + (c == c0 ? 1 : 0)) * kBM + prow; };
    constexpr int kBatch = 16;
    float acc[kPer];
#pragma unroll
    for (int d = 0; d < kPer; ++d) acc[d] = 0.f;
    float mx = -INFINITY, sum = 0.f;
    for (int s0 = c0; s0 <= c1; s0 += kBatch) {
        const int n = c1 + 1 - s0 < kBatch ? c1 + 1 - s0 : kBatch;
        const float ls = lane < n ? p.part_lse[row_of(s0 + lane)] : -INFINITY;
        float v[kBatch][kPer];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (i < n) {
                const float *src = p.part_o + row_of(s0 + i) * D + lane * kPer;
#pragma unroll
                for (int d = 0; d < kPer; ++d) v[i][d] = src[d];
            }
        float bm = ls;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
        const float m_new = fmaxf(mx, bm);
        const float old = mx == -INFINITY ? 0.f : expf(mx - m_new);
#pragma unroll
        for (int d = 0; d < kPer; ++d) acc[d] *= old;
        sum *= old;
        mx = m_new;
        const float wl = ls == -INFINITY ? 0.f : expf(ls - mx);
        sum += wl;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const float w = __shfl_sync(0xffffffffu, wl, i);
            if (i < n && w != 0.f) {
#pragma unroll
                for (int d = 0; d < kPer; ++d) acc[d] += w * v[i][d];
            }
        }
    }
    // every lane holds its own pieces' weights in `sum`
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // 0: the row saw no key
    uint32_t w[kPer / 2];
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) w[i] = pack2<kBF16>(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    store(w);
    if (lse_out != nullptr && lane == 0) *lse_out = sum == 0.f ? -INFINITY : mx + logf(sum);
}

}  // namespace gqa
