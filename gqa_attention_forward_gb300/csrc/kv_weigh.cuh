// The weight that each cached position receives (attn_kv_weigh): what an eviction by accumulated
// attention weight goes by.
//
// For the last T_s positions of sequence s, whose queries are packed rows [cu[s], cu[s+1]), and
// their attention's log-sum-exp, the call adds to the sums of every kv head
//   w_j (+)= sum_{t, g} exp(scale q_{t,g}.k_j - lse_{t,g})   over tokens t at or behind j
// and the G query heads of the kv head: the column sums of the softmax whose row sums are 1, which
// the online softmax of the page "从零开始写Qwen3" (deepseek.csdn.net/6a3201f8..., section
// "在线softmax") never holds.
//
// What bounds it: with few tokens HBM (K is read once, 2 D G T flops per key); with whole prompts
// the tensor cores and the exponentials alike (2 D flops and one exp2 per row and key, of which an
// SM does about 8192 and 32 a cycle: 512 cycles of each for 128 keys and 128 rows).
//
// Measured, GB300: 16 sequences of 2 to 8192 positions and a token each (Hq 32, Hkv 8, D 128) 35 us
// with the copy that resets the case, 1.5 us per 64 KB of K and SM while it streams (6.6 TB/s), 4 us
// until the first tile; the last 32 tokens of 32000 15 us; 12 whole prompts of 1 to 4096 (Hq 16) 80
// us, 0.87 PFLOP/s; one of 32768 (Hq 32) 3330 to 3400 us, 1.3 PFLOP/s; one of 512 beside 31 sequences of 32768
// with a token each 318 us, 6.66 TB/s.  A step of 256 keys and 128 rows takes 1800 to 2200 cycles, of
// which the tensor pipe and the exponentials are busy for about 1000 each, and its two halves, the
// issuer's waits, products and commits (1800) and the sums' barriers, TMEM loads and exponentials
// (1900), bound it alike: without the exponentials, with a quarter of the products or half of Q's loads
// the 12 prompts take the same time, with half of the sums' work 7% less.  (Two issuing threads 3 us
// more, K in TMEM as the A operand 2, the next step's scores loaded ahead 8.)
//
// The product is taken transposed, S^T = K Q^T: a TMEM lane, and so a thread, owns a key, and the
// sum over the rows is a sum over a thread's own columns, without shuffles, atomics or a second
// pass; the rows' log-sum-exps are the same for all threads and come from shared memory.  A unit is
// 256 keys of a kv head (two 128-key tiles that share every Q tile, two warpgroups each) against all
// row tiles that see one of them, so that every position's sum has one owner and a fixed order.
// Row tiles hold 128 / G tokens (row = token * G + head in the group).
//
// Units of up to 32 sequences are dealt to the CTAs by the number of their row tiles, most first (a
// sequence's blocks of keys have fewer and fewer, so that lane s of the scheduler finds sequence s's
// block of a level in closed form), large ones to the CTA with the least work, the rest in snake
// order; those of more sequences in the order of these, as a pass over all for each level would
// take too long (32 prompts of 1 to 4096, Hq 16: 296 us, 0.99 PFLOP/s; 33 of them 331, 0.91; 64 775, 0.90).
//
// Roles (640 threads): warp 0 MMA issuer, warp 1 TMA producer of Q, and the rows' log-sum-exps,
// warp 2 TMA producer of K (the lanes issue one page box each), warp 3 scheduler (and TMEM), and
// four warpgroups of sums, two to a key tile with 64 columns each (one alone needs 2300 cycles for
// 128 x 128 scores, mostly its own latencies, the products 504).  K has two buffers of a unit, Q a
// ring of three tiles.  TMEM: S^T of tile a, buffer b in columns [256 a + 128 b, + 128).  At a
// unit's end the second warpgroup of a tile hands its sums to the first through a column of its buffer.
//
// Rounding: all in fp32.  A warpgroup adds 64 columns of a row tile in 4 chains of 16, joins them (2
// sums) and adds one sum per row tile; the other's and the old value come last: a sum is off by at most
// (16 + 2 + row tiles + 2) 2^-24 of itself, beside what the scores and exponentials are off by.
#pragma once
#include <cuda.h>  // CUtensorMap

#include "attn_fwd_tree.cuh"
#include "kernel_common.cuh"
#include "kv_pages.cuh"

namespace gqa {

constexpr int kWgThreads = 640;
constexpr int kWgKeys = 2 * kBN;  // of a unit
// Units of so many row tiles and more are dealt one by one, to up to 256 CTAs, a few to each (every CTA
// works out all of it, about 80 ns a unit, in which the GPU does 11 row tiles).  For 12 prompts of 1
// to 4096 the longest share is then 64 row tiles and the mean 61; in snake order 82.
constexpr int kWgGreedy = 8, kWgRounds = 8, kWgLoads = 8;
constexpr int kWgQStages = 3, kWgSlots = 3, kWgLse = 3;
constexpr int kWgFewRows = 16;  // rows of the small Q box: with few tokens a full one is 32 KB beside 64 KB of K

struct WeighParams : Params {
    const int *cu, *table, *lens, *seqs;
    const float *lse_in;
    float *weights;  // of the layer: [n_rows][Hkv][positions]
    int n_seqs, total_q, Hkv, n_rows;
    int page, page_shift, n_pages, table_w;
    int rt, few;     // tokens of a row tile, of the small box
    int accumulate;
    const int *claim;  // of each row of the table the first entry of seqs that names it; null: few entries
};

struct WeighUnit {
    int valid;
    int row, kvh;
    int key0, L;    // first key of the unit, positions of the sequence
    int q0, T;      // packed row of the first token, tokens
    int base;       // positions before the tokens
    int m0, m1;     // row tiles
};

template <int D>
struct WeighLayout {
    static constexpr int kTileBytes = (D / 64) * kAtomBytes;
    static constexpr int kK = 0;  // two buffers of two tiles
    static constexpr int kQ = kK + 4 * kTileBytes;
    static constexpr int kLse = kQ + kWgQStages * kTileBytes;
    static constexpr int kBar = kLse + kWgLse * 512;
    // k_full[2], k_empty[2], q_full[S], q_empty[S], l_full[S], l_empty[S], s_full[2], s_empty[2], x_full[2][2], mma_done,
    // unit_full[slots], unit_empty[slots]
    static constexpr int kNumBars = 4 + 2 * kWgQStages + 2 * kWgLse + 4 + 4 + 1 + 2 * kWgSlots;
    static constexpr int kTmemSlot = kBar + kNumBars * 8;
    static constexpr int kAbort = kTmemSlot + 4;
    static constexpr int kUnits = kAbort + 4;
    static constexpr int kUsed = kUnits + kWgSlots * static_cast<int>(sizeof(WeighUnit));
    // more than half of an SM's shared memory: one CTA (all 512 TMEM columns) per SM
    static constexpr int kAlloc = (kUsed + 1024) > 118 * 1024 ? (kUsed + 1024) : 118 * 1024;
};
static_assert(WeighLayout<128>::kAlloc <= 227 * 1024, "shared memory of one CTA");

// 4-byte global -> shared copy.
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// S^T = K Q^T of 128 keys and N rows (K-major operands), for few rows; mma_qk with K in Q's place for 128.
template <int D, int kk = 0>
__device__ __forceinline__ void mma_kq(uint32_t td, uint32_t k_lo, uint32_t q_lo, uint32_t idesc) {
    if constexpr (kk < D / 16) {
        constexpr uint32_t off = (kk >> 2) * (kAtomBytes >> 4) + (kk & 3) * 2;
        const uint64_t hi = static_cast<uint64_t>(kDescHi) << 32;
        mma_f16_ss(td, hi | (k_lo + off), hi | (q_lo + off), idesc, kk > 0 ? 1u : 0u);
        mma_kq<D, kk + 1>(td, k_lo, q_lo, idesc);
    }
}

// The first entry of the list that names each row, for lists in which looking through the entries before
// takes longer than a launch (every CTA of the kernel below looks).
constexpr int kWgClaim = 64;
__global__ void __launch_bounds__(kPlanThreads) kv_claim_kernel(const KvPool c, const int *seqs, int n) {
    grid_launch_dependents();
    grid_dependency_wait();
    for (int i = threadIdx.x; i < n; i += kPlanThreads)
        if (seqs[i] >= 0 && seqs[i] < c.n_rows) c.claim[seqs[i]] = INT_MAX;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads)
        if (seqs[i] >= 0 && seqs[i] < c.n_rows) atomicMin(&c.claim[seqs[i]], i);
}

// tmQ: 3-D tensor map (D, Hq, tokens), box 64 x G x rt; tmF the same with a box of `few` tokens; tmK: 3-D map
// (D, page, n_pages * Hkv), box 64 x min(page, 128) x 1; all with the 128-byte swizzle.
template <int D, bool kBF16>
__global__ void __launch_bounds__(kWgThreads, 1)
    kv_weigh_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmF,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ WeighParams p) {
    using L = WeighLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const uint32_t sK = base + L::kK, sQ = base + L::kQ, sL = base + L::kLse;
    const uint32_t bar0 = base + L::kBar;
    constexpr int QS = kWgQStages, LS = kWgLse;
    auto k_full = [&](int b) { return bar0 + 8u * b; };
    auto k_empty = [&](int b) { return bar0 + 8u * (2 + b); };
    auto q_full = [&](int s) { return bar0 + 8u * (4 + s); };
    auto q_empty = [&](int s) { return bar0 + 8u * (4 + QS + s); };
    auto l_full = [&](int s) { return bar0 + 8u * (4 + 2 * QS + s); };
    auto l_empty = [&](int s) { return bar0 + 8u * (4 + 2 * QS + LS + s); };
    auto s_full = [&](int b) { return bar0 + 8u * (4 + 2 * QS + 2 * LS + b); };  // of both tiles
    auto s_empty = [&](int b) { return bar0 + 8u * (6 + 2 * QS + 2 * LS + b); };
    // tile a's sums have been handed over in buffer b: a barrier for each buffer, so that it cannot turn again
    // before the other warpgroup, which frees the buffer, has seen it
    auto x_full = [&](int a, int b) { return bar0 + 8u * (8 + 2 * QS + 2 * LS + 2 * a + b); };
    const uint32_t mma_done = bar0 + 8u * (12 + 2 * QS + 2 * LS);
    auto unit_full = [&](int s) { return bar0 + 8u * (13 + 2 * QS + 2 * LS + s); };
    auto unit_empty = [&](int s) { return bar0 + 8u * (13 + 2 * QS + 2 * LS + kWgSlots + s); };
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + L::kTmemSlot);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kAbort);
    WeighUnit *units = reinterpret_cast<WeighUnit *>(smem + L::kUnits);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    grid_launch_dependents();
    if (threadIdx.x == 32) {
        tma_prefetch_map(&tmQ);
        tma_prefetch_map(&tmF);
        tma_prefetch_map(&tmK);
    }
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int b = 0; b < 2; ++b) {
            mbar_init(k_full(b), 1);
            mbar_init(k_empty(b), 1);
            mbar_init(x_full(0, b), 4);
            mbar_init(x_full(1, b), 4);
            mbar_init(s_full(b), 1);
            mbar_init(s_empty(b), 16);  // one arrival per warp of sums
        }
        for (int s = 0; s < QS; ++s) {
            mbar_init(q_full(s), 1);
            mbar_init(q_empty(s), 1);
        }
        for (int s = 0; s < LS; ++s) {
            mbar_init(l_full(s), 32);  // the copies of each lane
            mbar_init(l_empty(s), 16);
        }
        mbar_init(mma_done, 1);
        for (int s = 0; s < kWgSlots; ++s) {
            mbar_init(unit_full(s), 1);
            mbar_init(unit_empty(s), 19);  // K, Q, MMA issuer, 16 warps of sums
        }
        fence_mbar_init();
    }
    if (warp == 3) {
        tmem_alloc(base + L::kTmemSlot, 512);
        tmem_relinquish();
    }
    // the set-up above overlaps the kernel before this one; its results are read from here on
    grid_dependency_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // a role's place in the units' slots
    struct Place {
        int slot = 0;
        uint32_t phase = 0;
        __device__ __forceinline__ void next() {
            if (++slot == kWgSlots) {
                slot = 0;
                phase ^= 1u;
            }
        }
    };
    auto tiles_of = [&](const WeighUnit &u) { return u.L - u.key0 > kBN ? 2 : 1; };

    if (warp == 3) {
        // -------------------------------------------------------- scheduler
        // 32 sequences at a time, a lane each: where they are, their blocks of 256 keys, units before them
        int s0 = -32, T = 0, len = 0, row = -1, q0 = 0, blocks = 0, incl = 0, block0 = 0;
        int before = 0, batch = 0;      // units before the 32, and of them
        long long tokens = 0;           // of the sequences before the 32
        bool bad = false;
        auto count = [&](int mine) {
            incl = mine * p.Hkv;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            batch = __shfl_sync(0xffffffffu, incl, 31);
        };
        auto load = [&]() {
            s0 += 32;
            before += batch;
            const int s = s0 + lane;
            T = blocks = 0;
            long long upto = 0;
            if (s < p.n_seqs) {
                const VlSpan q = vl_span(p.cu, s, p.total_q);
                row = p.seqs != nullptr ? p.seqs[s] : s;
                q0 = q.a;
                T = q.b - q.a;
                const bool in = row >= 0 && row < p.n_rows;
                len = in ? p.lens[row] : 0;
                // a sequence named before in the list would be added to by two units at once
                bool again = false;
                if (p.claim != nullptr)
                    again = in && p.claim[row] != s;
                else if (p.seqs != nullptr)
                    for (int j = 0; j < s; ++j) again |= p.seqs[j] == row;
                if (q.bad || !in || again || len < T || len > (static_cast<long long>(p.table_w) << p.page_shift)) {
                    bad = true;
                    T = 0;
                }
                upto = T;
            }
            // offsets that descend can overlap: no more rows than ascending ones can have
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            if (T > 0 && tokens + upto > p.total_q) {
                bad = true;
                T = 0;
            }
            tokens += __shfl_sync(0xffffffffu, upto, 31);
            if (T > 0) blocks = (len + kWgKeys - 1) / kWgKeys;
            count(blocks);
        };
        load();
        // the levels of up to 32 sequences: a lane's blocks [block0, block0 + on) are on the level
        const bool levels = p.n_seqs <= 32;
        const int all = blocks, tiles = (T + p.rt - 1) / p.rt, old = len - T;
        int level = INT_MAX, on = blocks;
        auto tiles_of_block = [&](int b) { return tiles - (b * kWgKeys > old ? (b * kWgKeys - old) / p.rt : 0); };
        // the first block of fewer than l tiles: it starts tiles - l + 1 of them or more behind the first token
        auto fewer = [&](int l) -> int {
            if (l > tiles) return 0;
            const long long from = old + static_cast<long long>(tiles - l + 1) * p.rt;
            return static_cast<int>((from + kWgKeys - 1) / kWgKeys);
        };
        auto next_level = [&]() -> bool {
            int b = fewer(level);
            const int mine = b < all ? tiles_of_block(b) : 0;
            level = __reduce_max_sync(0xffffffffu, mine);
            if (level == 0) return false;
            before += batch;
            block0 = b;
            on = mine == level ? (fewer(level) < all ? fewer(level) : all) - b : 0;
            count(on);
            return true;
        };
        bool more = true;
        // goes on to unit t (t never decreases, but for a new start); more: there is one
        auto seek = [&](int t) {
            if (levels) {
                while (more && t >= before + batch) more = next_level();
            } else {
                while (more && t >= before + batch) {
                    load();
                    on = blocks;
                    more = s0 < p.n_seqs;
                }
            }
        };
        auto restart = [&]() {
            level = INT_MAX;
            before = batch = 0;
            more = true;
        };
        Place at;
        auto emit = [&](int t) -> bool {  // unit t, or where there is no more the end
            if (!__all_sync(0xffffffffu, wait_bar(unit_empty(at.slot), at.phase ^ 1u, p, abort_flag))) return false;
            if (more) {
                const int src = __ffs(__ballot_sync(0xffffffffu, before + incl > t)) - 1;
                if (lane == src) {
                    const int in = t - before - (incl - on * p.Hkv);
                    WeighUnit &u = units[at.slot];
                    u.valid = 1;
                    u.row = row;
                    u.kvh = in % p.Hkv;
                    u.key0 = (block0 + in / p.Hkv) * kWgKeys;
                    u.L = len;
                    u.q0 = q0;
                    u.T = T;
                    u.base = len - T;
                    u.m0 = u.key0 > u.base ? (u.key0 - u.base) / p.rt : 0;
                    u.m1 = (T + p.rt - 1) / p.rt;
                }
            } else if (lane == 0) {
                units[at.slot].valid = 0;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(unit_full(at.slot));
            at.next();
            return true;
        };
        const int grid = static_cast<int>(gridDim.x), me = static_cast<int>(blockIdx.x);
        if (levels) restart();
        seek(0);
        // how units are dealt is one choice for all CTAs: it goes by the largest unit, not by a CTA's own first
        const bool greedy = levels && more && level >= kWgGreedy && grid <= 32 * kWgLoads;
        seek(me);
        bool ok = emit(me);
        if (ok && more) {
            int t = grid;
            if (greedy) {
                // A unit goes to the CTA with the least row tiles so far, which all CTAs work out alike: the first
                // ones in order, then one by one.  Lane l keeps CTAs l, l + 32, ..
                constexpr unsigned kNone = 0xFFFFFFu;
                unsigned load_of[kWgLoads];
#pragma unroll
                for (int e = 0; e < kWgLoads; ++e) load_of[e] = lane + 32 * e < grid ? 0u : kNone;
                restart();
                for (seek(0); more && before < grid; seek(before + batch)) {
#pragma unroll
                    for (int e = 0; e < kWgLoads; ++e)
                        if (lane + 32 * e >= before && lane + 32 * e < before + batch && lane + 32 * e < grid)
                            load_of[e] = static_cast<unsigned>(level);
                    if (before + batch >= grid) break;
                }
                for (; ok; ++t) {
                    seek(t);
                    if (!more || level < kWgGreedy || t >= kWgRounds * grid) break;
                    unsigned best = 0xFFFFFFFFu;
#pragma unroll
                    for (int e = 0; e < kWgLoads; ++e) {
                        const unsigned x = load_of[e] << 8 | static_cast<unsigned>(lane + 32 * e);
                        best = x < best ? x : best;
                    }
                    best = __reduce_min_sync(0xffffffffu, best);
                    const int c = static_cast<int>(best & 255u);
#pragma unroll
                    for (int e = 0; e < kWgLoads; ++e)
                        if (c == lane + 32 * e) {
                            const unsigned x = load_of[e] + static_cast<unsigned>(level);
                            load_of[e] = x < kNone ? x : kNone - 1u;
                        }
                    if (c == me) ok = emit(t);
                }
            }
            // the others in snake order, up to the end
            for (bool back = true; ok; t += grid, back = !back) {
                const int mine = t + (back ? grid - 1 - me : me);
                seek(mine);
                ok = emit(mine);
                if (!more) break;
            }
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicCAS(&g_error_code, 0, static_cast<int>(ATTN_ERR_SHAPE));
    } else if (warp == 2) {
        // -------------------------------------------------------- TMA producer of K
        constexpr int kAtoms = D / 64;
        const int box_rows = p.page < kBN ? p.page : kBN;
        const int boxes = (kBN / box_rows) * kAtoms;  // per tile, at most 16
        // lane b issues box b: atom b % kAtoms of page piece b / kAtoms of the unit's keys
        const int piece = lane / kAtoms, a = lane % kAtoms, key = piece * box_rows;
        Place at;
        int n = 0, kvh = 0, tiles = 0, page = 0, first = 0, L0 = 0;
        bool valid = false;
        auto take = [&]() -> bool {
            if (!__all_sync(0xffffffffu, wait_bar(unit_full(at.slot), at.phase, p, abort_flag))) return false;
            const WeighUnit &u = units[at.slot];
            valid = u.valid != 0;
            if (valid) {
                kvh = u.kvh;
                tiles = tiles_of(u);
                first = u.key0;
                L0 = u.L;
                page = lane < boxes * tiles && first + key < L0
                    ? p.table[static_cast<long long>(u.row) * p.table_w + ((first + key) >> p.page_shift)] : -1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(unit_empty(at.slot));
            at.next();
            return true;
        };
        bool ok = take();
        for (; ok && valid; ++n) {
            const int b = n & 1;
            if (!(ok = __all_sync(0xffffffffu, wait_bar(k_empty(b), ((n >> 1) & 1u) ^ 1u, p, abort_flag)))) break;
            if (lane == 0) mbar_arrive_expect_tx(k_full(b), static_cast<uint32_t>(tiles * L::kTileBytes));
            __syncwarp();
            if (lane < boxes * tiles) {
                int e = page;
                if (e < 0 || e >= p.n_pages) {
                    if (first + key < L0) atomicCAS(&g_error_code, 0, static_cast<int>(ATTN_ERR_PAGE));
                    e = p.n_pages;  // one past the last: reads as zeros
                }
                const int tile = key / kBN;
                tma_load_3d(sK + (2 * b + tile) * L::kTileBytes + a * kAtomBytes + (key & (kBN - 1)) * 128, &tmK, 64 * a,
                            (first + key) & (p.page - 1), e * p.Hkv + (e < p.n_pages ? kvh : 0), k_full(b));
            }
            __syncwarp();
            ok = take();
        }
        if (lane == 0) {
            // every copy has landed before the CTA exits (also after a timeout)
            if (n > 0) drain_bar(k_full((n - 1) & 1), ((n - 1) >> 1) & 1, p);
            if (n > 1) drain_bar(k_full(n & 1), ((n - 2) >> 1) & 1, p);
        }
        __syncwarp();
    } else if (warp == 1) {
        // -------------------------------------------------------- TMA producer of Q, log-sum-exps
        Place at;
        int s = 0, ls = 0, loads = 0;
        uint32_t ph = 0, lph = 0;
        long long off[4];  // of this lane's rows of a tile: token in the tile, head in the group
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = lane + 32 * e, t = r / p.group;
            off[e] = static_cast<long long>(r - t * p.group) * p.total_q + t;
        }
        bool ok = true;
        while (ok) {
            if (!(ok = __all_sync(0xffffffffu, wait_bar(unit_full(at.slot), at.phase, p, abort_flag)))) break;
            const WeighUnit u = units[at.slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(unit_empty(at.slot));
            at.next();
            if (!u.valid) break;
            for (int m = u.m0; m < u.m1; ++m) {
                const int tok0 = u.q0 + m * p.rt, left = u.T - m * p.rt;
                if (!(ok = __all_sync(0xffffffffu, wait_bar(q_empty(s), ph ^ 1u, p, abort_flag)))) break;
                if (!p.inject_stall) {
                    if (lane == 0) {
                        const bool few = left <= p.few;
                        mbar_arrive_expect_tx(q_full(s), static_cast<uint32_t>(p.group * (few ? p.few : p.rt)) * D * 2);
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
                            tma_load_3d(sQ + s * L::kTileBytes + x * kAtomBytes, few ? &tmF : &tmQ, 64 * x, u.kvh * p.group,
                                        tok0, q_full(s));
                    }
                    ++loads;
                }
                if (!(ok = __all_sync(0xffffffffu, wait_bar(l_empty(ls), lph ^ 1u, p, abort_flag)))) break;
                const int rows = (left < p.rt ? left : p.rt) * p.group;
                const float *from = p.lse_in + static_cast<long long>(u.kvh) * p.group * p.total_q + tok0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (lane + 32 * e < rows) cp_async_4(sL + ls * 512 + (lane + 32 * e) * 4, from + off[e]);
                cp_async_arrive(l_full(ls));
                if (++s == QS) {
                    s = 0;
                    ph ^= 1u;
                }
                if (++ls == LS) {
                    ls = 0;
                    lph ^= 1u;
                }
            }
        }
        cp_async_commit();
        cp_async_wait<0>();
        if (lane == 0)
            for (int st = 0; st < QS; ++st)  // the last load of each stage
                if (loads > st) drain_bar(q_full(st), ((loads - 1 - st) / QS) & 1, p);
        __syncwarp();
    } else if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------------- MMA issuer
            const uint32_t dk = desc_lo(sK, 16), dq = desc_lo(sQ, 16);
            constexpr uint32_t kTile16 = L::kTileBytes >> 4;
            Place at;
            int s = 0, n = 0;
            uint32_t ph = 0, step = 0;
            bool ok = true;
            while (ok) {
                if (!(ok = wait_bar(unit_full(at.slot), at.phase, p, abort_flag))) break;
                const WeighUnit &us = units[at.slot];
                const int valid = us.valid, m0 = us.m0, m1 = us.m1, T = us.T;
                mbar_arrive(unit_empty(at.slot));
                at.next();
                if (!valid) break;
                const int b = n & 1;
                if (!(ok = wait_bar(k_full(b), (n >> 1) & 1u, p, abort_flag))) break;
                for (int m = m0; m < m1 && ok; ++m) {
                    if (!(ok = wait_bar(q_full(s), ph, p, abort_flag))) break;
                    const int left = T - m * p.rt, rows = (left < p.rt ? left : p.rt) * p.group;
                    const uint32_t sb = step & 1u;
                    if (!(ok = wait_bar(s_empty(sb), ((step >> 1) & 1u) ^ 1u, p, abort_flag))) break;
                    tc_fence_after();
                    // (where the sequence ends in the first tile the second one's scores are never looked at)
                    const uint32_t td = tmem + 128u * sb, k_lo = dk + 2 * b * kTile16, q_lo = dq + s * kTile16;
                    if (rows > 64) {
                        mma_qk<D, kBF16>(td, k_lo, q_lo);
                        mma_qk<D, kBF16>(td + 256u, k_lo + kTile16, q_lo);
                    } else {
                        const uint32_t idesc = idesc_f16_f32acc(kBF16, 128, (rows + 15) & ~15, false);
                        mma_kq<D>(td, k_lo, q_lo, idesc);
                        mma_kq<D>(td + 256u, k_lo + kTile16, q_lo, idesc);
                    }
                    mma_commit(s_full(sb));
                    ++step;
                    mma_commit(q_empty(s));
                    if (++s == QS) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                mma_commit(k_empty(b));
                ++n;
            }
            // TMEM and shared memory stay alive until every issued MMA is done.
            mma_commit(mma_done);
            drain_bar(mma_done, 0, p);
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------- sums, a key per thread
        const int a = (warp - 4) >> 3, wq = warp & 3;
        const int half = ((warp - 4) >> 2) & 1;  // this warpgroup's columns: [64 half, 64 half + 64)
        const uint32_t tA = tmem + 256u * a + (static_cast<uint32_t>(wq * 32) << 16);
        const float c = p.scale_log2;
        const float2 c2 = make_float2(c, c), nl2 = make_float2(-1.4426950408889634f, -1.4426950408889634f);
        const long long width = static_cast<long long>(p.table_w) << p.page_shift;
        Place at;
        uint32_t step = 0, lph = 0, xph = 0;
        int ls = 0;
        bool ok = true;
        while (ok) {
            if (!(ok = __all_sync(0xffffffffu, wait_bar(unit_full(at.slot), at.phase, p, abort_flag)))) break;
            const WeighUnit u = units[at.slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(unit_empty(at.slot));
            at.next();
            if (!u.valid) break;
            const int warp_key = u.key0 + kBN * a + 32 * wq, key = warp_key + lane;
            const bool real = key < u.L, some = warp_key < u.L;
            float *w = p.weights + (static_cast<long long>(u.row) * p.Hkv + u.kvh) * width + key;
            // the sum so far is on its way while the scores are computed; a new token's position begins here
            float old = 0.f;
            if (half == 0 && p.accumulate && real && key < u.base) old = *w;
            const int most = u.T - u.m0 * p.rt;  // tokens of the unit's row tiles
            const bool both = (most < p.rt ? most : p.rt) * p.group > 64;  // the second warpgroup has columns
            float sum = 0.f;
            for (int m = u.m0; m < u.m1; ++m, ++step) {
                const float *lse = reinterpret_cast<const float *>(smem + L::kLse + ls * 512);
                const uint32_t sb = step & 1u, tS = tA + 128u * sb;
                if (!(ok = __all_sync(0xffffffffu, wait_bar(l_full(ls), lph, p, abort_flag)))) break;
                if (!(ok = __all_sync(0xffffffffu, wait_bar(s_full(sb), (step >> 1) & 1u, p, abort_flag)))) break;
                if (some) {
                    tc_fence_after();
                    __syncwarp();
                    const int left = u.T - m * p.rt, cols = (left < p.rt ? left : p.rt) * p.group;
                    // this key's columns are [c0, cols): those of tokens at or behind it
                    const int tok0 = u.base + m * p.rt;
                    auto first_col = [&](int k) -> int {
                        const int t = k - tok0;
                        return (t < 0 ? 0 : (t < p.rt ? t : p.rt)) * p.group;
                    };
                    const int c0 = first_col(key), c0_low = first_col(warp_key), c0_high = first_col(warp_key + 31);
                    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    // 32 columns: exp2(s c - lse log2 e) of four at a time
                    auto add = [&](const uint32_t (&s)[32], int q, bool whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 l4 = *reinterpret_cast<const float4 *>(lse + q + e);
                            const float2 n0 = fmul2(make_float2(l4.x, l4.y), nl2);
                            const float2 n1 = fmul2(make_float2(l4.z, l4.w), nl2);
                            float2 x0 = ffma2(make_float2(u2f(s[e]), u2f(s[e + 1])), c2, n0);
                            float2 x1 = ffma2(make_float2(u2f(s[e + 2]), u2f(s[e + 3])), c2, n1);
                            if (!whole) {
                                // a column that is not this key's adds nothing, whatever it holds
                                const int d = q + e;
                                if (d < c0 || d >= cols) x0.x = -INFINITY;
                                if (d + 1 < c0 || d + 1 >= cols) x0.y = -INFINITY;
                                if (d + 2 < c0 || d + 2 >= cols) x1.x = -INFINITY;
                                if (d + 3 < c0 || d + 3 >= cols) x1.y = -INFINITY;
                            }
                            acc[0] = fadd2(acc[0], make_float2(ex2_approx(x0.x), ex2_approx(x0.y)));
                            acc[1] = fadd2(acc[1], make_float2(ex2_approx(x1.x), ex2_approx(x1.y)));
                        }
                    };
                    const int q0 = 64 * half, q1 = cols < q0 + 64 ? cols : q0 + 64;
                    if (c0_high <= q0 && q1 == q0 + 64) {
                        // every key of the warp has all columns
                        uint32_t s[32];
                        tmem_ld32(tS + q0, s);
                        tmem_ld_wait(s);
                        add(s, q0, true);
                        tmem_ld32(tS + q0 + 32, s);
                        tmem_ld_wait(s);
                        add(s, q0 + 32, true);
                    } else {
#pragma unroll 1
                        for (int q = q0; q < q1; q += 32) {
                            if (c0_low >= q + 32) continue;  // no key of the warp has one of these
                            uint32_t s[32];
                            tmem_ld32(tS + q, s);
                            tmem_ld_wait(s);
                            add(s, q, false);
                        }
                    }
                    tc_fence_before();
                    acc[0] = fadd2(acc[0], acc[1]);
                    sum += acc[0].x + acc[0].y;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(l_empty(ls));
                if (++ls == LS) {
                    ls = 0;
                    lph ^= 1u;
                }
                if (half == 0 || !both || m + 1 < u.m1) {
                    if (lane == 0) mbar_arrive(s_empty(sb));
                } else {
                    // this one's sums are handed over in its last buffer, which the other then frees
                    uint32_t x[1] = {__float_as_uint(sum)};
                    tmem_st1(tS + 64u, x);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(x_full(a, sb));
                }
            }
            if (!ok) break;
            if (both && half == 0) {
                const uint32_t sb = (step - 1u) & 1u;
                if (!(ok = __all_sync(0xffffffffu, wait_bar(x_full(a, sb), (xph >> sb) & 1u, p, abort_flag)))) break;
                xph ^= 1u << sb;
                tc_fence_after();
                __syncwarp();
                uint32_t x[1];
                tmem_ld1(tA + 128u * sb + 64u, x);
                tmem_ld_wait(x);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_empty(sb));
                sum += u2f(x[0]);
            }
            if (half == 0 && real) *w = old + sum;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace gqa
