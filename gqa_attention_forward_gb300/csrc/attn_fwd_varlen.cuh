// Attention over packed sequences of different lengths (attn_fwd_varlen).
//
// The rows of all sequences lie one after another; sequence s owns query rows
// [cu_q[s], cu_q[s+1]) and keys [cu_k[s], cu_k[s+1]), both read on the device, so a call
// needs no host copy of the lengths and a captured call replays on new ones.  Per row i of
// sequence s:  O_i = sum_j softmax_j(scale q_i.k_j) v_j  over the keys j of s, and with the
// causal mask over j <= i + Nk_s - Nq_s; a row that sees no key gets O = 0, LSE = -inf.
// The online softmax is the one of the page "从零开始写Qwen3" (deepseek.csdn.net/6a3201f8...,
// sections "在线softmax" and "FlashAttention").
//
// What bounds it: 4 D flops per visible (row, key) pair and head on the tensor cores, of
// which the MMA issue takes most (two 128-row tiles per key tile keep the pipe busy while
// the softmax works); for short sequences the fill and drain of a unit's pipeline.
//
// Work unit: two 128-row query tiles that read the same keys.  With an even number of
// query heads per kv head these are two heads of one group over the same 128 rows: both
// tiles then visit the same key tiles and no causal step runs half empty (256 rows of one
// head waste one half step per unit, 1/6 of the work of a 512-token prompt) and a
// sequence of at most 128 rows still fills both.  With an odd group the tiles are rows
// [0,128) and [128,256) of one head, and the second is skipped where there is none.
//
// Order of the units: longest first over all sequences (the last block of a sequence sees
// the most keys), dealt to the persistent CTAs in snake order.  The scheduler warp finds
// unit u without a sorted list: blocks are enumerated by level, the number of key blocks
// that a block sees.  Under the causal mask each sequence has at most one block per level
// (its nqb blocks lie on the levels H - nqb + 1 .. H, H = ceil(Nk / block)), so the r-th
// block of a level is found with a ballot over the sequences.  A CTA's units only ever
// move down the levels.
//
// Roles (384 threads): warp 0 MMA issuer, warp 1 value guard (and TMEM), warp 2 TMA
// producer, warp 3 scheduler, warps 4-7 and 8-11 the softmax of tile 0 and 1; shared
// memory, TMEM and the K/V ring are laid out as in the equal-length kernel.
//
// Value guard.  A 128-row V box of the last key tile reaches into the next sequence (or
// into rows behind the last one, which may hold anything), and P = 0 times infinity or
// NaN is NaN.  The guard zeroes those rows in shared memory before P V reads them.  In
// tiles on the causal boundary it also looks for non-finite values: they are zeroed, their
// rows noted, and the epilogue adds them to exactly the rows that see the key.
#pragma once
#include <cuda.h>  // CUtensorMap

#include <climits>

#include "attn_fwd_ws.cuh"
#include "kernel_common.cuh"

namespace gqa {

constexpr int kVlSlots = 4;       // unit descriptors in flight
constexpr int kVlSeqCache = 2048; // sequences whose block counts are kept in shared memory
constexpr int kVlBadTiles = 4;    // key tiles of a unit that the guard may look at

struct VarlenParams : Params {
    const int *cu_q, *cu_k;  // device [n_seqs + 1]
    const uint8_t *v_ptr;    // V in global memory (the rare non-finite rows are read again)
    int n_seqs, total_q, total_k;
    int pair;                // 1: the tiles are two heads of a group; 0: two row tiles of a head
    int block_rows;          // query rows of a unit: 128 (pair) or 256
    int head_units;          // units per block of rows: Hq / 2 (pair) or Hq
    int q_head_y, k_head_y, v_head_y;  // tensor map order: 1 = (D, heads, rows), 0 = (D, rows, heads)
    long long o_row, o_head, v_row, v_head;  // strides in bytes
};

// One unit, as the scheduler hands it to the other roles.
struct VlUnit {
    int valid;   // 0: no more units
    int head;    // query head of tile 0
    int q0;      // packed row of the block's first query row
    int rows;    // query rows from q0 to the end of the sequence
    int k0;      // packed row of the sequence's first key
    int nk;      // keys of the sequence
    int rel;     // row r of the block sees keys j <= r + rel under the causal mask
    int bad;     // set by the guard: some bad_rows bit is set
    uint32_t bad_rows[kVlBadTiles][4];  // rows of the guarded V tiles with a non-finite value
};

template <int D>
struct VlLayout {
    using W = WsLayout<D>;
    static constexpr int kTileBytes = W::kTileBytes;
    static constexpr int kQ = W::kQ, kKV = W::kKV, kStage = W::kStage;
    static constexpr int kStageBytes = W::kStageBytes;
    static constexpr int kBar = kStage + 8 * kStageBytes;
    // q_full[2], q_empty, kv_full[S], kv_empty[S], s_full[2], p_full[2], o_full[2], mma_done,
    // v_ask, v_ok, unit_full[slots], unit_empty[slots]
    static constexpr int kNumBars = 2 + 1 + 2 * kStagesWs + 2 + 2 + 2 + 1 + 2 + 2 * kVlSlots;
    static constexpr int kFlags = kBar + kNumBars * 8;
    static constexpr int kTmemSlot = kFlags + 32;
    static constexpr int kAbort = kTmemSlot + 4;
    static constexpr int kAsk = kAbort + 4;
    static constexpr int kUnits = (kAsk + 4 + 15) & ~15;
    static constexpr int kSeqs = kUnits + kVlSlots * static_cast<int>(sizeof(VlUnit));
    static constexpr int kUsed = kSeqs + kVlSeqCache * 4;
    static constexpr int kAlloc = (kUsed + 1024) > 118 * 1024 ? (kUsed + 1024) : 118 * 1024;
};
static_assert(VlLayout<128>::kAlloc <= 227 * 1024, "shared memory of one CTA");

// Tile i of a unit: its rows, head and the key tiles [0, n) that it visits.
struct VlTile {
    int row0;   // first row of the tile within the block
    int valid;  // query rows of the tile (0: absent)
    int rel;    // row r of the tile sees keys j <= r + rel (causal)
    int n;      // key tiles
};
template <bool kCausal>
__device__ __forceinline__ VlTile vl_tile(const VarlenParams &p, const VlUnit &u, int i) {
    VlTile t;
    t.row0 = p.pair ? 0 : kBM * i;
    const int left = u.rows - t.row0;
    t.valid = left < 0 ? 0 : (left < kBM ? left : kBM);
    t.rel = u.rel + t.row0;
    int seen = u.nk;
    if (kCausal && t.rel + t.valid < seen) seen = t.rel + t.valid;
    t.n = (t.valid > 0 && seen > 0) ? (seen + kBN - 1) / kBN : 0;
    return t;
}
// First key tile that some row of the tile does not see whole.
template <bool kCausal>
__device__ __forceinline__ int vl_first_masked(const VlUnit &u, const VlTile &t) {
    int whole = u.nk;
    if (kCausal && t.rel + 1 < whole) whole = t.rel + 1;
    return whole > 0 ? whole / kBN : 0;
}

// Bounds of sequence s, whatever the offsets hold: 0 <= a <= b <= total.
struct VlSpan {
    int a, b;
    bool bad;
};
__device__ __forceinline__ VlSpan vl_span(const int *cu, int s, int total) {
    const int a0 = __ldg(cu + s), b0 = __ldg(cu + s + 1);
    const int a = a0 < 0 ? 0 : (a0 > total ? total : a0);
    const int b = b0 < a ? a : (b0 > total ? total : b0);
    return {a, b, a != a0 || b != b0};
}
// (blocks << 16 | key blocks) of sequence s
__device__ __forceinline__ uint32_t vl_blocks(const VarlenParams &p, int s) {
    const VlSpan q = vl_span(p.cu_q, s, p.total_q), k = vl_span(p.cu_k, s, p.total_k);
    const uint32_t nqb = static_cast<uint32_t>((q.b - q.a + p.block_rows - 1) / p.block_rows);
    const uint32_t nkb = static_cast<uint32_t>((k.b - k.a + p.block_rows - 1) / p.block_rows);
    return (nqb << 16) | nkb;
}

// Walks the levels of the unit order (one warp, all lanes in step).
template <bool kCausal>
struct VlWalk {
    const VarlenParams &p;
    const uint32_t *cache;
    int lane;
    int level = INT_MAX;  // current level; blocks [base, base + count) lie on it
    int base = 0, count = 0;

    __device__ __forceinline__ uint32_t info(int s) const {
        return s < kVlSeqCache ? cache[s] : vl_blocks(p, s);
    }
    // blocks of a sequence on a level
    __device__ __forceinline__ int on_level(uint32_t x, int lev) const {
        const int nqb = static_cast<int>(x >> 16), H = static_cast<int>(x & 0xFFFFu);
        if (kCausal) return (lev <= H && lev > H - nqb) ? 1 : 0;
        return lev == H ? nqb : 0;
    }
    __device__ __forceinline__ bool next_level() {
        int best = INT_MIN;
        for (int s = lane; s < p.n_seqs; s += 32) {
            const uint32_t x = info(s);
            const int nqb = static_cast<int>(x >> 16), H = static_cast<int>(x & 0xFFFFu);
            if (nqb == 0) continue;
            const int cand = H < level ? H : level - 1;
            if (kCausal ? cand > H - nqb : cand == H) best = best > cand ? best : cand;
        }
        best = __reduce_max_sync(0xffffffffu, best);
        if (best == INT_MIN) return false;
        base += count;
        level = best;
        int n = 0;
        for (int s = lane; s < p.n_seqs; s += 32) n += on_level(info(s), level);
        count = __reduce_add_sync(0xffffffffu, n);
        return true;
    }
    // Block b (b never decreases from call to call): its sequence and place, or false.
    __device__ __forceinline__ bool find(int b, int &seq, int &qb) {
        while (b >= base + count)
            if (!next_level()) return false;
        int r = b - base;
        for (int s0 = 0; s0 < p.n_seqs; s0 += 32) {
            const int s = s0 + lane;
            const uint32_t x = s < p.n_seqs ? info(s) : 0u;
            const int c = s < p.n_seqs ? on_level(x, level) : 0;
            int incl = c;  // blocks of sequences up to this lane
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            const int total = __shfl_sync(0xffffffffu, incl, 31);
            if (r < total) {
                const int src = __ffs(__ballot_sync(0xffffffffu, incl > r)) - 1;
                const uint32_t y = __shfl_sync(0xffffffffu, x, src);
                const int before = __shfl_sync(0xffffffffu, incl - c, src);
                const int nqb = static_cast<int>(y >> 16), H = static_cast<int>(y & 0xFFFFu);
                seq = s0 + src;
                qb = kCausal ? nqb - 1 - (H - level) : r - before;
                return true;
            }
            r -= total;
        }
        return false;
    }
};

// Packed 16-bit magnitudes: a value is infinite or NaN when its exponent bits are all set.
template <bool kBF16>
__device__ __forceinline__ bool nonfinite16(uint32_t h) {
    constexpr uint32_t kExp = kBF16 ? 0x7F80u : 0x7C00u;
    return (h & kExp) == kExp;
}

// The guard's work on one V tile in shared memory: rows at or past `rows` become zero;
// with `scan`, non-finite values of the rows before are zeroed and their rows noted.
template <int D, bool kBF16>
__device__ __forceinline__ bool vl_guard_tile(uint8_t *tile, int rows, bool scan, uint32_t *bad_rows, int lane) {
    constexpr int kAtoms = D / 64;
    constexpr uint32_t kInf = kBF16 ? 0x7F80u : 0x7C00u;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    bool any = false;
#pragma unroll
    for (int a = 0; a < kAtoms; ++a) {
        uint4 *atom = reinterpret_cast<uint4 *>(tile + a * kAtomBytes);  // 8 chunks of 16 bytes a row
        for (int i = rows * 8 + lane; i < kBN * 8; i += 32) atom[i] = zero;
        if (!scan) continue;
        uint32_t m0 = 0, m1 = 0;  // largest magnitudes, two 16-bit lanes each
#pragma unroll 8
        for (int i = lane; i < rows * 8; i += 32) {
            const uint4 x = atom[i];
            m0 = __vimax3_u16x2(m0, x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu);
            m1 = __vimax3_u16x2(m1, x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu);
        }
        m0 = __vmaxu2(m0, m1);
        if (!__any_sync(0xffffffffu, (m0 & 0xFFFFu) >= kInf || (m0 >> 16) >= kInf)) continue;
        any = true;
        for (int i = lane; i < rows * 8; i += 32) {
            uint4 x = atom[i];
            uint32_t *w = reinterpret_cast<uint32_t *>(&x);
            bool hit = false;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (nonfinite16<kBF16>(w[t] & 0xFFFFu)) w[t] &= 0xFFFF0000u, hit = true;
                if (nonfinite16<kBF16>(w[t] >> 16)) w[t] &= 0x0000FFFFu, hit = true;
            }
            if (hit) {
                atom[i] = x;
                atomicOr(&bad_rows[(i >> 3) >> 5], 1u << ((i >> 3) & 31));
            }
        }
    }
    return any;
}

// tmQ, tmK, tmV: 3-D tensor maps of the packed rows, box 64 columns x 128 rows of one head
// with the 128-byte swizzle; rows past the end of the tensor read as zeros.
template <int D, bool kBF16, bool kCausal>
__global__ void __launch_bounds__(kWsThreads, 1)
    attn_fwd_varlen_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const __grid_constant__ VarlenParams p) {
    using L = VlLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const uint32_t sQ = base + L::kQ, sKV = base + L::kKV;
    const uint32_t bar0 = base + L::kBar;
    auto q_full = [&](int i) { return bar0 + 8u * i; };
    const uint32_t q_empty = bar0 + 8u * 2;
    auto kv_full = [&](int s) { return bar0 + 8u * (3 + s); };
    auto kv_empty = [&](int s) { return bar0 + 8u * (3 + kStagesWs + s); };
    auto s_full = [&](int i) { return bar0 + 8u * (3 + 2 * kStagesWs + i); };
    auto p_full = [&](int i) { return bar0 + 8u * (5 + 2 * kStagesWs + i); };
    auto o_full = [&](int i) { return bar0 + 8u * (7 + 2 * kStagesWs + i); };
    const uint32_t mma_done = bar0 + 8u * (9 + 2 * kStagesWs);
    const uint32_t v_ask = bar0 + 8u * (10 + 2 * kStagesWs), v_ok = bar0 + 8u * (11 + 2 * kStagesWs);
    auto unit_full = [&](int s) { return bar0 + 8u * (12 + 2 * kStagesWs + s); };
    auto unit_empty = [&](int s) { return bar0 + 8u * (12 + 2 * kStagesWs + kVlSlots + s); };
    volatile int *ask = reinterpret_cast<volatile int *>(smem + L::kAsk);
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + L::kTmemSlot);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kAbort);
    volatile uint32_t *flags = reinterpret_cast<volatile uint32_t *>(smem + L::kFlags);
    auto split_flag = [&](int i, int w) -> volatile uint32_t & { return flags[4 * i + w]; };
    VlUnit *units = reinterpret_cast<VlUnit *>(smem + L::kUnits);
    uint32_t *seqs = reinterpret_cast<uint32_t *>(smem + L::kSeqs);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    grid_launch_dependents();
    if (threadIdx.x == 64) {
        tma_prefetch_map(&tmQ);
        tma_prefetch_map(&tmK);
        tma_prefetch_map(&tmV);
    }
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        mbar_init(q_full(0), 1);
        mbar_init(q_full(1), 1);
        mbar_init(q_empty, 1);
        for (int s = 0; s < kStagesWs; ++s) {
            mbar_init(kv_full(s), 1);
            mbar_init(kv_empty(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full(i), 1);
            mbar_init(p_full(i), 4);  // one arrival per softmax warp
            mbar_init(o_full(i), 1);
        }
        mbar_init(mma_done, 1);
        mbar_init(v_ask, 1);
        mbar_init(v_ok, 1);
        for (int s = 0; s < kVlSlots; ++s) {
            mbar_init(unit_full(s), 1);
            mbar_init(unit_empty(s), 11);  // producer, MMA issuer, guard, 8 softmax warps
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(base + L::kTmemSlot, kWsTmemCols);
        tmem_relinquish();
    }
    // the set-up above overlaps the kernel before this one; its results are read from here on
    grid_dependency_wait();
    for (int s = threadIdx.x; s < p.n_seqs && s < kVlSeqCache; s += kWsThreads) seqs[s] = vl_blocks(p, s);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < 4) {
        regs_dec<kRegsLow>();
        if (warp == 3) {
            // ---------------------------------------------------- scheduler
            VlWalk<kCausal> walk{p, seqs, lane};
            int slot = 0;
            uint32_t phase = 0;
            for (unsigned r = 0;; ++r) {
                const unsigned c = (r & 1u) ? (gridDim.x - 1u - blockIdx.x) : blockIdx.x;
                const unsigned t = r * gridDim.x + c;
                int seq = 0, qb = 0;
                const bool more =
                    walk.find(static_cast<int>(t / static_cast<unsigned>(p.head_units)), seq, qb);
                if (!__all_sync(0xffffffffu, wait_bar(unit_empty(slot), phase ^ 1u, p, abort_flag))) break;
                if (lane == 0) {
                    VlUnit &u = units[slot];
                    u.valid = more ? 1 : 0;
                    if (more) {
                        const VlSpan q = vl_span(p.cu_q, seq, p.total_q), k = vl_span(p.cu_k, seq, p.total_k);
                        const int Nq = q.b - q.a, Nk = k.b - k.a;
                        u.head = static_cast<int>(t % static_cast<unsigned>(p.head_units)) * (p.pair ? 2 : 1);
                        u.q0 = q.a + qb * p.block_rows;
                        u.rows = Nq - qb * p.block_rows;
                        u.k0 = k.a;
                        u.nk = Nk;
                        u.rel = qb * p.block_rows + Nk - Nq;
                        u.bad = 0;
                    }
                    mbar_arrive(unit_full(slot));
                }
                __syncwarp();
                if (!more) break;
                if (++slot == kVlSlots) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
            // offsets that do not ascend within the tensors were read as clamped: say so
            if (blockIdx.x == 0) {
                bool bad = false;
                for (int s = lane; s < p.n_seqs; s += 32)
                    bad |= vl_span(p.cu_q, s, p.total_q).bad || vl_span(p.cu_k, s, p.total_k).bad;
                if (bad) atomicCAS(&g_error_code, 0, static_cast<int>(ATTN_ERR_SHAPE));
            }
        } else if (warp == 2 && lane == 0) {
            // ---------------------------------------------------- TMA producer
            Ring ring;
            int slot = 0;
            uint32_t uphase = 0;
            uint32_t fph = 0, armed = 0;  // full barriers as in the equal-length kernel
            int q_loads[2] = {0, 0}, q_units = 0;
            bool ok = true;
            auto issue = [&](uint32_t dst, const CUtensorMap *tm, int head_y, int row, int head, uint32_t bar) {
#pragma unroll
                for (int a = 0; a < D / 64; ++a)
                    tma_load_3d(dst + a * kAtomBytes, tm, 64 * a, head_y ? head : row, head_y ? row : head, bar);
            };
            while (ok) {
                if (!wait_bar(unit_full(slot), uphase, p, abort_flag)) break;
                const VlUnit u = units[slot];
                mbar_arrive(unit_empty(slot));
                if (++slot == kVlSlots) {
                    slot = 0;
                    uphase ^= 1u;
                }
                if (!u.valid) break;
                const VlTile t0 = vl_tile<kCausal>(p, u, 0), t1 = vl_tile<kCausal>(p, u, 1);
                const int n = t0.n > t1.n ? t0.n : t1.n;
                if (n == 0) continue;
                const int kvh = u.head / p.group;
                // first K tile: its own full barrier
                if (!(ok = wait_bar(kv_empty(ring.s), ring.ph ^ 1u, p, abort_flag))) break;
                mbar_arrive_expect_tx(kv_full(ring.s), L::kTileBytes);
                armed |= 1u << ring.s;
                fph ^= 1u << ring.s;
                issue(sKV + ring.s * L::kTileBytes, &tmK, p.k_head_y, u.k0, kvh, kv_full(ring.s));
                ring.next();
                // Q: its buffers are free once the S products of the unit before are done
                if (!(ok = wait_bar(q_empty, (q_units & 1) ^ 1u, p, abort_flag))) break;
                ++q_units;
                if (!p.inject_stall) {
                    if (t0.n > 0) {
                        mbar_arrive_expect_tx(q_full(0), L::kTileBytes);
                        issue(sQ, &tmQ, p.q_head_y, u.q0, u.head, q_full(0));
                        ++q_loads[0];
                    }
                    if (t1.n > 0) {
                        mbar_arrive_expect_tx(q_full(1), L::kTileBytes);
                        issue(sQ + L::kTileBytes, &tmQ, p.q_head_y, u.q0 + t1.row0, u.head + (p.pair ? 1 : 0),
                              q_full(1));
                        ++q_loads[1];
                    }
                }
                // V_j, and K_{j+1} if any, on V_j's barrier
                for (int j = 0; j < n && ok; ++j) {
                    const bool two = j + 1 < n;
                    const int vs = ring.s;
                    if (!(ok = wait_bar(kv_empty(vs), ring.ph ^ 1u, p, abort_flag))) break;
                    Ring nr = ring;
                    nr.next();
                    if (two && !(ok = wait_bar(kv_empty(nr.s), nr.ph ^ 1u, p, abort_flag))) break;
                    mbar_arrive_expect_tx(kv_full(vs), L::kTileBytes * (two ? 2u : 1u));
                    armed |= 1u << vs;
                    fph ^= 1u << vs;
                    issue(sKV + vs * L::kTileBytes, &tmV, p.v_head_y, u.k0 + j * kBN, kvh, kv_full(vs));
                    ring.next();
                    if (two) {
                        issue(sKV + ring.s * L::kTileBytes, &tmK, p.k_head_y, u.k0 + (j + 1) * kBN, kvh, kv_full(vs));
                        ring.next();
                    }
                }
            }
            // every copy has landed before the CTA exits (also after a timeout)
#pragma unroll
            for (int st = 0; st < kStagesWs; ++st)
                if ((armed >> st) & 1u) drain_bar(kv_full(st), ((fph >> st) & 1u) ^ 1u, p);
            if (q_loads[0] > 0) drain_bar(q_full(0), (q_loads[0] - 1) & 1, p);
            if (q_loads[1] > 0) drain_bar(q_full(1), (q_loads[1] - 1) & 1, p);
        } else if (warp == 0 && lane == 0) {
            // ---------------------------------------------------- MMA issuer
            constexpr uint32_t idesc_qk = idesc_f16_f32acc(kBF16, 128, kBN, false);
            constexpr uint32_t idesc_pv = idesc_f16_f32acc(kBF16, 128, D, true);
            Ring ring;
            uint32_t fph = 0;
            auto wait_full = [&](int st) -> bool {
                const bool r = wait_bar(kv_full(st), (fph >> st) & 1u, p, abort_flag);
                fph ^= 1u << st;
                return r;
            };
            uint32_t pcount[2] = {0, 0}, qcount[2] = {0, 0}, vcount = 0;
            int slot = 0;
            uint32_t uphase = 0;
            bool ok = true;
            const uint64_t dq0 = sdesc_sw128(sQ, 16, 1024);
            const uint64_t dkv0 = sdesc_sw128(sKV, 16, 1024);
            const uint64_t dv0 = sdesc_sw128(sKV, kAtomBytes, 1024);
            auto qk = [&](int i, int kstage) {
                const uint64_t a = dq0 + static_cast<uint64_t>(i * (L::kTileBytes >> 4));
                const uint64_t b = dkv0 + static_cast<uint64_t>(kstage * (L::kTileBytes >> 4));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t off = (kk >> 2) * (kAtomBytes >> 4) + (kk & 3) * 2;
                    mma_f16_ss(tmem + 128u * i, a + off, b + off, idesc_qk, kk > 0);
                }
            };
            // O_i (+)= P_i V, with the P_lo pass on the lanes of the warps that split
            auto pv = [&](int i, int vstage, bool acc) {
                const uint64_t b0 = dv0 + static_cast<uint64_t>(vstage * (L::kTileBytes >> 4));
                const uint32_t ta = tmem + 128u * i, td = tmem + 256u + 128u * i;
                uint32_t lo_off[4];
                bool split = false;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const bool sw = split_flag(i, w) != 0;
                    lo_off[w] = sw ? 0u : ~0u;
                    split |= sw;
                }
                const int passes = split ? 2 : 1;
#pragma unroll 1
                for (int h = 0; h < passes; ++h) {
                    const uint32_t off[4] = {h ? lo_off[0] : 0u, h ? lo_off[1] : 0u, h ? lo_off[2] : 0u,
                                             h ? lo_off[3] : 0u};
#pragma unroll
                    for (int kk = 0; kk < kBN / 16; ++kk)
                        mma_f16_ts_lanes(td, ta + 64u * h + 8u * kk, b0 + kk * (2048 >> 4), idesc_pv, off,
                                         (acc || kk > 0 || h > 0) ? 1u : 0u);
                }
            };
            while (ok) {
                if (!wait_bar(unit_full(slot), uphase, p, abort_flag)) break;
                const VlUnit &us = units[slot];
                VlUnit u;
                u.valid = us.valid, u.rows = us.rows, u.nk = us.nk, u.rel = us.rel;
                mbar_arrive(unit_empty(slot));
                if (++slot == kVlSlots) {
                    slot = 0;
                    uphase ^= 1u;
                }
                if (!u.valid) break;
                const VlTile t0 = vl_tile<kCausal>(p, u, 0), t1 = vl_tile<kCausal>(p, u, 1);
                const int n0 = t0.n, n1 = t1.n, n = n0 > n1 ? n0 : n1;
                if (n == 0) continue;
                // tiles from here on pass the guard before P V reads them
                const int g0 = vl_first_masked<kCausal>(u, t0);
                if (!(ok = wait_full(ring.s))) break;
                if (n0 > 0) {
                    if (!(ok = wait_bar(q_full(0), qcount[0]++ & 1u, p, abort_flag))) break;
                    tc_fence_after();
                    qk(0, ring.s);
                    mma_commit(s_full(0));
                }
                if (n1 > 0) {
                    if (!(ok = wait_bar(q_full(1), qcount[1]++ & 1u, p, abort_flag))) break;
                    tc_fence_after();
                    qk(1, ring.s);
                    mma_commit(s_full(1));
                }
                mma_commit(kv_empty(ring.s));
                if (n == 1) mma_commit(q_empty);
                ring.next();
                for (int j = 0; j < n; ++j) {
                    const int vs = ring.s;
                    if (!(ok = wait_full(vs))) break;  // V_j, and K_{j+1} if any
                    if (j >= g0) {
                        // V_j lies in its stage: the guard looks at it while P is computed
                        *ask = vs;
                        mbar_arrive(v_ask);
                        if (!(ok = wait_bar(v_ok, vcount++ & 1u, p, abort_flag))) break;
                    }
                    tc_fence_after();
                    ring.next();
                    const bool more = j + 1 < n;
                    const int ks = ring.s;
                    if (j < n0) {
                        if (!(ok = wait_bar(p_full(0), pcount[0]++ & 1u, p, abort_flag))) break;
                        tc_fence_after();
                        pv(0, vs, j > 0);
                        if (j == n0 - 1) mma_commit(o_full(0));
                    }
                    if (j + 1 < n0) {
                        qk(0, ks);
                        mma_commit(s_full(0));
                    }
                    if (j < n1) {
                        if (!(ok = wait_bar(p_full(1), pcount[1]++ & 1u, p, abort_flag))) break;
                        tc_fence_after();
                        pv(1, vs, j > 0);
                        if (j == n1 - 1) mma_commit(o_full(1));
                    }
                    mma_commit(kv_empty(vs));
                    if (more) {
                        if (j + 1 < n1) {
                            qk(1, ks);
                            mma_commit(s_full(1));
                        }
                        mma_commit(kv_empty(ks));
                        // the unit's last S product is issued: Q may be replaced
                        if (j + 2 == n) mma_commit(q_empty);
                        ring.next();
                    }
                }
            }
            // TMEM and shared memory stay alive until every issued MMA is done.
            mma_commit(mma_done);
            drain_bar(mma_done, 0, p);
        } else if (warp == 1) {
            // ---------------------------------------------------- value guard
            // The issuer asks for each guarded tile once it has seen the tile arrive, and waits
            // for the answer: the guard needs no count of the ring's phases of its own.
            int slot = 0;
            uint32_t uphase = 0, asked = 0;
            while (true) {
                if (!__all_sync(0xffffffffu, wait_bar(unit_full(slot), uphase, p, abort_flag))) break;
                VlUnit &us = units[slot];
                VlUnit u;
                u.valid = us.valid, u.rows = us.rows, u.nk = us.nk, u.rel = us.rel;
                if (!u.valid) break;
                const VlTile t0 = vl_tile<kCausal>(p, u, 0), t1 = vl_tile<kCausal>(p, u, 1);
                const int n = t0.n > t1.n ? t0.n : t1.n, g0 = vl_first_masked<kCausal>(u, t0);
                if (lane < kVlBadTiles * 4) us.bad_rows[lane >> 2][lane & 3] = 0;
                __syncwarp();
                bool ok = true;
                for (int j = g0; j < n; ++j) {
                    if (!(ok = __all_sync(0xffffffffu, wait_bar(v_ask, asked & 1u, p, abort_flag)))) break;
                    ++asked;
                    const int left = u.nk - j * kBN;
                    const bool any = vl_guard_tile<D, kBF16>(smem + L::kKV + *ask * L::kTileBytes,
                                                             left < kBN ? left : kBN, kCausal,
                                                             us.bad_rows[(j - g0) & (kVlBadTiles - 1)], lane);
                    if (any && lane == 0) us.bad = 1;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(v_ok);
                }
                if (!ok) break;
                if (lane == 0) mbar_arrive(unit_empty(slot));
                if (++slot == kVlSlots) {
                    slot = 0;
                    uphase ^= 1u;
                }
            }
        }
        __syncwarp();
    } else {
        regs_inc<kRegsHigh>();
        // -------------------------------------------------------- softmax
        const int i = (warp - 4) >> 2;  // query tile of this warpgroup
        const int wq = warp & 3;
        const int r = wq * 32 + lane;  // row within the tile == TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t tS = tmem + 128u * i + lane_off;  // S_i, and P_i in its first 64 columns
        const uint32_t tO = tmem + 256u + 128u * i + lane_off;
        const uint32_t stage = base + L::kStage + static_cast<uint32_t>(warp - 4) * L::kStageBytes;
        const float c = p.scale_log2;
        uint32_t scount = 0, ocount = 0;
        int slot = 0;
        uint32_t uphase = 0;
        bool ok = true;
        while (ok) {
            if (!__all_sync(0xffffffffu, wait_bar(unit_full(slot), uphase, p, abort_flag))) break;
            const VlUnit &us = units[slot];
            VlUnit u;
            u.valid = us.valid, u.rows = us.rows, u.nk = us.nk, u.rel = us.rel;
            if (!u.valid) break;
            const VlTile t = vl_tile<kCausal>(p, u, i);
            const int first_masked = vl_first_masked<kCausal>(u, t);
            // m_ref: the max the probabilities are taken against (updated lazily);
            // m_top: the true running row max; l: running sum in units of 2^(m_ref*c).
            float m_ref = -INFINITY, m_top = -INFINITY, l = 0.f;
            for (int j = 0; j < t.n; ++j) {
                if (!__all_sync(0xffffffffu, wait_bar(s_full(i), scount & 1u, p, abort_flag))) {
                    ok = false;
                    break;
                }
                ++scount;
                tc_fence_after();
                __syncwarp();
                uint32_t s[128];
                if (j < first_masked) {
                    float mq[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        tmem_ld32_max(tS + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * q]), mq[q]);
                    tmem_ld_wait(s, mq);
                    m_top = fmaxf(m_top, fmax3(mq[0], mq[1], fmaxf(mq[2], mq[3])));
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        tmem_ld32(tS + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * q]));
                    tmem_ld_wait(s);
                    int lim = u.nk - 1;
                    if (kCausal && r + t.rel < lim) lim = r + t.rel;
                    lim -= j * kBN;  // row r keeps keys c <= lim of this tile
#pragma unroll
                    for (int cc = 0; cc < 128; ++cc)
                        if (cc > lim) s[cc] = __float_as_uint(-INFINITY);
                    float mx[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) mx[k] = fmaxf(u2f(s[2 * k]), u2f(s[2 * k + 1]));
#pragma unroll
                    for (int cc = 16; cc < 128; cc += 16)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mx[k] = fmax3(mx[k], u2f(s[cc + 2 * k]), u2f(s[cc + 2 * k + 1]));
                    m_top = fmaxf(m_top, fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]),
                                               fmaxf(mx[6], mx[7])));
                }
                float alpha = 1.f;
                bool rescale = false;
                if (m_ref == -INFINITY) {
                    m_ref = m_top;  // nothing seen so far: the accumulator holds zeros at most
                } else if ((m_top - m_ref) * c > kRescaleLog2) {
                    alpha = ex2_approx((m_ref - m_top) * c);
                    m_ref = m_top;
                    rescale = true;
                }
                // a row that has seen no key yet takes its weights, all 0, against 0
                const float mr = m_ref == -INFINITY ? 0.f : m_ref;
                const float2 c2 = make_float2(c, c);
                const float2 nmc2 = make_float2(-mr * c, -mr * c);
                float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int cc = 0; cc < 128; cc += 2) {
                    float2 e = ffma2(make_float2(u2f(s[cc]), u2f(s[cc + 1])), c2, nmc2);
                    e.x = ex2_approx(e.x);
                    e.y = ex2_approx(e.y);
                    acc[(cc >> 1) & 1] = fadd2(acc[(cc >> 1) & 1], e);
                    s[cc] = __float_as_uint(e.x);
                    s[cc + 1] = __float_as_uint(e.y);
                }
                const float2 sum2 = fadd2(acc[0], acc[1]);
                l = l * alpha + (sum2.x + sum2.y);
                // P = P_hi + P_lo for a warp with a row whose weight lies on few keys
                const bool need = r < t.valid && l * ex2_approx((m_ref - m_top) * c) < kSplitL;
                const bool split = __any_sync(0xffffffffu, need);
                if (lane == 0) split_flag(i, wq) = split ? 1u : 0u;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        pk[e] = pack2<kBF16>(u2f(s[32 * q + 2 * e]), u2f(s[32 * q + 2 * e + 1]));
                    tmem_st16(tS + 16 * q, pk);
                    if (split) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 h = unpack2<kBF16>(pk[e]);
                            pk[e] = pack2<kBF16>(u2f(s[32 * q + 2 * e]) - h.x, u2f(s[32 * q + 2 * e + 1]) - h.y);
                        }
                        tmem_st16(tS + 64 + 16 * q, pk);
                    }
                }
                if (__any_sync(0xffffffffu, rescale)) {
                    // O_i holds P_i V_{j-1} already (covered by the S_i(j) commit).
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
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(i));
            }
            if (!ok) break;
            // ---------------------------------------------------- epilogue
            const int head = us.head + (p.pair ? i : 0);
            const int qrow = us.q0 + t.row0;  // packed row of the tile's first row
            if (t.n > 0) {
                if (!__all_sync(0xffffffffu, wait_bar(o_full(i), ocount & 1u, p, abort_flag))) break;
                ++ocount;
                tc_fence_after();
                __syncwarp();
            }
            if (t.valid > wq * 32) {
                const bool bad = t.n > 0 && *reinterpret_cast<const volatile int *>(&us.bad) != 0;
                const float inv_l = l == 0.f ? 0.f : 1.f / l;  // 0: the row saw no key
                const int rd_row = lane >> 2, rd_c = lane & 3;
                uint8_t *otile = static_cast<uint8_t *>(p.o) + head * p.o_head + (qrow + wq * 32) * p.o_row;
                const int wvalid = t.valid - wq * 32;  // rows of this warp
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t o[32];
                    if (t.n > 0) {
                        tmem_ld32(tO + 32 * q, o);
                        tmem_ld_wait(o);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0u;
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(u2f(o[e]) * inv_l);
                    if (bad) {
                        // non-finite values that the guard took out of V, for the rows that see them
                        const int g0 = vl_first_masked<kCausal>(u, vl_tile<kCausal>(p, u, 0));
                        const uint8_t *vh = p.v_ptr + (us.head / p.group) * p.v_head;
                        int lim = u.nk - 1;
                        if (kCausal && r + t.rel < lim) lim = r + t.rel;
                        if (r >= t.valid) lim = -1;
                        for (int g = 0; g < kVlBadTiles; ++g)
                            for (int w = 0; w < 4; ++w)
                                for (uint32_t bits = us.bad_rows[g][w]; bits != 0; bits &= bits - 1) {
                                    const int key = (g0 + g) * kBN + 32 * w + __ffs(bits) - 1;
                                    if (key > lim) continue;
                                    const uint32_t *vr = reinterpret_cast<const uint32_t *>(
                                        vh + (us.k0 + key) * p.v_row + q * 64);
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        const uint32_t x = __ldg(vr + e);
                                        const float2 f = unpack2<kBF16>(x);
                                        if (nonfinite16<kBF16>(x & 0xFFFFu)) o[2 * e] = __float_as_uint(u2f(o[2 * e]) + f.x);
                                        if (nonfinite16<kBF16>(x >> 16)) o[2 * e + 1] = __float_as_uint(u2f(o[2 * e + 1]) + f.y);
                                    }
                                }
                    }
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = pack2<kBF16>(u2f(o[2 * e]), u2f(o[2 * e + 1]));
                    // whole 64-byte row segments through the warp's staging rows
                    __syncwarp();
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        st_shared_v4(stage + lane * 64 + ((v ^ ((lane >> 1) & 3)) << 4), w[4 * v], w[4 * v + 1],
                                     w[4 * v + 2], w[4 * v + 3]);
                    __syncwarp();
#pragma unroll
                    for (int s4 = 0; s4 < 4; ++s4) {
                        const int tr = 8 * s4 + rd_row;
                        const uint4 xv = ld_shared_v4(stage + tr * 64 + ((rd_c ^ ((tr >> 1) & 3)) << 4));
                        if (tr < wvalid) st_global_v4(otile + tr * p.o_row + q * 64 + rd_c * 16, xv.x, xv.y, xv.z, xv.w);
                    }
                }
                if (p.lse != nullptr && r < t.valid)
                    p.lse[static_cast<size_t>(head) * p.total_q + qrow + r] =
                        l == 0.f ? -INFINITY : (m_ref * c + log2f(l)) * 0.6931471805599453f;
            }
            // O_i is read; the next unit's first P_i V waits for this warpgroup's p_full, and
            // the descriptor may be replaced
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(unit_empty(slot));
            if (++slot == kVlSlots) {
                slot = 0;
                uphase ^= 1u;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kWsTmemCols);
    }
}

}  // namespace gqa
