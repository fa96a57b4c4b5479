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
// Units without keys are not handed out: the scheduler warp stores their zeros itself.  The
// producer, the issuer and the guard look one unit ahead, and the unit at work keeps its
// descriptor slot until its last V tile, which the producer loads after that look: a look past
// any number of units without keys would wait for slots that wait for it.  (Handing them out
// behind the others, to the softmax warps alone, takes a second walk and 58.6 us instead of 37.7
// for 8192 queries over 512 keys, Hq 32, D 128; not inlining the stores 67.1.)
//
// Roles (384 threads): warp 0 MMA issuer, warp 1 value guard (and TMEM), warp 2 TMA
// producer, warp 3 scheduler, warps 4-7 and 8-11 the softmax of tile 0 and 1.  Shared memory,
// TMEM and the K/V ring are laid out as in the equal-length kernel.  Units follow each other
// without a pause: the next unit's first K tile is loaded with the last V tile of the unit
// before, its first scores are computed right after that unit's last P V of the same tile,
// and a softmax warp stores O of a unit only after it has handed over the first weights of
// the next one, when the last P V has long finished.
//
// Rounding.  P is rounded to the input type, against a stale row max (weights up to 2^8 of the
// reference): half a step of each weight, the same as the output's own rounding.
//
// Window (attn_fwd_varlen_window).  A unit visits the key tiles of the first keys and those from the
// first key of its first row's window on; tiles that no row sees are neither loaded nor computed (4
// D flops per visible pair bound it in the same way, plus what the tiles on the three borders, the
// end of the first keys, the window's start and the diagonal, hold besides: with a window of 512 half
// of the steps).  Masked tiles go in one pass, as a word of bits per row and 32 columns: with windows
// they are too many of all tiles for the two passes of the plain kernel (12 prompts of 1 to 4096,
// Hq 16, D 128, window 512: 84.4 us in two passes, 82.1 in one; one prompt of 200, window 64, D 64
// 11.0 and 9.0; two of 16384 and 9001, Hq 32, window 2048 611 and 587, 1.37 PFLOP/s; the 12 prompts with
// D 64 69, where the kernel loads 512 bytes of spills in all).  Taking the first
// keys' tile as products of 16 ceil(n / 16) keys saves a sixth of the first case's MMAs and costs
// time (84.7): the steps' round trips between the roles bound short units, not their products.
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
constexpr int kVlSeqs = 2048;     // most sequences of one launch (their block counts lie in shared memory)
constexpr int kVlBadTiles = 4;    // key tiles of a unit that the guard may look at
// ... with a window: one where the first keys end, three at the window's start, three at the diagonal
constexpr int kVlBadTilesWin = 8;

struct VarlenParams : Params {
    const int *cu_q, *cu_k;  // device [n_seqs + 1]
    const uint8_t *v_ptr;    // V in global memory (the rare non-finite rows are read again)
    int n_seqs, total_q, total_k;  // n_seqs <= kVlSeqs
    int pair;                // 1: the tiles are two heads of a group; 0: two row tiles of a head
    int block_rows;          // query rows of a unit: 128 (pair) or 256
    int head_units;          // units per block of rows: Hq / 2 (pair) or Hq
    int most_blocks;         // blocks of rows that ascending offsets can have
    int window, sinks;       // window kernels: row at position p sees j <= p with j > p - window or j < sinks
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
    uint32_t bad_rows[kVlBadTilesWin][4];  // rows of the guarded V tiles with a non-finite value
};

template <int D>
struct VlLayout {
    using W = WsLayout<D>;
    static constexpr int kTileBytes = W::kTileBytes;
    static constexpr int kQ = W::kQ, kKV = W::kKV;
    static constexpr int kStageBytes = W::kStageBytes;  // epilogue staging of a softmax warp
    static constexpr int kStage = kKV + kStagesWs * kTileBytes;
    static constexpr int kBar = kStage + 8 * kStageBytes;
    // q_full[2], kv_full[S], kv_empty[S], s_full[2], p_full[2], o_full[2], o_empty[2], mma_done,
    // v_ok[2], unit_full[slots], unit_empty[slots]
    static constexpr int kNumBars = 2 + 2 * kStagesWs + 4 * 2 + 1 + 2 + 2 * kVlSlots;
    static constexpr int kTmemSlot = kBar + kNumBars * 8;
    static constexpr int kAbort = kTmemSlot + 4;
    static constexpr int kUnits = (kAbort + 4 + 15) & ~15;
    static constexpr int kSeqs = kUnits + kVlSlots * static_cast<int>(sizeof(VlUnit));
    static constexpr int kUsed = kSeqs + kVlSeqs * 4;
    static constexpr int kAlloc = (kUsed + 1024) > 118 * 1024 ? (kUsed + 1024) : 118 * 1024;
};
static_assert(VlLayout<128>::kAlloc <= 227 * 1024, "shared memory of one CTA");

// With a window, the key tiles that no row of a unit sees are left out: those between the tiles of
// the first `sinks` keys and the tile that holds the first key of the unit's first row's window.
// Steps j = 0, 1, .. of the unit then visit key tiles j, from the sinks' tiles on j + skip.
__device__ __forceinline__ int win_tiles(int keys) { return (keys + kBN - 1) / kBN; }
__device__ __forceinline__ int win_skip(int first_pos, int window, int sinks) {
    const int lo = first_pos - window + 1, gap = lo > 0 ? lo / kBN - win_tiles(sinks) : 0;
    return gap > 0 ? gap : 0;
}
template <bool kWindow>
__device__ __forceinline__ int win_key_tile(int j, int sinks, int skip) {
    if constexpr (!kWindow) return j;
    return j < win_tiles(sinks) ? j : j + skip;
}
// The steps whose tiles the rows at positions first_pos .. last_pos see whole, of keys 0 .. nk - 1
// (`nk`, or the first position that is not seen by all): steps below `sink` and in [w0, w1).
struct WinWhole {
    int sink, w0, w1;
    __device__ __forceinline__ bool operator()(int j) const { return j < sink || (j >= w0 && j < w1); }
};
__device__ __forceinline__ WinWhole win_whole(int nk, int first_pos, int last_pos, int window, int sinks, int skip) {
    const int end = first_pos + 1 < nk ? first_pos + 1 : nk;  // keys below are seen, but for the window
    WinWhole w;
    w.sink = end > 0 ? (sinks < end ? sinks : end) / kBN : 0;
    w.w0 = last_pos - window >= 0 ? (last_pos - window) / kBN + 1 - skip : 0;
    w.w1 = end > 0 ? end / kBN - skip : 0;
    return w;
}

// Tile i of a unit: its rows, head and the key tiles [0, n) that it visits.
struct VlTile {
    int row0;   // first row of the tile within the block
    int valid;  // query rows of the tile (0: absent)
    int rel;    // row r of the tile sees keys j <= r + rel (causal)
    int n;      // key tiles
    int skip;   // key tiles left out behind the first ones (0 without a window)
};
template <bool kCausal, bool kWindow>
__device__ __forceinline__ VlTile vl_tile(const VarlenParams &p, const VlUnit &u, int i) {
    VlTile t;
    t.row0 = p.pair ? 0 : kBM * i;
    const int left = u.rows - t.row0;
    t.valid = left < 0 ? 0 : (left < kBM ? left : kBM);
    t.rel = u.rel + t.row0;
    int seen = u.nk;
    if (kCausal && t.rel + t.valid < seen) seen = t.rel + t.valid;
    t.skip = kWindow ? win_skip(u.rel, p.window, p.sinks) : 0;
    t.n = (t.valid > 0 && seen > 0) ? (seen + kBN - 1) / kBN - t.skip : 0;
    return t;
}
// The steps of tile t whose keys all its rows see (window kernels).
__device__ __forceinline__ WinWhole vl_whole(const VarlenParams &p, const VlUnit &u, const VlTile &t) {
    return win_whole(u.nk, t.rel, t.rel + t.valid - 1, p.window, p.sinks, t.skip);
}
// The same for both tiles of a unit: the others pass the guard.
__device__ __forceinline__ WinWhole vl_unguarded(const VarlenParams &p, const VlUnit &u) {
    const int rows = u.rows < p.block_rows ? u.rows : p.block_rows;
    return win_whole(u.nk, u.rel, u.rel + rows - 1, p.window, p.sinks, win_skip(u.rel, p.window, p.sinks));
}
// Whether some row of a unit sees a key: of its rows, `rows` to the end of the sequence, the
// last one sees most.
template <bool kCausal>
__device__ __forceinline__ bool vl_has_keys(const VarlenParams &p, int rows, int nk, int rel) {
    return nk > 0 && (!kCausal || rel + (rows < p.block_rows ? rows : p.block_rows) > 0);
}
// Rows of one head that see no key (one warp): O = 0, LSE = -inf.
template <int D>
__device__ __forceinline__ void vl_store_blind(uint8_t *o, long long o_row, float *lse, int rows, int lane) {
    o += lane / (D / 8) * o_row + lane % (D / 8) * 16;
#pragma unroll 4
    for (int r = lane / (D / 8); r < rows; r += 32 / (D / 8)) {
        st_global_v4(o, 0u, 0u, 0u, 0u);
        o += 32 / (D / 8) * o_row;
    }
    if (lse != nullptr)
        for (int r = lane; r < rows; r += 32) lse[r] = -INFINITY;
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
template <bool kAhead = false>  // read ahead of grid_dependency_wait
__device__ __forceinline__ VlSpan vl_span(const int *cu, int s, int total) {
    const int a0 = ld_state<kAhead>(cu + s), b0 = ld_state<kAhead>(cu + s + 1);
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
    const uint32_t *blocks;  // vl_blocks of every sequence
    int lane;
    int level = INT_MAX;  // current level; blocks [base, base + count) lie on it
    int base = 0, count = 0;

    // blocks of a sequence on a level
    __device__ __forceinline__ int on_level(uint32_t x, int lev) const {
        const int nqb = static_cast<int>(x >> 16), H = static_cast<int>(x & 0xFFFFu);
        if (kCausal) return (lev <= H && lev > H - nqb) ? 1 : 0;
        return lev == H ? nqb : 0;
    }
    __device__ __forceinline__ bool next_level() {
        int best = INT_MIN;
        for (int s = lane; s < p.n_seqs; s += 32) {
            const uint32_t x = blocks[s];
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
        for (int s = lane; s < p.n_seqs; s += 32) n += on_level(blocks[s], level);
        count = __reduce_add_sync(0xffffffffu, n);
        return true;
    }
    // Block b (b never decreases from call to call): its sequence and place, or false.  Offsets
    // that descend can overlap, up to n_seqs times the rows: the walk ends at what ascending ones
    // can have.
    __device__ __forceinline__ bool find(int b, int &seq, int &qb) {
        if (b >= p.most_blocks) return false;
        while (b >= base + count)
            if (!next_level()) return false;
        int r = b - base;
        for (int s0 = 0; s0 < p.n_seqs; s0 += 32) {
            const int s = s0 + lane;
            const uint32_t x = s < p.n_seqs ? blocks[s] : 0u;
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

// The two products of a key tile, with the matrix descriptors of sdesc_sw128 put together in
// the instruction's own block: the upper word is a constant, the lower one (start address and
// leading offset, in 16-byte units) a base plus a constant, so that one register per operand is
// live and no descriptors are hoisted out of the issuer's loop (there they spilled).  What the
// kernel still spills is 12 bytes stored and 4 loaded at D = 128, 24 and 88 to 96 at D = 64, in all (with
// a window 12 and 4, 32 and 512).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // stride 1024 B, version 1, swizzle 128 B
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo_bytes) {
    return ((saddr & 0x3FFFFu) >> 4) | ((lbo_bytes >> 4) << 16);
}
// D[tmem] (+)= A[smem + off] B[smem + off]^T
template <uint32_t kIdesc, uint32_t kOff, bool kAcc>
__device__ __forceinline__ void mma_ss_at(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 x, y, h, i;\n\t.reg .b64 a, b;\n\t"
        "add.u32 x, %1, %5;\n\tadd.u32 y, %2, %5;\n\tmov.u32 h, %3;\n\tmov.u32 i, %4;\n\t"
        "mov.b64 a, {x, h};\n\tmov.b64 b, {y, h};\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, i, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "n"(kDescHi), "n"(kIdesc), "n"(kOff), "n"(kAcc ? 1 : 0)
        : "memory");
}
// D[tmem] (+)= A[tmem + off_a] B[smem + off]^T
template <uint32_t kIdesc, uint32_t kOffA, uint32_t kOff>
__device__ __forceinline__ void mma_ts_at(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 x, y, h, i;\n\t.reg .b64 b;\n\t"
        "add.u32 x, %1, %5;\n\tadd.u32 y, %2, %6;\n\tmov.u32 h, %3;\n\tmov.u32 i, %4;\n\t"
        "mov.b64 b, {y, h};\n\tsetp.ne.u32 p, %7, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, i, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "n"(kDescHi), "n"(kIdesc), "n"(kOffA), "n"(kOff), "r"(acc)
        : "memory");
}
// S = Q K^T of one 128 x 128 tile (K-major operands), and O (+)= P V (P in TMEM, V MN-major)
template <int D, bool kBF16, int kk = 0>
__device__ __forceinline__ void mma_qk(uint32_t td, uint32_t q_lo, uint32_t k_lo) {
    if constexpr (kk < D / 16) {
        mma_ss_at<idesc_f16_f32acc(kBF16, 128, kBN, false), (kk >> 2) * (kAtomBytes >> 4) + (kk & 3) * 2, (kk > 0)>(
            td, q_lo, k_lo);
        mma_qk<D, kBF16, kk + 1>(td, q_lo, k_lo);
    }
}
template <int D, bool kBF16, int kk = 0>
__device__ __forceinline__ void mma_pv(uint32_t to, uint32_t tp, uint32_t v_lo, uint32_t acc) {
    if constexpr (kk < kBN / 16) {
        mma_ts_at<idesc_f16_f32acc(kBF16, 128, D, true), 8u * kk, kk * (2048 >> 4)>(to, tp, v_lo, kk > 0 ? 1u : acc);
        mma_pv<D, kBF16, kk + 1>(to, tp, v_lo, acc);
    }
}

// Packed 16-bit magnitudes: a value is infinite or NaN when its exponent bits are all set.
template <bool kBF16>
__device__ __forceinline__ bool nonfinite16(uint32_t h) {
    constexpr uint32_t kExp = kBF16 ? 0x7F80u : 0x7C00u;
    return (h & kExp) == kExp;
}

// 0 * x + acc in both 16-bit halves: acc, or NaN from the first non-finite value on.
template <bool kBF16>
__device__ __forceinline__ uint32_t zero_times(uint32_t x, uint32_t acc) {
    uint32_t d;
    if constexpr (kBF16)
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(x), "r"(0u), "r"(acc));
    else
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(x), "r"(0u), "r"(acc));
    return d;
}

// Adds the non-finite values of a row of V to a stored row of O.
template <int D, bool kBF16>
__device__ __forceinline__ void add_nonfinite(uint8_t *o_row, const uint8_t *v_row) {
#pragma unroll 1
    for (int d = 0; d < D; ++d) {
        const uint32_t x = reinterpret_cast<const uint16_t *>(v_row)[d];
        if (!nonfinite16<kBF16>(x)) continue;
        volatile uint16_t *o = reinterpret_cast<volatile uint16_t *>(o_row) + d;
        *o = static_cast<uint16_t>(pack2<kBF16>(unpack2<kBF16>(*o).x + unpack2<kBF16>(x).x, 0.f));
    }
}

// As add_nonfinite, for a row of fp32 partial results.
template <int D, bool kBF16>
__device__ __forceinline__ void add_nonfinite_f32(float *o_row, const uint8_t *v_row) {
#pragma unroll 1
    for (int d = 0; d < D; ++d) {
        const uint32_t x = reinterpret_cast<const uint16_t *>(v_row)[d];
        volatile float *o = o_row + d;
        if (nonfinite16<kBF16>(x)) *o = *o + unpack2<kBF16>(x).x;
    }
}

// The guard's work on one V tile in shared memory: rows at or past `rows` become zero;
// with `scan`, non-finite values of the rows before are zeroed and their rows noted.  Rows [z0, z1)
// become zero, too.
template <int D, bool kBF16>
__device__ __forceinline__ bool vl_guard_tile(uint8_t *tile, int rows, bool scan, uint32_t *bad_rows, int lane,
                                              int z0 = 0, int z1 = 0) {
    constexpr int kAtoms = D / 64;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    bool any = false;
#pragma unroll
    for (int a = 0; a < kAtoms; ++a) {
        uint4 *atom = reinterpret_cast<uint4 *>(tile + a * kAtomBytes);  // 8 chunks of 16 bytes a row
        for (int i = rows * 8 + lane; i < kBN * 8; i += 32) atom[i] = zero;
        for (int i = z0 * 8 + lane; i < z1 * 8; i += 32) atom[i] = zero;
        if (!scan) continue;
        // 0 times a value, summed: NaN exactly where one is not finite.  The rows past the end are
        // zeros by now, so all 128 are taken, with a fixed count of loads in flight.
        __syncwarp();
        uint32_t sum[4] = {0u, 0u, 0u, 0u};
#pragma unroll 8
        for (int i = 0; i < kBN * 8 / 32; ++i) {
            const uint4 x = atom[i * 32 + lane];
            sum[0] = zero_times<kBF16>(x.x, sum[0]);
            sum[1] = zero_times<kBF16>(x.y, sum[1]);
            sum[2] = zero_times<kBF16>(x.z, sum[2]);
            sum[3] = zero_times<kBF16>(x.w, sum[3]);
        }
        if (!__any_sync(0xffffffffu, ((sum[0] | sum[1] | sum[2] | sum[3]) & 0x7FFF7FFFu) != 0)) continue;
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
// kWindow (causal): attn_fwd_varlen_window.
template <int D, bool kBF16, bool kCausal, bool kWindow>
__global__ void __launch_bounds__(kWsThreads, 1)
    attn_fwd_varlen_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const __grid_constant__ VarlenParams p) {
    static_assert(kCausal || !kWindow, "a window is causal");
    using L = VlLayout<D>;
    constexpr int kBad = kWindow ? kVlBadTilesWin : kVlBadTiles;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const uint32_t sQ = base + L::kQ, sKV = base + L::kKV;
    const uint32_t bar0 = base + L::kBar;
    auto q_full = [&](int i) { return bar0 + 8u * i; };
    auto kv_full = [&](int s) { return bar0 + 8u * (2 + s); };
    auto kv_empty = [&](int s) { return bar0 + 8u * (2 + kStagesWs + s); };
    auto s_full = [&](int i) { return bar0 + 8u * (2 + 2 * kStagesWs + i); };
    auto p_full = [&](int i) { return bar0 + 8u * (4 + 2 * kStagesWs + i); };
    auto o_full = [&](int i) { return bar0 + 8u * (6 + 2 * kStagesWs + i); };
    auto o_empty = [&](int i) { return bar0 + 8u * (8 + 2 * kStagesWs + i); };  // O_i has been read
    const uint32_t mma_done = bar0 + 8u * (10 + 2 * kStagesWs);
    auto v_ok = [&](int b) { return bar0 + 8u * (11 + 2 * kStagesWs + b); };  // stage 1, 3 has passed the guard
    auto unit_full = [&](int s) { return bar0 + 8u * (13 + 2 * kStagesWs + s); };
    auto unit_empty = [&](int s) { return bar0 + 8u * (13 + 2 * kStagesWs + kVlSlots + s); };
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + L::kTmemSlot);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kAbort);
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
        for (int s = 0; s < kStagesWs; ++s) {
            mbar_init(kv_full(s), 1);
            mbar_init(kv_empty(s), 1 + (s & 1));  // V (the odd stages) is freed by the issuer and the guard
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(v_ok(i), 1);
            mbar_init(q_full(i), 1);
            mbar_init(s_full(i), 1);
            mbar_init(p_full(i), 4);  // one arrival per softmax warp of the tile
            mbar_init(o_full(i), 1);
            mbar_init(o_empty(i), 4);
        }
        mbar_init(mma_done, 1);
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
    for (int s = threadIdx.x; s < p.n_seqs; s += kWsThreads) seqs[s] = vl_blocks(p, s);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < 4) {
        regs_dec<kRegsLow>();
        if (warp == 2 && lane == 0) {
            // ---------------------------------------------------- TMA producer
            // The ring holds K_0, then V_j and the K tile after it (K_{j+1}, or the next unit's
            // K_0) in pairs that complete V_j's barrier together, so that the issuer waits once
            // per key tile; every stage keeps its own phase bit (fph).
            struct Cur {
                int valid, n, n0, n1, q0, q1, head, k0, skip;
            };
            Ring ring;
            int slot = 0;
            uint32_t uphase = 0, fph = 0, armed = 0;
            uint32_t scores[2] = {0, 0};  // score tiles of the units before, per query tile
            int q_loads[2] = {0, 0};
            auto issue = [&](uint32_t dst, const CUtensorMap *tm, int head_y, int row, int head, uint32_t bar) {
#pragma unroll
                for (int a = 0; a < D / 64; ++a)
                    tma_load_3d(dst + a * kAtomBytes, tm, 64 * a, head_y ? head : row, head_y ? row : head, bar);
            };
            // the next unit (valid 0: none); it has keys, as every unit that is handed out
            auto fetch = [&](Cur &c) -> bool {
                if (!wait_bar(unit_full(slot), uphase, p, abort_flag)) return false;
                const VlUnit &u = units[slot];
                c.valid = u.valid;
                if (c.valid) {
                    const VlTile t0 = vl_tile<kCausal, kWindow>(p, u, 0), t1 = vl_tile<kCausal, kWindow>(p, u, 1);
                    c.n0 = t0.n;
                    c.n1 = t1.n;
                    c.n = t0.n > t1.n ? t0.n : t1.n;
                    c.q0 = u.q0;
                    c.q1 = u.q0 + t1.row0;
                    c.head = u.head;
                    c.k0 = u.k0;
                    c.skip = t0.skip;
                }
                mbar_arrive(unit_empty(slot));
                if (++slot == kVlSlots) {
                    slot = 0;
                    uphase ^= 1u;
                }
                return true;
            };
            auto load_q = [&](int i, const Cur &c) -> bool {
                if ((i ? c.n1 : c.n0) == 0) return true;
                // Q_i is free once the last score product of tile i is done; that barrier cannot
                // turn again before this load
                if (scores[i] > 0 && !wait_bar(s_full(i), (scores[i] - 1) & 1u, p, abort_flag)) return false;
                if (p.inject_stall) return true;
                mbar_arrive_expect_tx(q_full(i), L::kTileBytes);
                issue(sQ + i * L::kTileBytes, &tmQ, p.q_head_y, i ? c.q1 : c.q0, c.head + (i & p.pair), q_full(i));
                ++q_loads[i];
                return true;
            };
            Cur cur{}, nxt{};
            bool ok = fetch(cur);
            if (ok && cur.valid) {
                mbar_arrive_expect_tx(kv_full(0), L::kTileBytes);
                armed |= 1u;
                fph ^= 1u;
                issue(sKV, &tmK, p.k_head_y, cur.k0 + win_key_tile<kWindow>(0, p.sinks, cur.skip) * kBN,
                      cur.head / p.group, kv_full(0));
                ring.next();
                ok = load_q(0, cur) && load_q(1, cur);
            }
            while (ok && cur.valid) {
                const int kvh = cur.head / p.group;
                for (int j = 0; j < cur.n && ok; ++j) {
                    bool two = true;
                    int krow = cur.k0 + win_key_tile<kWindow>(j + 1, p.sinks, cur.skip) * kBN, khead = kvh;
                    if (j + 1 == cur.n) {
                        if (!(ok = fetch(nxt))) break;
                        two = nxt.valid != 0;
                        krow = nxt.k0 + win_key_tile<kWindow>(0, p.sinks, nxt.skip) * kBN;
                        khead = nxt.head / p.group;
                    }
                    const int vs = ring.s;
                    if (!(ok = wait_bar(kv_empty(vs), ring.ph ^ 1u, p, abort_flag))) break;
                    Ring nr = ring;
                    nr.next();
                    if (two && !(ok = wait_bar(kv_empty(nr.s), nr.ph ^ 1u, p, abort_flag))) break;
                    mbar_arrive_expect_tx(kv_full(vs), L::kTileBytes * (two ? 2u : 1u));
                    armed |= 1u << vs;
                    fph ^= 1u << vs;
                    issue(sKV + vs * L::kTileBytes, &tmV, p.v_head_y,
                          cur.k0 + win_key_tile<kWindow>(j, p.sinks, cur.skip) * kBN, kvh, kv_full(vs));
                    ring.next();
                    if (two) {
                        issue(sKV + ring.s * L::kTileBytes, &tmK, p.k_head_y, krow, khead, kv_full(vs));
                        ring.next();
                    }
                }
                if (!ok) break;
                scores[0] += cur.n0;
                scores[1] += cur.n1;
                cur = nxt;
                if (cur.valid) ok = load_q(0, cur) && load_q(1, cur);
            }
            // every copy has landed before the CTA exits (also after a timeout)
#pragma unroll
            for (int st = 0; st < kStagesWs; ++st)
                if ((armed >> st) & 1u) drain_bar(kv_full(st), ((fph >> st) & 1u) ^ 1u, p);
            if (q_loads[0] > 0) drain_bar(q_full(0), (q_loads[0] - 1) & 1, p);
            if (q_loads[1] > 0) drain_bar(q_full(1), (q_loads[1] - 1) & 1, p);
        } else if (warp == 0 && lane == 0) {
            // ---------------------------------------------------- MMA issuer
            struct Cur {
                int valid, n, n0, n1, g0;  // g0: tiles from here on pass the guard before P V reads them
                WinWhole w;                // with a window: all but these steps do
            };
            Ring ring;
            uint32_t fph = 0;
            auto wait_full = [&](int st) -> bool {
                const bool r = wait_bar(kv_full(st), (fph >> st) & 1u, p, abort_flag);
                fph ^= 1u << st;
                return r;
            };
            uint32_t pph = 0, qph = 0, oph = 0, vph = 0;  // phase bits of the tiles' barriers
            int slot = 0;
            uint32_t uphase = 0;
            const uint32_t dq0 = desc_lo(sQ, 16), dk0 = desc_lo(sKV, 16), dv0 = desc_lo(sKV, kAtomBytes);
            constexpr uint32_t kTile16 = L::kTileBytes >> 4;
            auto fetch = [&](Cur &c) -> bool {
                if (!wait_bar(unit_full(slot), uphase, p, abort_flag)) return false;
                const VlUnit &u = units[slot];
                c.valid = u.valid;
                if (c.valid) {
                    const VlTile t0 = vl_tile<kCausal, kWindow>(p, u, 0), t1 = vl_tile<kCausal, kWindow>(p, u, 1);
                    c.n0 = t0.n;
                    c.n1 = t1.n;
                    c.n = t0.n > t1.n ? t0.n : t1.n;
                    if constexpr (kWindow) c.w = vl_unguarded(p, u);
                    else c.g0 = vl_first_masked<kCausal>(u, t0);
                } else {
                    c.n0 = c.n1 = 0;
                }
                mbar_arrive(unit_empty(slot));
                if (++slot == kVlSlots) {
                    slot = 0;
                    uphase ^= 1u;
                }
                return true;
            };
            // The products are written out twice.  The loop over whole steps in the middle of a
            // long unit has its own, with both tiles unrolled: the issuer must not spend a cycle
            // between the products.  Everything else (first and last steps, masked tiles, the
            // change of unit, before the first unit a step without a V tile) shares one copy for
            // both tiles: instructions that run once per unit have left the cache by then, which
            // cost 3000 cycles per unit with a copy for each case.
            Cur cur{1, 1, 0, 0, INT_MAX, {1, 0, 0}}, nxt{};
            bool ok = true, start = true;
            while (ok && cur.valid) {
                // steps [1, inner) (with a window those from w.w0 on) are whole for both tiles, with no guard
                // and no change of unit
                int inner = (cur.n0 < cur.n1 ? cur.n0 : cur.n1) - 1;
                if constexpr (kWindow) {
                    if (cur.w.w1 < inner) inner = cur.w.w1;
                } else {
                    if (cur.g0 < inner) inner = cur.g0;
                }
                for (int j = 0; j < cur.n; ++j) {
                    if (kWindow ? j > 0 && j >= cur.w.w0 && j < inner : j == 1) {
                        for (; j < inner; ++j) {
                            const int vs = ring.s;
                            if (!(ok = wait_full(vs))) break;  // V_j and K_{j+1}
                            tc_fence_after();
                            ring.next();
                            const int ks = ring.s;
                            const uint32_t dv = dv0 + vs * kTile16, dk = dk0 + ks * kTile16;
                            if (!(ok = wait_bar(p_full(0), pph & 1u, p, abort_flag))) break;
                            tc_fence_after();
                            mma_pv<D, kBF16>(tmem + 256u, tmem, dv, 1u);
                            mma_qk<D, kBF16>(tmem, dq0, dk);
                            mma_commit(s_full(0));
                            if (!(ok = wait_bar(p_full(1), (pph >> 1) & 1u, p, abort_flag))) break;
                            pph ^= 3u;
                            tc_fence_after();
                            mma_pv<D, kBF16>(tmem + 384u, tmem + 128u, dv, 1u);
                            mma_commit(kv_empty(vs));
                            mma_qk<D, kBF16>(tmem + 128u, dq0 + kTile16, dk);
                            mma_commit(s_full(1));
                            mma_commit(kv_empty(ks));
                            ring.next();
                        }
                        if (!ok) break;
                    }
                    const int vs = ring.s;
                    if (!start) ring.next();
                    const int ks = ring.s;
                    const bool last = j + 1 == cur.n;
                    if (last && !(ok = fetch(nxt))) break;
                    if (start && !nxt.valid) break;
                    if (!(ok = wait_full(vs))) break;  // V_j and the K tile after it
                    if (kWindow ? !cur.w(j) : j >= cur.g0) {
                        const int b = vs >> 1;
                        if (!(ok = wait_bar(v_ok(b), (vph >> b) & 1u, p, abort_flag))) break;
                        vph ^= 1u << b;
                    }
#pragma unroll 1
                    for (int i = 0; i < 2; ++i) {
                        const int n_i = i ? cur.n1 : cur.n0;
                        const uint32_t td = tmem + 128u * i;
                        if (j < n_i) {
                            // O_i (+)= P_i V_j: P_i from the first 64 columns of S_i, V MN-major; a
                            // unit's first one waits until the O_i of the unit before has been read
                            if (!(ok = wait_bar(p_full(i), (pph >> i) & 1u, p, abort_flag))) break;
                            pph ^= 1u << i;
                            if (j == 0) {
                                if (!(ok = wait_bar(o_empty(i), ((oph >> i) & 1u) ^ 1u, p, abort_flag))) break;
                                oph ^= 1u << i;
                            }
                            tc_fence_after();
                            mma_pv<D, kBF16>(td + 256u, td, dv0 + vs * kTile16, j > 0 ? 1u : 0u);
                            if (j == n_i - 1) mma_commit(o_full(i));
                        }
                        if (i == 1 && !start) mma_commit(kv_empty(vs));
                        const bool first = last && (i ? nxt.n1 : nxt.n0) > 0;
                        if (j + 1 < n_i || first) {
                            if (first) {  // a unit's first scores: its Q tile must have arrived
                                if (!(ok = wait_bar(q_full(i), (qph >> i) & 1u, p, abort_flag))) break;
                                qph ^= 1u << i;
                            }
                            tc_fence_after();
                            mma_qk<D, kBF16>(td, dq0 + i * kTile16, dk0 + ks * kTile16);
                            mma_commit(s_full(i));
                        }
                    }
                    if (!ok) break;
                    if (!last || nxt.valid) {
                        mma_commit(kv_empty(ks));
                        ring.next();
                    }
                    start = false;
                }
                cur = nxt;
            }
            // TMEM and shared memory stay alive until every issued MMA is done.
            mma_commit(mma_done);
            drain_bar(mma_done, 0, p);
        } else if (warp == 1) {
            // ---------------------------------------------------- value guard
            // The t-th V tile of this CTA lies in stage 1 (t even) or 3 (t odd).  The guard sees
            // every one of them arrive, and a stage is loaded again only after the guard, too, has
            // released it, so it never misses a phase of the full barriers; it is ahead of the
            // issuer by up to two key tiles, so that its work is hidden behind theirs.
            int slot = 0;
            uint32_t uphase = 0, t = 0;
            bool ok = true;
            while (ok) {
                if (!__all_sync(0xffffffffu, wait_bar(unit_full(slot), uphase, p, abort_flag))) break;
                VlUnit &us = units[slot];
                VlUnit u;
                u.valid = us.valid, u.rows = us.rows, u.nk = us.nk, u.rel = us.rel;
                if (!u.valid) break;
                const VlTile t0 = vl_tile<kCausal, kWindow>(p, u, 0), t1 = vl_tile<kCausal, kWindow>(p, u, 1);
                const int n = t0.n > t1.n ? t0.n : t1.n, g0 = kWindow ? 0 : vl_first_masked<kCausal>(u, t0);
                const WinWhole w = kWindow ? vl_unguarded(p, u) : WinWhole{};
                int g = 0;  // guarded tiles so far
                if (lane < kBad * 4) us.bad_rows[lane >> 2][lane & 3] = 0;
                __syncwarp();
                for (int j = 0; j < n; ++j, ++t) {
                    const int b = t & 1u, vs = 1 + 2 * b;
                    if (!(ok = __all_sync(0xffffffffu, wait_bar(kv_full(vs), (t >> 1) & 1u, p, abort_flag)))) break;
                    if (kWindow ? !w(j) : j >= g0) {
                        const int left = u.nk - win_key_tile<kWindow>(j, p.sinks, t0.skip) * kBN;
                        const bool any = vl_guard_tile<D, kBF16>(smem + L::kKV + vs * L::kTileBytes,
                                                                 left < kBN ? left : kBN, kCausal,
                                                                 us.bad_rows[(kWindow ? g++ : j - g0) & (kBad - 1)], lane);
                        if (any && lane == 0) us.bad = 1;
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(v_ok(b));
                    }
                    if (lane == 0) mbar_arrive(kv_empty(vs));
                }
                if (!ok) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(unit_empty(slot));
                if (++slot == kVlSlots) {
                    slot = 0;
                    uphase ^= 1u;
                }
            }
        } else if (warp == 3) {
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
                const int head = static_cast<int>(t % static_cast<unsigned>(p.head_units)) * (p.pair ? 2 : 1);
                int q0 = 0, rows = 0, k0 = 0, nk = 0;
                if (more) {
                    const VlSpan q = vl_span(p.cu_q, seq, p.total_q), k = vl_span(p.cu_k, seq, p.total_k);
                    q0 = q.a + qb * p.block_rows;
                    rows = q.b - q0;
                    k0 = k.a;
                    nk = k.b - k.a;
                    if (!vl_has_keys<kCausal>(p, rows, nk, nk - rows)) {
                        for (int h = head; h <= head + p.pair; ++h)
                            vl_store_blind<D>(static_cast<uint8_t *>(p.o) + h * p.o_head + q0 * p.o_row, p.o_row,
                                              p.lse ? p.lse + static_cast<size_t>(h) * p.total_q + q0 : nullptr,
                                              rows < p.block_rows ? rows : p.block_rows, lane);
                        continue;
                    }
                }
                if (!__all_sync(0xffffffffu, wait_bar(unit_empty(slot), phase ^ 1u, p, abort_flag))) break;
                if (lane == 0) {
                    VlUnit &u = units[slot];
                    u.valid = more ? 1 : 0;
                    u.head = head;
                    u.q0 = q0;
                    u.rows = rows;
                    u.k0 = k0;
                    u.nk = nk;
                    u.rel = nk - rows;
                    u.bad = 0;
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
        int slot = -1, done_slot = -1;  // the unit at work, and the one whose O is still to be stored
        uint32_t uphase = 1;
        float done_m = 0.f, done_l = 0.f;
        int j = 0, n = 0, first_masked = 0, lim0 = 0;
        int pos = 0, skip = 0;  // with a window: this row's position, key tiles left out, steps seen whole
        WinWhole seen_whole{};
        // m_ref: the max the probabilities are taken against (updated lazily);
        // m_top: the true running row max; l: running sum in units of 2^(m_ref*c).
        float m_ref = -INFINITY, m_top = -INFINITY, l = 0.f;
        bool more = true;
        while (true) {
            if (j == n) {
                // the next unit; the one before has its last weights handed over
                done_slot = slot;
                done_m = m_ref;
                done_l = l;
                if (++slot == kVlSlots) slot = 0;
                if (slot == 0) uphase ^= 1u;
                if (!__all_sync(0xffffffffu, wait_bar(unit_full(slot), uphase, p, abort_flag))) break;
                VlUnit u;
                u.valid = units[slot].valid, u.rows = units[slot].rows, u.nk = units[slot].nk, u.rel = units[slot].rel;
                more = u.valid != 0;
                n = 0;
                if (more) {
                    const VlTile t = vl_tile<kCausal, kWindow>(p, u, i);
                    n = t.n;
                    if constexpr (kWindow) {
                        seen_whole = vl_whole(p, u, t);
                        pos = r + t.rel;
                        skip = t.skip;
                    } else {
                        first_masked = vl_first_masked<kCausal>(u, t);
                    }
                    lim0 = u.nk - 1;  // this row keeps the keys up to lim0
                    if (kCausal && r + t.rel < lim0) lim0 = r + t.rel;
                }
                j = 0;
                m_ref = m_top = -INFINITY;
                l = 0.f;
            }
            if (j < n) {
                if (!__all_sync(0xffffffffu, wait_bar(s_full(i), scount & 1u, p, abort_flag))) break;
                ++scount;
                tc_fence_after();
                __syncwarp();
                float alpha = 1.f;
                bool rescale = false;
                float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                const float2 c2 = make_float2(c, c);
                // takes the tile's max (in m_top) into the reference; what the weights are taken against
                auto reference = [&]() -> float2 {
                    if (m_ref == -INFINITY) {
                        m_ref = m_top;  // nothing seen so far: the accumulator holds zeros at most
                    } else if ((m_top - m_ref) * c > kRescaleLog2) {
                        alpha = ex2_approx((m_ref - m_top) * c);
                        m_ref = m_top;
                        rescale = true;
                    }
                    // a row that has seen no key yet takes its weights, all 0, against 0
                    const float mr = m_ref == -INFINITY ? 0.f : m_ref;
                    return make_float2(-mr * c, -mr * c);
                };
                // (with a window masked tiles are too many of all to be worth the two passes below)
                if (kWindow || j < first_masked) {
                    uint32_t s[128];
                    float mq[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        tmem_ld32_max(tS + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * q]), mq[q]);
                    tmem_ld_wait(s, mq);
                    if (kWindow && !seen_whole(j)) {
                        // this row sees column e where e <= lim and (e > from or e < sk)
                        const int col0 = win_key_tile<kWindow>(j, p.sinks, skip) * kBN;
                        const int lim = lim0 - col0, from = pos - p.window - col0, sk = p.sinks - col0;
                        auto below = [](int n) -> uint32_t { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); };
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t see = below(lim + 1 - 32 * q) & (~below(from + 1 - 32 * q) | below(sk - 32 * q));
                            if (__all_sync(0xffffffffu, see == ~0u)) continue;
                            mq[q] = -INFINITY;
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                if (!((see >> e) & 1u)) s[32 * q + e] = __float_as_uint(-INFINITY);
                                mq[q] = fmaxf(mq[q], u2f(s[32 * q + e]));
                            }
                        }
                    }
                    m_top = fmaxf(m_top, fmax3(mq[0], mq[1], fmaxf(mq[2], mq[3])));
                    const float2 nmc2 = reference();
#pragma unroll
                    for (int cc = 0; cc < 128; cc += 2) {
                        float2 e = ffma2(make_float2(u2f(s[cc]), u2f(s[cc + 1])), c2, nmc2);
                        e.x = ex2_approx(e.x);
                        e.y = ex2_approx(e.y);
                        acc[(cc >> 1) & 1] = fadd2(acc[(cc >> 1) & 1], e);
                        s[cc] = __float_as_uint(e.x);
                        s[cc + 1] = __float_as_uint(e.y);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            pk[e] = pack2<kBF16>(u2f(s[32 * q + 2 * e]), u2f(s[32 * q + 2 * e + 1]));
                        tmem_st16(tS + 16 * q, pk);
                    }
                } else {
                    // A masked tile, once or twice per unit: 32 columns at a time, in two passes over
                    // TMEM, which is few instructions to fetch each time (P, 16 columns of pairs,
                    // overwrites scores that have been read).
                    const int lim = lim0 - j * kBN;  // this row keeps the columns up to lim
                    // Of columns 32 q .. every row of the warp sees all for q < q_all and none for
                    // q >= q_none: on a causal diagonal all but one of the four steps need no selects.
                    const int lo = __reduce_min_sync(0xffffffffu, lim), hi = __reduce_max_sync(0xffffffffu, lim);
                    const int q_all = lo < 31 ? 0 : (lo + 1) >> 5, q_none = hi < 0 ? 0 : (hi >> 5) + 1;
#pragma unroll 1
                    for (int q = 0; q < 4 && q < q_none; ++q) {
                        uint32_t s[32];
                        if (q < q_all) {
                            float mq[1];
                            tmem_ld32_max(tS + 32 * q, s, mq[0]);
                            tmem_ld_wait(s, mq);
                            m_top = fmaxf(m_top, mq[0]);
                        } else {
                            tmem_ld32(tS + 32 * q, s);
                            tmem_ld_wait(s);
                            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                mx[e & 1] = fmaxf(mx[e & 1], e <= lim - 32 * q ? u2f(s[e]) : -INFINITY);
                            m_top = fmax3(m_top, mx[0], mx[1]);
                        }
                    }
                    const float2 nmc2 = reference();
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t s[32], pk[16];
                        if (q >= q_none) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) pk[e] = 0u;
                            tmem_st16(tS + 16 * q, pk);
                            continue;
                        }
                        tmem_ld32(tS + 32 * q, s);
                        tmem_ld_wait(s);
                        if (q >= q_all) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (e > lim - 32 * q) s[e] = __float_as_uint(-INFINITY);
                        }
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
                }
                const float2 sum2 = fadd2(acc[0], acc[1]);
                l = l * alpha + (sum2.x + sum2.y);
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
                ++j;
            }
            if (done_slot >= 0) {
                // ---------------------------------------------------- O of the unit before
                const VlUnit &us = units[done_slot];
                VlUnit u;
                u.rows = us.rows, u.nk = us.nk, u.rel = us.rel;
                const VlTile t = vl_tile<kCausal, kWindow>(p, u, i);
                const int wvalid = t.valid - wq * 32;  // rows of this warp
                if (t.n > 0) {
                    if (!__all_sync(0xffffffffu, wait_bar(o_full(i), ocount & 1u, p, abort_flag))) break;
                    ++ocount;
                    tc_fence_after();
                    __syncwarp();
                }
                uint32_t o[D];
                if (t.n > 0) {
#pragma unroll
                    for (int q = 0; q < D / 32; ++q)
                        tmem_ld32(tO + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&o[32 * q]));
                    tmem_ld_wait(o);
                    // O_i has been read: the next unit's first P_i V may overwrite it
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(o_empty(i));
                } else {
#pragma unroll
                    for (int e = 0; e < D; ++e) o[e] = 0u;
                    done_l = 0.f;
                }
                if (wvalid > 0) {
                    const float inv_l = done_l == 0.f ? 0.f : 1.f / done_l;  // 0: the row saw no key
                    const int head = us.head + (i & p.pair);
                    const long long qrow = us.q0 + t.row0 + wq * 32;
                    uint8_t *otile = static_cast<uint8_t *>(p.o) + head * p.o_head + qrow * p.o_row;
                    uint8_t *oto = otile + (lane >> 2) * p.o_row + (lane & 3) * 16;
#pragma unroll
                    for (int q = 0; q < D / 32; ++q) {
                        // 32 columns: each thread puts its row's 64 bytes into the staging rows (16-byte
                        // chunk v of row t at v ^ ((t >> 1) & 3): no bank conflict on either side), then
                        // lanes 4k .. 4k+3 store the 64 bytes of one row
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            w[e] = pack2<kBF16>(u2f(o[32 * q + 2 * e]) * inv_l, u2f(o[32 * q + 2 * e + 1]) * inv_l);
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            st_shared_v4(stage + lane * 64 + ((v ^ ((lane >> 1) & 3)) << 4), w[4 * v], w[4 * v + 1],
                                         w[4 * v + 2], w[4 * v + 3]);
                        __syncwarp();
#pragma unroll
                        for (int s4 = 0; s4 < 4; ++s4) {
                            const int tr = 8 * s4 + (lane >> 2);
                            const uint4 x = ld_shared_v4(stage + tr * 64 + (((lane & 3) ^ ((tr >> 1) & 3)) << 4));
                            if (tr < wvalid) st_global_v4(oto + 8 * s4 * p.o_row + q * 64, x.x, x.y, x.z, x.w);
                        }
                        __syncwarp();
                    }
                    if (p.lse != nullptr && lane < wvalid)
                        p.lse[static_cast<size_t>(head) * p.total_q + qrow + lane] =
                            done_l == 0.f ? -INFINITY : (done_m * c + log2f(done_l)) * 0.6931471805599453f;
                    // non-finite values that the guard took out of V, for the rows that see them: added
                    // to the stored row, whose other values they do not change
                    if (t.n > 0 && *reinterpret_cast<const volatile int *>(&us.bad) != 0 && lane < wvalid) {
                        const VlTile t0 = vl_tile<kCausal, kWindow>(p, u, 0);
                        const int g0 = kWindow ? 0 : vl_first_masked<kCausal>(u, t0) * kBN;
                        const WinWhole w = kWindow ? vl_unguarded(p, u) : WinWhole{};
                        const uint8_t *vh = p.v_ptr + (us.head / p.group) * p.v_head + us.k0 * p.v_row;
                        int lim = u.nk - 1;
                        if (kCausal && r + t.rel < lim) lim = r + t.rel;
                        int step = -1, tile0 = 0;  // with a window: the step of guarded tile g >> 2, its first key
#pragma unroll 1
                        for (int g = 0; g < kBad * 4; ++g) {
                            if (kWindow && (g & 3) == 0) {
                                do ++step; while (w(step));
                                tile0 = win_key_tile<kWindow>(step, p.sinks, t0.skip) * kBN;
                            }
#pragma unroll 1
                            for (uint32_t bits = us.bad_rows[g >> 2][g & 3]; bits != 0; bits &= bits - 1) {
                                const int key = (kWindow ? tile0 + 32 * (g & 3) : g0 + 32 * g) + __ffs(bits) - 1;
                                if (key <= lim && (!kWindow || key > r + t.rel - p.window || key < p.sinks))
                                    add_nonfinite<D, kBF16>(otile + lane * p.o_row, vh + key * p.v_row);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(unit_empty(done_slot));
                done_slot = -1;
            }
            if (!more) break;
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
