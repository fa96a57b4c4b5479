// Cutting sequences of the cache back to a given length (attn_kv_evict).
//
// A sequence of L positions, more than keep = sinks + heavy + recent, keeps in every layer and kv
// head its first `sinks`, its last `recent` and, of those between, the `heavy` ones with the
// largest weight (equal ones: the lowest positions), in their order; which ones differs from head to
// head.  Their rows of K and V and their weights move up to positions 0 .. keep - 1, the weights
// behind become 0, and the sequence's pages behind its new end are given back.
//
// What bounds it: the kept rows, read and written once each (4 D bytes a row of K and of V in all),
// and 4 bytes for each weight.
//
// A cluster of 1 to 8 blocks per (sequence, layer, kv head).  Finding the heaviest is a selection on
// the weights' bits (a non-negative float orders as its bits do), a byte at a time: each block counts
// a part of the positions, and adds up the others' counts from their shared memory.  Each then
// leaves a bit per position of its part: above the border, or equal to it.  From these bits every block
// lists all kept positions in order, 8192 bits at a time, and moves its share of the columns of
// their rows (all of K or V, or a part of a row of at least 32 bytes): blocks of a cluster never touch
// the same bytes.  Within a block a row never moves up past one that is still to be read: kept rows
// ascend, and place d takes a row from position d or behind, so that the rows of a step are stored
// once all of the step's loads have been issued, while the next step's are under way.
//
// Measured, GB300, captured, with the copies that start each pass from the same state (5 and 28 us;
// without weights 2): 16 sequences of 65 to 8192 to 1024 positions in 4 layers of 8 heads 103 us, in 20
// layers 418 (6.3 TB/s without those copies; before its rows move a block spends about 20 us on the choice,
// which the rows of other blocks hide where there are more of them than fit at once); 16 of 2048 to
// 4000 to 2048 without weights 168 and 760 (6.6 TB/s, near the copy rate); 65000 to 16016 148 us, in 32
// layers 810.
#pragma once
#include <cooperative_groups.h>

#include "kv_pages.cuh"

namespace gqa {

constexpr int kEvThreads = 256, kEvWarps = kEvThreads / 32;
constexpr int kEvPer = 16;                     // weights that a thread has on their way
constexpr int kEvList = 4096;                  // kept positions listed before their rows move
constexpr int kEvPart = 32768;                 // positions whose bits a block holds
constexpr int kEvMove = 4;                     // 16-byte chunks a thread moves in a step
constexpr int kEvBins = 256, kEvPasses = 4;    // a byte of the weights at a time
constexpr int kEvClusterMost = 8;

struct KvEvict {
    const int *seqs;
    float *weights;  // [n_layers][n_rows][Hkv][table_w * page], or null (heavy 0)
    int n, sinks, heavy, recent;
    long long keep;
};

struct EvictShared {
    int bins[kEvPasses][kEvBins];
    union {
        struct {
            uint32_t src[kEvList];  // kept positions, and then their rows within the layer
            float w[kEvList];
        };
        uint32_t keys[2 * kEvList];  // while the heaviest are looked for: of this block's part, where they fit
    };
    uint2 bits[kEvPart / 32];  // of this block's part: above the border, equal to it
    int scan[2][kEvWarps];
    int pages[kEvList / 16 + 1];  // of the places that the listed rows go to
    int found[2];
    int still;  // listed rows that stay where they are
};

// What a weight orders by: NaN and negative ones as 0.
__device__ __forceinline__ uint32_t evict_key(float w) { return w > 0.f ? __float_as_uint(w) : 0u; }

__device__ __forceinline__ int evict_seq(const KvEvict &x, int i) { return x.seqs != nullptr ? x.seqs[i] : i; }

// Sum of the warps' x before this one, `total` that of all.  All threads call it, with the two buffers in turn.
__device__ __forceinline__ int evict_warps(int x, int *sm, int &total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) sm[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kEvWarps; ++w) {
        const int y = sm[w];
        before += w < warp ? y : 0;
        all += y;
    }
    total = all;
    return before;
}

// What becomes of entry i of the list: its sequence s and length, and whether it is cut.  The block
// looks at the pages that it would write (which must not be shared) and read.
enum EvictVerdict { kEvNothing = 0, kEvCut = 1 };
__device__ __forceinline__ int evict_verdict(const KvPool &c, const KvEvict &x, int i, int &s, int &len, bool report) {
    s = evict_seq(x, i);
    int wrong = 0;  // 1: shape, 2: page
    len = 0;
    if (s < 0 || s >= c.n_rows) {
        wrong = 1;
    } else {
        len = c.lens[s];
        if (len < 0 || len > (static_cast<long long>(c.table_w) << c.page_shift)) wrong = 1;
        if (x.seqs != nullptr)
            for (int j = threadIdx.x; j < i; j += kEvThreads)
                if (x.seqs[j] == s) wrong = 1;  // named before in the list
    }
    wrong = __syncthreads_or(wrong);
    if (wrong != 0 || len <= x.keep) {
        if (wrong != 0 && report && threadIdx.x == 0) kv_error(ATTN_ERR_SHAPE);
        return kEvNothing;
    }
    const int keep = static_cast<int>(x.keep);
    const int j0 = x.sinks >> c.page_shift, j1 = (len + c.page - 1) >> c.page_shift;
    const int written = keep > x.sinks ? (keep + c.page - 1) >> c.page_shift : j0;
    for (int j = j0 + static_cast<int>(threadIdx.x); j < j1; j += 4 * kEvThreads) {
        int p[4], r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = kv_row(c, s)[j + e * kEvThreads < j1 ? j + e * kEvThreads : j];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = c.refs[p[e] < 0 || p[e] >= c.n_pages ? 0 : p[e]];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (p[e] < 0 || p[e] >= c.n_pages || (j + e * kEvThreads < written && r[e] != 1)) wrong = 2;
    }
    if (__syncthreads_or(wrong)) {
        if (report && threadIdx.x == 0) kv_error(ATTN_ERR_PAGE);
        return kEvNothing;
    }
    return kEvCut;
}

// Positions of a block's part of m: a multiple of 32, so that none shares a word of bits with the next.
__device__ __forceinline__ int evict_part(int m, int C) { return ((m + C - 1) / C + 31) & ~31; }

// The heavy-th largest key of w[0 .. m), and how many equal ones are among the heaviest (`ties`), by all
// blocks of the cluster.
__device__ __forceinline__ uint32_t evict_select(const float *w, int m, int heavy, EvictShared &sm, int &ties) {
    const auto cluster = cooperative_groups::this_cluster();
    const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int part = evict_part(m, C), j0 = rank * part, j1 = j0 + part < m ? j0 + part : m;
    const bool cached = part <= 2 * kEvList;
    for (int b = threadIdx.x; b < kEvPasses * kEvBins; b += kEvThreads) (&sm.bins[0][0])[b] = 0;
    __syncthreads();
    uint32_t prefix = 0;
    int left = heavy;
#pragma unroll 1
    for (int pass = 0; pass < kEvPasses; ++pass) {
        const int shift = 24 - 8 * pass;
        int *bins = sm.bins[pass];
        auto count = [&](uint32_t k) {
            if (pass == 0 || k >> (shift + 8) == prefix) atomicAdd(&bins[k >> shift & 255u], 1);
        };
        if (pass > 0 && cached) {
            for (int y = threadIdx.x; y < j1 - j0; y += 4 * kEvThreads) {
                uint32_t k[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) k[e] = sm.keys[y + e * kEvThreads < j1 - j0 ? y + e * kEvThreads : y];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (y + e * kEvThreads < j1 - j0) count(k[e]);
            }
        } else {
            for (int j = j0; j < j1; j += kEvPer * kEvThreads) {
                float v[kEvPer];  // (a load under a condition would be waited for before the next is issued)
#pragma unroll
                for (int e = 0; e < kEvPer; ++e) {
                    const int y = j + e * kEvThreads + static_cast<int>(threadIdx.x);
                    v[e] = w[y < j1 ? y : j1 - 1];
                }
#pragma unroll
                for (int e = 0; e < kEvPer; ++e) {
                    const int y = j + e * kEvThreads + static_cast<int>(threadIdx.x);
                    if (y >= j1) continue;
                    const uint32_t k = evict_key(v[e]);
                    if (cached) sm.keys[y - j0] = k;
                    count(k);
                }
            }
        }
        if (C == 1) __syncthreads(); else cluster.sync();
        // from the largest bin down, one a thread
        const int bin = kEvBins - 1 - static_cast<int>(threadIdx.x);
        int n[kEvClusterMost], total;
#pragma unroll
        for (int r = 0; r < kEvClusterMost; ++r) n[r] = r < C && bin >= 0 ? *cluster.map_shared_rank(bins + bin, r) : 0;
#pragma unroll
        for (int r = 1; r < kEvClusterMost; ++r) n[0] += n[r];
        const int incl = warp_scan(n[0], threadIdx.x & 31);
        const int above = evict_warps(__shfl_sync(0xffffffffu, incl, 31), sm.scan[pass & 1], total) + incl - n[0];
        if (above < left && above + n[0] >= left) {
            sm.found[0] = bin;
            sm.found[1] = left - above;
        }
        __syncthreads();
        prefix = prefix << 8 | static_cast<uint32_t>(sm.found[0]);
        left = sm.found[1];
    }
    ties = left;
    return prefix;
}

// kChoose: heavy is not 0.  Blocks per SM: with a choice 3 (80 registers, no spills); with 4 (64 registers,
// which spill) the 16 sequences take 109 us instead of 103, and 65000 positions 173 instead of 148.  Without
// one 4: 167 us, although 64 registers spill 28 bytes (48 loaded); with 3 175.
template <bool kChoose>
__global__ void __launch_bounds__(kEvThreads, kChoose ? 3 : 4) kv_evict_kernel(const KvPool c, const KvEvict x) {
    extern __shared__ __align__(16) uint8_t evict_raw[];
    EvictShared &sm = *reinterpret_cast<EvictShared *>(evict_raw);
    const auto cluster = cooperative_groups::this_cluster();
    const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    grid_launch_dependents();
    grid_dependency_wait();
    const int problem = static_cast<int>(blockIdx.x) / C, per_seq = c.n_layers * c.Hkv;
    const int i = problem / per_seq, rest = problem - i * per_seq;
    const int layer = rest / c.Hkv, head = rest - layer * c.Hkv;
    int s, len;
    const bool first = rest == 0 && rank == 0;
    const int verdict = evict_verdict(c, x, i, s, len, first);
    if (first && threadIdx.x == 0) c.need[i] = verdict;
    if (verdict != kEvCut) return;  // as all blocks of the cluster
    const int keep = static_cast<int>(x.keep), middle = len - x.recent;  // [sinks, middle) are chosen from
    const long long width = static_cast<long long>(c.table_w) << c.page_shift;
    float *w = x.weights == nullptr
        ? nullptr : x.weights + ((static_cast<long long>(layer) * c.n_rows + s) * c.Hkv + head) * width;
    int ties = 0;
    uint32_t border = 0;
    if constexpr (kChoose) border = evict_select(w + x.sinks, middle - x.sinks, x.heavy, sm, ties);
    const int *row = kv_row(c, s);
    auto row_of = [&](int page, int pos) -> uint32_t {  // of a position in that page, within the layer
        return (static_cast<uint32_t>(page) * c.Hkv + head) * c.page + (pos & (c.page - 1));
    };
    // this block's columns of a row: `cols` chunks of 16 bytes of K (or V) from `col0` on, and the same of V
    // where the cluster is one block
    const int cols = C == 1 ? c.row16 : 2 * c.row16 / C, cut = rank * cols;
    const size_t layer16 = static_cast<size_t>(layer) * c.n_pages * c.Hkv * c.page * c.row16;
    uint4 *pool = (cut < c.row16 ? c.k : c.v) + layer16 + (cut & (c.row16 - 1));
    const int shift = __ffs(cols) - 1, per_step = kEvMove * kEvThreads >> shift;
    int dst0 = x.sinks, fill = 0;  // kept positions that are listed, for places dst0 on
    const int choices = kChoose ? middle - x.sinks : 0, lane = threadIdx.x & 31;
    int c0 = 0, i0 = 0;        // positions chosen from so far, words of bits of those at work
    int equal0 = 0, turn = 0;  // equal ones seen so far
    while (true) {
        // n more kept positions: those of the next words of bits, or behind all of them the last ones
        const bool choose = kChoose && c0 < choices;
        const int m = choices - c0 < C * kEvPart ? choices - c0 : C * kEvPart, part = evict_part(m, C);
        if (choose && i0 == 0) {
            const int j0 = rank * part, j1 = j0 + part < m ? j0 + part : m;
            const bool cached = choices == m && part <= 2 * kEvList;  // as evict_select left them
            if (c0 > 0) cluster.sync();  // the bits have been read
            for (int j = j0 + static_cast<int>(threadIdx.x - lane); j < j1; j += kEvPer * kEvThreads) {
                uint32_t k[kEvPer];
                if (cached) {
#pragma unroll
                    for (int e = 0; e < kEvPer; ++e) {
                        const int y = j + e * kEvThreads + lane;
                        k[e] = sm.keys[(y < j1 ? y : j1 - 1) - j0];
                    }
                } else {
                    float v[kEvPer];
#pragma unroll
                    for (int e = 0; e < kEvPer; ++e) {
                        const int y = j + e * kEvThreads + lane;
                        v[e] = w[x.sinks + c0 + (y < j1 ? y : j1 - 1)];
                    }
#pragma unroll
                    for (int e = 0; e < kEvPer; ++e) k[e] = evict_key(v[e]);
                }
#pragma unroll
                for (int e = 0; e < kEvPer; ++e) {
                    const int y = j + e * kEvThreads;
                    if (y >= j1) break;
                    const uint32_t gt = __ballot_sync(0xffffffffu, y + lane < j1 && k[e] > border);
                    const uint32_t eq = __ballot_sync(0xffffffffu, y + lane < j1 && k[e] == border);
                    if (lane == 0 && y < j1) sm.bits[(y - j0) >> 5] = make_uint2(gt, eq);
                }
            }
            if (C == 1) __syncthreads(); else cluster.sync();
        }
        int n = x.recent, first_k = 0, pos0 = 0;
        uint32_t bits = 0u;
        if (choose) {
            // a word of 32 positions a thread
            const int words = (m + 31) >> 5, part_words = part >> 5, wi = i0 + static_cast<int>(threadIdx.x);
            uint2 bit = make_uint2(0u, 0u);
            if (wi < words) bit = cluster.map_shared_rank(sm.bits, wi / part_words)[wi % part_words];
            const int both = __popc(bit.x) << 16 | __popc(bit.y), incl = warp_scan(both, lane);
            int total;
            const int before = evict_warps(__shfl_sync(0xffffffffu, incl, 31), sm.scan[turn], total) + incl - both;
            turn ^= 1;
            // of the equal ones the first `ties` in all
            const int equal = equal0 + (before & 0xFFFF), left = ties - equal, taken = equal0 < ties ? equal0 : ties;
            first_k = (before >> 16) + (equal < ties ? equal : ties) - taken;
            bits = left > 0 ? bit.y : 0u;
            while (__popc(bits) > left && bits != 0u) bits &= ~(0x80000000u >> __clz(bits));
            bits |= bit.x;
            equal0 += total & 0xFFFF;
            n = (total >> 16) + (equal0 < ties ? equal0 : ties) - taken;
            pos0 = x.sinks + c0 + 32 * wi;
            i0 += kEvThreads;
            if (i0 >= words) {
                i0 = 0;
                c0 += m;
            }
        }
        for (int k = 0; k < n || (!choose && fill > 0);) {
            // numbers k to k1 - 1 of them are listed
            const int k1 = k + (kEvList - fill < n - k ? kEvList - fill : n - k), at = fill - k;
            if (choose) {
                int y = first_k;
                for (uint32_t rest = bits; rest != 0u && y < k1; rest &= rest - 1u, ++y)
                    if (y >= k) sm.src[at + y] = pos0 + __ffs(rest) - 1;
            } else {
                for (int y = k + static_cast<int>(threadIdx.x); y < k1; y += kEvThreads) sm.src[at + y] = middle + y;
            }
            fill += k1 - k;
            k = k1;
            if (fill == kEvList || (!choose && k == n)) {
                // ------------------------------------------------ the listed rows move up
                const int place0 = dst0 >> c.page_shift, place1 = (dst0 + fill + c.page - 1) >> c.page_shift;
                for (int j = place0 + static_cast<int>(threadIdx.x); j < place1; j += kEvThreads) sm.pages[j - place0] = row[j];
                if (threadIdx.x == 0) sm.still = 0;
                __syncthreads();  // all are listed
                // the weights, a block its share; positions become rows
                const int r1 = rank * kEvThreads + static_cast<int>(threadIdx.x);
                if (w != nullptr)
                    for (int r0 = r1; r0 < fill; r0 += 4 * C * kEvThreads) {
                        float v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int r = r0 + e * C * kEvThreads;
                            v[e] = w[sm.src[r < fill ? r : r0]];
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (r0 + e * C * kEvThreads < fill) sm.w[r0 + e * C * kEvThreads] = v[e];
                    }
                __syncthreads();
                int still = 0;
                for (int r0 = threadIdx.x; r0 < fill; r0 += 4 * kEvThreads) {
                    int pos[4], page[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        pos[e] = static_cast<int>(sm.src[r0 + e * kEvThreads < fill ? r0 + e * kEvThreads : r0]);
                        page[e] = row[pos[e] >> c.page_shift];
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (r0 + e * kEvThreads < fill) {
                            sm.src[r0 + e * kEvThreads] = row_of(page[e], pos[e]);
                            still += pos[e] == dst0 + r0 + e * kEvThreads ? 1 : 0;
                        }
                }
                // those before the first position that goes are where they belong
                still = __reduce_add_sync(0xffffffffu, still);
                if (lane == 0 && still > 0) atomicAdd(&sm.still, still);
                if (w != nullptr) cluster.sync(); else __syncthreads();  // their weights have been read
                still = sm.still;
                if (w != nullptr)
                    for (int r = r1; r < fill; r += C * kEvThreads) w[dst0 + r] = sm.w[r];
                for (int half = 0; half < (C == 1 ? 2 : 1); ++half) {
                    uint4 *p = half == 0 ? pool : c.v + layer16;
                    auto fetch = [&](int r0, uint4 (&v)[kEvMove]) {
#pragma unroll
                        for (int e = 0; e < kEvMove; ++e) {
                            const int y = e * kEvThreads + static_cast<int>(threadIdx.x), r = r0 + (y >> shift);
                            if (r < fill) v[e] = p[static_cast<size_t>(sm.src[r]) * c.row16 + (y & (cols - 1))];
                        }
                    };
                    auto place = [&](int r) { return row_of(sm.pages[((dst0 + r) >> c.page_shift) - place0], dst0 + r); };
                    auto store = [&](int r0, const uint4 (&v)[kEvMove]) {
#pragma unroll
                        for (int e = 0; e < kEvMove; ++e) {
                            const int y = e * kEvThreads + static_cast<int>(threadIdx.x), r = r0 + (y >> shift);
                            if (r < fill) p[static_cast<size_t>(place(r)) * c.row16 + (y & (cols - 1))] = v[e];
                        }
                    };
                    uint4 a[kEvMove], b[kEvMove];
                    fetch(still, a);
                    for (int r0 = still; r0 < fill; r0 += 2 * per_step) {
                        fetch(r0 + per_step, b);
                        __syncthreads();  // rows that these places hold have been read
                        store(r0, a);
                        fetch(r0 + 2 * per_step, a);
                        __syncthreads();
                        store(r0 + per_step, b);
                    }
                }
                __syncthreads();  // the list is free
                dst0 += fill;
                fill = 0;
            }
        }
        if (!choose) break;
    }
    // (with no weights the blocks need not wait for each other; with them none may leave while another
    // reads its counts, and the last weights have been read)
    if (w != nullptr) {
        cluster.sync();
        for (int j = keep + rank * kEvThreads + static_cast<int>(threadIdx.x); j < len; j += C * kEvThreads) w[j] = 0.f;
    }
}

// Lengths, page tables and references of the sequences that were cut: a block each.
__global__ void __launch_bounds__(256) kv_evict_end_kernel(const KvPool c, const KvEvict x) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int i = blockIdx.x;
    if (c.need[i] != kEvCut) return;
    const int s = evict_seq(x, i), keep = static_cast<int>(x.keep);
    for (int j = ((keep + c.page - 1) >> c.page_shift) + static_cast<int>(threadIdx.x); j < c.table_w; j += 256) {
        const int p = kv_row(c, s)[j];
        if (p < 0) continue;
        kv_row(c, s)[j] = -1;
        if (p >= c.n_pages || atomicSub(&c.refs[p], 1) <= 0) {
            if (p < c.n_pages) atomicAdd(&c.refs[p], 1);
            kv_error(ATTN_ERR_PAGE);
        }
    }
    if (threadIdx.x == 0) c.lens[s] = keep;
}

}  // namespace gqa
