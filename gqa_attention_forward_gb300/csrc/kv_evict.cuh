// Cutting sequences of the cache back to a budget (attn_kv_evict).
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
// One block per (sequence, layer, kv head).  The heaviest are found by selecting on the weights'
// bits (a non-negative float orders as its bits do), 11, 11 and 10 at a time; then the positions are
// walked in order, the kept ones of 2048 listed, and their rows moved.  A row never moves up past
// one that is still to be read: kept rows ascend, and place d takes a row from position d or behind.
#pragma once
#include "kv_pages.cuh"

namespace gqa {

constexpr int kEvThreads = kPlanThreads;
constexpr int kEvList = 2 * kEvThreads;  // positions listed at a time
constexpr int kEvBins = 2048;

struct KvEvict {
    const int *seqs;
    float *weights;  // [n_layers][n_rows][Hkv][table_w * page], or null (heavy 0)
    int n, sinks, heavy, recent;
    long long keep;
};

// What a weight orders by: NaN and negative ones as 0.
__device__ __forceinline__ uint32_t evict_key(float w) { return w > 0.f ? __float_as_uint(w) : 0u; }

__device__ __forceinline__ int evict_seq(const KvEvict &x, int i) { return x.seqs != nullptr ? x.seqs[i] : i; }

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
    for (int j = j0 + static_cast<int>(threadIdx.x); j < j1; j += kEvThreads) {
        const int p = kv_row(c, s)[j];
        if (p < 0 || p >= c.n_pages || (j < written && c.refs[p] != 1)) wrong = 2;
    }
    if (__syncthreads_or(wrong)) {
        if (report && threadIdx.x == 0) kv_error(ATTN_ERR_PAGE);
        return kEvNothing;
    }
    return kEvCut;
}

// The heavy-th largest of m keys: how many equal ones are among the heaviest (`ties`).  bins: kEvBins ints,
// sm: 33 ints of shared memory.
template <typename F>
__device__ __forceinline__ uint32_t evict_select(int m, int heavy, F key_of, int *bins, int *sm, int &ties) {
    __shared__ int found[2];
    uint32_t prefix = 0;
    int left = heavy;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
        for (int b = threadIdx.x; b < kEvBins; b += kEvThreads) bins[b] = 0;
        __syncthreads();
        for (int j = threadIdx.x; j < m; j += kEvThreads) {
            const uint32_t k = key_of(j);
            if (pass == 0 || k >> (shift + bits) == prefix) atomicAdd(&bins[k >> shift & ((1u << bits) - 1u)], 1);
        }
        __syncthreads();
        // from the largest bin down, two a thread
        const int hi = kEvBins - 1 - 2 * static_cast<int>(threadIdx.x);
        const int n0 = bins[hi], n1 = bins[hi - 1];
        int total;
        const int above = block_scan(n0 + n1, sm, total);
        if (above < left && above + n0 + n1 >= left) {
            const bool first = above + n0 >= left;
            found[0] = first ? hi : hi - 1;
            found[1] = left - above - (first ? 0 : n0);
        }
        __syncthreads();
        prefix = prefix << bits | static_cast<uint32_t>(found[0]);
        left = found[1];
        __syncthreads();
    }
    ties = left;
    return prefix;
}

__global__ void __launch_bounds__(kEvThreads) kv_evict_kernel(const KvPool c, const KvEvict x) {
    __shared__ int sm[33], bins[kEvBins];
    __shared__ int list[kEvList];      // positions that are kept
    __shared__ float wlist[kEvList];   // their weights
    grid_launch_dependents();
    grid_dependency_wait();
    const int per_seq = c.n_layers * c.Hkv;
    const int i = static_cast<int>(blockIdx.x) / per_seq, rest = static_cast<int>(blockIdx.x) - i * per_seq;
    const int layer = rest / c.Hkv, head = rest - layer * c.Hkv;
    int s, len;
    const int verdict = evict_verdict(c, x, i, s, len, rest == 0);
    if (rest == 0 && threadIdx.x == 0) c.need[i] = verdict;
    if (verdict != kEvCut) return;
    const int keep = static_cast<int>(x.keep), middle = len - x.recent;  // [sinks, middle) are chosen from
    const long long width = static_cast<long long>(c.table_w) << c.page_shift;
    float *w = x.weights == nullptr
        ? nullptr : x.weights + ((static_cast<long long>(layer) * c.n_rows + s) * c.Hkv + head) * width;
    int ties = 0;
    uint32_t border = 0;
    if (x.heavy > 0)
        border = evict_select(middle - x.sinks, x.heavy, [&](int j) { return evict_key(w[x.sinks + j]); }, bins, sm, ties);
    const int *row = kv_row(c, s);
    const size_t layer16 = static_cast<size_t>(layer) * c.n_pages * c.Hkv * c.page * c.row16;
    auto chunk_of = [&](int pos) -> size_t {  // first 16-byte chunk of a position's row
        return layer16 + ((static_cast<size_t>(row[pos >> c.page_shift]) * c.Hkv + head) * c.page + (pos & (c.page - 1))) * c.row16;
    };
    int dst0 = x.sinks, equal0 = 0;  // places taken, equal ones seen so far
    for (int at = x.heavy > 0 ? x.sinks : middle; at < len; at += kEvList) {
        // two positions a thread: kept, and of those equal to the border
        const int pos = at + 2 * static_cast<int>(threadIdx.x);
        int gt[2], eq[2];
        float wv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            gt[e] = eq[e] = 0;
            wv[e] = 0.f;
            if (pos + e >= len) continue;
            if (w != nullptr) wv[e] = w[pos + e];
            if (pos + e >= middle) {
                gt[e] = 1;
            } else {
                const uint32_t k = evict_key(wv[e]);
                gt[e] = k > border ? 1 : 0;
                eq[e] = k == border ? 1 : 0;
            }
        }
        int total;
        const int before = block_scan((gt[0] + gt[1]) | (eq[0] + eq[1]) << 16, sm, total);
        int equal = equal0 + (before >> 16);
        const int taken = equal0 < ties ? equal0 : ties;  // of the equal ones before this chunk
        int place = (before & 0xFFFF) + (equal < ties ? equal : ties) - taken;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (gt[e] || (eq[e] && equal < ties)) {
                list[place] = pos + e;
                wlist[place] = wv[e];
                ++place;
            }
            equal += eq[e];
        }
        equal0 += total >> 16;
        const int count = (total & 0xFFFF) + (equal0 < ties ? equal0 : ties) - taken;
        __syncthreads();
        // 8 chunks of 16 bytes a thread: rows of K, then of V
        const int per_row = 2 * c.row16, step = 8 * kEvThreads / per_row;
        for (int r0 = 0; r0 < count; r0 += step) {
            uint4 v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int y = e * kEvThreads + static_cast<int>(threadIdx.x), r = r0 + y / per_row, ch = y % per_row;
                if (r < count && list[r] != dst0 + r)
                    v[e] = (ch < c.row16 ? c.k : c.v)[chunk_of(list[r]) + (ch < c.row16 ? ch : ch - c.row16)];
            }
            __syncthreads();  // rows that these places hold have been read
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int y = e * kEvThreads + static_cast<int>(threadIdx.x), r = r0 + y / per_row, ch = y % per_row;
                if (r < count && list[r] != dst0 + r)
                    (ch < c.row16 ? c.k : c.v)[chunk_of(dst0 + r) + (ch < c.row16 ? ch : ch - c.row16)] = v[e];
            }
        }
        if (w != nullptr)
            for (int r = threadIdx.x; r < count; r += kEvThreads) w[dst0 + r] = wlist[r];
        dst0 += count;
    }
    if (w != nullptr) {
        __syncthreads();
        for (int j = keep + static_cast<int>(threadIdx.x); j < len; j += kEvThreads) w[j] = 0.f;
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
