// The pages of a key/value cache: extending, appending, accepting, copying, forking, freeing
// and compacting (attn_kv_*).
//
// State, all on the device: K and V pools [n_layers][n_pages][Hkv][page][D] of 2-byte
// elements; a page table [n_rows][table_w] whose row s lists the pages of sequence s from its
// first position on, -1 behind the last; lens[s]; and refs[p], the number of table entries
// that name page p.  A page is free exactly when refs is 0 (no list of free pages is kept),
// and pages are taken lowest index first, so that every call's result is determined by its
// inputs and the pool stays dense at its front.
//
// What bounds these: the moved rows at copy bandwidth (each is read and written once, 16
// bytes per lane, 4 KB in flight per warp); for small calls the latency of one or two
// dependent launches.  The bookkeeping of a call is one CTA: it needs an ordered choice of
// free pages (a prefix sum over refs), which is 4 bytes a page, against 128 KB and more of
// data for each page that is then moved.
//
// Indexes from device memory (sequences, pages, path positions) are checked before use; one
// out of range, a page that another sequence shares and would be written, or a pool without
// enough free pages sets the device error word and leaves that sequence as it was.
#pragma once
#include <cooperative_groups.h>

#include <climits>

#include "kernel_common.cuh"

namespace gqa {

struct KvPool {
    uint4 *k, *v;
    int *table, *lens, *refs;
    int n_layers, n_pages, page, page_shift, Hkv, row16, n_rows, table_w;  // row16: 16-byte chunks of a row
    // scratch: list [n_pages], map [n_pages], claim [n_rows], need [n_rows], pairs [3 n_rows], count
    int *list, *map, *claim, *need, *pairs, *count;
};

constexpr int kPlanThreads = 1024;

__device__ __forceinline__ void kv_error(attn_status_t e) { atomicCAS(&g_error_code, 0, static_cast<int>(e)); }

__device__ __forceinline__ int *kv_row(const KvPool &c, int s) { return c.table + static_cast<size_t>(s) * c.table_w; }

__device__ __forceinline__ int warp_scan(int x, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// Exclusive prefix sum over the block (kPlanThreads threads); `total` gets the sum.
// sm: 33 ints of shared memory.  All threads call it.
__device__ __forceinline__ int block_scan(int x, int *sm, int &total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int incl = warp_scan(x, lane);
    __syncthreads();  // the last call's readers of sm are done
    if (lane == 31) sm[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const int w = sm[lane], s = warp_scan(w, lane);
        sm[lane] = s - w;
        if (lane == 31) sm[32] = s;
    }
    __syncthreads();
    total = sm[32];
    return sm[warp] + incl - x;
}

// Writes the pages p of [p0, p1) whose refs are (free: zero, else not zero), in ascending
// order, to list, at most `most` of them; returns how many there are (counting stops in the
// chunk in which `most` is reached).  All threads of the block call it.
template <bool kFree>
__device__ __forceinline__ int kv_list(const int *refs, int p0, int p1, int most, int *list, int *sm) {
    int found = 0;
    for (int at = p0; at < p1 && found < most; at += 4 * kPlanThreads) {
        const int p = at + 4 * static_cast<int>(threadIdx.x);
        int r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = p + i < p1 ? refs[p + i] : 0;
        int n = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) n += p + i < p1 && (r[i] == 0) == kFree ? 1 : 0;
        int total, k = found + block_scan(n, sm, total);
        if (list != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (p + i < p1 && (r[i] == 0) == kFree) {
                    if (k < most) list[k] = p + i;
                    ++k;
                }
        }
        found += total;
    }
    return found;
}

// need[0 .. n) becomes its exclusive prefix sum; returns the sum (clamped to INT_MAX / 2).
__device__ __forceinline__ int kv_offsets(int *need, int n, int *sm) {
    int before = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + static_cast<int>(threadIdx.x);
        const int x = i < n ? need[i] : 0;
        int total;
        const int off = block_scan(x, sm, total);
        if (i < n) need[i] = before + off;
        before = before > INT_MAX / 2 - total ? INT_MAX / 2 : before + total;
    }
    __syncthreads();
    return before;
}

// Room for n_new[i] more positions of sequence seqs[i]: pages for them, lens grown.  One
// block, a warp per sequence.  Requests are served in order; from the first on that the
// free pages do not hold, nothing changes (ATTN_ERR_POOL).
__global__ void __launch_bounds__(kPlanThreads) kv_extend_kernel(const KvPool c, const int *seqs, const int *n_new, int n) {
    __shared__ int sm[33];
    grid_launch_dependents();
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int s = seqs != nullptr ? seqs[i] : i;
        if (s >= 0 && s < c.n_rows) c.claim[s] = INT_MAX;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int s = seqs != nullptr ? seqs[i] : i;
        if (s >= 0 && s < c.n_rows) atomicMin(&c.claim[s], i);
    }
    __syncthreads();
    // a request in range, of a sequence not asked for before: its columns [j0, j1)
    auto columns = [&](int i, int &s, int &len, int &j0, int &j1) -> bool {
        s = seqs != nullptr ? seqs[i] : i;
        if (s < 0 || s >= c.n_rows || c.claim[s] != i) return false;
        len = c.lens[s];
        const int more = n_new[i];
        const long long to = static_cast<long long>(len) + more;
        if (len < 0 || more < 0 || to > (static_cast<long long>(c.table_w) << c.page_shift)) return false;
        j0 = (len + c.page - 1) >> c.page_shift;
        j1 = static_cast<int>((to + c.page - 1) >> c.page_shift);
        return true;
    };
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        int s, len, j0, j1, miss = 0;
        const bool fine = columns(i, s, len, j0, j1);
        bool past = false;  // a page that the sequence has kept is none of the pool
        if (fine)
            for (int j = j0 + lane; j < j1; j += 32) {
                const int p = kv_row(c, s)[j];
                miss += p < 0 ? 1 : 0;
                past |= p >= c.n_pages;
            }
        miss = __reduce_add_sync(0xffffffffu, miss);
        past = __any_sync(0xffffffffu, past);
        if (lane == 0) {
            c.need[i] = past ? 0 : miss;
            if (past) c.claim[s] = -1;  // refused: no request of the list
            if (!fine || past) kv_error(fine ? ATTN_ERR_PAGE : ATTN_ERR_SHAPE);
        }
    }
    __syncthreads();
    const int want = kv_offsets(c.need, n, sm);
    const int have = kv_list<true>(c.refs, 0, c.n_pages, want < c.n_pages ? want : c.n_pages, c.list, sm);
    __syncthreads();
    if (have < want && threadIdx.x == 0) kv_error(ATTN_ERR_POOL);
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        int s, len, j0, j1;
        if (!columns(i, s, len, j0, j1)) continue;
        const int off = c.need[i], past = i + 1 < n ? c.need[i + 1] : want;
        if (past > have) continue;
        int k = off;
        for (int j = j0; j < j1; j += 32) {
            const bool miss = j + lane < j1 && kv_row(c, s)[j + lane] < 0;
            const unsigned m = __ballot_sync(0xffffffffu, miss);
            if (miss) {
                const int p = c.list[k + __popc(m & ((1u << lane) - 1u))];
                kv_row(c, s)[j + lane] = p;
                c.refs[p] = 1;
            }
            k += __popc(m);
        }
        __syncwarp();
        if (lane == 0) c.lens[s] = len + n_new[i];
    }
}

// Children take the lengths of their parents and a free page for the last page that is not
// full; pairs lists what kv_move_kernel<kMoveFork> then copies, beside the table entries of the
// full pages and their references, which one block would take too long over.  A request is
// refused as a whole before anything is written: all pages of its parent are looked at first, as
// a long context has thousands of them by a warp per request (4 entries per lane in flight) of the
// blocks behind the first of a cluster; the first plans (a captured beam step of 96 children 16.9
// us, 17.4 where the first looks, too, and 15.9 without looking).
constexpr int kForkCtas = 8;
__global__ void __cluster_dims__(kForkCtas, 1, 1) __launch_bounds__(kPlanThreads)
    kv_fork_kernel(const KvPool c, const int *parents, const int *children, int n) {
    __shared__ int sm[33];
    grid_launch_dependents();
    grid_dependency_wait();
    auto in = [&](int s) { return s >= 0 && s < c.n_rows; };
    constexpr int kFine = -1, kRefused = -2, kNoPage = -3;  // in pairs[3 i]
    if (blockIdx.x != 0) {
        constexpr int kWarps = kPlanThreads / 32;
        const int lane = threadIdx.x & 31;
        for (int i = (blockIdx.x - 1) * kWarps + (threadIdx.x >> 5); i < n; i += (kForkCtas - 1) * kWarps) {
            const int a = parents[i], len = in(a) ? c.lens[a] : -1;
            int verdict = kRefused;
            if (len >= 0 && len <= (static_cast<long long>(c.table_w) << c.page_shift)) {
                const int pages = static_cast<int>((static_cast<long long>(len) + c.page - 1) >> c.page_shift);
                const int *row = kv_row(c, a);
                bool hole = false;
                for (int j = lane; j < pages; j += 128) {
                    int p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] = j + 32 * e < pages ? row[j + 32 * e] : 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) hole |= p[e] < 0 || p[e] >= c.n_pages;
                }
                verdict = __any_sync(0xffffffffu, hole) ? kNoPage : kFine;
            }
            if (lane == 0) c.pairs[3 * i] = verdict;
        }
        cooperative_groups::this_cluster().sync();
        return;
    }
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int a = parents[i], b = children[i];
        if (in(a)) c.claim[a] = INT_MAX;
        if (in(b)) c.claim[b] = INT_MAX;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads)
        if (in(children[i])) atomicMin(&c.claim[children[i]], i);
    cooperative_groups::this_cluster().sync();  // the parents have been looked at
    // each child once, empty, and no child of this call a parent of it
    auto fine = [&](int i, int &a, int &b) -> bool {
        a = parents[i];
        b = children[i];
        return in(a) && in(b) && c.claim[b] == i && c.claim[a] == INT_MAX;
    };
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        int a, b;
        const int verdict = c.pairs[3 * i];
        const bool right = fine(i, a, b) && c.lens[b] == 0 && kv_row(c, b)[0] < 0 && verdict != kRefused;
        const bool ok = right && verdict == kFine;
        c.need[i] = ok && (c.lens[a] & (c.page - 1)) != 0 ? 1 : 0;
        c.pairs[3 * i] = ok ? kFine : kRefused;
        if (!ok) kv_error(right ? ATTN_ERR_PAGE : ATTN_ERR_SHAPE);
    }
    __syncthreads();
    const int want = kv_offsets(c.need, n, sm);
    const int have = kv_list<true>(c.refs, 0, c.n_pages, want < c.n_pages ? want : c.n_pages, c.list, sm);
    __syncthreads();
    if (have < want && threadIdx.x == 0) kv_error(ATTN_ERR_POOL);
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int off = c.need[i], past = i + 1 < n ? c.need[i + 1] : want;
        if (c.pairs[3 * i] == kRefused) continue;
        if (past > have) {
            c.pairs[3 * i] = kRefused;
            continue;
        }
        const int a = parents[i], b = children[i], len = c.lens[a];
        if (past > off) {
            const int p = c.list[off], full = len >> c.page_shift;
            c.pairs[3 * i] = kv_row(c, a)[full];
            c.pairs[3 * i + 1] = p;
            c.pairs[3 * i + 2] = len & (c.page - 1);
            kv_row(c, b)[full] = p;
            c.refs[p] = 1;
        }
        c.lens[b] = len;
    }
}

// One reference less for each page of the sequences, whose rows become empty.
__global__ void __launch_bounds__(256) kv_free_kernel(const KvPool c, const int *seqs, int n) {
    grid_launch_dependents();
    grid_dependency_wait();
    const long long total = static_cast<long long>(n) * c.table_w;
    for (long long t = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; t < total; t += 256ll * gridDim.x) {
        const int i = static_cast<int>(t / c.table_w), j = static_cast<int>(t % c.table_w);
        const int s = seqs[i];
        if (s < 0 || s >= c.n_rows) {
            if (j == 0) kv_error(ATTN_ERR_SHAPE);
            continue;
        }
        if (j == 0) c.lens[s] = 0;
        // an exchange, so that a sequence named twice gives its pages back once
        const int p = atomicExch(&kv_row(c, s)[j], -1);
        if (p < 0) continue;
        if (p >= c.n_pages || atomicSub(&c.refs[p], 1) <= 0) {
            if (p < c.n_pages) atomicAdd(&c.refs[p], 1);
            kv_error(ATTN_ERR_PAGE);
        }
    }
}

// The k-th free page below the number of live pages is to take the contents of the k-th
// live page at or above it: list holds the holes, map[p] the new place of a moved page,
// pairs of kv_move_kernel are (movers[k], holes[k]) with movers in the upper half of list.
__global__ void __launch_bounds__(kPlanThreads) kv_compact_kernel(const KvPool c, int *live_out) {
    __shared__ int sm[33];
    grid_launch_dependents();
    grid_dependency_wait();
    const int live = kv_list<false>(c.refs, 0, c.n_pages, INT_MAX, nullptr, sm);
    int *movers = c.list + (c.n_pages >> 1);
    const int half = c.n_pages >> 1;  // holes, and movers, are at most half of the pages
    const int m = kv_list<true>(c.refs, 0, live, half, c.list, sm);
    kv_list<false>(c.refs, live, c.n_pages, half, movers, sm);
    // an entry that names a free page, which no table should, stays what it is
    for (int p = live + static_cast<int>(threadIdx.x); p < c.n_pages; p += kPlanThreads) c.map[p] = p;
    __syncthreads();
    for (int k = threadIdx.x; k < m; k += kPlanThreads) {
        const int from = movers[k], to = c.list[k];
        c.map[from] = to;
        c.refs[to] = c.refs[from];
        c.refs[from] = 0;
    }
    if (threadIdx.x == 0) {
        c.count[0] = m;
        c.count[1] = live;
        if (live_out != nullptr) *live_out = live;
    }
}

// Table entries that name a moved page name its new place.
__device__ __forceinline__ void kv_rename(const KvPool &c, long long first, long long step) {
    const int live = c.count[1];
    const long long entries = static_cast<long long>(c.n_rows) * c.table_w;
    for (long long t = first; t < entries; t += step) {
        const int p = c.table[t];
        if (p >= live && p < c.n_pages) c.table[t] = c.map[p];
    }
}

// The full pages of forked sequences: one reference more each.
__device__ __forceinline__ void kv_share(const KvPool &c, const int *parents, const int *children, int n,
                                         long long first, long long step) {
    const long long entries = static_cast<long long>(n) * c.table_w;
    for (long long t = first; t < entries; t += step) {
        const int i = static_cast<int>(t / c.table_w), j = static_cast<int>(t - static_cast<long long>(i) * c.table_w);
        if (c.pairs[3 * i] == -2) continue;  // refused
        const int b = children[i];
        if (j >= c.lens[b] >> c.page_shift) continue;
        const int p = kv_row(c, parents[i])[j];
        if (p < 0 || p >= c.n_pages) continue;  // (changed since it was looked at, against the rules)
        atomicAdd(&c.refs[p], 1);
        kv_row(c, b)[j] = p;
    }
}

enum KvMove { kMoveCopy, kMoveFork, kMoveCompact };

// Copies rows of pages in every layer, K and V: a warp moves up to 4 KB of one head of one
// page at a time.  kMoveCopy: pages src[i] -> dst[i]; kMoveFork: the pairs of kv_fork_kernel
// for parents src, children dst, and their tables; kMoveCompact: the movers and holes of
// kv_compact_kernel, and the table entries renamed.
template <KvMove kMove>
__global__ void __launch_bounds__(256) kv_move_kernel(const KvPool c, const int *src, const int *dst, int n) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const long long wid = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5), warps = 8ll * gridDim.x;
    if (kMove == kMoveCompact) {
        n = c.count[0];
        kv_rename(c, static_cast<long long>(blockIdx.x) * 256 + threadIdx.x, 256ll * gridDim.x);
    }
    if (kMove == kMoveFork)
        kv_share(c, src, dst, n, static_cast<long long>(blockIdx.x) * 256 + threadIdx.x, 256ll * gridDim.x);
    const int head16 = c.page * c.row16;         // 16-byte chunks of one head of a page
    const int segs = (head16 + 255) >> 8;        // of 4 KB
    const unsigned per = static_cast<unsigned>(c.n_layers) * 2u * c.Hkv * segs;  // segments per page
    const size_t page16 = static_cast<size_t>(c.Hkv) * head16, layer16 = page16 * c.n_pages;
    const long long total = static_cast<long long>(n) * per;
    for (long long t = wid; t < total; t += warps) {
        const int i = static_cast<int>(t / per);
        unsigned x = static_cast<unsigned>(t - static_cast<long long>(i) * per);
        int a, b, rows = c.page;
        if (kMove == kMoveCopy) {
            a = src[i];
            b = dst[i];
            if (a < 0 || a >= c.n_pages || b < 0 || b >= c.n_pages) {
                if (x == 0 && lane == 0) kv_error(ATTN_ERR_PAGE);
                continue;
            }
        } else if (kMove == kMoveFork) {
            a = c.pairs[3 * i];
            if (a < 0) continue;
            b = c.pairs[3 * i + 1];
            rows = c.pairs[3 * i + 2];
        } else {
            a = c.list[(c.n_pages >> 1) + i];
            b = c.list[i];
        }
        const unsigned seg = x % segs;
        x /= segs;
        const unsigned head = x % c.Hkv;
        x /= c.Hkv;
        uint4 *pool = (x & 1u) ? c.v : c.k;
        const size_t at = (x >> 1) * layer16 + static_cast<size_t>(head) * head16;
        const int left = rows * c.row16 - static_cast<int>(seg << 8);  // chunks from this segment on
        const uint4 *from = pool + at + a * page16 + (seg << 8);
        uint4 *to = pool + at + b * page16 + (seg << 8);
        uint4 r[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e * 32 + lane < left) r[e] = from[e * 32 + lane];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e * 32 + lane < left) to[e * 32 + lane] = r[e];
    }
}

// Rows of new tokens into their pages: sequence s's tokens [cu[s], cu[s+1]) are its last
// positions.  A warp per token: it asks for the token's rows (all heads, K and V, 16 bytes a
// lane) and looks for their place, a chain of dependent loads, while they are on their way.
struct KvAppend {
    const uint4 *k, *v;                        // of the layer's new rows
    long long k_row, k_head, v_row, v_head;    // strides in 16-byte chunks
    const int *cu, *seqs;
    int n, total, layer;
};
// Where token t's rows go (one warp): page * Hkv * page rows + row within the page, or -1 (behind the last
// sequence, or refused).
__device__ __forceinline__ long long append_place(const KvPool &c, const KvAppend &x, int t) {
    int lo = 0, hi = x.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (x.cu[mid] <= t) lo = mid; else hi = mid;
    }
    const int a = x.cu[lo], b = x.cu[lo + 1];
    if (t < a || t >= b) return -1;
    const int s = x.seqs != nullptr ? x.seqs[lo] : lo;
    bool again = false;  // named before in the list
    if (x.seqs != nullptr) {
        for (int j = threadIdx.x & 31; j < lo; j += 32) again |= x.seqs[j] == s;
        again = __any_sync(0xffffffffu, again);
    }
    if (s < 0 || s >= c.n_rows || again) {
        kv_error(ATTN_ERR_SHAPE);
        return -1;
    }
    const int len = c.lens[s], pos = len - (b - t);
    // none of a sequence's rows where it has fewer positions than new tokens, or where its
    // offsets leave the new rows
    if (a < 0 || b > x.total || static_cast<long long>(b) - a > len || (pos >> c.page_shift) >= c.table_w) {
        kv_error(ATTN_ERR_SHAPE);
        return -1;
    }
    const int p = kv_row(c, s)[pos >> c.page_shift];
    if (p < 0 || p >= c.n_pages || c.refs[p] != 1) {
        kv_error(ATTN_ERR_PAGE);  // no page, or one that another sequence shares
        return -1;
    }
    return static_cast<long long>(p) * c.Hkv * c.page + (pos & (c.page - 1));
}

// (4 blocks per SM: 13419 tokens take 22.0 us at the 3 that 78 registers leave, 20.6 at 64 registers)
__global__ void __launch_bounds__(256, 4) kv_append_kernel(const KvPool c, const KvAppend x) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int t = static_cast<int>(blockIdx.x) * 8 + static_cast<int>(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= x.total) return;
    const unsigned row = static_cast<unsigned>(c.Hkv) * c.row16;  // chunks of a token, K or V
    const size_t layer16 = static_cast<size_t>(x.layer) * c.n_pages * c.Hkv * c.page * c.row16;
    long long at = 0;
    for (unsigned i0 = lane; i0 < 2u * row + lane; i0 += 32u * 8u) {
        uint4 r[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const unsigned i = i0 + 32u * e;
            if (i >= 2u * row) continue;
            const bool v = i >= row;
            const unsigned y = v ? i - row : i, head = y / c.row16, ch = y - head * c.row16;
            r[e] = (v ? x.v + t * x.v_row + head * x.v_head : x.k + t * x.k_row + head * x.k_head)[ch];
        }
        if (i0 == static_cast<unsigned>(lane)) at = append_place(c, x, t);  // the rows are on their way
        if (at < 0) return;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const unsigned i = i0 + 32u * e;
            if (i >= 2u * row) continue;
            const bool v = i >= row;
            const unsigned y = v ? i - row : i, head = y / c.row16, ch = y - head * c.row16;
            (v ? c.v : c.k)[layer16 + (at + static_cast<long long>(head) * c.page) * c.row16 + ch] = r[e];
        }
    }
}

// Keeps the accepted path of each tree: the row of tree token path[i][j] moves to position
// base + j (base: the positions before the tree) in every layer, and the sequence ends
// behind the path.  The path ascends, so path[j] >= j and a row is never overwritten before
// it is read, as long as one thread moves a column's rows in order (8 are read, then
// written, at a time).  A cluster of kAcceptCtas blocks per sequence shares the columns; the
// length is written once all of them have read it.
constexpr int kAcceptCtas = 8, kAcceptMost = 128;
__global__ void __cluster_dims__(kAcceptCtas, 1, 1) __launch_bounds__(256)
    kv_accept_kernel(const KvPool c, const int *cu, const int *seqs, const int *path, int path_w, const int *taken) {
    __shared__ long long from[kAcceptMost], to[kAcceptMost];  // row within a layer
    __shared__ int moves, bad;
    grid_launch_dependents();
    grid_dependency_wait();
    const int i = blockIdx.x / kAcceptCtas, rank = blockIdx.x % kAcceptCtas;
    const int s = seqs != nullptr ? seqs[i] : i;
    const int T = cu[i + 1] - cu[i], m = taken[i];
    if (threadIdx.x == 0) {
        moves = 0;
        bad = 0;
    }
    // a sequence named before in the list is refused: its length may be changing by now
    int again = 0;
    if (seqs != nullptr)
        for (int j = threadIdx.x; j < i; j += 256) again |= seqs[j] == s ? 1 : 0;
    again = __syncthreads_or(again);
    int base = 0;
    bool fine = again == 0 && s >= 0 && s < c.n_rows && T >= 0 && T <= kAcceptMost && m >= 0 && m <= T && m <= path_w;
    if (fine) {
        base = c.lens[s] - T;
        fine = base >= 0 && ((base + T + c.page - 1) >> c.page_shift) <= c.table_w;
    }
    if (fine && threadIdx.x < m) {
        const int j = threadIdx.x;
        const int at = path[static_cast<size_t>(i) * path_w + j];
        const int prev = j > 0 ? path[static_cast<size_t>(i) * path_w + j - 1] : -1;
        // (each entry on its own, before it is an index: one that ascends from a negative one is
        // negative, too, and lies before the tree)
        if (at < 0 || at <= prev || at >= T) {
            atomicExch(&bad, 1);  // not an ascending path within the tree
        } else {
            const int ps = base + at, pd = base + j;
            const int a = kv_row(c, s)[ps >> c.page_shift], b = kv_row(c, s)[pd >> c.page_shift];
            if (a < 0 || a >= c.n_pages || b < 0 || b >= c.n_pages || (at != j && c.refs[b] != 1)) {
                atomicExch(&bad, 2);
            } else {
                from[j] = static_cast<long long>(a) * c.Hkv * c.page + (ps & (c.page - 1));
                to[j] = static_cast<long long>(b) * c.Hkv * c.page + (pd & (c.page - 1));
                if (at != j) atomicAdd(&moves, 1);
            }
        }
    }
    __syncthreads();
    if (!fine || bad) {
        if (rank == 0 && threadIdx.x == 0) kv_error(bad == 2 ? ATTN_ERR_PAGE : ATTN_ERR_SHAPE);
        fine = false;
    }
    if (fine && moves > 0) {
        const int stay = m - moves;  // an ascending path: tokens 0 .. stay-1 are where they belong
        const size_t layer16 = static_cast<size_t>(c.n_pages) * c.Hkv * c.page * c.row16;
        const unsigned cols = static_cast<unsigned>(c.n_layers) * 2u * c.Hkv * c.row16;
        for (unsigned x = rank * 256u + threadIdx.x; x < cols; x += 256u * kAcceptCtas) {
            const unsigned ch = x % c.row16, y = x / c.row16, head = y % c.Hkv, z = y / c.Hkv;
            uint4 *pool = ((z & 1u) ? c.v : c.k) + (z >> 1) * layer16 + ch;
            const long long hrow = static_cast<long long>(head) * c.page;
            for (int j0 = stay; j0 < m; j0 += 8) {
                uint4 r[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (j0 + e < m) r[e] = pool[(from[j0 + e] + hrow) * c.row16];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (j0 + e < m) pool[(to[j0 + e] + hrow) * c.row16] = r[e];
            }
        }
    }
    cooperative_groups::this_cluster().sync();  // every block has read the length
    if (fine && rank == 0 && threadIdx.x == 0) c.lens[s] = base + m;
}

}  // namespace gqa
