/*
 * gqa_attn.h -- C ABI of the GB300 (sm_103a) fused grouped-query attention
 * forward library (libgqa_attn.so).
 *
 * The operation is the fused attention forward of the page "从零开始写Qwen3"
 * (deepseek.csdn.net/6a3201f8..., section "FlashAttention": O_i is the sum over
 * key blocks j of softmax(mask(Q_i K_j^T / sqrt(D))) V_j, computed with the
 * online-softmax update of section "在线softmax" so that no N x N score matrix
 * is ever stored), with
 *   - grouped-query heads: query head hq reads key/value head
 *     hq / (Hq / Hkv) of the same batch entry (same section's kernel: the
 *     flattened (b, q_head) index divided by the group count);
 *   - the optional causal mask j <= i on absolute row indices (same section:
 *     positions with offsets_qm >= offsets_kk are kept); with Nq query rows
 *     over Nk keys (attn_fwd_kv and the calls built on it) the query rows are
 *     the last Nq positions, so row i keeps keys j <= i + Nk - Nq;
 *   - the natural-log log-sum-exp of each masked, scaled score row,
 *     lse = max_j s_ij + ln(sum_j exp(s_ij - max_j s_ij)), written as fp32.
 *
 * Arithmetic: Q K^T and P V on the tensor cores with fp32 accumulation;
 * running max, running sum and the output accumulator in fp32 (page
 * "从零开始写Qwen3", deepseek.csdn.net/6a31faef..., section "改进点4-去掉多余的
 * 转换"); the probabilities P are rounded to the input type before the P V
 * product; O is rounded once, to nearest even, at the end.
 */
#ifndef GQA_ATTN_H
#define GQA_ATTN_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of q, k, v and o. */
typedef enum {
    ATTN_F16 = 0,  /* IEEE binary16 */
    ATTN_BF16 = 1  /* bfloat16 */
} attn_dtype_t;

typedef enum {
    ATTN_OK = 0,
    ATTN_ERR_NULL = 1,     /* q, k, v or o is NULL while the problem is non-empty */
    ATTN_ERR_SHAPE = 2,    /* negative size, Hkv < 1, Hq % Hkv != 0, a size too
                              large for 32-bit tile coordinates, or scale not
                              finite and > 0 */
    ATTN_ERR_HEADDIM = 3,  /* D is not 64 or 128 */
    ATTN_ERR_DTYPE = 4,    /* dtype is not ATTN_F16 / ATTN_BF16 */
    ATTN_ERR_ALIGN = 5,    /* q, k, v or o not 16-byte aligned, or lse not 4-byte aligned */
    ATTN_ERR_LAUNCH = 6,   /* a CUDA runtime / driver call failed (see attn_last_cuda_error) */
    ATTN_ERR_TIMEOUT = 7,  /* a bounded in-kernel wait ran out (reported by
                              attn_last_device_error) */
    ATTN_ERR_NODEVICE = 8, /* no CUDA device of compute capability 10.3 is current */
    ATTN_ERR_SCRATCH = 9,  /* attn_fwd_decode_noalloc: the problem needs more scratch
                              than the library's fixed device buffer holds;
                              attn_fwd_tree: the workspace is too small */
    ATTN_ERR_PAGE = 10,    /* (attn_last_device_error) a page table entry is missing or out
                              of range, or names a shared page that would be written */
    ATTN_ERR_POOL = 11     /* (attn_last_device_error) the pool has not enough free pages */
} attn_status_t;

/*
 * attn_fwd -- O = softmax(mask(Q K^T * scale)) V and LSE, one kernel launch.
 *
 * q    device pointer, [B, Hq,  N, D] contiguous (row-major, D fastest), dtype
 * k    device pointer, [B, Hkv, N, D] contiguous, dtype
 * v    device pointer, [B, Hkv, N, D] contiguous, dtype
 * o    device pointer, [B, Hq,  N, D] contiguous, dtype (written)
 * lse  device pointer, [B, Hq, N] fp32 (written), or NULL to skip it
 * B, Hq, Hkv, N   batch, query heads, key/value heads (Hq % Hkv == 0), sequence
 *                 length (keys and queries have the same length N)
 * D      head dimension, 64 or 128
 * scale  logit scale, finite and > 0 (1/sqrt(D) for standard attention)
 * causal nonzero: keep only keys j <= i for query row i (top-left aligned)
 * dtype  ATTN_F16 or ATTN_BF16 for q, k, v and o
 * stream CUDA stream (cudaStream_t) the kernel is launched on; NULL = legacy
 *        default stream
 *
 * Ownership: the caller owns every buffer; the library allocates no device
 * memory per call and keeps no pointer after the call returns.  o must not
 * overlap q, k or v.
 * Asynchrony: returns after the launch is queued on `stream`; results are
 * ready when the stream reaches that point.  The call never synchronises.
 * CUDA graphs: a call can be captured into a CUDA graph (one kernel node; the
 * node keeps the pointers, sizes and scale of the captured call).  The first
 * call of each (D, dtype, causal) variant on a device sets the kernel's shared
 * memory limit, which is not a stream operation: make one such call before
 * capturing, as with any library that configures itself on first use.
 * Errors: argument errors are returned before anything is launched and leave
 * o and lse untouched.  An empty problem (B, Hq or N equal to 0) launches
 * nothing and returns ATTN_OK.  A wait inside the kernel that runs out of time
 * makes the kernel stop early and record ATTN_ERR_TIMEOUT, which
 * attn_last_device_error reports; o and lse are then undefined.
 */
attn_status_t attn_fwd(const void *q, const void *k, const void *v, void *o, float *lse,
                       int B, int Hq, int Hkv, int N, int D, float scale, int causal,
                       attn_dtype_t dtype, void *stream);

/*
 * attn_fwd_kv -- as attn_fwd, for Nq query rows attending over Nk keys (a
 * block of new tokens over a longer key/value sequence, e.g. a chunk of a
 * prefill or a decode step over a cache).  The derivation page's kernel
 * ("从零开始写Qwen3", deepseek.csdn.net/6a3201f8..., section "FlashAttention")
 * keeps the query and key lengths apart; this call does too.
 *
 * q, o   [B, Hq,  Nq, D];  k, v  [B, Hkv, Nk, D];  lse  [B, Hq, Nq] or NULL
 * causal nonzero: the query rows are the last Nq positions of the Nk-long
 *        sequence (bottom-right alignment): row i keeps keys j <= i + Nk - Nq.
 *        With Nq == Nk this is attn_fwd's mask j <= i.
 * Errors: as attn_fwd, plus ATTN_ERR_SHAPE when Nk == 0 while Nq > 0, or when
 *        causal and Nq > Nk (some query row would see no key).  Nq == 0 is an
 *        empty problem (nothing launched, ATTN_OK).
 * attn_fwd(..., N, ...) is attn_fwd_kv(..., N, N, ...).
 */
attn_status_t attn_fwd_kv(const void *q, const void *k, const void *v, void *o, float *lse,
                          int B, int Hq, int Hkv, int Nq, int Nk, int D, float scale,
                          int causal, attn_dtype_t dtype, void *stream);

/*
 * attn_fwd_kv_split -- attn_fwd_kv with a caller workspace that lets the library
 * balance the last round of its schedule.
 *
 * The persistent kernel deals 256-row items to one CTA per SM in rounds.  When
 * every item has the same length (no mask, or a chunk of queries over a much
 * longer key sequence) and the last round holds at most half a round of items,
 * each of those items is cut into up to 8 key ranges; the pieces (the partial
 * O / l in fp32 and the partial log-sum-exp of every row) go to the workspace,
 * and the warp that computes the last piece of its rows merges them:
 * lse = log sum_s exp(lse_s), O = sum_s exp(lse_s - lse) O_s -- the online-softmax
 * update of page "从零开始写Qwen3" (deepseek.csdn.net/6a3201f8..., section
 * "在线softmax"), applied across CTAs.  The result equals attn_fwd_kv's up to
 * rounding.
 *
 * Arguments, layout, masks and errors: as attn_fwd_kv, plus
 * workspace        device pointer, 256-byte aligned, or NULL; workspace_bytes its
 *                  size.  attn_fwd_kv_split_workspace gives the size the plan needs
 *                  (0 when nothing is cut, e.g. causal problems with Nq == Nk,
 *                  whose items already differ in length).  With a NULL or smaller
 *                  workspace, or when nothing is cut, the call is attn_fwd_kv.
 * Contents: the workspace needs no initial value; its counters carry the launch's
 *   sequence number, so stale contents are recognised.  A captured call replays
 *   correctly as long as no replay of it has timed out (ATTN_ERR_TIMEOUT); after a
 *   timeout, capture the call again or clear the workspace.
 * Races: calls that can run at the same time must not share a workspace.
 * ATTN_ERR_ALIGN also when workspace is not 256-byte aligned.
 */
attn_status_t attn_fwd_kv_split_workspace(int B, int Hq, int Hkv, int Nq, int Nk, int D, int causal,
                                          size_t *bytes);
attn_status_t attn_fwd_kv_split(const void *q, const void *k, const void *v, void *o, float *lse,
                                int B, int Hq, int Hkv, int Nq, int Nk, int D, float scale,
                                int causal, attn_dtype_t dtype, void *workspace,
                                size_t workspace_bytes, void *stream);

/*
 * attn_fwd_decode -- the same function as attn_fwd_kv, computed by a kernel
 * for short query blocks over long key sequences (decode steps, small chunks).
 *
 * The Hq / Hkv query heads that share a kv head have adjacent rows, so their
 * Hq/Hkv * Nq query rows are stacked into 128-row tiles and every K/V tile is
 * read once per kv head (grouped-query packing).  The key range is cut into
 * splits, one CTA each, so that few kv heads still fill the GPU; the splits'
 * partial results are merged through their log-sum-exp by a second kernel
 * (the online-softmax merge of the derivation page "从零开始写Qwen3",
 * deepseek.csdn.net/6a3201f8..., section "在线softmax", applied across CTAs).
 *
 * Arguments as attn_fwd_kv, plus:
 * workspace        device pointer, 16-byte aligned, or NULL; scratch for the
 *                  partial results, owned by the caller, used by the two
 *                  kernels this call queues on `stream` and free again once
 *                  the stream has passed them.  Nothing in it needs to start
 *                  at any value.
 * workspace_bytes  its size.  The call uses as many splits as it wants and
 *                  the workspace holds (attn_fwd_decode_workspace gives the
 *                  size for all it wants); with NULL or too little for two
 *                  splits it runs one split, which needs no workspace.
 * Two calls that run at the same time must not share a workspace.
 * Errors: as attn_fwd_kv; ATTN_ERR_ALIGN also for a misaligned workspace.
 */
attn_status_t attn_fwd_decode(const void *q, const void *k, const void *v, void *o, float *lse,
                              int B, int Hq, int Hkv, int Nq, int Nk, int D, float scale,
                              int causal, attn_dtype_t dtype, void *workspace,
                              size_t workspace_bytes, void *stream);

/*
 * Workspace bytes attn_fwd_decode uses for this problem on the current device
 * when given enough (0 when it would run one split).  Writes *bytes; returns
 * argument errors as attn_fwd_kv, ATTN_ERR_NULL for bytes == NULL and
 * ATTN_ERR_NODEVICE without an sm_103 device.
 */
attn_status_t attn_fwd_decode_workspace(int B, int Hq, int Hkv, int Nq, int Nk, int D,
                                        size_t *bytes);

/*
 * attn_fwd_decode_noalloc -- attn_fwd_decode for callers that cannot allocate
 * device memory (an allocator-free runtime, a captured graph that must not own
 * buffers, a call site that only receives q, k, v, o and lse).  The pages have
 * no counterpart: their kernels keep everything on chip and need no scratch;
 * the key splits of attn_fwd_decode do.
 *
 * Instead of a caller workspace the call uses a buffer that the library
 * itself holds in device memory: ATTN_NOALLOC_SCRATCH_BYTES (16 MiB) per
 * device, a static array of this library's module, so nothing is allocated
 * on any call.  The split plan is the one attn_fwd_decode chooses with an
 * unlimited workspace, so both calls give the same bits.  That plan needs at
 * most (number of SMs) * 128 * (D + 1) * 4 bytes (10 MB on 152 SMs), so the
 * buffer covers every problem on devices with up to 254 SMs; a plan that needs
 * more (e.g. one forced by attn_test_force_splits) returns ATTN_ERR_SCRATCH
 * before anything is launched.
 *
 * Arguments, layout, masks and errors: as attn_fwd_kv.
 * Setup: the first call on a device that passes argument validation looks
 *   up the buffer's address (not a stream operation), whether or not its plan
 *   splits the keys; make one such call on each device before capturing calls
 *   into a CUDA graph.
 * Contents: nothing in the buffer needs to start at any value; each call
 *   writes every part it reads.
 * Races: all calls on one device share the buffer.  Calls queued on one
 *   stream are ordered and safe; calls that can run at the same time (other
 *   streams, concurrently replayed graphs) race on it and give undefined
 *   results.
 */
#define ATTN_NOALLOC_SCRATCH_BYTES (16u << 20)
attn_status_t attn_fwd_decode_noalloc(const void *q, const void *k, const void *v, void *o,
                                      float *lse, int B, int Hq, int Hkv, int Nq, int Nk, int D,
                                      float scale, int causal, attn_dtype_t dtype, void *stream);

/*
 * attn_fwd_host -- attn_fwd_kv for inputs and outputs in host memory: copies Q,
 * K, V in, computes, copies O and LSE out, overlapping the three.
 *
 * The B * Hkv (batch, kv head) groups are contiguous in every tensor (a group's
 * Hq / Hkv query heads are adjacent), so the call cuts them into up to 8 chunks
 * of consecutive groups: chunk c + 1 is copied in on one library stream while
 * chunk c is computed on `stream` and chunk c - 1 is copied out on another.
 * The pages have no counterpart (their benchmarks start from device tensors).
 *
 * q_h, k_h, v_h       host inputs, layouts as attn_fwd_kv; page-locked memory
 *                     makes the copies asynchronous (pageable memory works but
 *                     serialises them)
 * o_h, lse_h          host outputs (lse_h NULL exactly when lse_d is NULL)
 * q_d ... lse_d       device buffers of the same sizes, owned by the caller;
 *                     they hold the inputs and results when the call is done
 * stream              the call is ordered after earlier work on `stream`, and
 *                     later work on `stream` waits for its last copy out; the
 *                     call returns without waiting.  Host outputs are valid
 *                     once `stream` has passed that point.
 * Set-up: the first call on a device creates the library's two copy streams
 *   and its events (not memory; kept for the life of the process).
 * Errors: as attn_fwd_kv; ATTN_ERR_NULL for a missing host pointer.
 */
attn_status_t attn_fwd_host(const void *q_h, const void *k_h, const void *v_h, void *o_h,
                            float *lse_h, void *q_d, void *k_d, void *v_d, void *o_d, float *lse_d,
                            int B, int Hq, int Hkv, int Nq, int Nk, int D, float scale, int causal,
                            attn_dtype_t dtype, void *stream);

/*
 * attn_fwd_varlen -- attention over packed sequences of different lengths (the
 * prompts of a batch, without padding).
 *
 * Sequence s owns query rows [cu_q[s], cu_q[s+1]) of q, o and lse and rows
 * [cu_k[s], cu_k[s+1]) of k and v.  Each of its rows attends over its keys
 * only; with the causal mask the queries are the last Nq_s positions of the
 * Nk_s-long sequence, as in attn_fwd_kv, so row i sees keys j <= i + Nk_s - Nq_s.
 * A row that sees no key (causal with Nq_s > Nk_s, or no keys at all) gets
 * o = 0 and lse = -inf.
 *
 * q, o    [total_q, Hq, D], k, v  [total_k, Hkv, D], 16-byte aligned; other layouts
 *         through `strides`
 * lse     [Hq, total_q] fp32 (written), or NULL
 * cu_q, cu_k  device pointers, [n_seqs + 1] ints that ascend from 0; the lengths are
 *         read on the device, so a captured call replays on new ones.  cu_k NULL: the
 *         keys' offsets are cu_q's (total_k == total_q).  Lengths of zero are allowed.
 *         Rows behind the last sequence are left as they are, and nothing in them, nor
 *         in another sequence, reaches a result (not even infinities or NaN); within a
 *         sequence a non-finite value of V reaches exactly the rows that see its key.
 * strides host pointer, NULL for the layouts above, or 8 element strides {q row, q head,
 *         k row, k head, v row, v head, o row, o head}, each a multiple of 8 and at
 *         least D, the larger of a pair a multiple of the smaller and no two rows
 *         overlapping ([heads, rows, D], or heads cut from one projection's output)
 * Rounding: the weights are rounded once to the input type, half a step of each: o is off by
 *         at most u |o| + u sum_j p_j |v_j| and fp32 terms (u 2^-8 for bf16, 2^-11 for fp16;
 *         for fp16 2^-25 |v_j| more for each weight below 2^-14, the smallest normal number).
 *         attn_fwd and attn_fwd_kv keep a second term of the weights where a row's sum is
 *         small, and come nearer there; lse is fp32 in all of them.
 * Limits: total_q and total_k at most 65535 * 128.
 * Errors: as attn_fwd_kv (no error for Nq_s > Nk_s); ATTN_ERR_SHAPE for strides.
 *         Offsets that descend or leave the tensors are clamped, with no more work done
 *         than ascending ones can be, and attn_last_device_error reports ATTN_ERR_SHAPE.
 * Graphs, streams and ownership: as attn_fwd, one launch per 2048 sequences; no workspace.
 */
attn_status_t attn_fwd_varlen(const void *q, const void *k, const void *v, void *o, float *lse,
                              const int *cu_q, const int *cu_k, int n_seqs, int total_q,
                              int total_k, int Hq, int Hkv, int D, const long long *strides,
                              float scale, int causal, attn_dtype_t dtype, void *stream);

/*
 * attn_fwd_varlen_window -- attn_fwd_varlen with the causal mask and a sliding window: the row
 * at position pos = i + Nk_s - Nq_s of sequence s sees the keys j <= pos with j > pos - window
 * (itself and the window - 1 before it) or j < sinks (the first keys, which stay visible).
 *
 * window  at least 1; one of total_k or more is the causal mask alone.  sinks: at least 0.
 * Key tiles that no row of a block sees are neither loaded nor computed.
 * Everything else, rounding, values in masked places, limits and errors among it: as
 * attn_fwd_varlen with causal set; ATTN_ERR_SHAPE also for window < 1 or sinks < 0.
 */
attn_status_t attn_fwd_varlen_window(const void *q, const void *k, const void *v, void *o, float *lse,
                                     const int *cu_q, const int *cu_k, int n_seqs, int total_q,
                                     int total_k, int Hq, int Hkv, int D, const long long *strides,
                                     float scale, int window, int sinks, attn_dtype_t dtype,
                                     void *stream);

/*
 * A paged key/value cache.  All pointers are device memory owned by the caller.
 *
 * k, v    pools [n_layers, n_pages, Hkv, page, D] contiguous, dtype, 16-byte aligned
 * table   [n_rows, table_width]: row s lists the pages of sequence s from its first
 *         position on, -1 behind the last; position j lies in row j % page of page
 *         table[s][j / page].  The same page index serves every layer, K and V.
 * lens    [n_rows] positions of each sequence
 * refs    [n_pages] number of table entries that name the page; 0: the page is free
 * scratch attn_kv_scratch bytes that the calls on this cache use; needs no value
 * page    positions per page, a power of two from 16 to 4096
 * An empty cache is table = -1, lens = 0, refs = 0.
 *
 * The calls below read their lists on the device and never synchronise; calls on
 * one cache must be ordered (one stream, or events): they change its state and
 * share its scratch.  Sequences are rows of the table; a list names each at most
 * once unless said otherwise.  Where a list, a table or the state is wrong, the
 * sequence is left as it was and attn_last_device_error reports ATTN_ERR_SHAPE
 * (an index or length out of range, a sequence named twice), ATTN_ERR_PAGE or
 * ATTN_ERR_POOL.  An empty list launches nothing.  All can be captured.
 */
typedef struct {
    void *k, *v;
    int *table, *lens, *refs, *scratch;
    int n_layers, n_pages, page, Hkv, D, n_rows, table_width;
    attn_dtype_t dtype;
} attn_kv_cache_t;

/* Bytes of a cache's scratch. */
attn_status_t attn_kv_scratch(int n_pages, int n_rows, size_t *bytes);

/* Makes room for n_new[i] more positions of sequence seqs[i] (i, when seqs is NULL):
 * takes the free pages that are missing, lowest index first, and grows lens.  Requests
 * are served in order; from the first one on that the free pages do not hold, nothing
 * changes (ATTN_ERR_POOL). */
attn_status_t attn_kv_extend(const attn_kv_cache_t *cache, const int *seqs, const int *n_new,
                             int n, void *stream);

/* Writes the keys and values of new tokens into their pages of one layer.  Packed rows
 * [cu[i], cu[i+1]) of k_new, v_new [total, Hkv, D] are the last positions of sequence
 * seqs[i] (i, when NULL), whose lens already counts them (attn_kv_extend).  strides: NULL,
 * or 4 element strides {k row, k head, v row, v head}, multiples of 8.  Rows whose page is
 * missing, out of range or shared with another sequence are not written (ATTN_ERR_PAGE; the
 * sequence's other rows are), nor the rows of a sequence that was named before in the list
 * (ATTN_ERR_SHAPE). */
attn_status_t attn_kv_append(const attn_kv_cache_t *cache, int layer, const void *k_new,
                             const void *v_new, const long long *strides, const int *cu,
                             const int *seqs, int n, int total, void *stream);

/* Keeps the accepted tokens of drafted trees, in every layer.  The last
 * T = cu[i+1] - cu[i] <= 128 positions of sequence seqs[i] (i, when NULL) are its tree's
 * tokens; path[i][0 .. taken[i]) are the accepted ones, ascending.  Their rows move to the
 * positions right behind those before the tree, and the sequence ends there; its pages
 * stay with it.  path is [n, path_width].  A sequence named again stays as its first entry
 * leaves it (ATTN_ERR_SHAPE). */
attn_status_t attn_kv_accept(const attn_kv_cache_t *cache, const int *cu, const int *seqs,
                             const int *path, int path_width, const int *taken, int n,
                             void *stream);

/* Copies the contents of page src[i] to page dst[i], in every layer.  A page named in dst
 * must not be named again in src or dst. */
attn_status_t attn_kv_copy(const attn_kv_cache_t *cache, const int *src, const int *dst, int n,
                           void *stream);

/* children[i], an empty sequence, becomes a copy of parents[i]: it shares its parent's full
 * pages, and its own last page, where that is not full, is a copy in the lowest free page.
 * A parent may be named many times, a child once, and no child as a parent.  Served in
 * order as attn_kv_extend. */
attn_status_t attn_kv_fork(const attn_kv_cache_t *cache, const int *parents, const int *children,
                           int n, void *stream);

/* Empties the sequences: one reference less for each of their pages.  A sequence may be
 * named twice.  Entries of its row that name no page of the pool, or one that has no
 * references, are dropped with the others (ATTN_ERR_PAGE). */
attn_status_t attn_kv_free(const attn_kv_cache_t *cache, const int *seqs, int n, void *stream);

/* Moves the live pages to the front of the pool, so that they are pages 0 .. live - 1: the
 * k-th live page at or past `live` takes the place of the k-th free one before it, and the
 * table is rewritten.  live: device pointer that receives their number, or NULL. */
attn_status_t attn_kv_compact(const attn_kv_cache_t *cache, int *live, void *stream);

/*
 * attn_fwd_tree -- attention of drafted token trees over a paged cache; with one
 * token per sequence, the decoding step over pages.
 *
 * The last T = cu[i+1] - cu[i] <= 128 positions of sequence seqs[i] (i, when seqs is NULL)
 * are the tokens of its tree, already in the cache (attn_kv_extend, attn_kv_append); their
 * queries are packed rows [cu[i], cu[i+1]).  Token t sees every position before the tree,
 * its ancestors and itself.  The Hq / Hkv heads of a kv head and the tokens of a tree share
 * each K/V tile, and the key tiles of all sequences are shared out evenly over the GPU; cut
 * pieces are merged by a second kernel.
 *
 * q, o      [total_q, Hq, D], cache->dtype, 16-byte aligned; strides: NULL, or 4 element
 *           strides {q row, q head, o row, o head} as in attn_fwd_varlen, rows outside heads
 *           in q
 * lse       [Hq, total_q] fp32, or NULL
 * parents   device [total_q]: the index within its tree of each token's parent, less than
 *           its own, or -1 for a child of the last position before the tree.  NULL: a chain
 *           (each token follows the one before it), the causal mask.
 * cu, seqs  device pointers; a sequence may be named twice
 * workspace device pointer, 16-byte aligned, attn_fwd_tree_workspace bytes; needs no
 *           value.  Calls that can run at the same time must not share it.
 * Rows behind the last tree are left as they are.  Rows of a page past the sequence's end
 * may hold anything; a non-finite value of V at a tree's position reaches exactly the tokens
 * that see it, and one before the tree all of them.  Rounding as in attn_fwd_varlen.
 * Errors: as attn_fwd_kv, ATTN_ERR_SHAPE for Hq / Hkv > 128, ATTN_ERR_SCRATCH for a small
 * workspace; attn_last_device_error reports a tree of more than 128 tokens or of more than
 * the sequence's positions and bad offsets or sequences (ATTN_ERR_SHAPE), whose rows are then
 * undefined, and missing pages (ATTN_ERR_PAGE), which read as zeros.
 */
attn_status_t attn_fwd_tree_workspace(int n_seqs, int D, size_t *bytes);
attn_status_t attn_fwd_tree(const void *q, const attn_kv_cache_t *cache, int layer, void *o,
                            float *lse, const int *cu, const int *seqs, const int *parents,
                            int n_seqs, int total_q, int Hq, const long long *strides,
                            float scale, void *workspace, size_t workspace_bytes, void *stream);

/*
 * attn_fwd_tree_window -- attn_fwd_tree with a sliding window; with one token per sequence, the
 * decoding step over the window.
 *
 * A token with d ancestors in its tree stands at position pos = base + d, base being the number
 * of positions before the tree, and sees what a sequence of those before the tree, its ancestors
 * and itself would show it: positions before the tree j > pos - window or j < sinks; itself and
 * its nearest window - 1 ancestors; and ancestors that stand at a position below sinks.
 *
 * window  at least 1; one of table_width * page or more is attn_fwd_tree.  sinks: at least 0.
 * Positions count the rows that the cache holds: where attn_kv_evict has cut a sequence, its
 * rows have moved up (see its note on rotary positions).  Of the pages, those that hold a part of
 * a run of 128 positions (from a multiple of 128) of which some token sees one are read; the
 * others may be missing.
 * Everything else: as attn_fwd_tree; ATTN_ERR_SHAPE also for window < 1 or sinks < 0.
 */
attn_status_t attn_fwd_tree_window(const void *q, const attn_kv_cache_t *cache, int layer, void *o,
                                   float *lse, const int *cu, const int *seqs, const int *parents,
                                   int n_seqs, int total_q, int Hq, const long long *strides,
                                   float scale, int window, int sinks, void *workspace,
                                   size_t workspace_bytes, void *stream);

/*
 * The weights of cached positions, and eviction by them: a cache of bounded size.
 *
 * weights [n_layers][n_rows][Hkv][table_width * page] fp32, device, 4-byte aligned, owned by the
 * caller: entry j of a sequence's row is the attention weight that its position j has received, in
 * one layer, from the query heads of one kv head.  The library keeps no copy of it: a program
 * that forks a sequence copies its row, one that compacts pages need do nothing.
 *
 * attn_kv_weigh -- adds what the last T = cu[i+1] - cu[i] positions of sequence seqs[i] (i, when
 * NULL) pay, a chain of any length up to the whole sequence:
 *   weights[j] (+)= sum over those tokens t at or behind j, and the Hq / Hkv heads,
 *                   of exp(scale q_t . k_j - lse_t)
 * Their queries are packed rows [cu[i], cu[i+1]) of q, their keys are in the cache.
 *
 * q           [total_q, Hq, D], cache->dtype, 16-byte aligned; strides: NULL, or 2 element strides
 *             {row, head}, rows outside heads
 * lse         [Hq, total_q] fp32: what attn_fwd_varlen or attn_fwd_tree gave for these rows and
 *             all keys up to their own (of a call with a window the sums would not be weights)
 * accumulate  the sums of the positions before the T tokens go on where they stood; 0: they begin at
 *             zero.  Those of the tokens' own positions begin at zero in either case.  Entries
 *             behind the sequence, and sequences without tokens, are left as they are.
 * Scores and sums are fp32, each position's in a fixed order: one result for the same inputs.  A
 * key or query that a pair does not join (a later token, rows behind the end) never matters.
 * Limits: n sequences of the table's width have less than 2^30 / Hkv blocks of 256 positions.
 * Errors: as attn_fwd_tree; attn_last_device_error reports ATTN_ERR_SHAPE for offsets, lengths
 * and sequences out of range, T above the sequence's length and a sequence named twice (its first
 * entry counts), whose weights are then left as they were, and ATTN_ERR_PAGE for a missing page,
 * whose positions' weights are then undefined.  After ATTN_ERR_TIMEOUT the layer's weights of all
 * listed sequences, up to their ends, are undefined (some may hold the new sums and some the old ones):
 * restore them, or weigh from zero, before they are added to or evicted by again.
 */
attn_status_t attn_kv_weigh(const attn_kv_cache_t *cache, int layer, const void *q, const float *lse,
                            float *weights, const int *cu, const int *seqs, int n, int total_q,
                            int Hq, const long long *strides, float scale, int accumulate,
                            void *stream);

/* Cuts sequences seqs[i] (i, when NULL) of more than sinks + heavy + recent positions back to
 * that many.  In every layer and kv head the first `sinks` and the last `recent` stay, and of
 * those between the `heavy` largest in weights (equal ones: the lowest positions; NaN and negative
 * ones count as 0), in their order: their rows of K and V and their weights move up, so that a
 * position's row then differs from head to head, but all have one length.  Weights behind the new
 * end, up to the old one, become 0; rows there stay as they are; the pages behind it are given back.
 * weights may be NULL when heavy is 0 (the oldest positions behind the first go).
 * Rows behind the first position that goes move up, whether one goes or many: let sequences grow
 * between calls.  A sequence of no more positions is left as it is, its pages too.  Pages from that of
 * position `sinks` to the new end are written and must not be shared (those of whole pages of first positions
 * may be): ATTN_ERR_PAGE, also for one that is missing up to the old end; ATTN_ERR_SHAPE for a
 * sequence or length out of range and the second entry of a sequence named twice.
 * Rotary positions: a row keeps the rotation that its key was written with, while lengths, windows and
 * first keys count the rows of the cache.  Where new tokens go on with positions of their own (and not with
 * the cut length), the program keeps count of them.
 * Limits (ATTN_ERR_SHAPE): n * n_layers * Hkv below 2^28, rows of a layer (n_pages * Hkv * page) below 2^32. */
attn_status_t attn_kv_evict(const attn_kv_cache_t *cache, const int *seqs, int n, float *weights,
                            int sinks, int heavy, int recent, void *stream);

/* Static, human-readable name of a status code. */
const char *attn_status_str(attn_status_t status);

/*
 * Synchronises `stream`, then returns and clears the error word that kernels
 * of this library set on the current device (ATTN_OK if none), together with
 * the mark that makes the other CTAs of a launch that gave up exit early.  A
 * CUDA error raised by the synchronisation itself is returned as
 * ATTN_ERR_LAUNCH.  Call it while no other launch of this library is running
 * on the device.
 */
attn_status_t attn_last_device_error(void *stream);

/* Text of the last CUDA error this library saw on the calling thread ("" if none). */
const char *attn_last_cuda_error(void);

/* Library version, e.g. 0x000100 for 0.1.0. */
int attn_version(void);

/*
 * Test hooks for the failure path (process-wide, affect later launches).
 *
 * attn_test_set_wait_timeout_ns: limit of every bounded in-kernel wait, in
 *   nanoseconds; 0 restores the default (4 s).
 * attn_test_inject_stall: nonzero makes later launches skip the load of the
 *   query tile, so the MMA warp's wait on it can only end by running out; the
 *   kernel then records ATTN_ERR_TIMEOUT, drains its own copies in flight,
 *   frees its TMEM and returns.  0 restores normal launches.
 * Neither hook faults, traps or hangs the GPU.
 */
void attn_test_set_wait_timeout_ns(unsigned long long ns);
void attn_test_inject_stall(int enable);

/*
 * attn_test_select_kernel: 0 (default) = persistent warp-specialised kernel
 *   (two 128-row query tiles per work item, P kept in TMEM); 1 = the simpler
 *   kernel with one CTA per 128-row query tile and P staged in shared memory.
 *   Both compute the same operation; the second exists to cross-check the first.
 */
void attn_test_select_kernel(int which);

/* attn_test_force_splits: n > 0 makes attn_fwd_decode and attn_fwd_decode_noalloc
 * use n key splits (as far as the key tiles and the workspace allow); 0 restores
 * their own choice. */
void attn_test_force_splits(int n_splits);

/* attn_test_set_item_order: work-item order of the persistent kernel (the
 * default one of attn_fwd / attn_fwd_kv).  0 (default) = the longest causal
 * row blocks first across all heads, the query heads of a GQA group adjacent;
 * 1 = kv-group major: every row block of one (batch, kv head) group, longest
 * first, before the next group, so that one group's K/V is live in L2 at a
 * time (the grid order of page "从零开始写Qwen3", deepseek.csdn.net/6a31faef...,
 * section "改进1-使用正确的grid").  Both orders compute every item once and give
 * the same bits; the hook exists to measure one against the other. */
void attn_test_set_item_order(int order);

#ifdef __cplusplus
}
#endif

#endif /* GQA_ATTN_H */
