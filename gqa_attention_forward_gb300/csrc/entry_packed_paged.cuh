// Host side of the packed-sequence attention and of the paged cache: checks, launch plans
// and launches of attn_fwd_varlen, attn_fwd_tree and attn_kv_*.  Included once, by
// attn_fwd.cu, whose device check, error text and launch counters it uses.
#pragma once

#include "attn_fwd_tree.cuh"
#include "attn_fwd_varlen.cuh"
#include "kv_pages.cuh"

namespace {

bool misaligned(const void *ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) != 0; }

// Launch with the dependent-launch attribute: the kernel's set-up overlaps the tail of the
// kernel before it, for which it waits (griddepcontrol.wait) before it reads memory.
template <typename... KArgs, typename... Args>
attn_status_t launch_dependent(void (*kern)(KArgs...), unsigned grid, unsigned block, size_t smem, cudaStream_t s,
                               Args... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e != cudaSuccess) {
        note_cuda_error(e, "kernel launch");
        return ATTN_ERR_LAUNCH;
    }
    return ATTN_OK;
}

// A stride pair (elements) of a [rows, heads, D] or [heads, rows, D] tensor: multiples of 8
// elements, no overlap of neighbours, the larger a multiple of the smaller (what a tensor map
// describes).  The stride of an axis of one entry is not looked at.
bool strides_ok(long long row, long long head, long long rows, long long heads, int D) {
    if (rows > 1 && (row < D || row % 8 != 0)) return false;
    if (heads > 1 && (head < D || head % 8 != 0)) return false;
    if (rows > 1 && heads > 1) {
        const long long big = row > head ? row : head, small = row > head ? head : row;
        if (big % small != 0 || big < small * (row > head ? heads : rows)) return false;
    }
    return row < (1ll << 36) && head < (1ll << 36);
}

// Tensor map of packed rows, box 64 columns x box_rows rows x box_heads heads, the axes in
// ascending order of their strides; *head_y is 1 when the head axis comes first, as it does
// in any case for a box of several heads.
bool encode_packed_map(CUtensorMap *map, const void *base, bool bf16, int D, long long rows, long long heads,
                       long long row_stride, long long head_stride, int box_rows, int box_heads, int *head_y) {
    auto enc = tensor_map_encoder();
    if (enc == nullptr) return false;
    if (heads <= 1) head_stride = D;
    if (rows <= 1) row_stride = head_stride * heads;
    const bool hy = head_stride <= row_stride;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(hy ? heads : rows),
                                static_cast<cuuint64_t>(hy ? rows : heads)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(hy ? head_stride : row_stride) * 2,
                                   static_cast<cuuint64_t>(hy ? row_stride : head_stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(hy ? box_heads : box_rows),
                               static_cast<cuuint32_t>(hy ? box_rows : box_heads)};
    const cuuint32_t elem[3] = {1, 1, 1};
    *head_y = hy ? 1 : 0;
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
               const_cast<void *>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map of a pool [n_pages * Hkv, page, D], box 64 columns x min(page, 128) rows.
bool encode_pool_map(CUtensorMap *map, const void *base, bool bf16, int D, int page, long long slices) {
    auto enc = tensor_map_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(page), static_cast<cuuint64_t>(slices)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(page) * D * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(page < gqa::kBN ? page : gqa::kBN), 1};
    const cuuint32_t elem[3] = {1, 1, 1};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
               const_cast<void *>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

attn_status_t no_map() {
    std::snprintf(t_last_cuda_error, sizeof(t_last_cuda_error), "cuTensorMapEncodeTiled failed");
    return ATTN_ERR_LAUNCH;
}

// The fields of Params that the waits and the softmax of every kernel use.
void common_params(gqa::Params &prm, void *o, float *lse, int Hq, int Hkv, float scale) {
    prm.o = o;
    prm.lse = lse;
    prm.group = Hq / Hkv;
    prm.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    prm.seq = g_launch_seq.fetch_add(1);
    prm.timeout_ns = g_timeout_ns.load();
    prm.inject_stall = g_inject_stall.load();
}

template <int D, bool BF16, bool CAUSAL>
attn_status_t launch_varlen(int dev, int kid, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                            const gqa::VarlenParams &prm, unsigned grid, cudaStream_t s) {
    auto kern = gqa::attn_fwd_varlen_kernel<D, BF16, CAUSAL>;
    constexpr int smem = gqa::VlLayout<D>::kAlloc;
    if (attn_status_t st = set_smem_limit(dev, 24 + kid, kern, smem); st != ATTN_OK) return st;
    return launch_dependent(kern, grid, gqa::kWsThreads, smem, s, tq, tk, tv, prm);
}

template <int D, bool BF16>
attn_status_t launch_tree(int dev, int kid, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                          const gqa::TreeParams &prm, unsigned grid, cudaStream_t s) {
    auto kern = gqa::attn_fwd_tree_kernel<D, BF16>;
    constexpr int smem = gqa::TreeLayout<D>::kAlloc;
    if (attn_status_t st = set_smem_limit(dev, 32 + kid, kern, smem); st != ATTN_OK) return st;
    if (attn_status_t st = launch_dependent(kern, grid, gqa::kTreeThreads, smem, s, tq, tk, tv, prm);
        st != ATTN_OK)
        return st;
    if (prm.plan != nullptr)
        return launch_dependent(gqa::attn_tree_merge_kernel<D, BF16>, static_cast<unsigned>(prm.total_q) * prm.Hq, 32, 0,
                                s, prm);
    constexpr unsigned per_cta = gqa::kBM / gqa::kMergeCtaRows;
    return launch_dependent(gqa::attn_tree_merge_ctas_kernel<D, BF16>, grid * per_cta, gqa::kMergeCtaThreads, 0, s, prm);
}

// Least weight of a CTA's share in the tree kernel (a unit weighs its key tiles and two more).
constexpr int kTreeMinShare = 2;

int log2_of(int x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

attn_status_t check_cache(const attn_kv_cache_t *c) {
    if (c == nullptr) return ATTN_ERR_NULL;
    if (c->n_layers < 1 || c->n_pages < 1 || c->Hkv < 1 || c->n_rows < 1 || c->table_width < 1) return ATTN_ERR_SHAPE;
    if (c->page < 16 || c->page > 4096 || (c->page & (c->page - 1)) != 0) return ATTN_ERR_SHAPE;
    if (c->n_rows > (1 << 26)) return ATTN_ERR_SHAPE;  // lists of sequences: grids and 32-bit indexes
    if (c->D != 64 && c->D != 128) return ATTN_ERR_HEADDIM;
    if (c->dtype != ATTN_F16 && c->dtype != ATTN_BF16) return ATTN_ERR_DTYPE;
    // 32-bit tile coordinates, positions and row numbers
    if (static_cast<long long>(c->n_pages) * c->Hkv > INT_MAX / 2 ||
        static_cast<long long>(c->table_width) * c->page > INT_MAX / 2 ||
        static_cast<long long>(c->n_rows) * c->table_width > INT_MAX ||
        static_cast<long long>(c->n_layers) * 2 * c->Hkv * c->page * c->D > INT_MAX)
        return ATTN_ERR_SHAPE;
    if (!c->k || !c->v || !c->table || !c->lens || !c->refs || !c->scratch) return ATTN_ERR_NULL;
    if (misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(c->table, 4) || misaligned(c->lens, 4) ||
        misaligned(c->refs, 4) || misaligned(c->scratch, 4))
        return ATTN_ERR_ALIGN;
    return ATTN_OK;
}

gqa::KvPool pool_of(const attn_kv_cache_t *c) {
    gqa::KvPool p = {};
    p.k = static_cast<uint4 *>(c->k);
    p.v = static_cast<uint4 *>(c->v);
    p.table = c->table;
    p.lens = c->lens;
    p.refs = c->refs;
    p.n_layers = c->n_layers;
    p.n_pages = c->n_pages;
    p.page = c->page;
    p.page_shift = log2_of(c->page);
    p.Hkv = c->Hkv;
    p.row16 = c->D / 8;
    p.n_rows = c->n_rows;
    p.table_w = c->table_width;
    p.list = c->scratch;
    p.map = p.list + c->n_pages;
    p.claim = p.map + c->n_pages;
    p.need = p.claim + c->n_rows;
    p.pairs = p.need + c->n_rows;
    p.count = p.pairs + 3ll * c->n_rows;
    return p;
}

// Checks shared by the cache's calls on lists of n entries; *empty when there is nothing to do.
attn_status_t check_list(const attn_kv_cache_t *c, int n, bool &empty) {
    empty = n == 0;
    if (attn_status_t st = check_cache(c); st != ATTN_OK) return st;
    return n < 0 ? ATTN_ERR_SHAPE : ATTN_OK;
}

// Grid of kv_move_kernel: its warps' 4 KB segments, at most 32 blocks of 8 warps per SM; more
// blocks than are resident at once keep the memory busier than a loop in each of few (a 600 MB
// compaction, the ranges of three runs: 198 to 208 us with 8 blocks per SM, 191 to 201 with 16, 193
// to 195 with 32, 192 to 197 with 64).
unsigned move_grid(const gqa::KvPool &p, long long pages, int sms) {
    const long long segs = pages * p.n_layers * 2 * p.Hkv * ((p.page * p.row16 + 255) / 256);
    const long long blocks = (segs + 7) / 8, most = 32ll * sms;
    return static_cast<unsigned>(blocks < most ? (blocks > 0 ? blocks : 1) : most);
}

}  // namespace

extern "C" {

attn_status_t attn_fwd_varlen(const void *q, const void *k, const void *v, void *o, float *lse, const int *cu_q,
                              const int *cu_k, int n_seqs, int total_q, int total_k, int Hq, int Hkv, int D,
                              const long long *strides, float scale, int causal, attn_dtype_t dtype, void *stream) {
    if (n_seqs < 0 || total_q < 0 || total_k < 0 || Hq < 0 || Hkv < 1 || Hq % Hkv != 0) return ATTN_ERR_SHAPE;
    if (!(std::isfinite(scale) && scale > 0.f)) return ATTN_ERR_SHAPE;
    if (D != 64 && D != 128) return ATTN_ERR_HEADDIM;
    if (dtype != ATTN_F16 && dtype != ATTN_BF16) return ATTN_ERR_DTYPE;
    if (cu_k == nullptr && total_k != total_q) return ATTN_ERR_SHAPE;
    if (n_seqs == 0 || Hq == 0 || total_q == 0) return ATTN_OK;
    if (!q || !o || !cu_q || (total_k > 0 && (!k || !v))) return ATTN_ERR_NULL;
    if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) || misaligned(lse, 4) ||
        misaligned(cu_q, 4) || misaligned(cu_k, 4))
        return ATTN_ERR_ALIGN;
    // rows [total, heads, D] unless strides say otherwise
    const long long st[8] = {strides ? strides[0] : static_cast<long long>(Hq) * D,  strides ? strides[1] : D,
                             strides ? strides[2] : static_cast<long long>(Hkv) * D, strides ? strides[3] : D,
                             strides ? strides[4] : static_cast<long long>(Hkv) * D, strides ? strides[5] : D,
                             strides ? strides[6] : static_cast<long long>(Hq) * D,  strides ? strides[7] : D};
    if (!strides_ok(st[0], st[1], total_q, Hq, D) || !strides_ok(st[2], st[3], total_k, Hkv, D) ||
        !strides_ok(st[4], st[5], total_k, Hkv, D) || !strides_ok(st[6], st[7], total_q, Hq, D))
        return ATTN_ERR_SHAPE;
    gqa::VarlenParams prm = {};
    prm.pair = (Hq / Hkv) % 2 == 0 ? 1 : 0;
    prm.block_rows = prm.pair ? 128 : 256;
    prm.head_units = prm.pair ? Hq / 2 : Hq;
    // block counts of a sequence are kept in 16 bits, unit numbers in 32
    const long long units = (static_cast<long long>(total_q) / prm.block_rows + n_seqs) * prm.head_units;
    if (total_q > 65535ll * 128 || total_k > 65535ll * 128 || units > INT_MAX / 2) return ATTN_ERR_SHAPE;
    int dev = 0;
    if (attn_status_t e = check_device(&dev); e != ATTN_OK) return e;
    common_params(prm, o, lse, Hq, Hkv, scale);
    prm.v_ptr = static_cast<const uint8_t *>(v);
    prm.total_q = total_q;
    prm.total_k = total_k;
    prm.v_row = st[4] * 2;
    prm.v_head = st[5] * 2;
    prm.o_row = st[6] * 2;
    prm.o_head = st[7] * 2;
    const bool bf16 = dtype == ATTN_BF16;
    CUtensorMap tq, tk, tv;
    // without keys the K and V maps are never used: any valid one will do
    const bool keys = total_k > 0;
    if (!encode_packed_map(&tq, q, bf16, D, total_q, Hq, st[0], st[1], 128, 1, &prm.q_head_y) ||
        !encode_packed_map(&tk, keys ? k : q, bf16, D, keys ? total_k : 1, keys ? Hkv : 1, st[2], st[3], 128, 1,
                           &prm.k_head_y) ||
        !encode_packed_map(&tv, keys ? v : q, bf16, D, keys ? total_k : 1, keys ? Hkv : 1, st[4], st[5], 128, 1,
                           &prm.v_head_y))
        return no_map();
    const unsigned grid = static_cast<unsigned>(units < g_dev_sms[dev] ? units : g_dev_sms[dev]);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int kid = (D == 128 ? 4 : 0) + (bf16 ? 2 : 0) + (causal ? 1 : 0);
    auto launch = [&]() {
        switch (kid) {
            case 0: return launch_varlen<64, false, false>(dev, kid, tq, tk, tv, prm, grid, s);
            case 1: return launch_varlen<64, false, true>(dev, kid, tq, tk, tv, prm, grid, s);
            case 2: return launch_varlen<64, true, false>(dev, kid, tq, tk, tv, prm, grid, s);
            case 3: return launch_varlen<64, true, true>(dev, kid, tq, tk, tv, prm, grid, s);
            case 4: return launch_varlen<128, false, false>(dev, kid, tq, tk, tv, prm, grid, s);
            case 5: return launch_varlen<128, false, true>(dev, kid, tq, tk, tv, prm, grid, s);
            case 6: return launch_varlen<128, true, false>(dev, kid, tq, tk, tv, prm, grid, s);
            default: return launch_varlen<128, true, true>(dev, kid, tq, tk, tv, prm, grid, s);
        }
    };
    // at most kVlSeqs sequences per launch; a launch leaves the rows of the others alone
    for (int s0 = 0; s0 < n_seqs; s0 += gqa::kVlSeqs) {
        prm.cu_q = cu_q + s0;
        prm.cu_k = (cu_k ? cu_k : cu_q) + s0;
        prm.n_seqs = n_seqs - s0 < gqa::kVlSeqs ? n_seqs - s0 : gqa::kVlSeqs;
        prm.most_blocks = total_q / prm.block_rows + prm.n_seqs;
        if (attn_status_t e = launch(); e != ATTN_OK) return e;
    }
    return ATTN_OK;
}

attn_status_t attn_fwd_tree_workspace(int n_seqs, int D, size_t *bytes) {
    if (bytes == nullptr) return ATTN_ERR_NULL;
    *bytes = 0;
    if (n_seqs < 0) return ATTN_ERR_SHAPE;
    if (D != 64 && D != 128) return ATTN_ERR_HEADDIM;
    int dev = 0;
    if (attn_status_t st = check_device(&dev); st != ATTN_OK) return st;
    const size_t rows = static_cast<size_t>(g_dev_sms[dev]) * 2 * gqa::kBM;
    const int launch_seqs = n_seqs < gqa::kTreeSeqs ? n_seqs : gqa::kTreeSeqs;
    const size_t plan = (static_cast<size_t>(launch_seqs) + 1) * sizeof(int), starts = g_dev_sms[dev] * sizeof(int4);
    *bytes = rows * (D + 1) * sizeof(float) + (plan > starts ? plan : starts);
    return ATTN_OK;
}

attn_status_t attn_fwd_tree(const void *q, const attn_kv_cache_t *cache, int layer, void *o, float *lse, const int *cu,
                            const int *seqs, const int *parents, int n_seqs, int total_q, int Hq,
                            const long long *strides, float scale, void *workspace, size_t workspace_bytes,
                            void *stream) {
    if (attn_status_t st = check_cache(cache); st != ATTN_OK) return st;
    const int Hkv = cache->Hkv, D = cache->D;
    if (n_seqs < 0 || total_q < 0 || Hq < 0 || Hq % Hkv != 0 || Hq / Hkv > 128) return ATTN_ERR_SHAPE;
    if (layer < 0 || layer >= cache->n_layers) return ATTN_ERR_SHAPE;
    if (!(std::isfinite(scale) && scale > 0.f)) return ATTN_ERR_SHAPE;
    if (n_seqs == 0 || total_q == 0 || Hq == 0) return ATTN_OK;
    if (!q || !o || !cu || !workspace) return ATTN_ERR_NULL;
    if (misaligned(q, 16) || misaligned(o, 16) || misaligned(lse, 4) || misaligned(cu, 4) || misaligned(seqs, 4) ||
        misaligned(parents, 4) || misaligned(workspace, 16))
        return ATTN_ERR_ALIGN;
    if (seqs == nullptr && n_seqs > cache->n_rows) return ATTN_ERR_SHAPE;
    const long long st[4] = {strides ? strides[0] : static_cast<long long>(Hq) * D, strides ? strides[1] : D,
                             strides ? strides[2] : static_cast<long long>(Hq) * D, strides ? strides[3] : D};
    if (!strides_ok(st[0], st[1], total_q, Hq, D) || !strides_ok(st[2], st[3], total_q, Hq, D)) return ATTN_ERR_SHAPE;
    // a box of tokens x heads lies token by token in the tile: tokens are the outer axis of q
    if (total_q > 1 && Hq > 1 && st[0] < st[1]) return ATTN_ERR_SHAPE;
    gqa::TreeParams prm = {};
    prm.rt = 128 / (Hq / Hkv);
    // weight of the longest sequence with the largest tree in the kernel's list
    const long long key_tiles = (static_cast<long long>(cache->table_width) * cache->page + 127) / 128;
    const long long seq_weight = (gqa::kTreeMax + prm.rt - 1) / prm.rt * (key_tiles + 2) * Hkv;
    if (seq_weight > INT_MAX / 2 || static_cast<long long>(total_q) * Hq > INT_MAX) return ATTN_ERR_SHAPE;
    int dev = 0;
    if (attn_status_t e = check_device(&dev); e != ATTN_OK) return e;
    size_t need = 0;
    if (attn_status_t e = attn_fwd_tree_workspace(n_seqs, D, &need); e != ATTN_OK) return e;
    if (workspace_bytes < need) return ATTN_ERR_SCRATCH;
    common_params(prm, o, lse, Hq, Hkv, scale);
    const size_t layer_bytes = static_cast<size_t>(cache->n_pages) * Hkv * cache->page * D * 2;
    const uint8_t *kp = static_cast<const uint8_t *>(cache->k) + layer * layer_bytes;
    const uint8_t *vp = static_cast<const uint8_t *>(cache->v) + layer * layer_bytes;
    prm.table = cache->table;
    prm.lens = cache->lens;
    prm.parents = parents;
    prm.v_ptr = vp;
    prm.total_q = total_q;
    prm.Hq = Hq;
    prm.Hkv = Hkv;
    prm.n_rows = cache->n_rows;
    prm.page = cache->page;
    prm.page_shift = log2_of(cache->page);
    prm.n_pages = cache->n_pages;
    prm.table_w = cache->table_width;
    prm.min_share = kTreeMinShare;
    prm.o_row = st[2] * 2;
    prm.o_head = st[3] * 2;
    const int sms = g_dev_sms[dev];
    prm.part_o = static_cast<float *>(workspace);
    prm.part_lse = prm.part_o + static_cast<size_t>(sms) * 2 * gqa::kBM * D;
    void *plan = prm.part_lse + static_cast<size_t>(sms) * 2 * gqa::kBM;
    if (total_q * Hq <= gqa::kMergeRows)
        prm.plan = static_cast<int *>(plan);
    else
        prm.starts = static_cast<int4 *>(plan);
    const bool bf16 = cache->dtype == ATTN_BF16;
    CUtensorMap tq, tk, tv;
    int head_y = 0;
    const long long slices = static_cast<long long>(cache->n_pages) * Hkv;
    if (!encode_packed_map(&tq, q, bf16, D, total_q, Hq, st[0], st[1], prm.rt, prm.group, &head_y) || head_y != 1 ||
        !encode_pool_map(&tk, kp, bf16, D, cache->page, slices) || !encode_pool_map(&tv, vp, bf16, D, cache->page, slices))
        return no_map();
    const long long most = (static_cast<long long>(total_q) / prm.rt + n_seqs) * Hkv * (key_tiles + 2);
    const unsigned grid = static_cast<unsigned>(most < sms ? most : sms);
    prm.grid = static_cast<int>(grid);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int kid = (D == 128 ? 2 : 0) + (bf16 ? 1 : 0);
    auto launch = [&]() {
        switch (kid) {
            case 0: return launch_tree<64, false>(dev, kid, tq, tk, tv, prm, grid, s);
            case 1: return launch_tree<64, true>(dev, kid, tq, tk, tv, prm, grid, s);
            case 2: return launch_tree<128, false>(dev, kid, tq, tk, tv, prm, grid, s);
            default: return launch_tree<128, true>(dev, kid, tq, tk, tv, prm, grid, s);
        }
    };
    // at most kTreeSeqs sequences per launch, and no more than the list's 32-bit weights hold
    // whatever the device offsets are; a launch leaves the tokens of the others alone
    const int step = static_cast<int>(seq_weight * gqa::kTreeSeqs > INT_MAX / 2 ? INT_MAX / 2 / seq_weight : gqa::kTreeSeqs);
    for (int s0 = 0; s0 < n_seqs; s0 += step) {
        prm.cu = cu + s0;
        prm.seqs = seqs != nullptr ? seqs + s0 : nullptr;
        prm.seq0 = s0;
        prm.n_seqs = n_seqs - s0 < step ? n_seqs - s0 : step;
        if (attn_status_t e = launch(); e != ATTN_OK) return e;
    }
    return ATTN_OK;
}

attn_status_t attn_kv_scratch(int n_pages, int n_rows, size_t *bytes) {
    if (bytes == nullptr) return ATTN_ERR_NULL;
    *bytes = 0;
    if (n_pages < 1 || n_rows < 1) return ATTN_ERR_SHAPE;
    *bytes = (2ull * n_pages + 5ull * n_rows + 2) * sizeof(int);
    return ATTN_OK;
}

attn_status_t attn_kv_extend(const attn_kv_cache_t *cache, const int *seqs, const int *n_new, int n, void *stream) {
    int dev = 0;
    bool empty = false;
    if (attn_status_t st = check_list(cache, n, empty); st != ATTN_OK || empty) return st;
    if (!n_new) return ATTN_ERR_NULL;
    if (n > cache->n_rows) return ATTN_ERR_SHAPE;
    if (misaligned(seqs, 4) || misaligned(n_new, 4)) return ATTN_ERR_ALIGN;
    if (attn_status_t st = check_device(&dev); st != ATTN_OK) return st;
    return launch_dependent(gqa::kv_extend_kernel, 1, gqa::kPlanThreads, 0, static_cast<cudaStream_t>(stream),
                            pool_of(cache), seqs, n_new, n);
}

attn_status_t attn_kv_append(const attn_kv_cache_t *cache, int layer, const void *k_new, const void *v_new,
                             const long long *strides, const int *cu, const int *seqs, int n, int total, void *stream) {
    int dev = 0;
    bool empty = false;
    if (attn_status_t st = check_list(cache, n, empty); st != ATTN_OK || empty) return st;
    if (layer < 0 || layer >= cache->n_layers || total < 0) return ATTN_ERR_SHAPE;
    if (total == 0) return ATTN_OK;
    if (!k_new || !v_new || !cu) return ATTN_ERR_NULL;
    if (misaligned(k_new, 16) || misaligned(v_new, 16) || misaligned(cu, 4) || misaligned(seqs, 4)) return ATTN_ERR_ALIGN;
    const long long D = cache->D, row = cache->Hkv * D;
    const long long st[4] = {strides ? strides[0] : row, strides ? strides[1] : D, strides ? strides[2] : row,
                             strides ? strides[3] : D};
    for (int i = 0; i < 4; ++i) {
        if ((i % 2 == 0 ? total : cache->Hkv) == 1) continue;  // the stride of an axis of one entry
        if (st[i] < 0 || st[i] % 8 != 0 || st[i] >= (1ll << 36)) return ATTN_ERR_SHAPE;
    }
    if (attn_status_t e = check_device(&dev); e != ATTN_OK) return e;
    const gqa::KvAppend x = {static_cast<const uint4 *>(k_new), static_cast<const uint4 *>(v_new), st[0] / 8, st[1] / 8,
                             st[2] / 8, st[3] / 8, cu, seqs, n, total, layer};
    return launch_dependent(gqa::kv_append_kernel, static_cast<unsigned>((static_cast<long long>(total) + 7) / 8), 256, 0,
                            static_cast<cudaStream_t>(stream), pool_of(cache), x);
}

attn_status_t attn_kv_accept(const attn_kv_cache_t *cache, const int *cu, const int *seqs, const int *path, int path_width,
                             const int *taken, int n, void *stream) {
    int dev = 0;
    bool empty = false;
    if (attn_status_t st = check_list(cache, n, empty); st != ATTN_OK || empty) return st;
    if (!cu || !path || !taken) return ATTN_ERR_NULL;
    if (n > cache->n_rows || path_width < 1) return ATTN_ERR_SHAPE;
    if (misaligned(cu, 4) || misaligned(seqs, 4) || misaligned(path, 4) || misaligned(taken, 4)) return ATTN_ERR_ALIGN;
    if (attn_status_t st = check_device(&dev); st != ATTN_OK) return st;
    return launch_dependent(gqa::kv_accept_kernel, static_cast<unsigned>(n) * gqa::kAcceptCtas, 256, 0,
                            static_cast<cudaStream_t>(stream), pool_of(cache), cu, seqs, path, path_width, taken);
}

attn_status_t attn_kv_copy(const attn_kv_cache_t *cache, const int *src, const int *dst, int n, void *stream) {
    int dev = 0;
    bool empty = false;
    if (attn_status_t st = check_list(cache, n, empty); st != ATTN_OK || empty) return st;
    if (!src || !dst) return ATTN_ERR_NULL;
    if (misaligned(src, 4) || misaligned(dst, 4)) return ATTN_ERR_ALIGN;
    if (attn_status_t st = check_device(&dev); st != ATTN_OK) return st;
    const gqa::KvPool p = pool_of(cache);
    return launch_dependent(gqa::kv_move_kernel<gqa::kMoveCopy>, move_grid(p, n, g_dev_sms[dev]), 256, 0,
                            static_cast<cudaStream_t>(stream), p, src, dst, n);
}

attn_status_t attn_kv_fork(const attn_kv_cache_t *cache, const int *parents, const int *children, int n, void *stream) {
    int dev = 0;
    bool empty = false;
    if (attn_status_t st = check_list(cache, n, empty); st != ATTN_OK || empty) return st;
    if (!parents || !children) return ATTN_ERR_NULL;
    if (n > cache->n_rows) return ATTN_ERR_SHAPE;
    if (misaligned(parents, 4) || misaligned(children, 4)) return ATTN_ERR_ALIGN;
    if (attn_status_t st = check_device(&dev); st != ATTN_OK) return st;
    const gqa::KvPool p = pool_of(cache);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (attn_status_t st = launch_dependent(gqa::kv_fork_kernel, gqa::kForkCtas, gqa::kPlanThreads, 0, s, p, parents, children, n);
        st != ATTN_OK)
        return st;
    return launch_dependent(gqa::kv_move_kernel<gqa::kMoveFork>, move_grid(p, n, g_dev_sms[dev]), 256, 0, s, p, parents,
                            children, n);
}

attn_status_t attn_kv_free(const attn_kv_cache_t *cache, const int *seqs, int n, void *stream) {
    int dev = 0;
    bool empty = false;
    if (attn_status_t st = check_list(cache, n, empty); st != ATTN_OK || empty) return st;
    if (!seqs) return ATTN_ERR_NULL;
    if (misaligned(seqs, 4)) return ATTN_ERR_ALIGN;
    if (attn_status_t st = check_device(&dev); st != ATTN_OK) return st;
    const long long blocks = (static_cast<long long>(n) * cache->table_width + 255) / 256, most = 4ll * g_dev_sms[dev];
    return launch_dependent(gqa::kv_free_kernel, static_cast<unsigned>(blocks < most ? blocks : most), 256, 0,
                            static_cast<cudaStream_t>(stream), pool_of(cache), seqs, n);
}

attn_status_t attn_kv_compact(const attn_kv_cache_t *cache, int *live, void *stream) {
    int dev = 0;
    if (attn_status_t st = check_cache(cache); st != ATTN_OK) return st;
    if (misaligned(live, 4)) return ATTN_ERR_ALIGN;
    if (attn_status_t st = check_device(&dev); st != ATTN_OK) return st;
    const gqa::KvPool p = pool_of(cache);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (attn_status_t st = launch_dependent(gqa::kv_compact_kernel, 1, gqa::kPlanThreads, 0, s, p, live); st != ATTN_OK)
        return st;
    return launch_dependent(gqa::kv_move_kernel<gqa::kMoveCompact>, move_grid(p, (p.n_pages + 1) / 2, g_dev_sms[dev]), 256,
                            0, s, p, static_cast<const int *>(nullptr), static_cast<const int *>(nullptr), 0);
}

}  // extern "C"
