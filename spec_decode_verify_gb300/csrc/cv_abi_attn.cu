// C ABI of the attention layers' operators: attention over a paged cache, draft verification, query and key norms with
// rotation, and the cache's pages.  Every check runs on the host before anything is launched.
#include <cstdint>
#include <cstring>

#include "convverify.h"
#include "cv_attn.h"
#include "cv_host.h"

namespace {

using cvk::aligned16;
using cvk::device_limits;
using cvk::launch_pdl;

constexpr int kMaxHeads = 4096, kMaxLayers = 4096, kMaxPage = 65536, kMaxHeadDim = 256, kMaxVocab = 1 << 24;
constexpr int64_t kMaxTokens = 0x7fffffff - 255;  // the end of a tile that begins within them is an int too
constexpr int64_t kMaxStride = 1LL << 38;  // elements: a tensor map's strides are below 2^40 bytes
constexpr unsigned kPolls = 65536;         // of up to 20 us each

int esize_of(int dtype) { return dtype == CV_BF16 ? 2 : 4; }

int check_cache(const cv_cache &c, bool pointers, bool counts) {
    if (c.dtype != CV_F32 && c.dtype != CV_BF16) return CV_ERR_DTYPE;
    if (c.n_layers < 1 || c.n_layers > kMaxLayers || c.n_pages < 1 || c.page_size < 1 || c.page_size > kMaxPage ||
        c.n_kv_heads < 1 || c.n_kv_heads > kMaxHeads || c.n_slots < 1 || c.max_pages < 1 ||
        (int64_t)c.max_pages * c.page_size > kMaxTokens)
        return CV_ERR_SHAPE;
    if (c.head_dim < 1 || c.head_dim > kMaxHeadDim) return CV_ERR_HEAD_DIM;
    const int64_t strides[] = {c.k_layer_stride, c.k_page_stride, c.k_row_stride, c.k_head_stride,
                               c.v_layer_stride, c.v_page_stride, c.v_row_stride, c.v_head_stride};
    for (int64_t s : strides)
        if (s < 0) return CV_ERR_STRIDE;
    if (c.table_stride < c.max_pages && c.n_slots > 1) return CV_ERR_STRIDE;
    if (pointers && (!c.page_table || !c.k || !c.v)) return CV_ERR_NULL_POINTER;
    if (pointers && counts && (!c.held || !c.refs)) return CV_ERR_NULL_POINTER;
    return CV_OK;
}

cvk::CacheView view(const cv_cache &c) {
    return {c.k, c.v, c.k_layer_stride, c.k_page_stride, c.k_row_stride, c.k_head_stride, c.v_layer_stride,
            c.v_page_stride, c.v_row_stride, c.v_head_stride, c.n_layers, c.n_pages, c.page_size, c.n_kv_heads,
            c.head_dim, c.n_slots, c.max_pages, c.page_table, c.table_stride, c.held, c.refs};
}

// Whether a cache tensor's rows are whole 16-byte pieces at 16-byte addresses.
bool rows16(const void *p, int64_t layer, int64_t page, int64_t row, int64_t head, const cv_cache &c) {
    const int es = esize_of(c.dtype);
    return aligned16(p) && c.head_dim * es % 16 == 0 && (c.n_layers == 1 || layer * es % 16 == 0) && page * es % 16 == 0 &&
           (c.page_size == 1 || row * es % 16 == 0) && (c.n_kv_heads == 1 || head * es % 16 == 0);
}

// Clears err where kernels OR their bits into it.
int clear_err(int32_t *err, int n_seq, cudaStream_t stream) {
    return err && cudaMemsetAsync(err, 0, sizeof(int32_t) * (size_t)n_seq, stream) != cudaSuccess ? CV_ERR_LAUNCH : CV_OK;
}

// ---- attention

int check_attention(const cv_tree_attention_args *a, bool pointers) {
    if (!a) return CV_ERR_NULL_ARGS;
    const int rc = check_cache(a->cache, false, false);
    if (rc != CV_OK) return rc;
    if (a->n_seq < 0 || a->n_seq > 65535 || a->n_heads < 1 || a->n_heads > kMaxHeads) return CV_ERR_SHAPE;
    if (a->T < 1 || a->T > CV_MAX_T) return CV_ERR_TOKENS;
    if (a->n_heads % a->cache.n_kv_heads != 0) return CV_ERR_HEAD_DIM;
    if (a->cu_draft && a->total_tokens < 0) return CV_ERR_SHAPE;
    const int64_t strides[] = {a->q_seq_stride, a->q_tok_stride, a->q_head_stride, a->out_seq_stride, a->out_tok_stride,
                               a->out_head_stride};
    for (int64_t s : strides)
        if (s < 0) return CV_ERR_STRIDE;
    if (!pointers || a->n_seq == 0) return CV_OK;
    if (a->cu_draft && a->total_tokens == 0) return a->err && !a->cache_len ? CV_ERR_NULL_POINTER : CV_OK;
    if (!a->q || !a->out || !a->cache_len || !a->cache.k || !a->cache.v || !a->cache.page_table) return CV_ERR_NULL_POINTER;
    if (a->out == a->q || a->out == a->cache.k || a->out == a->cache.v) return CV_ERR_ALIAS;
    return CV_OK;
}

// What a unit takes beside its tiles, in tiles, when the blocks' runs are made equal; device us with 0, 1, 2 and 3 of them, sequences of n/2 to n
// cached tokens.  Tensor cores: 128 x 8 drafts of 32/4 heads of 128, n = 8k, 282, 280, 279, 278; 100 x 4 of 16/8 heads of 64, 1k, 91, 87, 86, 86; 300
// x 1 of 16/8 heads, 300, 170, 167, 161, 165.  fp32 products: 100 x 1 of 32/8 heads, 1k, 123, 119, 120, 122; 13 x 1 of 64/8, 3k, 89, 90, 90, 94; 16 x
// 8 of 32/4, 2k, 191, 191, 202, 202; 23 x 1 of 4/2 heads of 64, 2.3k, 19.1, 18.3, 18.3, 18.3.
constexpr int kTcUnitCost = 3, kSimtUnitCost = 1;

struct AttnPlan {
    cvk::AttnSimt simt;
    cvk::AttnTc tc;
    bool on_tc, pair;
    int dp, rows, keys, parts, unit_cost, page_rows, tok;
    bool cut;
    int64_t bytes;
};

// What the tensor-core kernel's copies need: 16-byte rows, pages of whole groups of 8 rows that fit into tiles or are made of
// them, a positive scale (its masks are minus infinity before the scale).
bool tc_takes(const cv_tree_attention_args *a, int keys) {
    const cv_cache &c = a->cache;
    const int G = a->n_heads / c.n_kv_heads;
    auto dim = [](int64_t stride, int64_t n) { return n == 1 || (stride > 0 && stride % 8 == 0 && stride < kMaxStride); };
    return c.dtype == CV_BF16 && c.head_dim % 8 == 0 && G <= 128 && a->scale > 0.f && a->scale < 1e30f && c.page_size % 8 == 0 &&
           (c.page_size % keys == 0 || keys % c.page_size == 0) && aligned16(c.k) && aligned16(c.v) && aligned16(a->q) &&
           dim(c.k_page_stride, c.n_pages) && dim(c.k_row_stride, c.page_size) && dim(c.k_head_stride, c.n_kv_heads) &&
           dim(c.v_page_stride, c.n_pages) && dim(c.v_row_stride, c.page_size) && dim(c.v_head_stride, c.n_kv_heads) &&
           dim(a->q_head_stride, a->n_heads) && dim(a->q_tok_stride, a->cu_draft ? a->total_tokens : a->T) &&
           (a->cu_draft || dim(a->q_seq_stride, a->n_seq));
}

// Kernels from the most particular one down that a plan may use.
enum { kAnyAlignment, kWholePieces, kTensorCores };
AttnPlan plan_attention(const cv_tree_attention_args *a, int best = kTensorCores) {
    const cv_cache &c = a->cache;
    const int es = esize_of(c.dtype), G = a->n_heads / c.n_kv_heads, d = c.head_dim;
    AttnPlan pl;
    const cvk::DeviceLimits lim = device_limits();
    pl.dp = d <= 64 ? 64 : d <= 128 ? 128 : d <= 192 ? 192 : 256;
    pl.tok = G <= 128 ? (a->T < 128 / G ? a->T : 128 / G) : 1;
    // More rows than one tile of 128: two row tiles a unit, so that a tile of keys is read once for both.  Device us with one and with a unit
    // each: 17 drafts of 64/8 heads over 100k 107 and 139, 64 x 17 over 2k-4k 235 and 297, 32 x 128 of 32/8 heads over 2k-4k 272 and 333, 4 x 128 over
    // 4k-8k 97 and 97; heads of 64: 88 and 106, 185 and 236, 219 and 259.  Where a block has few tiles a unit each is faster (17 drafts over 20k
    // 45 and 37, 9 of 16/1 heads over 700 18.3 and 14.6), but how many there are stands in the lengths, on the device.  Tensor memory
    // has room for two up to 128 channels.
    pl.pair = pl.dp <= 128 && a->T > pl.tok;
    pl.tc = cvk::attn_tc_kernel(pl.dp, pl.pair);
    pl.on_tc = best >= kTensorCores && tc_takes(a, pl.tc.keys);
    if (pl.on_tc) {
        pl.keys = pl.tc.keys;
        pl.rows = pl.tok * G * (pl.pair ? 2 : 1);
        pl.page_rows = c.page_size < pl.keys ? c.page_size : pl.keys;
        pl.parts = lim.sms, pl.unit_cost = kTcUnitCost;
    } else {
        const bool vec = rows16(c.k, 0, c.k_page_stride, c.k_row_stride, c.k_head_stride, c) &&
                         rows16(c.v, 0, c.v_page_stride, c.v_row_stride, c.v_head_stride, c) && aligned16(a->q) &&
                         a->q_seq_stride * es % 16 == 0 && a->q_tok_stride * es % 16 == 0 && a->q_head_stride * es % 16 == 0;
        if (pl.dp == 192) pl.dp = 256;
        // Up to 8 rows share too little for a tile in shared memory.  Device us there and in registers, n/2 to n cached tokens: fp32, 13 tokens
        // of 64/8 heads of 128, n = 3k, 182 and 90, 16 of 8/8 heads of 256, 4k, 520 and 160, 23 of 4/2 heads of 64, 2.3k, 29 and 18, 32 x 2 of 32/8 heads
        // of 64, 2k, 151 and 75; bf16 in pages of 20: 177 and 85, 501 and 141, 29 and 18, and 32 x 4 of 16/8 heads, 4k, 482 and 221.  Of those in
        // registers, units of 4 rows and of 8: 16 tokens of 8/8 heads of 256, 4k, 160 and 254, 64 of 32/8 heads, 4k, 274 and 415, 64 of 16/8 heads of
        // 64, 147 and 220; with 8, 6 and 5 rows a kv head, in two units of 4: 108 and 90, 108 and 89, 84 and 75.
        const int64_t rows = (int64_t)a->T * G;
        const bool few = best >= kWholePieces && vec && rows <= cvk::kFewRows;
        pl.rows = !few ? cvk::kSimtRows : rows <= 4 ? 4 : 8;
        pl.simt = few ? cvk::attn_few_kernel(c.dtype == CV_BF16, pl.dp, pl.rows) : cvk::attn_simt_kernel(c.dtype == CV_BF16, pl.dp, vec);
        pl.keys = pl.simt.keys;
        const int resident = few && pl.dp > 128 ? 1 : lim.smem_per_sm / (pl.simt.smem_bytes + 1024);
        pl.parts = lim.sms * (resident < 1 ? 1 : resident > 2 ? 2 : resident);
        pl.unit_cost = kSimtUnitCost;
    }
    // tiles there can be at most: fewer blocks are enough for fewer
    const int64_t tiles = ((int64_t)c.max_pages * c.page_size + pl.keys - 1) / pl.keys;
    const int64_t units = (int64_t)a->n_seq * c.n_kv_heads * (((int64_t)a->T * G + pl.rows - 1) / pl.rows);
    if (units * tiles < pl.parts) pl.parts = (int)(units * tiles);
    pl.cut = tiles > 1;
    pl.bytes = pl.cut ? 2LL * pl.parts * cvk::part_floats((pl.rows + 3) / 4 * 4, pl.dp) * 4 : 0;
    return pl;
}

// A map of rows of d channels in boxes of 64 channels by `b1` x `b2` rows of the next two dimensions.
bool encode4(CUtensorMap *map, const void *p, int d, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t n3, int64_t s3, int b1,
             int b2) {
    const auto encode = cvk::encode_tiled();
    if (!encode) return false;
    const cuuint64_t any = (cuuint64_t)(d + 7) / 8 * 16;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)n1, (cuuint64_t)n2, (cuuint64_t)n3};
    const cuuint64_t strides[3] = {n1 > 1 ? (cuuint64_t)s1 * 2 : any, n2 > 1 ? (cuuint64_t)s2 * 2 : any, n3 > 1 ? (cuuint64_t)s3 * 2 : any};
    const cuuint32_t box[4] = {64, (cuuint32_t)b1, (cuuint32_t)b2, 1}, step[4] = {1, 1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Of the call, without its kernel's plan and tensor maps.
cvk::AttnParams attention_params(const cv_tree_attention_args *a) {
    const cv_cache &c = a->cache;
    cvk::AttnParams p;
    std::memset(&p, 0, sizeof p);
    p.n_seq = a->n_seq, p.T = a->T, p.total = a->total_tokens, p.n_heads = a->n_heads, p.G = a->n_heads / c.n_kv_heads;
    p.scale = a->scale * 1.4426950408889634f;
    p.polls = a->wait_polls == 0 ? kPolls : a->wait_polls < 0 ? 0u : (unsigned)a->wait_polls;
    p.c = view(c);
    p.q = a->q, p.q_seq = a->q_seq_stride, p.q_tok = a->q_tok_stride, p.q_head = a->q_head_stride;
    p.out = a->out, p.o_seq = a->out_seq_stride, p.o_tok = a->out_tok_stride, p.o_head = a->out_head_stride;
    p.cu = a->cu_draft, p.parent = a->parent, p.len = a->cache_len, p.idx = a->cache_idx, p.err = a->err;
    return p;
}

int launch_attention(const cv_tree_attention_args *a, cudaStream_t stream) {
    const cv_cache &c = a->cache;
    const AttnPlan pl = plan_attention(a);
    if (pl.bytes > 0 && (!a->workspace || reinterpret_cast<uintptr_t>(a->workspace) % 256 != 0 || a->workspace_bytes < pl.bytes))
        return CV_ERR_WORKSPACE;
    cvk::AttnMaps mp;
    std::memset(&mp, 0, sizeof mp);
    cvk::AttnParams &p = mp.a;
    p = attention_params(a);
    p.rows = pl.rows, p.pad = (pl.rows + 3) / 4 * 4, p.keys = pl.keys, p.dp = pl.dp, p.parts = pl.parts, p.unit_cost = pl.unit_cost;
    p.ws = pl.cut ? reinterpret_cast<float *>(a->workspace) : nullptr;
    if (pl.on_tc) {
        const int64_t tokens = a->cu_draft ? a->total_tokens : a->T, seqs = a->cu_draft ? 1 : a->n_seq;
        if (!encode4(&mp.q, a->q, c.head_dim, a->n_heads, a->q_head_stride, tokens, a->q_tok_stride, seqs, a->q_seq_stride, p.G, pl.tok) ||
            !encode4(&mp.k, c.k, c.head_dim, c.page_size, c.k_row_stride, c.n_kv_heads, c.k_head_stride, c.n_pages, c.k_page_stride,
                     pl.page_rows, 1) ||
            !encode4(&mp.v, c.v, c.head_dim, c.page_size, c.v_row_stride, c.n_kv_heads, c.v_head_stride, c.n_pages, c.v_page_stride,
                     pl.page_rows, 1))
            return CV_ERR_LAUNCH;
        mp.page_rows = pl.page_rows, mp.tok = pl.tok;
        mp.o_vec = aligned16(a->out) && a->out_seq_stride % 8 == 0 && a->out_tok_stride % 8 == 0 && a->out_head_stride % 8 == 0;
    }
    const int rc = clear_err(a->err, a->n_seq, stream);
    if (rc != CV_OK) return rc;
    if (pl.on_tc) {
        if (cvk::ensure_smem(reinterpret_cast<const void *>(pl.tc.fn), pl.tc.smem_bytes) != cudaSuccess) return CV_ERR_LAUNCH;
        if (launch_pdl(pl.tc.fn, dim3((unsigned)pl.parts), dim3((unsigned)pl.tc.threads), pl.tc.smem_bytes, stream, mp) != cudaSuccess)
            return CV_ERR_LAUNCH;
    } else {
        if (cvk::ensure_smem(reinterpret_cast<const void *>(pl.simt.fn), pl.simt.smem_bytes) != cudaSuccess) return CV_ERR_LAUNCH;
        if (launch_pdl(pl.simt.fn, dim3((unsigned)pl.parts), dim3(cvk::kSimtThreads), pl.simt.smem_bytes, stream, p) != cudaSuccess)
            return CV_ERR_LAUNCH;
    }
    if (pl.cut) {
        const dim3 grid((unsigned)pl.parts, (unsigned)cvk::kAttnJoinY, 2);
        if (launch_pdl(cvk::attn_join_kernel(c.dtype == CV_BF16, pl.dp), grid, dim3(cvk::kAttnJoinThreads), 0, stream, p) != cudaSuccess)
            return CV_ERR_LAUNCH;
    }
    return cudaGetLastError() == cudaSuccess ? CV_OK : CV_ERR_LAUNCH;
}

// Packed rows of which there are none: a block that looks at every sequence and finds no work.
int launch_no_attention(const cv_tree_attention_args *a, cudaStream_t stream) {
    if (!a->err) return CV_OK;
    cvk::AttnParams p = attention_params(a);
    const cvk::AttnSimt k = cvk::attn_simt_kernel(a->cache.dtype == CV_BF16, 64, false);
    p.rows = p.pad = cvk::kSimtRows, p.keys = k.keys, p.dp = 64, p.parts = 1;
    const int rc = clear_err(a->err, a->n_seq, stream);
    if (rc != CV_OK) return rc;
    if (cvk::ensure_smem(reinterpret_cast<const void *>(k.fn), k.smem_bytes) != cudaSuccess) return CV_ERR_LAUNCH;
    if (launch_pdl(k.fn, dim3(1), dim3(cvk::kSimtThreads), k.smem_bytes, stream, p) != cudaSuccess) return CV_ERR_LAUNCH;
    return cudaGetLastError() == cudaSuccess ? CV_OK : CV_ERR_LAUNCH;
}

// ---- draft verification

int check_sample(const cv_draft_verify_args *a) {
    if (!a) return CV_ERR_NULL_ARGS;
    if (a->dtype != CV_F32 && a->dtype != CV_BF16) return CV_ERR_DTYPE;
    if (a->n_seq < 0 || a->n_seq > 65535 || a->vocab < 1 || a->vocab > kMaxVocab || (a->cu_draft && a->total_tokens < 0))
        return CV_ERR_SHAPE;
    if (a->T < 1 || a->T > CV_MAX_T) return CV_ERR_TOKENS;
    if (a->draft_probs && a->parent) return CV_ERR_LAYOUT;
    if (a->probs_seq_stride < 0 || a->probs_tok_stride < 0 || a->draft_seq_stride < 0 || a->draft_tok_stride < 0)
        return CV_ERR_STRIDE;
    if (a->n_seq == 0) return CV_OK;
    const bool rows = !a->cu_draft || a->total_tokens > 0;
    if ((rows && (!a->probs || !a->tokens)) || !a->uniforms || !a->accept_len || !a->out_tokens) return CV_ERR_NULL_POINTER;
    const void *outs[] = {a->accept_len, a->accept_node, a->path, a->out_tokens, a->err};
    const void *ins[] = {a->probs, a->draft_probs, a->tokens, a->parent, a->uniforms, a->cu_draft, a->cache_idx};
    for (int i = 0; i < 5; ++i) {
        if (!outs[i]) continue;
        for (const void *in : ins)
            if (outs[i] == in) return CV_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (outs[i] == outs[j]) return CV_ERR_ALIAS;
    }
    return CV_OK;
}

// ---- query and key norms

int check_rope(const cv_qk_norm_rope_args *a) {
    if (!a) return CV_ERR_NULL_ARGS;
    if (a->dtype != CV_F32 && a->dtype != CV_BF16) return CV_ERR_DTYPE;
    if (a->n_seq < 0 || a->n_seq > 65535 || a->n_heads < 0 || a->n_heads > kMaxHeads || a->n_kv_heads < 0 ||
        a->n_kv_heads > kMaxHeads || (a->cu && a->total_tokens < 0))
        return CV_ERR_SHAPE;
    if (a->T < 0) return CV_ERR_TOKENS;
    if (a->head_dim < 1 || a->head_dim > kMaxHeadDim || a->rot_dim < 0 || a->rot_dim > a->head_dim || a->rot_dim % 2 != 0)
        return CV_ERR_HEAD_DIM;
    const bool paged = a->cache.page_table != nullptr;
    if (paged) {
        const int rc = check_cache(a->cache, true, false);
        if (rc != CV_OK) return rc;
        if (a->cache.dtype != a->dtype) return CV_ERR_DTYPE;
        if (a->cache.n_kv_heads != a->n_kv_heads || a->cache.head_dim != a->head_dim) return CV_ERR_HEAD_DIM;
        if (!a->cache_len) return CV_ERR_NULL_POINTER;
    }
    const int64_t strides[] = {a->q_seq_stride, a->q_tok_stride, a->q_head_stride, a->q_out_seq_stride, a->q_out_tok_stride,
                               a->q_out_head_stride, a->k_seq_stride, a->k_tok_stride, a->k_head_stride, a->k_out_seq_stride,
                               a->k_out_tok_stride, a->k_out_head_stride, a->v_seq_stride, a->v_tok_stride, a->v_head_stride,
                               a->cos_sin_stride};
    for (int64_t s : strides)
        if (s < 0) return CV_ERR_STRIDE;
    if (a->rot_dim > 0 && (a->n_positions < 1 || (a->n_positions > 1 && a->cos_sin_stride < a->rot_dim))) return CV_ERR_STRIDE;
    if (a->n_seq == 0 || a->T == 0 || (a->cu && a->total_tokens == 0)) return CV_OK;
    if ((a->n_heads > 0 && (!a->q || !a->q_out)) || (a->n_kv_heads > 0 && (!a->k || (!a->k_out && !paged))) ||
        (a->rot_dim > 0 && (!a->cos_sin || (!a->positions && !a->cache_len))) || (a->v && !paged))
        return CV_ERR_NULL_POINTER;
    // an output over its own input has to have its strides
    auto over = [](const void *out, const void *in, int64_t so, int64_t si, int64_t to, int64_t ti, int64_t ho, int64_t hi) {
        return out && out == in && (so != si || to != ti || ho != hi);
    };
    if (over(a->q_out, a->q, a->cu ? 0 : a->q_out_seq_stride, a->cu ? 0 : a->q_seq_stride, a->q_out_tok_stride, a->q_tok_stride,
             a->q_out_head_stride, a->q_head_stride) ||
        over(a->k_out, a->k, a->cu ? 0 : a->k_out_seq_stride, a->cu ? 0 : a->k_seq_stride, a->k_out_tok_stride, a->k_tok_stride,
             a->k_out_head_stride, a->k_head_stride))
        return CV_ERR_ALIAS;
    const void *outs[] = {a->n_heads > 0 ? a->q_out : nullptr, a->k_out, paged ? a->cache.k : nullptr, paged ? a->cache.v : nullptr};
    const void *ins[] = {a->q, a->k, a->v, a->q_weight, a->k_weight, a->cos_sin};
    for (int i = 0; i < 4; ++i) {
        if (!outs[i]) continue;
        for (int j = 0; j < 6; ++j)
            if (outs[i] == ins[j] && !(i == j && i < 2)) return CV_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (outs[i] == outs[j]) return CV_ERR_ALIAS;
    }
    return CV_OK;
}

int launch_rope(const cv_qk_norm_rope_args *a, cudaStream_t stream) {
    const bool paged = a->cache.page_table != nullptr;
    const int es = esize_of(a->dtype);
    cvk::RopeParams p;
    std::memset(&p, 0, sizeof p);
    p.n_seq = a->n_seq, p.T = a->T, p.n_heads = a->n_heads, p.n_kv = a->n_kv_heads, p.d = a->head_dim, p.total = a->total_tokens;
    p.rot = a->rot_dim, p.pairs = a->pairs != 0, p.norm = a->norm != 0, p.n_pos = a->n_positions, p.eps = a->eps;
    p.tokens = a->T == 0 ? 0 : a->cu ? (long long)a->total_tokens : (long long)a->n_seq * a->T;
    // without a row to work on the sequences' flags are all there is to do
    const bool flags_only = p.tokens == 0 || a->n_heads + a->n_kv_heads == 0;
    if (flags_only && !a->err) return CV_OK;
    p.q = a->q, p.k = a->k, p.v = a->n_kv_heads > 0 ? a->v : nullptr, p.wq = a->q_weight, p.wk = a->k_weight;
    p.q_out = a->q_out, p.k_out = a->k_out;
    p.q_seq = a->q_seq_stride, p.q_tok = a->q_tok_stride, p.q_head = a->q_head_stride;
    p.qo_seq = a->q_out_seq_stride, p.qo_tok = a->q_out_tok_stride, p.qo_head = a->q_out_head_stride;
    p.k_seq = a->k_seq_stride, p.k_tok = a->k_tok_stride, p.k_head = a->k_head_stride;
    p.ko_seq = a->k_out_seq_stride, p.ko_tok = a->k_out_tok_stride, p.ko_head = a->k_out_head_stride;
    p.v_seq = a->v_seq_stride, p.v_tok = a->v_tok_stride, p.v_head = a->v_head_stride;
    p.cs = a->cos_sin, p.cs_row = a->cos_sin_stride;
    p.pos = a->positions, p.cu = a->cu, p.len = a->cache_len, p.idx = a->cache_idx, p.err = a->err;
    p.paged = paged;
    if (paged) p.c = view(a->cache);
    // pieces of 8 channels at 16-byte addresses, in pairs of pieces
    auto rows = [&](const void *x, int64_t seq, int64_t tok, int64_t head) {
        return !x || (aligned16(x) && seq * es % 16 == 0 && tok * es % 16 == 0 && head * es % 16 == 0);
    };
    const bool vec = !flags_only && a->head_dim % 16 == 0 && a->rot_dim % 16 == 0 && rows(p.q, p.q_seq, p.q_tok, p.q_head) &&
                     rows(p.q_out, p.qo_seq, p.qo_tok, p.qo_head) && rows(p.k, p.k_seq, p.k_tok, p.k_head) &&
                     rows(p.k_out, p.ko_seq, p.ko_tok, p.ko_head) && rows(p.v, p.v_seq, p.v_tok, p.v_head) &&
                     aligned16(p.wq) && aligned16(p.wk) && aligned16(p.cs) && p.cs_row % 4 == 0 &&
                     (!paged || (rows(p.c.k, p.c.k_page, p.c.k_row, p.c.k_head) && rows(p.c.v, p.c.v_page, p.c.v_row, p.c.v_head)));
    const long long sms = device_limits().sms;
    long long blocks;
    if (vec) {
        p.lanes = 1;
        while (p.lanes * 16 < a->head_dim) p.lanes *= 2;
        // Groups that share a token's heads: as many as are resident at once (2 blocks an SM), at most one a head (1024
        // tokens of 20 heads: 12.3 us with 4, 14 with 1, 20 with 16); one where the tokens alone are as many (30,822 tokens: 143 us,
        // with 4 groups a token 168).
        const long long per = cvk::kRopeThreads / p.lanes, heads = p.n_heads + p.n_kv + (p.v ? p.n_kv : 0);
        const long long fit = 2 * sms * per / p.tokens, most = fit > 1 ? fit : 1;
        p.groups = (int)(most < heads ? most : heads);
        blocks = (p.tokens * p.groups + per - 1) / per;
    } else {
        // enough tokens a block for all its threads, fewer while that leaves SMs without one
        p.block_tokens = cvk::kRopeTokens;
        while (p.block_tokens > 1 && (p.tokens + p.block_tokens - 1) / p.block_tokens < 4 * sms) p.block_tokens /= 2;
        blocks = p.tokens == 0 ? 1 : (p.tokens + p.block_tokens - 1) / p.block_tokens;
    }
    if (blocks > 0x7fffffff) return CV_ERR_SHAPE;
    const int rc = clear_err(a->err, a->n_seq, stream);
    if (rc != CV_OK) return rc;
    const auto k = cvk::rope_kernel(a->dtype == CV_BF16, vec);
    const int smem = vec ? cvk::rope_smem(a->dtype == CV_BF16) : 0;
    if (cvk::ensure_smem(reinterpret_cast<const void *>(k), smem) != cudaSuccess) return CV_ERR_LAUNCH;
    if (launch_pdl(k, dim3((unsigned)blocks), dim3(cvk::kRopeThreads), smem, stream, p) != cudaSuccess) return CV_ERR_LAUNCH;
    return cudaGetLastError() == cudaSuccess ? CV_OK : CV_ERR_LAUNCH;
}

// ---- pages

// Bytes an access of a copy between rows can have.
int copy_bytes(const cv_cache &c) {
    return rows16(c.k, c.k_layer_stride, c.k_page_stride, c.k_row_stride, c.k_head_stride, c) &&
                   rows16(c.v, c.v_layer_stride, c.v_page_stride, c.v_row_stride, c.v_head_stride, c)
               ? 16
               : esize_of(c.dtype);
}

// Pieces of one position's rows in all layers' K and V.
int64_t copy_pieces(const cv_cache &c) {
    return 2LL * c.n_layers * c.n_kv_heads * (c.head_dim * esize_of(c.dtype) / copy_bytes(c));
}

int check_compact(const cv_cache_compact_args *a) {
    if (!a) return CV_ERR_NULL_ARGS;
    if (a->n_seq < 0 || a->n_seq > 65535) return CV_ERR_SHAPE;
    if (a->T < 1 || a->T > CV_MAX_T) return CV_ERR_TOKENS;
    const int rc = check_cache(a->cache, a->n_seq > 0, false);
    if (rc != CV_OK || a->n_seq == 0) return rc;
    if (copy_pieces(a->cache) > 0x7fffffff) return CV_ERR_SHAPE;
    if (!a->cache_len || !a->path || !a->accept_len) return CV_ERR_NULL_POINTER;
    if (a->cache.k == a->cache.v) return CV_ERR_ALIAS;
    const void *outs[] = {a->new_len, a->err};
    const void *ins[] = {a->cache_len, a->path, a->accept_len, a->cache_idx, a->cache.page_table};
    for (const void *o : outs)
        for (const void *in : ins)
            if (o && o == in) return CV_ERR_ALIAS;
    return a->err && a->err == a->new_len ? CV_ERR_ALIAS : CV_OK;
}

int check_pages(const cv_cache_pages_args *a, bool fork, bool needs_tokens, bool copies) {
    if (!a) return CV_ERR_NULL_ARGS;
    if (a->n_seq < 0 || a->n_seq > cvk::kMaxPageSeqs) return CV_ERR_SHAPE;
    const int rc = check_cache(a->cache, a->n_seq > 0, true);
    if (rc != CV_OK || a->n_seq == 0) return rc;
    if (copies && copy_pieces(a->cache) > 0x7fffffff) return CV_ERR_SHAPE;
    if ((needs_tokens && !a->n_tokens) || (fork && !a->src_idx)) return CV_ERR_NULL_POINTER;
    if (copies && a->cache.k == a->cache.v) return CV_ERR_ALIAS;
    const void *outs[] = {a->err, a->cache.page_table, a->cache.held, a->cache.refs};
    const void *ins[] = {a->idx, a->src_idx, a->n_tokens, a->cache_len};
    for (int i = 0; i < 4; ++i) {
        if (!outs[i]) continue;
        for (const void *in : ins)
            if (outs[i] == in) return CV_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (outs[i] == outs[j]) return CV_ERR_ALIAS;
    }
    return CV_OK;
}

cvk::PagesParams pages_params(const cv_cache_pages_args *a) {
    cvk::PagesParams p;
    std::memset(&p, 0, sizeof p);
    p.n_seq = a->n_seq, p.c = view(a->cache);
    p.idx = a->idx, p.src = a->src_idx, p.n_tok = a->n_tokens, p.err = a->err;
    return p;
}

int launch_take(const cvk::PagesParams &p, int op, cudaStream_t stream) {
    const int smem = cvk::pages_take_smem(p.n_seq);
    const auto k = cvk::pages_take_kernel(op);
    if (cvk::ensure_smem(reinterpret_cast<const void *>(k), smem) != cudaSuccess) return CV_ERR_LAUNCH;
    return launch_pdl(k, dim3(1), dim3(cvk::kTakeThreads), smem, stream, p) == cudaSuccess ? CV_OK : CV_ERR_LAUNCH;
}

int done() { return cudaGetLastError() == cudaSuccess ? CV_OK : CV_ERR_LAUNCH; }

// A kernel that copies rows, a cluster a sequence.
int launch_copies(cvk::PagesParams p, const cv_cache_pages_args *a, cvk::PagesKernel (*kernel)(int bytes), cudaStream_t stream) {
    const int bytes = copy_bytes(a->cache);
    p.esize = esize_of(a->cache.dtype), p.chunks = a->cache.head_dim * p.esize / bytes;
    if (launch_pdl(kernel(bytes), dim3((unsigned)a->n_seq * cvk::kForkCluster), dim3(cvk::kPagesThreads), 0, stream, p) != cudaSuccess)
        return CV_ERR_LAUNCH;
    return done();
}

}  // namespace

extern "C" {

int cv_tree_attention_workspace(const cv_tree_attention_args *args, int64_t *bytes) {
    if (!bytes) return CV_ERR_NULL_POINTER;
    const int rc = check_attention(args, false);
    if (rc != CV_OK) return rc;
    *bytes = 0;
    if (args->n_seq == 0) return CV_OK;
    // NULL pointers count as aligned; the call's own may be aligned to less and take another kernel
    const bool known = args->q && args->cache.k && args->cache.v;
    for (int best = kTensorCores; best >= (known ? kTensorCores : kAnyAlignment); --best) {
        const int64_t n = plan_attention(args, best).bytes;
        *bytes = *bytes > n ? *bytes : n;
    }
    return CV_OK;
}

int cv_tree_attention(const cv_tree_attention_args *args, void *stream) {
    const int rc = check_attention(args, true);
    if (rc != CV_OK) return rc;
    if (args->n_seq == 0) return CV_OK;
    if (args->cu_draft && args->total_tokens == 0) return launch_no_attention(args, reinterpret_cast<cudaStream_t>(stream));
    return launch_attention(args, reinterpret_cast<cudaStream_t>(stream));
}

int cv_draft_verify(const cv_draft_verify_args *args, void *stream) {
    const int rc = check_sample(args);
    if (rc != CV_OK) return rc;
    if (args->n_seq == 0) return CV_OK;
    // blocks a sequence: as many as are resident at once (115 sequences of 128,000 tokens: 38 us in 4 blocks each, 43 in 8, 52 in 2)
    int cluster = cvk::kSampleCluster;
    while (cluster > 1 && (int64_t)args->n_seq * cluster > (int64_t)cvk::kSampleBlocks * device_limits().sms) cluster /= 2;
    cvk::SampleParams p{args->n_seq, args->T, args->vocab, args->total_tokens, cluster, args->probs, args->draft_probs,
                        args->probs_seq_stride, args->probs_tok_stride, args->draft_seq_stride, args->draft_tok_stride,
                        args->tokens, args->parent, args->uniforms, args->cu_draft, args->cache_idx, args->accept_len,
                        args->accept_node, args->path, args->out_tokens, args->err};
    cudaStream_t on = reinterpret_cast<cudaStream_t>(stream);
    const int clear = clear_err(args->err, args->n_seq, on);
    if (clear != CV_OK) return clear;
    const auto k = cvk::sample_kernel(args->dtype == CV_BF16);
    if (cvk::launch_pdl_cluster(k, dim3((unsigned)(args->n_seq * cluster)),
                                dim3(cvk::kSampleThreads), cluster, on, p) != cudaSuccess)
        return CV_ERR_LAUNCH;
    return done();
}

int cv_qk_norm_rope(const cv_qk_norm_rope_args *args, void *stream) {
    const int rc = check_rope(args);
    if (rc != CV_OK) return rc;
    if (args->n_seq == 0) return CV_OK;
    return launch_rope(args, reinterpret_cast<cudaStream_t>(stream));
}

int cv_cache_compact(const cv_cache_compact_args *args, void *stream) {
    const int rc = check_compact(args);
    if (rc != CV_OK) return rc;
    if (args->n_seq == 0) return CV_OK;
    cvk::PagesParams p;
    std::memset(&p, 0, sizeof p);
    p.n_seq = args->n_seq, p.T = args->T, p.c = view(args->cache);
    p.idx = args->cache_idx, p.len = args->cache_len, p.path = args->path, p.accept = args->accept_len;
    p.new_len = args->new_len, p.err = args->err;
    const int bytes = copy_bytes(args->cache);
    p.esize = esize_of(args->cache.dtype), p.chunks = args->cache.head_dim * p.esize / bytes;
    // a piece a thread, but no more blocks than are resident (4 an SM): a block's start costs as much as several pieces
    const int64_t items = copy_pieces(args->cache);
    int64_t blocks = (items + cvk::kPagesThreads - 1) / cvk::kPagesThreads;
    const int64_t most = 4LL * device_limits().sms / args->n_seq;
    if (blocks > most) blocks = most > 1 ? most : 1;
    if (launch_pdl(cvk::pages_compact_kernel(bytes), dim3((unsigned)blocks, (unsigned)args->n_seq), dim3(cvk::kPagesThreads), 0,
                   reinterpret_cast<cudaStream_t>(stream), p) != cudaSuccess)
        return CV_ERR_LAUNCH;
    return done();
}

int cv_cache_reserve(const cv_cache_pages_args *args, void *stream) {
    const int rc = check_pages(args, false, true, args && args->cache_len);
    if (rc != CV_OK) return rc;
    if (args->n_seq == 0) return CV_OK;
    cvk::PagesParams p = pages_params(args);
    p.len = args->cache_len;
    const int take = launch_take(p, p.len ? cvk::kPagesOwn : cvk::kPagesReserve, reinterpret_cast<cudaStream_t>(stream));
    if (take != CV_OK || !p.len) return take != CV_OK ? take : done();
    return launch_copies(p, args, cvk::pages_own_kernel, reinterpret_cast<cudaStream_t>(stream));
}

int cv_cache_fork(const cv_cache_pages_args *args, void *stream) {
    const int rc = check_pages(args, true, true, true);
    if (rc != CV_OK) return rc;
    if (args->n_seq == 0) return CV_OK;
    const cvk::PagesParams p = pages_params(args);
    const int take = launch_take(p, cvk::kPagesFork, reinterpret_cast<cudaStream_t>(stream));
    return take != CV_OK ? take : launch_copies(p, args, cvk::pages_fork_kernel, reinterpret_cast<cudaStream_t>(stream));
}

int cv_cache_free(const cv_cache_pages_args *args, void *stream) {
    const int rc = check_pages(args, false, false, false);
    if (rc != CV_OK) return rc;
    if (args->n_seq == 0) return CV_OK;
    const cvk::PagesParams p = pages_params(args);
    if (launch_pdl(cvk::pages_free_kernel(), dim3((unsigned)args->n_seq), dim3(cvk::kPagesThreads), 0,
                   reinterpret_cast<cudaStream_t>(stream), p) != cudaSuccess)
        return CV_ERR_LAUNCH;
    return done();
}

}  // extern "C"
