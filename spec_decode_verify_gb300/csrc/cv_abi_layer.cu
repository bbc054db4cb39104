// C ABI of the operators beside the conv: linear attention (prompts, single tokens and drafts) and the
// block norms.  As for the conv, every check runs on the host before anything is launched.
#include <cuda.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "convverify.h"
#include "cv_host.h"
#include "cv_linattn.h"
#include "cv_norm.h"

namespace {

using cvk::device_limits;
using cvk::launch_pdl;

constexpr int kMaxHeads = 4096;
constexpr int kMaxHeadDim = 256;
constexpr int kMaxNormDim = 65536;
constexpr int kNormGroupBlocks = 8;  // resident blocks of norm_groups per SM
constexpr int kNormGroupGrid = 16;   // its blocks per SM, at most

bool aligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
int esize_of(int dtype) { return dtype == CV_BF16 ? 2 : 4; }

// ---- linear attention

int check_run(const cv_linattn_tokens &r) {
    const int64_t strides[] = {r.q_seq_stride, r.q_tok_stride, r.q_head_stride, r.k_seq_stride, r.k_tok_stride,
                               r.k_head_stride, r.v_seq_stride, r.v_tok_stride, r.v_head_stride, r.decay_seq_stride,
                               r.decay_tok_stride, r.gain_seq_stride, r.gain_tok_stride};
    for (int64_t s : strides)
        if (s < 0) return CV_ERR_STRIDE;
    if (r.cu && r.total_tokens < 0) return CV_ERR_SHAPE;
    return CV_OK;
}

// Whether a run holds any token at all (buffers may be NULL otherwise).
bool run_empty(const cv_linattn_tokens &r) { return r.T == 0 || (r.cu && r.total_tokens == 0); }

int check_linattn(const cv_linattn_args *a, bool step, bool pointers) {
    if (!a) return CV_ERR_NULL_ARGS;
    if (a->dtype != CV_F32 && a->dtype != CV_BF16) return CV_ERR_DTYPE;
    if (a->n_seq < 0 || a->n_seq > 65535 || a->n_slots < 1 || a->n_heads < 1 || a->n_heads > kMaxHeads)
        return CV_ERR_SHAPE;
    if (a->dk < 1 || a->dk > kMaxHeadDim || a->dv < 1 || a->dv > kMaxHeadDim || a->n_qk_heads < 1 ||
        a->n_heads % a->n_qk_heads != 0)
        return CV_ERR_HEAD_DIM;
    if (a->tok.T < 0 || (step && (a->tok.T > CV_MAX_T || a->prev.T < 0 || a->prev.T > CV_MAX_T))) return CV_ERR_TOKENS;
    int rc = check_run(a->tok);
    if (rc == CV_OK && step) rc = check_run(a->prev);
    if (rc != CV_OK) return rc;
    if (a->out_seq_stride < 0 || a->out_tok_stride < 0 || a->out_head_stride < 0 || a->state_slot_stride < 0 ||
        a->state_head_stride < 0)
        return CV_ERR_STRIDE;
    // heads and slots of the state must not overlap
    if (a->n_heads > 1 && a->state_head_stride < (int64_t)a->dk * a->dv) return CV_ERR_STRIDE;
    if (a->n_slots > 1 && a->state_slot_stride < (int64_t)a->dk * a->dv) return CV_ERR_STRIDE;
    if (!pointers || a->n_seq == 0) return CV_OK;
    if (!a->state || !aligned(a->state, 4)) return CV_ERR_NULL_POINTER;
    if (!step && !a->tok.cu) return CV_ERR_NULL_POINTER;
    if (!run_empty(a->tok)) {
        if (!a->tok.q || !a->tok.k || !a->tok.v || !a->tok.log_decay || !a->out) return CV_ERR_NULL_POINTER;
        const void *in[] = {a->tok.q, a->tok.k, a->tok.v, a->tok.log_decay, a->tok.gain, a->state};
        for (const void *p : in)
            if (a->out == p) return CV_ERR_ALIAS;
    }
    if (step && a->prev.T > 0) {
        if (!a->accept_len) return CV_ERR_NULL_POINTER;
        if (!run_empty(a->prev) && (!a->prev.k || !a->prev.v || !a->prev.log_decay)) return CV_ERR_NULL_POINTER;
    }
    return CV_OK;
}

// n elements at every multiple of n channels may be loaded at once.
bool rows_of(int n, const void *p, int64_t seq, int64_t tok, int64_t head, bool packed, int d, int es) {
    return d % n == 0 && aligned(p, n * es) && (packed || seq % n == 0) && tok % n == 0 && head % n == 0;
}

cvk::LinattnRun make_run(const cv_linattn_tokens &t, const cv_linattn_args *a, bool with_q) {
    const int es = esize_of(a->dtype);
    cvk::LinattnRun r;
    std::memset(&r, 0, sizeof r);
    r.q = t.q, r.q_seq = t.q_seq_stride, r.q_tok = t.q_tok_stride, r.q_head = t.q_head_stride;
    r.k = t.k, r.k_seq = t.k_seq_stride, r.k_tok = t.k_tok_stride, r.k_head = t.k_head_stride;
    r.v = t.v, r.v_seq = t.v_seq_stride, r.v_tok = t.v_tok_stride, r.v_head = t.v_head_stride;
    r.g = t.log_decay, r.g_seq = t.decay_seq_stride, r.g_tok = t.decay_tok_stride;
    r.b = t.gain, r.b_seq = t.gain_seq_stride, r.b_tok = t.gain_tok_stride;
    r.cu = t.cu, r.T = t.T, r.total = t.total_tokens;
    auto all = [&](int n) {
        return rows_of(n, t.k, r.k_seq, r.k_tok, r.k_head, t.cu, a->dk, es) &&
               rows_of(n, t.v, r.v_seq, r.v_tok, r.v_head, t.cu, a->dv, es) &&
               (!with_q || rows_of(n, t.q, r.q_seq, r.q_tok, r.q_head, t.cu, a->dk, es));
    };
    r.vec = all(4);
    r.vec16 = all(16 / es);
    return r;
}

cvk::LinattnParams make_linattn(const cv_linattn_args *a, bool step) {
    cvk::LinattnParams p;
    std::memset(&p, 0, sizeof p);
    p.tok = make_run(a->tok, a, true);
    if (step) p.prev = make_run(a->prev, a, false);
    p.skip = a->skip;
    p.out = a->out, p.o_seq = a->out_seq_stride, p.o_tok = a->out_tok_stride, p.o_head = a->out_head_stride;
    p.state = a->state, p.st_slot = a->state_slot_stride, p.st_head = a->state_head_stride;
    p.cache_idx = a->cache_idx, p.has_init = a->has_initial_state, p.err = a->err;
    p.accept = step ? a->accept_len : nullptr;
    p.n_seq = a->n_seq, p.n_heads = a->n_heads, p.n_qk = a->n_qk_heads, p.dk = a->dk, p.dv = a->dv;
    p.n_slots = a->n_slots;
    p.bf16 = a->dtype == CV_BF16;
    p.update = step ? a->update_state != 0 : 1;
    p.st_vec = a->dv % 4 == 0 && aligned(a->state, 16) && a->state_slot_stride % 4 == 0 && a->state_head_stride % 4 == 0;
    p.o_vec = rows_of(4, a->out, a->out_seq_stride, a->out_tok_stride, a->out_head_stride, a->tok.cu, a->dv,
                      esize_of(a->dtype));
    p.scale = a->scale;
    p.polls = a->wait_polls == 0 ? cvk::kPolls : a->wait_polls < 0 ? 0u : (unsigned)a->wait_polls;
    return p;
}

constexpr int kMinPieceTokens = 32;  // of a prompt cut for the recurrent kernel
constexpr int kMaxPieces = 64;

// The recurrent kernel's launch.
struct StepPlan {
    bool stream;  // the streaming kernel
    int vs, slices, tg, pieces, piece_len;
    long long units, resident;
};
int64_t step_workspace(const cv_linattn_args *a, const StepPlan &pl) {
    const int64_t states = pl.pieces > 1 ? (int64_t)a->n_seq * a->n_heads * pl.pieces : 0;
    return states * a->dk * a->dv * 4 + (states * 4 + 255) / 256 * 256;
}

StepPlan plan_step(const cv_linattn_args *a, const cvk::LinattnParams &p, bool step) {
    StepPlan pl;
    const long long heads = (long long)a->n_seq * a->n_heads, sms = device_limits().sms;
    const int most = step && a->prev.T > a->tok.T ? a->prev.T : a->tok.T;
    pl.stream = p.st_vec && a->dk <= 128 && (run_empty(a->tok) || p.tok.vec16) &&
                (!step || run_empty(a->prev) || p.prev.vec16);
    pl.tg = most <= 1 ? 1 : cvk::kStepMaxGroup;
    pl.pieces = 1, pl.piece_len = 0;
    // Blocks share the products of their tokens' q and k, so runs of tokens take 128 columns (128 x 8 drafts of 48
    // heads: 172 us, 201 with 64); single tokens have one product, and smaller blocks overlap better (64 tokens of
    // 32 heads: 22.4 us, 24.2 with 128).
    pl.vs = pl.stream && pl.tg > 1 ? 128 : 64;
    while (pl.vs > 32 && pl.vs / 2 >= a->dv) pl.vs /= 2;
    // Few heads and long prompts: the length is cut into pieces that fill the resident blocks.  A cut costs a
    // pass for the pieces' own states and their join, so two pieces are not worth it.
    const int64_t longest = a->tok.T < a->tok.total_tokens ? a->tok.T : a->tok.total_tokens;
    if (!step && pl.stream) {
        // pieces that are resident at once; each sequence's last is half a piece on average
        const int64_t slots = sms * (256 / pl.vs) / ((int64_t)a->n_heads * ((a->dv + pl.vs - 1) / pl.vs));
        const int64_t halves = 2 * slots - a->n_seq, per = slots / a->n_seq;
        int64_t len = longest;
        if (a->n_seq > cvk::kStepMaxCounted) len = per > 0 ? (longest + per - 1) / per : longest;
        else if (halves > 0) len = (2 * a->tok.total_tokens + halves - 1) / halves;
        if (len < kMinPieceTokens) len = kMinPieceTokens;
        if (len < (longest + kMaxPieces - 1) / kMaxPieces) len = (longest + kMaxPieces - 1) / kMaxPieces;
        len = (len + cvk::kStepMaxGroup - 1) / cvk::kStepMaxGroup * cvk::kStepMaxGroup;
        const int64_t n = (longest + len - 1) / len;
        if (n > 2) pl.pieces = (int)n, pl.piece_len = (int)len;
    }
    // the widest slice of a head whose grid still gives every SM two blocks
    while (pl.vs > 32 && heads * pl.pieces * ((a->dv + pl.vs - 1) / pl.vs) < 2 * sms) pl.vs /= 2;
    pl.slices = (a->dv + pl.vs - 1) / pl.vs;
    pl.units = heads * pl.pieces * pl.slices;
    pl.resident = sms * (256 / pl.vs);  // the streaming kernel's registers allow 16 warps per SM
    return pl;
}

int launch_recurrent(const cv_linattn_args *a, bool step, cudaStream_t stream) {
    cvk::LinattnParams p = make_linattn(a, step);
    const StepPlan pl = plan_step(a, p, step);
    if (pl.units > 0x7fffffff) return CV_ERR_SHAPE;
    p.slices = pl.slices, p.pieces = pl.pieces, p.piece_len = pl.piece_len;
    const cvk::StepKernel k = pl.stream ? cvk::stream_kernel(pl.vs / 16, a->dk, pl.tg, p.bf16)
                                        : cvk::step_kernel(pl.vs, a->dk, pl.tg);
    if (cvk::ensure_smem(reinterpret_cast<const void *>(k.fn), k.smem_bytes) != cudaSuccess) return CV_ERR_LAUNCH;
    const dim3 grid((unsigned)(pl.stream && pl.units > pl.resident ? pl.resident : pl.units));
    const dim3 block(pl.stream ? 2 * pl.vs : cvk::kStepThreads);
    if (pl.pieces > 1) {
        if (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < step_workspace(a, pl))
            return CV_ERR_WORKSPACE;
        const int64_t states = (int64_t)a->n_seq * a->n_heads;
        p.ws_state = reinterpret_cast<float *>(a->workspace);
        p.ws_decay = p.ws_state + states * pl.pieces * a->dk * a->dv;
        cvk::LinattnParams own = p;  // the tokens as a run to advance over, from zero
        own.prev = p.tok, own.tok.T = 0, own.tok.cu = nullptr, own.accept = nullptr;
        own.own_states = 1, own.update = 0;
        if (launch_pdl(k.fn, grid, block, k.smem_bytes, stream, own) != cudaSuccess) return CV_ERR_LAUNCH;
        const int64_t parts = ((int64_t)a->dk * a->dv + cvk::kStateJoinThreads - 1) / cvk::kStateJoinThreads;
        if (launch_pdl(cvk::state_join_kernel(), dim3((unsigned)(states * parts)), dim3(cvk::kStateJoinThreads), 0, stream,
                       p) != cudaSuccess)
            return CV_ERR_LAUNCH;
    }
    if (launch_pdl(k.fn, grid, block, k.smem_bytes, stream, p) != cudaSuccess) return CV_ERR_LAUNCH;
    return cudaGetLastError() == cudaSuccess ? CV_OK : CV_ERR_LAUNCH;
}

// The chunked kernel's launch for these arguments; pieces 0: the recurrent kernel takes them.
struct ChunkPlan {
    int pieces, seg_len;
    long long ws_states;  // states of pieces that go through the workspace
    int dv_pad;
};
// Prompts of at most so many tokens go to the recurrent kernel, more where there are heads for every SM
// (measured, 32 heads of 128, recurrent / chunked: 1 prompt of 8 tokens 7.6 / 9.1 us, of 16 11.3 / 9.2; 64 prompts
// of 16 tokens 104 / 132 us, of 24 144 / 134).
constexpr int kShortFew = 8, kShortMany = 16;
constexpr int64_t kMaxStride = 1LL << 38;  // elements: a tensor map's strides are below 2^40 bytes

// A map of [tokens][heads][d] bf16 rows read in boxes of 128 tokens of one head's 64 channels.
bool encode_rows(CUtensorMap *map, const void *p, int d, int heads, int64_t tokens, int64_t head, int64_t tok) {
    const auto encode = cvk::encode_tiled();
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? head : d) * 2, (cuuint64_t)tok * 2};
    const cuuint32_t box[3] = {64, 1, cvk::kChunk}, step[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

ChunkPlan plan_chunks(const cv_linattn_args *a) {
    ChunkPlan pl{0, 0, 0, a->dv <= 64 ? 64 : 128};
    const cv_linattn_tokens &t = a->tok;
    // what the copies by TMA (q, k, v) and of 16 bytes (out, state) need
    auto rows8 = [](const void *p, int64_t tok, int64_t head) {
        return aligned(p, 16) && tok % 8 == 0 && head % 8 == 0 && tok > 0 && tok < kMaxStride && head < kMaxStride;
    };
    if (a->dtype != CV_BF16 || a->dk % 8 != 0 || a->dv % 8 != 0 || a->dk > 128 || a->dv > 128 ||
        (a->n_qk_heads > 1 && (t.q_head_stride == 0 || t.k_head_stride == 0)) || (a->n_heads > 1 && t.v_head_stride == 0) ||
        !rows8(t.q, t.q_tok_stride, t.q_head_stride) || !rows8(t.k, t.k_tok_stride, t.k_head_stride) ||
        !rows8(t.v, t.v_tok_stride, t.v_head_stride) || !rows8(a->out, a->out_tok_stride, a->out_head_stride) ||
        !aligned(a->state, 16) || a->state_slot_stride % 4 != 0 || a->state_head_stride % 4 != 0)
        return pl;
    const int64_t longest = t.T < t.total_tokens ? t.T : t.total_tokens;
    const int64_t whole = (longest + cvk::kChunk - 1) / cvk::kChunk * cvk::kChunk;
    const int64_t heads = (int64_t)a->n_seq * a->n_heads, sms = device_limits().sms;
    if (longest <= (heads > sms ? kShortMany : kShortFew)) return pl;
    pl.pieces = 1;
    pl.seg_len = (int)(whole > 0 ? whole : cvk::kChunk);
    // Few heads: cut the length into pieces.  A cut costs a pass over k and v for the pieces' own states and their
    // join.  The estimate is in tenths of a us, from measured launches (128 columns): 5.7 us and 3.6 us a chunk of the
    // fullest SM uncut; cut 13.5 us, 5.2 us a chunk, 0.35 us a piece of the join and 4.5 us for each further piece
    // that an SM takes (1 prompt of 32k tokens, 6 heads: 85 us in 24 pieces; 4.1k tokens, 4 heads: 28 us in 33).
    // (It was not fitted to the kernel for 64 columns, which takes it too.)
    // Lengths are on the device, so the fullest SM is estimated from their sum.
    const int64_t chunks = whole / cvk::kChunk, mean = (a->n_heads * t.total_tokens / cvk::kChunk + sms - 1) / sms;
    int64_t best = 57 + 36 * (chunks > mean ? chunks : mean);
    for (int64_t n = 2; n <= chunks && n <= sms && heads * n <= 8 * sms;) {
        const int64_t len = (chunks + n - 1) / n;
        n = (chunks + len - 1) / len;
        int64_t full = a->n_seq * n, units = full;
        if (a->n_seq <= cvk::kChunkMaxSorted) {  // (otherwise pieces past a sequence's end take their turns too)
            const int64_t of = t.total_tokens / (len * cvk::kChunk);
            full = of < full ? of : full;
            units = of + a->n_seq < units ? of + a->n_seq : units;
        }
        int64_t fullest = len;
        if (a->n_heads * units > sms) {
            const int64_t rounds = (a->n_heads * full + sms - 1) / sms * len, spread = mean + (len + 1) / 2;
            fullest = rounds > spread ? rounds : spread;
        }
        const int64_t cost = 135 + 52 * fullest + 45 * ((a->n_heads * units - 1) / sms) + 7 * n / 2;
        if (cost < best) {
            best = cost;
            pl.pieces = (int)n, pl.seg_len = (int)(len * cvk::kChunk), pl.ws_states = heads * n;
        }
        if (len == 1) break;
        n = (chunks + len - 2) / (len - 1);
    }
    return pl;
}

int64_t chunk_workspace(const cv_linattn_args *a, const ChunkPlan &pl) {
    if (pl.ws_states == 0) return 0;
    return pl.ws_states * (cvk::kChunk * pl.dv_pad * 4) + ((pl.ws_states + a->n_seq) * 4 + 255) / 256 * 256;
}

int launch_chunks(const cv_linattn_args *a, const ChunkPlan &pl, cudaStream_t stream) {
    cvk::LinattnChunkParams p;
    std::memset(&p, 0, sizeof p);
    p.a = make_linattn(a, false);
    p.n_segs = pl.pieces;
    p.seg_len = pl.seg_len;
    const int64_t units = (int64_t)a->n_seq * a->n_heads * pl.pieces, sms = device_limits().sms;
    if (units > 0x7fffffff) return CV_ERR_SHAPE;
    p.units = (int)units;
    p.sort = (units > sms || pl.pieces > 1) && a->n_seq <= cvk::kChunkMaxSorted;
    p.dv_pad = pl.dv_pad;
    if (pl.ws_states > 0) {
        if (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < chunk_workspace(a, pl))
            return CV_ERR_WORKSPACE;
        p.ws_state = reinterpret_cast<float *>(a->workspace);
        p.ws_decay = p.ws_state + pl.ws_states * cvk::kChunk * pl.dv_pad;
        p.ws_left = reinterpret_cast<int *>(p.ws_decay + pl.ws_states);
    }
    const cv_linattn_tokens &t = a->tok;
    if (t.total_tokens > 0 &&
        (!encode_rows(&p.q_map, t.q, a->dk, a->n_qk_heads, t.total_tokens, t.q_head_stride, t.q_tok_stride) ||
         !encode_rows(&p.k_map, t.k, a->dk, a->n_qk_heads, t.total_tokens, t.k_head_stride, t.k_tok_stride) ||
         !encode_rows(&p.v_map, t.v, a->dv, a->n_heads, t.total_tokens, t.v_head_stride, t.v_tok_stride)))
        return CV_ERR_LAUNCH;
    const cvk::ChunkKernel k = cvk::chunk_kernel(a->dv);
    if (cvk::ensure_smem(reinterpret_cast<const void *>(k.fn), k.smem_bytes) != cudaSuccess) return CV_ERR_LAUNCH;
    // the kernel ORs its bits into err
    if (a->err && cudaMemsetAsync(a->err, 0, sizeof(int32_t) * (size_t)a->n_seq, stream) != cudaSuccess)
        return CV_ERR_LAUNCH;
    const dim3 grid((unsigned)(units < sms ? units : sms)), block(cvk::kChunkThreads);
    if (pl.ws_states > 0) {
        p.state_only = 1;
        if (launch_pdl(k.fn, grid, block, k.smem_bytes, stream, p) != cudaSuccess) return CV_ERR_LAUNCH;
        p.state_only = 0;
        const unsigned parts = (unsigned)(a->n_seq * (int64_t)a->n_heads * (pl.dv_pad / 4));
        if (launch_pdl(cvk::chunk_join_kernel(), dim3(parts), dim3(cvk::kJoinThreads), 0, stream, p) != cudaSuccess)
            return CV_ERR_LAUNCH;
    }
    if (launch_pdl(k.fn, grid, block, k.smem_bytes, stream, p) != cudaSuccess) return CV_ERR_LAUNCH;
    return cudaGetLastError() == cudaSuccess ? CV_OK : CV_ERR_LAUNCH;
}

// ---- block norm

int check_norm(const cv_norm_args *a) {
    if (!a) return CV_ERR_NULL_ARGS;
    if (a->dtype != CV_F32 && a->dtype != CV_BF16) return CV_ERR_DTYPE;
    if (a->residual && a->residual_dtype != a->dtype && a->residual_dtype != CV_F32) return CV_ERR_DTYPE;
    if (a->rows < 0 || a->dim < 1 || a->dim > kMaxNormDim) return CV_ERR_SHAPE;
    if (a->group < 0 || (a->group > 0 && a->dim % a->group != 0) || (a->group == 0 && a->post_weight))
        return CV_ERR_HEAD_DIM;
    if (a->gate && a->gate_act != CV_GATE_SILU && a->gate_act != CV_GATE_SIGMOID) return CV_ERR_LAYOUT;
    if (a->y_stride < 0 || a->gate_stride < 0 || a->residual_stride < 0) return CV_ERR_STRIDE;
    if ((a->out && a->rows > 1 && a->out_stride < a->dim) ||
        (a->residual && a->rows > 1 && a->residual_out_stride < a->dim))
        return CV_ERR_STRIDE;
    if (a->rows == 0) return CV_OK;
    if (!a->y || (a->residual ? !a->residual_out : !a->out)) return CV_ERR_NULL_POINTER;
    if (a->out) {
        if (a->out == a->residual || a->out == a->residual_out || a->out == a->post_weight || a->out == a->pre_weight ||
            a->out == a->channel_scale || (a->out == a->y && a->out_stride != a->y_stride) ||
            (a->out == a->gate && a->out_stride != a->gate_stride))
            return CV_ERR_ALIAS;
    }
    if (a->residual &&
        (a->residual_out == a->y || a->residual_out == a->gate || a->residual_out == a->post_weight ||
         a->residual_out == a->pre_weight || a->residual_out == a->channel_scale ||
         (a->residual_out == a->residual && a->residual_out_stride != a->residual_stride)))
        return CV_ERR_ALIAS;
    return CV_OK;
}

// A row buffer that may be absent: accesses of `bytes` at every multiple of them.
bool vec_row(const void *p, int64_t stride, int64_t rows, int es, int bytes) {
    return !p || (aligned(p, bytes) && (rows <= 1 || (stride * es) % bytes == 0));
}

// norm_row, more than kNormRowMany rows an SM: threads a row while elements a thread allow it, so that several rows
// share an SM (7324 rows of 8192, bf16: 99 us with 256 threads, 152 with 512; 300 rows of 4096: 4.9 against 3.8).
constexpr int kNormRowWide = 256, kNormRowMany = 4;
constexpr int kNormRowAhead = 16;  // rows an SM from which the next rows are prefetched

int launch_norm(const cv_norm_args *a, cudaStream_t stream) {
    const int es = esize_of(a->dtype), V = 16 / es;
    const bool res = a->residual != nullptr, res32 = res && a->residual_dtype == CV_F32;
    cvk::NormParams p;
    std::memset(&p, 0, sizeof p);
    p.rows = a->rows, p.dim = a->dim, p.group = a->group;
    p.gate_act = a->gate_act, p.gate_first = a->gate_first != 0;
    p.eps = a->eps, p.scale = a->scale;
    p.y = a->y, p.gate = a->gate, p.post = a->post_weight;
    p.res = a->residual, p.cs = res ? a->channel_scale : nullptr, p.pre = res ? a->pre_weight : nullptr;
    p.out = a->out, p.res_out = res ? a->residual_out : nullptr;
    p.y_row = a->y_stride, p.gate_row = a->gate_stride, p.res_row = a->residual_stride;
    p.res_out_row = a->residual_out_stride, p.out_row = a->out_stride;
    // whether every tensor allows accesses of n elements
    auto runs = [&](int n) {
        const int rs = res32 ? 4 : es, b = n * es, rb = n * rs < 16 ? n * rs : 16;
        return vec_row(p.y, p.y_row, a->rows, es, b) && vec_row(p.gate, p.gate_row, a->rows, es, b) &&
               vec_row(p.out, p.out_row, a->rows, es, b) && vec_row(p.res, p.res_row, a->rows, rs, rb) &&
               vec_row(p.res_out, p.res_out_row, a->rows, rs, rb) && vec_row(p.post, 0, 1, es, b) &&
               vec_row(p.cs, 0, 1, es, b) && vec_row(p.pre, 0, 1, es, b);
    };
    const bool vec = runs(V);
    const bool bf16 = a->dtype == CV_BF16;

    // narrow groups without a residual: up to 32 lanes a group
    if (!res && a->group > 0) {
        const bool v = vec && a->group % V == 0;
        const int per = v ? V : 1, most = v ? 2 : 4;
        if (a->group <= 32 * per * most) {
            const int need = (a->group + per - 1) / per;  // accesses a group
            p.lanes = 1;
            while (p.lanes < 32 && p.lanes < need) p.lanes *= 2;
            const long long groups = a->rows * (a->dim / a->group);
            const int nv = (need + p.lanes - 1) / p.lanes, per_block = cvk::kNormGroupThreads / p.lanes;
            p.flat = a->rows == 1 || (a->y_stride == a->dim && a->out_stride == a->dim && (!a->gate || a->gate_stride == a->dim));
            if (p.flat) p.y_row = p.gate_row = p.out_row = a->group;
            const long long sms = device_limits().sms;
            // several groups a thread once that leaves every SM a full set of blocks
            const int unroll = v && nv == 1 && groups >= sms * kNormGroupBlocks * per_block * cvk::kNormUnroll ? cvk::kNormUnroll : 1;
            const long long blocks = (groups + per_block * unroll - 1) / (per_block * unroll), cap = sms * kNormGroupGrid;
            const auto k = cvk::norm_groups_kernel(bf16, v, nv, unroll);
            if (launch_pdl(k, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(cvk::kNormGroupThreads), 0, stream,
                           p) != cudaSuccess)
                return CV_ERR_LAUNCH;
            return cudaGetLastError() == cudaSuccess ? CV_OK : CV_ERR_LAUNCH;
        }
    }
    const unsigned grid = (unsigned)(a->rows < 0x7fffffff ? a->rows : 0x7fffffff);
    const int v = vec && a->dim % V == 0 ? V : a->dim % 2 == 0 && runs(2) ? 2 : 1;
    if ((a->group == 0 || a->group == a->dim) && a->dim <= cvk::kNormRowThreads * cvk::norm_row_elems(v)) {
        const int64_t sms = device_limits().sms;
        const bool many = a->rows > kNormRowMany * sms;
        p.ahead = a->rows > kNormRowAhead * sms ? sms : a->rows;
        int elems = 8, rows = 1;
        while (elems < cvk::norm_row_elems(v) && elems * (many && v > 2 ? kNormRowWide : cvk::kNormRowThreads) < a->dim)
            elems *= many && v == 8 ? 4 : 2;  // 16 of bf16 keep too few loads in flight (rows of 4096: 133 us, 32: 93)
        // A warp a row, several rows a block (30000 residual rows of 64, bf16: 15.5 us; a block of one warp for each:
        // 31).  16-byte accesses stop at 8 elements a thread: above, a block a row with the next rows prefetched is
        // faster (rows of 512: 39 us against 45).
        if (many && a->dim <= (v > 2 ? 8 : 16) * 32) elems = a->dim <= 8 * 32 ? 8 : 16, rows = kNormRowWide / 32;
        const int threads = (a->dim + elems - 1) / elems;
        const int64_t blocks = (a->rows + rows - 1) / rows;
        if (launch_pdl(cvk::norm_row_kernel(bf16, res32, v, elems), dim3((unsigned)(blocks < 0x7fffffff ? blocks : 0x7fffffff)),
                       dim3((threads + 31) / 32 * 32, rows), 0,
                       stream, p) != cudaSuccess)
            return CV_ERR_LAUNCH;
        return cudaGetLastError() == cudaSuccess ? CV_OK : CV_ERR_LAUNCH;
    }
    const int groups = a->group > 0 ? a->dim / a->group : 0, smem = (cvk::kNormAnyThreads / 32 + groups) * 4;
    const auto k = cvk::norm_any_kernel(bf16, res32);
    if (smem > device_limits().smem_per_block) return CV_ERR_SMEM;
    if (cvk::ensure_smem(reinterpret_cast<const void *>(k), smem) != cudaSuccess) return CV_ERR_LAUNCH;
    if (launch_pdl(k, dim3(grid), dim3(cvk::kNormAnyThreads), smem, stream, p) != cudaSuccess) return CV_ERR_LAUNCH;
    return cudaGetLastError() == cudaSuccess ? CV_OK : CV_ERR_LAUNCH;
}

}  // namespace

extern "C" {

int cv_linattn_workspace(const cv_linattn_args *args, int64_t *bytes) {
    if (!bytes) return CV_ERR_NULL_POINTER;
    const int rc = check_linattn(args, false, false);
    if (rc != CV_OK) return rc;
    *bytes = 0;
    if (args->n_seq == 0) return CV_OK;
    // NULL pointers count as aligned, which either kernel may take: the call's own may be aligned to less and
    // leave the chunked kernel, so the size then covers both (unaligned rows need none).
    const cv_linattn_tokens &t = args->tok;
    const bool known = t.q && t.k && t.v && args->out && args->state;
    const ChunkPlan pl = plan_chunks(args);
    if (pl.pieces > 0) *bytes = chunk_workspace(args, pl);
    if (pl.pieces == 0 || !known) {
        const int64_t step = step_workspace(args, plan_step(args, make_linattn(args, false), false));
        *bytes = *bytes > step ? *bytes : step;
    }
    return CV_OK;
}

int cv_linattn_prefill(const cv_linattn_args *args, void *stream) {
    const int rc = check_linattn(args, false, true);
    if (rc != CV_OK) return rc;
    if (args->n_seq == 0) return CV_OK;
    const ChunkPlan pl = plan_chunks(args);
    if (pl.pieces > 0) return launch_chunks(args, pl, reinterpret_cast<cudaStream_t>(stream));
    return launch_recurrent(args, false, reinterpret_cast<cudaStream_t>(stream));
}

int cv_linattn_step(const cv_linattn_args *args, void *stream) {
    const int rc = check_linattn(args, true, true);
    if (rc != CV_OK) return rc;
    if (args->n_seq == 0) return CV_OK;
    return launch_recurrent(args, true, reinterpret_cast<cudaStream_t>(stream));
}

int cv_block_norm(const cv_norm_args *args, void *stream) {
    const int rc = check_norm(args);
    if (rc != CV_OK) return rc;
    if (args->rows == 0) return CV_OK;
    return launch_norm(args, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
