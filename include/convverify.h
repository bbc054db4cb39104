/*
 * convverify.h -- C ABI of the batched speculative-verify causal depthwise conv1d update.
 *
 * One verify call runs, for n_seq sequences of T draft tokens each, the conv update of a hybrid
 * GDN/KDA/Mamba2 layer over all T positions in one launch, and writes every per-token rollback
 * snapshot of the conv window; one commit call later restores the state of the accepted prefix.
 *
 * Sources (the pages this library follows):
 *   [atlas-batched]  Atlas spark_model API doc, fn gdn_verify_fused_conv_kn_batched: one launch
 *                    covers the K draft positions, the kernel itself stores each position's
 *                    rollback snapshot into a strided buffer, the state ends on the committed
 *                    window, and the batch over n_seq (per-sequence strides) matches n separate
 *                    calls bit for bit.
 *   [sglang-46184]   sglang pull request #46184 (dedup conv window tile store), sections
 *                    "Motivation" and "Modifications": the deduplicated [dim, T+K-2] window row
 *                    seen as an overlapping [T, dim, K-1] view whose step stride equals its
 *                    column stride; the window of step t starts at column t of the row that
 *                    follows the first committed column with x_0 .. x_{T-1}; padded rows store
 *                    nothing; the tests cover an accepted-token offset into the state.
 *   [kda-mod]        Atlas spark_model/layers/glm5next_kda/mod.rs: conv1d with SiLU, then an L2
 *                    normalisation of the q|k channels alone (V untouched), eps under the root; decode_k snapshot
 *                    t = state after row t, which a partial accept rewinds to.
 *
 * Conventions for every entry point:
 *   - Strides are in ELEMENTS and must be >= 0.  The channel stride of x, out and weight is 1, and
 *     the column stride of conv_state is 1.
 *   - Every data pointer is a DEVICE pointer (or managed memory) unless stated otherwise.  The
 *     caller owns every buffer: the library allocates, frees and synchronises nothing, launches
 *     asynchronously on `stream`, and keeps no pointer after it returns.
 *   - `stream` is a cudaStream_t passed as void*; NULL means the legacy default stream.
 *   - Invalid arguments are reported by a negative status before anything is launched; nothing is
 *     written then.  Problems that only the device can see (a cache slot or state offset out of
 *     range, an accept count out of range) are reported per sequence through the optional `err`
 *     array, and that sequence is left untouched.  No kernel traps.  The kernels that stage data
 *     through bulk copies wait for them with bounded waits (wait_polls below): a wait that gives
 *     up flags CV_SEQ_TIMEOUT for every sequence the block did not finish, and the kernel returns
 *     with its context intact.
 */
#ifndef CONVVERIFY_H
#define CONVVERIFY_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define CV_API __attribute__((visibility("default")))
#else
#define CV_API
#endif

#define CV_ABI_VERSION 12
#define CV_MAX_T 128 /* draft tokens per verify call */

typedef enum cv_dtype {
    CV_F32 = 0,  /* IEEE binary32 */
    CV_BF16 = 1  /* bfloat16; arithmetic in fp32, outputs rounded to nearest even */
} cv_dtype;

/* cv_verify_args.state_dtype: the dtype of conv_state and the snapshots. */
#define CV_STATE_SAME 0 /* the dtype of x (a zero-initialised struct asks for no mixing) */
#define CV_STATE_F32 1  /* fp32 state with bf16 x */
#define CV_STATE_BF16 2 /* bf16 state with fp32 x */

typedef enum cv_window_layout {
    /* window element (s, t, c, k) at s*win_seq_stride + t*win_step_stride + c*win_ch_stride
       + k*win_col_stride: the [n_seq, T, dim, W-1] intermediates of [atlas-batched]. */
    CV_WINDOW_DENSE = 1,
    /* the deduplicated row of [sglang-46184]: element (s, t, c, k) at s*win_seq_stride
       + (t+k)*win_col_stride + c*win_ch_stride, i.e. one [dim, T+W-2] row per sequence whose
       column q holds input q+1 of [committed window, x_0 .. x_{T-1}].  win_step_stride must
       equal win_col_stride. */
    CV_WINDOW_DEDUP = 2,
    /* history-row state: no window buffer (window may be NULL; the win_* strides are ignored).
       The state row is the deduplicated row itself: the call reads the committed window at
       columns [o, o+W-1) of conv_state[slot][c] and then writes columns [0, T+W-2) of that row
       with [full[1 .. W-2], x_0 .. x_{T-1}], so snapshot t sits at columns [t, t+W-1).  The next
       call passes state_off[s] = accept_len[s] - 1 and no commit runs (a reading of the
       [sglang-46184] slot row together with its accepted-token state offset).  Needs
       state_cols >= T+W-2; columns at and above T+W-2 are not touched.  cv_conv_commit rejects
       this layout.  Only this layout accepts column-major state rows (state_col_stride != 1:
       [n_slots, state_cols, dim] storage seen as [n_slots, dim, state_cols], like the pool's
       axis-0 window layout of [sglang-46184]), with which the call reads W-1 columns and writes
       T+W-2 columns, each a contiguous run of channels. */
    CV_WINDOW_HISTORY = 3,
    /* recompute rollback ([memra-engine] ssm_conv_ring_rebuild_dc): no window buffer (window may
       be NULL; the win_* strides are ignored).  The verify writes the outputs only -- no
       snapshots, and conv_state is not written, so it keeps the pre-verify window.  The matching
       cv_conv_commit (same layout) then rebuilds the state from that window and the verify's x:
       conv_state[slot][c][k] = full[a+k], the value snapshot a-1 would hold. */
    CV_WINDOW_RECOMPUTE = 4
} cv_window_layout;

/* Status codes returned by the entry points. */
enum {
    CV_OK = 0,
    CV_ERR_NULL_ARGS = -1,    /* args pointer is NULL */
    CV_ERR_NULL_POINTER = -2, /* a required buffer pointer is NULL */
    CV_ERR_SHAPE = -3,        /* n_seq outside 0..65535, dim < 1, n_slots < 1, state_cols < W-1,
                                 or state_cols < T+W-2 in the history layout */
    CV_ERR_TOKENS = -4,       /* T outside 1..CV_MAX_T */
    CV_ERR_WIDTH = -5,        /* conv width outside 2..4 */
    CV_ERR_DTYPE = -6,        /* dtype not a cv_dtype */
    CV_ERR_HEAD_DIM = -7,     /* qk_channels > 0 and head_dim not a power of two in 8..256, or
                                 qk_channels not a multiple of head_dim, or qk_channels > dim;
                                 linear attention: dk or dv outside 1..256, or n_heads not a
                                 multiple of n_qk_heads; block norm: group not a divisor of dim */
    CV_ERR_LAYOUT = -8,       /* unknown layout, DEDUP with win_step_stride != win_col_stride,
                                 HISTORY passed to cv_conv_commit, or column-major state rows
                                 outside HISTORY */
    CV_ERR_STRIDE = -9,       /* a negative stride, or state rows that overlap (state_ch_stride <
                                 state_cols with dim > 1; column-major rows: state_ch_stride != 1
                                 or state_col_stride < dim) */
    CV_ERR_ALIAS = -10,       /* out or window has the same base address as x, conv_state or weight,
                                 or out and window share a base address */
    CV_ERR_LAUNCH = -11,      /* the CUDA launch failed (cudaGetLastError after the launch) */
    CV_ERR_SMEM = -12,        /* the tile does not fit in shared memory for any block size */
    CV_ERR_WORKSPACE = -13    /* the workspace is NULL, misaligned or smaller than the call needs */
};

/* Per-sequence bits written to err[s] (0 = fine or padded). */
#define CV_SEQ_BAD_SLOT 1   /* cache slot >= n_slots */
#define CV_SEQ_BAD_OFFSET 2 /* state offset < 0 or offset + W-1 > state_cols */
#define CV_SEQ_BAD_ACCEPT 4 /* accept count outside 1..T (commit only) */
#define CV_SEQ_TIMEOUT 8    /* a bounded wait for a bulk copy gave up: the sequence may be partly
                               written (every sequence whose data the block had not finished) */
#define CV_SEQ_BAD_SPAN 16  /* prefill: token span invalid or longer than max_seqlen; packed
                               verify / commit: draft span invalid or longer than T */
#define CV_SEQ_BAD_TREE 32  /* tree verify: a draft token's parent outside [-1, t); cache_compact: a path that does not
                               rise, or leaves the drafts */
#define CV_SEQ_BAD_LENGTH 64    /* paged cache: a length < 0, or past what the page table row (or the held pages) can hold */
#define CV_SEQ_BAD_PAGE 128     /* paged cache: a page outside [0, n_pages) where the call needs one */
#define CV_SEQ_BAD_TOKEN 256    /* draft_verify: a draft token outside [0, vocab) */
#define CV_SEQ_BAD_PROBS 512    /* draft_verify: the weights to sample from add up to 0, or to 4 and more */
#define CV_SEQ_NO_PAGES 1024    /* cache_reserve, cache_fork: not enough free pages */
#define CV_SEQ_BAD_POSITION 2048 /* qk_norm_rope: a position outside the table of angles */
#define CV_SEQ_SHARED_PAGE 4096 /* qk_norm_rope, cache_compact: a page to be written that more than one slot holds (with refs) */

/*
 * cv_conv_verify -- [atlas-batched] fused multi-token verify, batched over sequences.
 *
 * For every sequence s with slot = cache_idx ? cache_idx[s] : s and slot >= 0, and every channel
 * c, let o = state_off ? state_off[s] : 0 and
 *     full = [conv_state[slot][c][o .. o+W-2], x[s][0][c], ..., x[s][T-1][c]]     (W-1+T values)
 * Then for every token t:
 *     acc   = bias[c] (or 0) + sum_{j=0}^{W-1} weight[c][j] * full[t+j]   fp32, bias first, taps in
 *                                                                         order, each product
 *                                                                         rounded (exact for bf16)
 *     y     = acc / (1 + exp(-acc))                                      SiLU [kda-mod]
 *     for c < qk_channels: y *= 1/sqrt(sum over c's head_dim group of y^2 + l2_eps)   [kda-mod]
 *     out[s][t][c] = y rounded once to dtype
 *                    (SiLU and the normalisation use fast hardware approximations: the outputs
 *                    match the exact expressions to within 1e-5 relative (+1e-7) in fp32 and
 *                    2 ulp in bf16, and are identical for every launch path and batch split)
 *     snapshot (s, t, c, k) = full[t+1+k], k < W-1      raw bit copy, dense or dedup layout
 * and finally conv_state[slot][c][0 .. W-2] = full[T .. T+W-2] (the committed window, equal to
 * snapshot T-1); state columns >= W-1 keep their values (packed rows wider than the window may be
 * written back whole with those columns' own bits, so nothing else may write them during the
 * call).  In the CV_WINDOW_HISTORY layout the
 * snapshots go into the state row instead (columns [0, T+W-2), see the layout) and no window
 * buffer is written; in the CV_WINDOW_RECOMPUTE layout neither snapshots nor the state are
 * written.  A sequence with slot < 0 is padding: its
 * out rows, window rows and every state slot are left untouched ([sglang-46184]).
 *
 * Arguments (all in cv_verify_args):
 *   n_seq, T, dim      sequences (0 = nothing to do), draft tokens 1..CV_MAX_T, channels >= 1
 *   width              conv width W in 2..4 (the window is held in registers)
 *   qk_channels        leading channels that are L2-normalised (0 = none); multiple of head_dim
 *   head_dim           L2 group size when qk_channels > 0: power of two, 8..256
 *   dtype              cv_dtype of x, out, weight and bias (and of conv_state and window unless
 *                      state_dtype says otherwise)
 *   l2_eps             added to the group's sum of squares inside the square root
 *   x                  [n_seq][T][dim] read-only; element (s,t,c) at s*x_seq_stride + t*x_tok_stride + c
 *                      (x may be a strided slice of a wider projection output)
 *   out                [n_seq][T][dim] write-only; (s,t,c) at s*out_seq_stride + t*out_tok_stride + c
 *   conv_state         [n_slots][dim][state_cols] read-modify-write in place;
 *                      (slot,c,k) at slot*state_slot_stride + c*state_ch_stride + k*state_col_stride
 *                      (state_col_stride 0 or 1: columns contiguous, state_ch_stride >= state_cols;
 *                      else only in CV_WINDOW_HISTORY, with state_ch_stride == 1 and
 *                      state_col_stride >= dim: column-major rows, else CV_ERR_STRIDE /
 *                      CV_ERR_LAYOUT)
 *   cache_idx          int32 [n_seq] device array or NULL (slot = s); negative = padded sequence
 *   state_off          int32 [n_seq] device array or NULL (0): column where the committed window is
 *                      read, the num_accept_tokens offset of [sglang-46184]
 *   weight             [dim][W] contiguous, read-only; weight[c][W-1] multiplies the newest input
 *   bias               [dim] read-only, or NULL
 *   window             snapshot buffer, write-only, laid out as window_layout says (NULL allowed
 *                      and ignored for CV_WINDOW_HISTORY and CV_WINDOW_RECOMPUTE)
 *   err                int32 [n_seq] device array or NULL: receives the CV_SEQ_* bits of each
 *                      sequence (0 for fine and for padded sequences).  On the pipelined path the
 *                      library clears it (an asynchronous memset on `stream`) before the kernel ORs
 *                      the bits in, since several blocks report for one sequence.
 *   wait_polls         limit of each unit's first wait for its bulk copies on the pipelined path
 *                      (path 3): 0 = the default (2^20 polls of mbarrier.try_wait, far beyond any
 *                      copy's latency), n > 0 = n polls, negative = no poll at all, so the wait
 *                      gives up at once.  Nonzero values exist to exercise the timeout path: the
 *                      block flags CV_SEQ_TIMEOUT for the unit's sequence and for those of every
 *                      later unit it owns, waits (with the default limit) for the copies it has in
 *                      flight, and returns; the other sequences are computed as usual.  Other paths
 *                      ignore it.
 *   state_dtype        CV_STATE_SAME, or the other dtype for conv_state and window (mixed dtypes,
 *                      [sglang-46184] "Accuracy Tests"): inputs are widened exactly for the
 *                      arithmetic; snapshots and state receive x converted to the state dtype
 *                      (exact widening bf16 -> fp32, or round to nearest even fp32 -> bf16 with any
 *                      NaN becoming the quiet NaN 0x7fc0).  Mixed calls take the pipelined kernel
 *                      (path 3) for T <= 8 with packed buffers, the general kernel otherwise.
 *   parent             int32 [n_seq][T] device array (row-major, contiguous) or NULL (a chain):
 *                      tree verify ([sglang-46184] "Scope": tree verify keeps dense windows).  Token
 *                      t's parent p in [-1, t) (-1: the committed window); its conv sees the
 *                      parent's window followed by x_t, and snapshot t is window(t) =
 *                      [window(p)[1 .. W-2], x_t].  The state is left on window(T-1).  The commit
 *                      restores the accepted path's last node: accept_len = its index + 1.  Needs
 *                      the dense layout and one dtype; a parent outside [-1, t) flags
 *                      CV_SEQ_BAD_TREE.
 *   cu_draft           int32 [n_seq + 1] device array or NULL: packed ragged drafts ([sglang-46184]
 *                      "Related upstream work": target verify on packed ragged tokens, the tile
 *                      store covering the packed rows).  Sequence s then owns rows
 *                      [cu_draft[s], cu_draft[s+1]) of x and out -- row r at r*x_tok_stride and
 *                      r*out_tok_stride; x_seq_stride and out_seq_stride are ignored -- and its T_s
 *                      rows are verified exactly as a verify of T_s tokens: T_s outputs, snapshots
 *                      t < T_s (dense steps >= T_s and dedup columns >= T_s+W-2 are not written),
 *                      and the state left on full[T_s .. T_s+W-2].  T is the largest T_s and sizes
 *                      the window buffer (dense [n_seq][T][dim][W-1], dedup [n_seq][dim][T+W-2],
 *                      history rows >= T+W-2).  T_s = 0 writes no output and no snapshot (the
 *                      state receives the committed window; in the history layout nothing is
 *                      written).  A span that is reversed, leaves [0, total_tokens) or holds more
 *                      than T rows flags CV_SEQ_BAD_SPAN and leaves the sequence untouched.  Chains
 *                      only: cu_draft with parent is CV_ERR_LAYOUT.  With packed 16-byte-aligned
 *                      buffers the pipelined kernel runs it (one dtype), otherwise the general one.
 *   total_tokens       rows of x and out with cu_draft (>= 0); x and out may be NULL when it is 0
 * Preconditions the library cannot check: distinct sequences use distinct slots; out and window do
 * not overlap themselves, each other, x, conv_state or weight.
 * Returns CV_OK after the launch is queued, or a negative CV_ERR_* code with nothing launched.
 */
typedef struct cv_verify_args {
    int32_t n_seq, T, dim, width, qk_channels, head_dim;
    int32_t dtype; /* cv_dtype */
    float l2_eps;
    const void *x;
    int64_t x_seq_stride, x_tok_stride;
    void *out;
    int64_t out_seq_stride, out_tok_stride;
    void *conv_state;
    int32_t n_slots, state_cols;
    int64_t state_slot_stride, state_ch_stride;
    const int32_t *cache_idx;
    const int32_t *state_off;
    const void *weight;
    const void *bias;
    void *window;
    int32_t window_layout; /* cv_window_layout */
    int32_t wait_polls;    /* limit of the bounded waits (see above); 0 = the default */
    int64_t win_seq_stride, win_step_stride, win_ch_stride, win_col_stride;
    int32_t *err;
    int32_t state_dtype; /* CV_STATE_* */
    const int32_t *parent;
    const int32_t *cu_draft; /* packed ragged drafts: int32 [n_seq + 1] device array, or NULL */
    int32_t total_tokens;    /* rows of x and out when cu_draft is given */
    int64_t state_col_stride; /* conv_state column stride; 0 or 1 = columns contiguous */
} cv_verify_args;

CV_API int cv_conv_verify(const cv_verify_args *args, void *stream);

/*
 * cv_conv_commit -- restore the state of the accepted prefix ([sglang-46184] "Motivation": the
 * window exists so the state can be rolled back to the accepted prefix; [kda-mod] decode_k:
 * snapshot t is the state after row t, which a partial accept rewinds to).
 *
 * For every sequence s with slot = cache_idx ? cache_idx[s] : s, slot >= 0, and a = accept_len[s]
 * read on the device (no host round trip), 1 <= a <= T:
 *     conv_state[slot][c][k] = snapshot (s, a-1, c, k)      for every c < dim, k < W-1
 * a = T rewrites the state with the value it already holds.  State columns >= W-1 keep their
 * values (packed rows wider than the window may be written back whole with those columns' own
 * bits, so nothing else may write them during the call).  A sequence whose a is out of range
 * gets CV_SEQ_BAD_ACCEPT in err[s] and is untouched.  Packed deduplicated rows are staged by a
 * bulk copy per block with a bounded wait (wait_polls, as in cv_verify_args; a timeout flags
 * CV_SEQ_TIMEOUT and leaves the block's channels unwritten); that kernel ORs its bits into err,
 * which the library clears first with an asynchronous memset on `stream`.  Rows laid out
 * transposed (win_ch_stride = 1, 16-byte-aligned columns) are read by plain loads of the accepted
 * columns alone.  The window must be the one the matching
 * cv_conv_verify wrote (same layout and strides).
 *
 * CV_WINDOW_RECOMPUTE: there is no window; x (with x_seq_stride, x_tok_stride, channel stride 1)
 * must be the input of the matching verify, unchanged since, and the state still holds the
 * pre-verify window in columns [0, W-1) (the verify leaves it alone in this layout).  With
 * full = [conv_state[slot][c][0 .. W-2], x[s][0][c] .. x[s][T-1][c]], the commit sets
 * conv_state[slot][c][k] = full[a+k] for k < W-1; each state row is read before it is written.
 * With cu_draft (the matching verify's packed spans) the accept count of sequence s must lie in
 * 1..T_s, an invalid span flags CV_SEQ_BAD_SPAN, and a sequence with T_s = 0 has nothing to commit
 * (skipped, err 0); in the recompute layout its x rows start at row cu_draft[s] (x_tok_stride;
 * total_tokens rows).
 * CV_WINDOW_HISTORY has nothing to commit and returns CV_ERR_LAYOUT.  dtype here is the dtype of
 * conv_state and window (with mixed dtypes, the state's); the recompute layout needs x in it too.
 */
typedef struct cv_commit_args {
    int32_t n_seq, T, dim, width;
    int32_t dtype; /* cv_dtype */
    int32_t n_slots;
    void *conv_state;
    int64_t state_slot_stride, state_ch_stride;
    int32_t state_cols;
    int32_t window_layout; /* cv_window_layout */
    const int32_t *cache_idx;
    const void *window;
    int64_t win_seq_stride, win_step_stride, win_ch_stride, win_col_stride;
    const int32_t *accept_len; /* int32 [n_seq] device array, required */
    int32_t *err;              /* int32 [n_seq] device array or NULL */
    /* CV_WINDOW_RECOMPUTE only (ignored otherwise): the verify's input [n_seq][T][dim] */
    const void *x;
    int64_t x_seq_stride, x_tok_stride;
    const int32_t *cu_draft; /* the matching verify's packed draft spans, or NULL */
    int32_t total_tokens;    /* rows of x (recompute layout) when cu_draft is given */
    int32_t wait_polls;      /* limit of the packed-dedup commit's bounded wait, as in cv_verify_args */
} cv_commit_args;

CV_API int cv_conv_commit(const cv_commit_args *args, void *stream);

/*
 * cv_conv_prefill -- the conv over whole prompts, packed back to back ([kda-mod], the layer's
 * prefill path: conv + SiLU over every prompt token, then the L2 normalisation of q|k).
 *
 * Sequence s owns tokens [cu_seqlens[s], cu_seqlens[s+1]) of x and out (L = its length, 0
 * allowed).  With slot = cache_idx ? cache_idx[s] : s and slot >= 0, for every channel c:
 *     full = [w0, x[cu_seqlens[s]][c], ..., x[cu_seqlens[s]+L-1][c]]      (W-1+L values)
 * where w0 = conv_state[slot][c][0 .. W-2] if has_initial_state[s] (or has_initial_state is
 * NULL), else W-1 zeros.  Token t's output is computed exactly as cv_conv_verify's output for
 * token t (conv, SiLU, the L2 normalisation of the q|k groups applied to the fp32 values, one
 * rounding), and afterwards conv_state[slot][c][0 .. W-2] = full[L .. L+W-2] (the last W-1
 * inputs, raw bits).  State columns >= W-1 are not touched; a sequence with slot < 0 touches
 * nothing.  Device-side problems go to err[s]: CV_SEQ_BAD_SLOT, or CV_SEQ_BAD_SPAN when the span
 * is reversed, leaves [0, total_tokens) or is longer than max_seqlen; that sequence is untouched.
 *
 * Arguments (all in cv_prefill_args):
 *   n_seq, dim, width, qk_channels, head_dim, dtype, l2_eps   as for cv_conv_verify
 *   total_tokens       rows of x and out (>= 0)
 *   max_seqlen         host-side bound on every L (sizes the grid), >= 0
 *   x                  [total_tokens][dim] read-only; token stride x_tok_stride, channel stride 1
 *   out                [total_tokens][dim] write-only; token stride out_tok_stride, channel stride 1
 *   cu_seqlens         int32 [n_seq + 1] device array (required)
 *   conv_state         [n_slots][dim][state_cols], column stride 1, read-modify-write
 *   cache_idx, has_initial_state, err   int32 [n_seq] device arrays or NULL
 *   weight, bias       [dim][W] and [dim] (bias may be NULL)
 * Returns CV_OK after the launch is queued, or a negative CV_ERR_* code with nothing launched.
 */
typedef struct cv_prefill_args {
    int32_t n_seq, dim, width, qk_channels, head_dim;
    int32_t dtype; /* cv_dtype */
    float l2_eps;
    int32_t total_tokens, max_seqlen;
    const void *x;
    int64_t x_tok_stride;
    void *out;
    int64_t out_tok_stride;
    const int32_t *cu_seqlens;
    void *conv_state;
    int32_t n_slots, state_cols;
    int64_t state_slot_stride, state_ch_stride;
    const int32_t *cache_idx;
    const int32_t *has_initial_state;
    const void *weight;
    const void *bias;
    int32_t *err;
} cv_prefill_args;

CV_API int cv_conv_prefill(const cv_prefill_args *args, void *stream);

/*
 * cv_verify_plan -- validate `args` exactly as cv_conv_verify does and report the launch it would
 * make, without touching the GPU.  grid = (grid_x, grid_y), block = threads, dynamic shared
 * memory = smem_bytes; a unit of work is channels_per_block channels of one sequence (one unit per
 * block, or, on the persistent paths 3 and 5, a stream of units per block).  path says
 * which kernel runs: 3 = persistent pipelined kernel (packed buffers and packed state rows, T a
 * compile-time constant; grid_y = 1 and each block walks (sequence, channel block) units),
 * 1 = packed buffers with T a compile-time constant (T <= 17 for bf16, <= 8 for fp32),
 * 2 = packed buffers, dense window, larger T in chunks of 8 tokens, 0 = the general kernel (any
 * strides), 5 = tree verify (parent given; persistent blocks of one or two warps walk (sequence,
 * 256 channels) units, staging each unit's committed windows, x rows and parents in one of `stages`
 * shared-memory buffers; grid_y = 1).  Host pointer `plan` must not be NULL.  Returns the same status
 * cv_conv_verify would return before launching.
 */
typedef struct cv_launch_plan {
    int32_t grid_x, grid_y, threads, smem_bytes, channels_per_block, path;
    int32_t stages; /* paths 3 and 5: unit buffers per block (loads in flight); 0 otherwise */
    int32_t token_groups; /* path 2: thread groups splitting the draft tokens (the block's y size); 1 otherwise */
} cv_launch_plan;

CV_API int cv_verify_plan(const cv_verify_args *args, cv_launch_plan *plan);

/*
 * Linear attention with a decay for each head, the recurrence that follows the conv in a hybrid
 * layer.  Every value head h keeps a state S [dk][dv] in fp32 and reads the q|k head
 * h * n_qk_heads / n_heads (integer division).  One token does
 *     S   <- exp(g) S + b k v^T         g = log_decay[h], b = gain[h] (1 without gain)
 *     out  = scale * S^T q + skip[h] v  (no last term without skip)
 * with the updated state.  Sums, decays, gains and the state are fp32, and out is rounded once to dtype.
 * g may be -infinity (the state is dropped: exp(g) = 0), it is meant to be <= 0.
 * Precision: cv_linattn_step, and cv_linattn_prefill of fp32 tokens, do every product in fp32.
 * cv_linattn_prefill of bf16 tokens (prompts of more than 8 to 16 tokens, dk and dv multiples of 8 up
 * to 128, 16-byte aligned rows) multiplies on tensor cores, whose operands are bf16: the products q.k with their
 * decays, and the copy of the state that q reads, are rounded to bf16 too (2^-8 of a term; together
 * with the rounding of out 2.3e-3 of the outputs' norm, where that rounding alone leaves 1.7e-3), and the
 * keys that enter the state hold 16 bits (2^-17 of a term, 3e-6 of the state's norm at any
 * length).  On the way its sums are up to 2^80 times what they add to an output, so finite terms
 * |b (q.k) v| above 2^47 may give infinities.  fp32 tokens avoid all of this.
 * Values that are not finite reach what depends on them and nothing else: an output is then a NaN or an
 * infinity as the order of its sums has it, an element of the state what the recurrence leaves.
 *
 * cv_linattn_tokens holds one run of tokens per sequence: T tokens for each of the n_seq sequences
 * (cu NULL; token t of sequence s at s*seq_stride + t*tok_stride) or, with cu (int32 [n_seq + 1]
 * device array), rows [cu[s], cu[s+1]) packed back to back (the seq strides are ignored), at most T
 * of them and all within [0, total_tokens).  Strides are in elements; the innermost stride of q, k
 * and v is 1, and that of log_decay and gain (fp32, [.., n_heads]) is 1 too.  q, k and v may be
 * slices of one conv output row.
 */
typedef struct cv_linattn_tokens {
    int32_t T;            /* tokens per sequence (cu NULL), or the largest count (cu) */
    int32_t total_tokens; /* rows with cu */
    const int32_t *cu;
    const void *q, *k, *v;
    int64_t q_seq_stride, q_tok_stride, q_head_stride;
    int64_t k_seq_stride, k_tok_stride, k_head_stride;
    int64_t v_seq_stride, v_tok_stride, v_head_stride;
    const float *log_decay;
    int64_t decay_seq_stride, decay_tok_stride;
    const float *gain; /* or NULL (1) */
    int64_t gain_seq_stride, gain_tok_stride;
} cv_linattn_tokens;

/*
 * Arguments of cv_linattn_prefill and cv_linattn_step.
 *   n_seq, n_heads, n_qk_heads   sequences 0..65535; value heads 1..4096, a multiple of the q|k heads
 *   dk, dv             1..256: channels of q and k, and of v and out, per head
 *   dtype              cv_dtype of q, k, v and out
 *   tok                the tokens.  prefill: cu is required (prompts packed back to back, any length
 *                      up to T).  step: T is 0..CV_MAX_T; 0 = no tokens (only the commit of prev)
 *   skip               fp32 [n_heads] or NULL
 *   out                write-only, rows as tok's: (s, t, h, c) at s*out_seq_stride (cu: no such term)
 *                      + t*out_tok_stride + h*out_head_stride + c
 *   state              fp32 [n_slots][n_heads][dk][dv], read-modify-write: element (slot, h, i, j) at
 *                      slot*state_slot_stride + h*state_head_stride + i*dv + j
 *   cache_idx          int32 [n_seq] or NULL (slot = s); negative = padded sequence: nothing of it is
 *                      read or written
 *   has_initial_state  int32 [n_seq] or NULL (all have one): 0 starts from a zero state, the slot's
 *                      old content is not read
 *   err                int32 [n_seq] or NULL: CV_SEQ_* bits (0 for fine and padded sequences).  A
 *                      flagged sequence is left untouched (CV_SEQ_TIMEOUT apart: see wait_polls)
 * step only:
 *   prev               the previous step's drafts (q is not read; T = 0: none) and accept_len, int32
 *                      [n_seq], how many of them were accepted, 0..T_s (else CV_SEQ_BAD_ACCEPT): the
 *                      state is first advanced over those tokens and written, then the outputs of tok
 *                      are computed from it
 *   update_state       nonzero: the state is left after all of tok's tokens (decoding).  Zero: the
 *                      outputs only (a verify, committed as prev of the next call)
 * prefill only:
 *   workspace          device buffer of at least the bytes cv_linattn_workspace reports, 256-byte
 *                      aligned; its content means nothing before and after the call.  NULL when 0
 *   wait_polls         limit of each bounded wait of the kernel for bf16 prompts, in polls of up to
 *                      20 us: 0 = the default (65536), negative = none.  A wait that gives up ends
 *                      its block's work and flags CV_SEQ_TIMEOUT for all sequences that the block
 *                      had a part of; their outputs and states may be partly written, unless the
 *                      prompt was cut into pieces and failed in the first pass over them: then the
 *                      sequence is left untouched
 * Preconditions the library cannot check: distinct sequences use distinct slots; out and state do not
 * overlap an input, each other, or the workspace.
 */
typedef struct cv_linattn_args {
    int32_t n_seq, n_heads, n_qk_heads, dk, dv;
    int32_t dtype; /* cv_dtype */
    float scale;
    int32_t n_slots;
    cv_linattn_tokens tok;
    const float *skip;
    void *out;
    int64_t out_seq_stride, out_tok_stride, out_head_stride;
    float *state;
    int64_t state_slot_stride, state_head_stride;
    const int32_t *cache_idx;
    const int32_t *has_initial_state;
    int32_t *err;
    cv_linattn_tokens prev;
    const int32_t *accept_len;
    int32_t update_state;
    int32_t wait_polls; /* prefill: limit of its bounded waits; 0 = the default */
    void *workspace;
    int64_t workspace_bytes;
} cv_linattn_args;

/* cv_linattn_prefill -- outputs of whole prompts and their final states (update_state and prev are
 * ignored; the state is always left after the last token; an empty prompt leaves it, or writes zeros
 * without an initial state). */
CV_API int cv_linattn_prefill(const cv_linattn_args *args, void *stream);

/* cv_linattn_workspace -- validates args as cv_linattn_prefill does (pointers apart) and sets *bytes
 * to the workspace that call needs on the current device (0 = none).  Which kernel runs depends on the
 * alignment of q, k, v, out and state: with those pointers as the call will have them the size
 * is the call's own; where any of them is NULL it is enough for any pointers. */
CV_API int cv_linattn_workspace(const cv_linattn_args *args, int64_t *bytes);

/* cv_linattn_step -- one new token or a run of draft tokens per sequence, after the commit of the
 * previous step's accepted drafts (see prev and update_state).  With T = 0 only the commit runs. */
CV_API int cv_linattn_step(const cv_linattn_args *args, void *stream);

/*
 * cv_block_norm -- the RMS norms around a block, fused with its gate and its scaled residual.  For
 * every row of dim channels, all in fp32 with one rounding per output:
 *     a = y                                      gate act(z) = z*sigmoid(z) or sigmoid(z)
 *     a = a * act(z)                             with a gate and gate_first
 *     a = a / sqrt(mean over its group of a^2 + eps) * post_weight    with group > 0
 *     a = a * act(z)                             with a gate otherwise
 *     without residual:  out = a
 *     with residual:     r = residual + scale * channel_scale * a
 *                        residual_out = r        and, unless out is NULL,
 *                        out = r / sqrt(mean over the row of r^2 + eps) * pre_weight
 *   rows, dim          rows >= 0 (0 = nothing to do), dim 1..65536
 *   group              0 = no first norm, else a divisor of dim (group = dim: one norm over the row);
 *                      a row of more than about 58,000 groups is CV_ERR_SMEM
 *   post_weight        [group] (shared by the groups, needs group > 0) or NULL; pre_weight, channel_scale [dim] or NULL
 *   dtype              cv_dtype of y, gate, out and the weights; residual_dtype that of residual and
 *                      residual_out (dtype, or CV_F32 beside bf16)
 *   *_stride           row strides in elements; channels are contiguous
 * out may be y or gate, and residual_out may be residual, each with equal base and stride (every
 * row is read before it is written); any other overlap is undefined.
 */
enum { CV_GATE_SILU = 0, CV_GATE_SIGMOID = 1 };
typedef struct cv_norm_args {
    int64_t rows;
    int32_t dim, group;
    int32_t dtype, residual_dtype; /* cv_dtype */
    int32_t gate_act, gate_first;  /* CV_GATE_* */
    float eps, scale;
    const void *y;
    int64_t y_stride;
    const void *gate; /* or NULL */
    int64_t gate_stride;
    const void *post_weight;
    const void *residual; /* or NULL */
    int64_t residual_stride;
    void *residual_out;
    int64_t residual_out_stride;
    const void *channel_scale;
    const void *pre_weight;
    void *out;
    int64_t out_stride;
} cv_norm_args;

CV_API int cv_block_norm(const cv_norm_args *args, void *stream);

/*
 * The attention layers of a hybrid model: a cache of K and V in pages, attention of drafted tokens over it, the
 * norms and rotation before it, the acceptance of drafts, and the pages' bookkeeping.
 *
 * cv_cache describes one cache.  Token position x of slot r stands in row x % page_size of page
 * page_table[r][x / page_size].  K and V are [n_layers][n_pages][page_size][n_kv_heads][head_dim], every stride but
 * the innermost (1) free; the layer strides are used by cv_cache_compact and cv_cache_fork alone, the other calls read
 * and write layer 0 (pass the layer's own address).  page_table entries past those a call needs are not read.
 *   held   int32 [n_slots]: pages of each slot (reserve, fork, free; else may be NULL)
 *   refs   int32 [n_pages]: slots that hold each page, 0 = free (reserve, fork, free; else may be NULL).  Where it is given,
 *          cv_qk_norm_rope and cv_cache_compact write into no page that more than one slot holds; without it that is the caller's to see to.
 * Preconditions the library cannot check: distinct sequences of a call use distinct slots, except where a call only reads the cache;
 * calls that change a cache, its table or its counts are ordered with the calls that use them; k and v do not overlap each other or an
 * input.
 * Sizes: n_layers 1..4096, n_pages 1..2^31-1, page_size 1..65536, n_kv_heads 1..4096, head_dim 1..256, n_slots >= 1,
 * max_pages >= 1, max_pages * page_size <= 2^31 - 256 (else CV_ERR_SHAPE; head_dim: CV_ERR_HEAD_DIM).
 */
typedef struct cv_cache {
    void *k, *v;
    int64_t k_layer_stride, k_page_stride, k_row_stride, k_head_stride;
    int64_t v_layer_stride, v_page_stride, v_row_stride, v_head_stride;
    int32_t n_layers, n_pages, page_size, n_kv_heads, head_dim, n_slots, max_pages;
    int32_t dtype; /* cv_dtype of k and v */
    int32_t *page_table;
    int64_t table_stride; /* of its rows, >= max_pages */
    int32_t *held, *refs;
} cv_cache;

/*
 * cv_tree_attention -- attention of T drafted tokens per sequence, a chain or a tree of them, over the cache.  With
 * slot r = cache_idx ? cache_idx[s] : s, L = cache_len[s] and T_s drafts, whose K and V stand at positions L .. L+T_s-1
 * already, every draft t and head h (which reads kv head h * n_kv_heads / n_heads):
 *     w_j = scale * q[t][h] . k_j        for j < L, and for j = L + u with u = t or u an ancestor of t
 *     out[t][h] = sum_j exp(w_j) v_j / sum_j exp(w_j)
 * A draft's parent is in [-1, t) (-1: the cached tokens alone precede it); without parent token t follows t-1 (a
 * causal run: a decoded token with T = 1).  Nothing of any other position reaches an output, whatever stands there.
 * Products and sums are fp32 and out is rounded once; bf16 calls on the tensor cores also round exp(w_j - max) to
 * bf16 (2^-8 of a term at most), as the operand of the second product.
 *   n_seq 0..65535, T 1..CV_MAX_T (the largest T_s), n_heads 1..4096, a multiple of n_kv_heads
 *   q, out             [n_seq][T][n_heads][head_dim], or with cu_draft [total_tokens][n_heads][head_dim]; dtype = the cache's
 *   cu_draft           int32 [n_seq + 1] or NULL; sequence s owns rows [cu_draft[s], cu_draft[s+1]); a row of several sequences (where
 *                      cu_draft falls) receives values of any of them
 *   parent             int32 [n_seq][T], with cu_draft [total_tokens]; or NULL
 *   cache_len          int32 [n_seq]; cache_idx int32 [n_seq] or NULL, negative = padded (nothing is read or written)
 *   err                int32 [n_seq] or NULL: CV_SEQ_BAD_SLOT, _BAD_SPAN, _BAD_LENGTH (L < 0 or L + T_s beyond the table's
 *                      row), also of calls without a row; _BAD_PAGE, _BAD_TREE, _TIMEOUT; a flagged sequence's out is left untouched (after a
 *                      timeout it may be partly written)
 *   workspace          device buffer of at least cv_tree_attention_workspace bytes, 256-byte aligned; its content
 *                      means nothing before and after the call.  NULL when 0
 *   wait_polls         limit of the kernel's bounded waits: 0 = the default, negative = none
 */
typedef struct cv_tree_attention_args {
    int32_t n_seq, T, n_heads, total_tokens;
    float scale;
    int32_t wait_polls;
    cv_cache cache;
    const void *q;
    int64_t q_seq_stride, q_tok_stride, q_head_stride;
    void *out;
    int64_t out_seq_stride, out_tok_stride, out_head_stride;
    const int32_t *cu_draft, *parent, *cache_len, *cache_idx;
    int32_t *err;
    void *workspace;
    int64_t workspace_bytes;
} cv_tree_attention_args;

CV_API int cv_tree_attention(const cv_tree_attention_args *args, void *stream);

/* cv_tree_attention_workspace -- validates args (pointers apart) and sets *bytes to the workspace the call needs on
 * the current device, for q, out, k and v aligned as given (NULL counts as any alignment). */
CV_API int cv_tree_attention_workspace(const cv_tree_attention_args *args, int64_t *bytes);

/*
 * cv_draft_verify -- which drafted tokens stand, and the token after them.  Row t of probs is the target's distribution
 * after draft t.  Token 0 is the last step's token and stands.  From node c = 0 the walk goes on:
 *     children of c: the drafts whose parent is c, in order; one whose token an earlier one of them has is passed over
 *     with draft_probs (a chain only; row t is what token t was drawn from, row 0 is not read): the child stands iff
 *         uniforms[s][c] * draft_probs[child][token] < probs[c][token]
 *     without: a child stands iff uniforms[s][c] < the sum of probs[c][token] over it and the children before it
 *     the first child that stands is the next c; without one the walk ends
 * and the new token is sampled from the weights w at its end:
 *     no child there: probs[c];   with draft_probs: max(probs[c] - draft_probs[child], 0)
 *     without: probs[c], the children's tokens left out;   where all w are 0: probs[c]
 *     new = the lowest token whose cumulative weight exceeds uniforms[s][T] * the sum of w
 * Weights are summed exactly, in units of 2^-60 (values are cut off there, and at 2; what is not above 0, NaN among it,
 * counts as 0).  Comparisons are made in 64 bits, on the values as they are.  A uniform counts as within [0, 1).
 *   n_seq 0..65535, T 1..CV_MAX_T, vocab 1..2^24; dtype of probs and draft_probs, innermost stride 1
 *   tokens             int32 [n_seq][T] (cu_draft: [total_tokens]); parent likewise or NULL (a chain)
 *   uniforms           fp32 [n_seq][T + 1] contiguous
 *   accept_len         int32 [n_seq]: tokens that stand, 1..T_s (cv_conv_commit's and cv_linattn_step's, for a chain)
 *   accept_node        int32 [n_seq] or NULL: 1 + the last one's index (cv_conv_commit's accept_len, for a tree)
 *   path               int32 [n_seq][T] or NULL: their indexes in order, then -1
 *   out_tokens         int32 [n_seq][T]: the tokens after token 0 that stand, the new token, then -1
 *   err                CV_SEQ_BAD_SLOT is not raised (cache_idx only marks padding); _BAD_SPAN (also T_s = 0), _BAD_TREE (token 0 must have
 *                      parent -1), _BAD_TOKEN (tokens 1 .. T_s-1), _BAD_PROBS.  A flagged sequence is left untouched
 */
typedef struct cv_draft_verify_args {
    int32_t n_seq, T, vocab, dtype, total_tokens;
    const void *probs;
    int64_t probs_seq_stride, probs_tok_stride;
    const void *draft_probs;
    int64_t draft_seq_stride, draft_tok_stride;
    const int32_t *tokens, *parent;
    const float *uniforms;
    const int32_t *cu_draft, *cache_idx;
    int32_t *accept_len, *accept_node, *path, *out_tokens, *err;
} cv_draft_verify_args;

CV_API int cv_draft_verify(const cv_draft_verify_args *args, void *stream);

/*
 * cv_qk_norm_rope -- the RMS norm of each query and key head and the rotation of its first rot_dim channels by the
 * token's position, with K and V written into the cache's pages in the same pass.  In fp32, rounded once:
 *     y = x / sqrt(mean over head_dim of x^2 + eps) * weight       (norm != 0; weight NULL: 1;  norm = 0: y = x)
 *     (y[a], y[b]) = (y[a] cos - y[b] sin, y[b] cos + y[a] sin)    pair i: a = i, b = i + rot_dim/2; pairs != 0: a = 2i, b = 2i+1
 * with cos = cos_sin[position][i] and sin = cos_sin[position][rot_dim/2 + i], position = positions of the token, or
 * cache_len[s] + t without them.
 *   tokens             [n_seq][T], or with cu [total_tokens] packed, T then bounds a sequence's length; a row of several sequences (where cu
 *                      falls) goes to each one's cache, and to q_out and k_out for the last of them
 *   q, q_out           .. [n_heads][head_dim] (q_out may be q); k .. [n_kv_heads][head_dim]
 *   k_out              like k, or NULL;  cache (page_table not NULL): K goes to position cache_len[s] + t, and so does v,
 *                      .. [n_kv_heads][head_dim], unrounded, unless NULL.  One of k_out and the cache is needed unless n_kv_heads = 0
 *   cos_sin            fp32 [n_positions][rot_dim], row stride cos_sin_stride; rot_dim even, 0..head_dim (0: NULL)
 *   err                _BAD_SLOT, _BAD_SPAN, _BAD_LENGTH (also of calls without a row): the sequence is left untouched; _BAD_PAGE, _SHARED_PAGE,
 *                      _BAD_POSITION: the tokens concerned are left out
 */
typedef struct cv_qk_norm_rope_args {
    int32_t n_seq, T, n_heads, n_kv_heads, head_dim, dtype, total_tokens, rot_dim, pairs, norm, n_positions;
    float eps;
    const void *q;
    int64_t q_seq_stride, q_tok_stride, q_head_stride;
    void *q_out;
    int64_t q_out_seq_stride, q_out_tok_stride, q_out_head_stride;
    const void *k;
    int64_t k_seq_stride, k_tok_stride, k_head_stride;
    void *k_out;
    int64_t k_out_seq_stride, k_out_tok_stride, k_out_head_stride;
    const void *v;
    int64_t v_seq_stride, v_tok_stride, v_head_stride;
    const void *q_weight, *k_weight;
    const float *cos_sin;
    int64_t cos_sin_stride;
    const int32_t *positions, *cu, *cache_len, *cache_idx;
    cv_cache cache;
    int32_t *err;
} cv_qk_norm_rope_args;

CV_API int cv_qk_norm_rope(const cv_qk_norm_rope_args *args, void *stream);

/*
 * cv_cache_compact -- the accepted path of each sequence moved to its place: rows L + path[s][i] of every layer's K and V
 * go to L + i, i < accept_len[s] (0..T), L = cache_len[s]; new_len[s] = L + accept_len[s] unless NULL (it may not be
 * cache_len).  path int32 [n_seq][T] rises and lies in [0, T).  The pages written must be the slot's alone.
 * err: _BAD_SLOT, _BAD_ACCEPT, _BAD_TREE, _BAD_LENGTH, _BAD_PAGE, _SHARED_PAGE; the sequence is left untouched.
 */
typedef struct cv_cache_compact_args {
    int32_t n_seq, T;
    cv_cache cache;
    const int32_t *cache_len, *path, *accept_len, *cache_idx;
    int32_t *new_len, *err;
} cv_cache_compact_args;

CV_API int cv_cache_compact(const cv_cache_compact_args *args, void *stream);

/*
 * The pages' bookkeeping, on the device.  A page is free while refs is 0; new pages are the free ones with the lowest
 * numbers, given to the call's sequences in order.  n_seq 0..4096.  A slot that an earlier sequence of the same call
 * names too is CV_SEQ_BAD_SLOT (for a fork: as a destination), a negative one is passed over.
 *
 * cv_cache_reserve   slot idx[s] (NULL: s) grows to ceil(n_tokens[s] / page_size) pages if it holds fewer.  The sequences are served in
 *                    order while the free pages last: CV_SEQ_NO_PAGES for the first whose need, added to those before it,
 *                    exceeds them, and for all with a need after it.  With cache_len, positions cache_len[s] .. n_tokens[s] - 1 then
 *                    stand in pages that the slot alone holds: of those that it holds already, one that another slot held too before
 *                    the call is replaced by a new page (before the growth's, in order), with a copy of its rows before
 *                    cache_len[s] (every layer's K and V).  cache_len[s] is at most what the held pages hold (CV_SEQ_BAD_LENGTH).
 * cv_cache_fork      slot idx[s], which holds nothing, gets the first n_tokens[s] tokens of slot src_idx[s]: full pages are
 *                    shared, the rest of a last one is copied into a new page (every layer's K and V).  The sources are
 *                    read as they were before the call: a destination may not be a source too (CV_SEQ_BAD_SLOT).  A source with a page
 *                    that is not there among those tokens' (CV_SEQ_BAD_PAGE) takes no new page.
 * cv_cache_free      slot idx[s] lets go of its pages past those of its first n_tokens[s] tokens (NULL: 0).  Their table
 *                    entries become -1.  A page that it keeps in part may be a shared one: cv_cache_reserve with cache_len makes it the slot's
 *                    own before more tokens are written.
 * err: _BAD_SLOT (also a destination that holds pages), _BAD_LENGTH, _BAD_PAGE, _NO_PAGES; the slot is left as it was.
 */
typedef struct cv_cache_pages_args {
    int32_t n_seq;
    cv_cache cache;
    const int32_t *idx, *src_idx, *n_tokens;
    int32_t *err;
    const int32_t *cache_len; /* reserve: or NULL */
} cv_cache_pages_args;

CV_API int cv_cache_reserve(const cv_cache_pages_args *args, void *stream);
CV_API int cv_cache_fork(const cv_cache_pages_args *args, void *stream);
CV_API int cv_cache_free(const cv_cache_pages_args *args, void *stream);

/* cv_status_string -- a static, NUL-terminated description of a status code (never NULL). */
CV_API const char *cv_status_string(int status);

/* cv_abi_version -- CV_ABI_VERSION of the built library. */
CV_API int cv_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* CONVVERIFY_H */
