// Internal: parameters and kernel tables of the linear-attention kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace cvk {

// One run of tokens per sequence (cv_linattn_tokens).
struct LinattnRun {
    const void *q, *k, *v;
    long long q_seq, q_tok, q_head;
    long long k_seq, k_tok, k_head;
    long long v_seq, v_tok, v_head;
    const float *g;
    long long g_seq, g_tok;
    const float *b;
    long long b_seq, b_tok;
    const int *cu;
    int T, total;
    int vec;  // rows of q, k and v allow loads of 4 elements at multiples of 4 (checked on the host)
    int vec16;  // and of 16 bytes at every multiple of 16 bytes
};

struct LinattnParams {
    LinattnRun tok, prev;
    const float *skip;
    void *out;
    long long o_seq, o_tok, o_head;
    float *state;
    long long st_slot, st_head;
    const int *cache_idx;
    const int *has_init;
    const int *accept;
    int *err;
    int n_seq, n_heads, n_qk, dk, dv, n_slots;
    int bf16;    // dtype of q, k, v and out: bf16, else fp32
    int update;  // leave the state after the tokens
    int o_vec;   // out allows 4 elements at once at multiples of 4 (checked on the host)
    int st_vec;  // state rows allow 16-byte accesses (checked on the host)
    int slices;  // column slices of a head's state, one block each
    // long prompts of few heads: pieces a sequence is cut into (1: whole), their length in tokens, and whether
    // this launch makes the pieces' own states (and decays) instead of outputs
    int pieces, piece_len, own_states;
    float *ws_state;  // [sequence][head][pieces][dk][dv]: the state before each piece of a cut sequence
    float *ws_decay;  // [sequence][head][pieces]: over a piece
    float scale;
    unsigned polls;  // limit of the chunked kernel's waits
};

constexpr int kStepThreads = 256;
constexpr int kStepMaxGroup = 8;  // tokens per pass over the state tile, at most

// Shared memory of linattn_step<VS, R, TG>, in floats: q, k [rows][TG], v [TG][VS], the warps' partial
// outputs [row groups][TG][VS], the token products [TG][TG], the decays and gains [TG] each.
__host__ __device__ constexpr int step_smem_floats(int VS, int R, int TG) {
    return 2 * (R * (kStepThreads / (VS / 4))) * TG + TG * VS + 4 * kStepThreads * TG + TG * TG + 2 * TG;
}

using LinattnKernel = void (*)(LinattnParams);

// The recurrent kernel for slices of VS columns, TG tokens a pass.
struct StepKernel {
    LinattnKernel fn;
    int smem_bytes;
};
// Any alignment; vs: 64 or 32; tg: 1 or kStepMaxGroup; dk <= 256.
StepKernel step_kernel(int vs, int dk, int tg);
// Rows aligned to 16 bytes; blocks of 2, 4 or 8 warps of 16 columns each; dk <= 128; tg: 1 or kStepMaxGroup.
StepKernel stream_kernel(int warps, int dk, int tg, bool bf16);

// Turns the pieces' own states into the states the next pieces start from.
LinattnKernel state_join_kernel();
constexpr int kStateJoinThreads = 128;

// Shared memory of linattn_stream, in bytes from its start: the state tile, two buffers of raw rows (k, q
// and v of TG tokens, each row 16 bytes longer than it is to spread the banks; decays, gains), the products
// of the group's tokens, and the units at hand.
struct StepUnit {
    int s, h, slice, piece;
    int n_tok, row0, n_prev, prow0, status;
    bool on, init, update;
    const float *from;  // the head's state before the unit (init), and after it
    float *to;
};
struct StreamLayout {
    int raw, raw_bytes, products, ring, bytes;
    __host__ __device__ static constexpr int row_bytes(int d, bool bf16) { return d * (bf16 ? 2 : 4) + 16; }
    __host__ __device__ constexpr StreamLayout(int warps, int R, int TG, bool bf16)
        : raw(R * warps * 32 * 16),
          raw_bytes(TG * (2 * row_bytes(8 * R, bf16) + row_bytes(16 * warps, bf16)) + (TG * 8 + 15) / 16 * 16),
          products(raw + 2 * raw_bytes),
          ring((products + TG * TG * 4 + 7) / 8 * 8),
          bytes(ring + 4 * (int)sizeof(StepUnit)) {}
};

// The chunked kernel for prompts (bf16, dk and dv multiples of 8 up to 128).
constexpr int kChunk = 128;            // tokens a chunk
constexpr int kChunkThreads = 768;     // 20 warps of the four large roles, 4 more
constexpr int kChunkMaxSorted = 64;    // sequences whose pieces are counted and taken longest first
constexpr int kStepMaxCounted = 32;    // the same of the recurrent kernel
struct LinattnChunkParams {
    CUtensorMap q_map, k_map, v_map;  // [token][head][channel], boxes of 128 x 1 x 64, 128-byte swizzle
    LinattnParams a;
    int n_segs;      // pieces a sequence is cut into, at most
    int seg_len;     // tokens a piece, a multiple of kChunk
    int units;       // sequences * pieces * heads
    int sort;        // count only the pieces that there are, and take long ones first
    int dv_pad;      // columns of a state in the workspace (64 or 128)
    int state_only;  // the pieces' own states into the workspace, instead of outputs
    float *ws_state;  // [sequence][head][n_segs][dv / 4][128] groups of 4 columns of a state row, before each piece
    float *ws_decay;  // [sequence][head][n_segs]: over a piece
    int *ws_left;     // [sequence]: nonzero where a piece's own state was not made (a wait gave up)
};
constexpr unsigned kPolls = 1u << 16;  // of a wait by default, up to 20 us each
using LinattnChunkKernel = void (*)(LinattnChunkParams);
struct ChunkKernel {
    LinattnChunkKernel fn;
    int smem_bytes;
};
ChunkKernel chunk_kernel(int dv);
// Turns the pieces' own states in the workspace into the states the next pieces start from.
LinattnChunkKernel chunk_join_kernel();
constexpr int kJoinThreads = 128;

}  // namespace cvk
