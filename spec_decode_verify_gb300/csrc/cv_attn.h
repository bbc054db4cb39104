// Internal: parameters and kernel tables of the attention layers' operators (attention over a paged cache, draft
// verification, query and key norms with rotation, the cache's pages).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace cvk {

// A cache in pages; strides in elements.
struct CacheView {
    void *k, *v;
    long long k_layer, k_page, k_row, k_head, v_layer, v_page, v_row, v_head;
    int n_layers, n_pages, page, n_kv, d, n_slots, max_pages;
    int *table;
    long long table_row;
    int *held, *refs;
};

// ---- attention
struct AttnParams {
    int n_seq, T, total, n_heads, G;  // G: query heads of a kv head
    float scale;                      // times log2(e)
    unsigned polls;
    CacheView c;
    const void *q;
    void *out;
    long long q_seq, q_tok, q_head, o_seq, o_tok, o_head;
    const int *cu, *parent, *len, *idx;
    int *err;
    // A unit of work is up to `rows` rows (draft, query head of the group) of one kv head of one sequence over all its keys,
    // in tiles of `keys` of them.  All units' work, in a row, is cut into `parts` equal runs, one a block; a unit's work is its tiles
    // and up to unit_cost more, what its beginning and end take, in tiles.
    int rows, keys, dp, parts, unit_cost;
    int pad;    // rows of a partial result: rows, a multiple of 4
    float *ws;  // two partial results a block, or NULL where no unit can be cut
};
struct AttnMaps {
    AttnParams a;
    CUtensorMap q, k, v;
    int page_rows;   // rows of a copy's box: of a page, at most a tile
    int tok;         // drafts of a row tile
    int o_vec;       // out allows 16-byte accesses
};
constexpr int kSimtRows = 32, kSimtThreads = 256;
constexpr int kFewRows = 8, kFewThreads = 256, kFewKeys = 64;  // rows at most, keys a tile
constexpr int kPartHead = 16;  // ints before a partial's maxima, sums and outputs, each of them 16-byte aligned
__host__ __device__ constexpr long long part_floats(int pad, int dp) { return kPartHead + 2 * pad + (long long)pad * dp; }

using AttnKernel = void (*)(AttnParams);
using AttnTcKernel = void (*)(AttnMaps);
struct AttnSimt {
    AttnKernel fn;
    int smem_bytes, keys;
};
struct AttnTc {
    AttnTcKernel fn;
    int smem_bytes, keys, threads;
};
AttnSimt attn_simt_kernel(bool bf16, int dp, bool vec);
AttnSimt attn_few_kernel(bool bf16, int dp, int rows);  // rows: 4 or 8
AttnTc attn_tc_kernel(int dp, bool two);  // two: units of two row tiles (up to 128 channels)
AttnKernel attn_join_kernel(bool bf16, int dp);
constexpr int kAttnJoinThreads = 256, kAttnJoinY = 4;

// ---- draft verification
struct SampleParams {
    int n_seq, T, vocab, total, cluster;  // cluster: blocks a sequence
    const void *p, *q;
    long long p_seq, p_tok, q_seq, q_tok;
    const int *tok, *parent;
    const float *u;
    const int *cu, *idx;
    int *accept, *node, *path, *out, *err;
};
using SampleKernel = void (*)(SampleParams);
constexpr int kSampleThreads = 384, kSampleBlocks = 4, kSampleCluster = 8;  // threads, blocks an SM, blocks a sequence at most
SampleKernel sample_kernel(bool bf16);

// ---- query and key norms with the rotation
struct RopeParams {
    int n_seq, T, n_heads, n_kv, d, total, rot, pairs, norm, n_pos;
    float eps;
    long long tokens;
    const void *q, *k, *v, *wq, *wk;
    void *q_out, *k_out;
    long long q_seq, q_tok, q_head, qo_seq, qo_tok, qo_head, k_seq, k_tok, k_head, ko_seq, ko_tok, ko_head, v_seq, v_tok, v_head;
    const float *cs;
    long long cs_row;
    const int *pos, *cu, *len, *idx;
    int *err;
    CacheView c;
    int paged;
    int lanes, groups;     // norm_rope: lanes of a group, groups that share a token's heads
    int block_tokens;      // norm_rope_any
};
using RopeKernel = void (*)(RopeParams);
constexpr int kRopeThreads = 256, kRopeTokens = 16;
RopeKernel rope_kernel(bool bf16, bool vec);
int rope_smem(bool bf16);  // of the kernel for 16-byte pieces

// ---- the cache's pages
struct PagesParams {
    int n_seq, T;
    CacheView c;
    const int *idx, *src, *n_tok;          // reserve, fork, free
    const int *len;                        // compact, reserve
    const int *path, *accept;              // compact
    int *new_len, *err;
    int esize, chunks;                     // copies: pieces of a head's row
};
enum { kPagesReserve, kPagesOwn, kPagesFork };  // growth, growth with lengths, forks
using PagesKernel = void (*)(PagesParams);
constexpr int kTakeThreads = 1024, kMaxPageSeqs = 4096, kPagesThreads = 256, kForkCluster = 8;
PagesKernel pages_take_kernel(int op);          // new pages: one block
PagesKernel pages_fork_kernel(int bytes);       // shares and copies; bytes an access
PagesKernel pages_own_kernel(int bytes);        // copies of shared pages that are to be written
PagesKernel pages_free_kernel();
PagesKernel pages_compact_kernel(int bytes);
int pages_take_smem(int n_seq);

}  // namespace cvk
