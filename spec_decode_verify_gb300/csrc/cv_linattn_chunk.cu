// Linear attention with a decay for each head over prompts: chunked form on the tensor cores.
//
// Mathematics.  For a chunk of C = 128 tokens with G_i = sum_{u<=i} g_u and the state S before it,
//   out_i = scale * exp(G_i) ( S^T q_i + sum_{j<=i} A_ij v_j ),      A_ij = exp(-G_j) b_j (q_i . k_j)
//   S'    = exp(G_C) S + K'^T V,                                     K'_j = exp(G_C - G_j) b_j k_j
// so a chunk is five products of 128 x 128 x 128: Q K^T, Q S, A V, and K'^T V twice, because K' is
// written as a high and a low bf16 part (together 16 significant bits).  K'^T V is summed from zero and added
// to S in fp32: the tensor cores cut their sums off towards zero, so products onto S itself lost 5e-7 of
// it a chunk (64 chunks of slow decays: off by 3.1e-5; now 9e-7 to 3e-6 at any length).  A and the copy of S
// that Q S reads are rounded to bf16, as the outputs are.
// exp(-G_j) grows with the decay: a chunk that decays by more than 2^80 takes, block of 32 tokens by
// block, A_ij = scale exp(G_i - G_j) b_j (q_i . k_j) instead: between two blocks from sums over the tokens between i and
// j alone, inside a block from the difference of two sums over the block.  Log decays below -200 count
// as -200 (exp(-200) is 0 in fp32), so after m such tokens in a block these differences are off by up to 2^-16 m in
// log2, a token: with 16 of them 2^-12, and 0.3 % at most over the 15 tokens that are left, about what the
// rounding of A to bf16 does.  The exponents of K' are sums over the tokens after j, so a large decay early in a
// chunk costs later tokens no precision there.
//
// Layout.  A block (one per SM) takes units (sequence, head, piece of its length) and walks each unit's
// chunks; every role below runs the same stream of chunks, so the next unit's loads and products
// start while the last one's outputs are still being written.
//   scores  4 warps, a row a thread: Q K^T from tensor memory, times the decays, back to it as A
//   state   4 warps, a row of S a thread: S times the last chunk's decay plus its K'^T V, both in tensor memory,
//           back there in fp32 and as a bf16 copy to shared memory
//   output  4 warps, a row a thread: out from Q S and A V, rounded, through the dead v tile to memory
//   keys    8 warps, half a token a thread: K' as a high and a low part from the k tile
//   decays  1 warp: sums of the log decays and the weights made of them, ahead of the others
//   load    2 threads: q, k, v tiles by TMA in the 128-byte swizzle, channels past the end zero
//   issue   1 thread: all products, in the order Q K^T, Q S, K'^T V (64 columns after the others, so that the
//           state warps begin the next chunk meanwhile: 311 us, 320 in one), A V
// Shared memory: v in two stages, k, q, both parts of K' and the copy of S once (32 KB each at 128 channels).
// Tensor memory: Q K^T (then A) 128 columns, S and two buffers of dv columns each, which take turns as Q S + A V
// and, between two chunks' outputs, as K'^T V.
//
// Measured: 8 prompts of 1.5k-5.8k tokens, 48 heads of 128 x 128: 317 us, 3.3 TB/s (HBM's floor is 156 us), tensor
// pipe 32 % and issue slots 45 % busy.  A chunk takes 3.6 us of an SM; its products need 1.7 us of the tensor
// pipe.  What bounds it is the longest cycle through the roles, K'^T V -> S -> Q S, and the shared memory that all
// of them read and write: about 600 KB a chunk (the operands of the products 288, tiles in and out 160, K' made of
// k 96, the copy of S 32, the look for NaN in v 32), 2.4 us at 128 bytes a cycle.
//
// Every wait is bounded; one that gives up ends the block's work, flags its sequences and returns.  Where pieces' own
// states were not made, the join notes their sequences and the launch for the outputs leaves those out.
#include "cv_linattn.h"
#include "cv_tcgen05.cuh"

namespace cvk {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinLog2 = -200.0f * kLog2e;
constexpr float kDrop = -150.0f;  // log2 of a decay that is 0 in fp32
constexpr float kNoDecay = -1.0f;  // in the place of a piece's decay (>= 0 or NaN): it was not made
constexpr float kStrong = -80.0f;  // log2 of a chunk's decay from which on A is made block by block
constexpr int kTileQK = kChunk * 256;  // bytes of a q or k tile: two blocks of 64 channels

// Barriers, in order (8 bytes each), then the small arrays.
struct ChunkShared {
    uint64_t v_full[2], v_empty[2];
    uint64_t g_full[2], g_empty[2], out[2], out_free[2];
    uint64_t key_empty, k_full, k_empty, q_full, scores, a_ready, keys, q_used, s_init, s_ready, s_done[2], s_used, last;
    uint32_t tmem;
    int dead;
    // why the chunk's Q S and A V are kept apart: 1 it decays by more than 2^80, 2 its v holds a NaN or inf; and from
    // bit 8 on, in which groups of 8 columns v does.  4, beside 1: a token drops the state.
    int apart[2];
    // The work of sorted launches: first the full pieces, sequence by sequence (first: the number before a
    // sequence's own), then the shorter rests, longest first (order: their sequences).  Uncut, all are rests.
    uint8_t order[kChunkMaxSorted];
    uint16_t first[kChunkMaxSorted + 1];
    int full, units;
    // Of a chunk: each token's sum of log2 decays up to it (over the chunk, or over its block of 32 where the
    // chunk decays by more than 2^80), its weight as a column of A, the blocks' sums, and its weight in K'.
    // Tokens past the end: no decay, no weight.
    alignas(16) float G[2][kChunk];
    alignas(16) float col[2][kChunk];
    alignas(16) float tot[2][4];
    alignas(16) float key[kChunk];
};

static_assert(sizeof(ChunkShared) <= 3072, "what 227 KB leave beside the tiles");

template <int DV>
__host__ __device__ constexpr int chunk_smem_bytes() {
    return 4 * kTileQK + 3 * kChunk * DV * 2 + (int)sizeof(ChunkShared);
}

struct Unit {
    int s, h, hq, seg, slot, row0, n, chunks;
    bool on, init, last;
    bool cut;  // one of several pieces: its state before it is in the workspace
};

__device__ __forceinline__ Unit unit_of(const LinattnChunkParams &p, const ChunkShared *sh, int idx) {
    Unit u;
    const LinattnParams &a = p.a;
    u.h = idx % a.n_heads;
    const int r = idx / a.n_heads;
    if (p.n_segs == 1) {
        u.seg = 0, u.s = p.sort ? sh->order[r] : r;
    } else if (!p.sort) {
        u.seg = r % p.n_segs, u.s = r / p.n_segs;
    } else if (r >= sh->full) {
        u.s = sh->order[r - sh->full];
        u.seg = sh->first[u.s + 1] - sh->first[u.s];
    } else {
        int lo = 0, hi = a.n_seq - 1;  // the last sequence whose first piece is at most r
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (sh->first[mid] <= r) lo = mid;
            else hi = mid - 1;
        }
        u.s = lo, u.seg = r - sh->first[lo];
    }
    u.hq = (int)((unsigned)u.h * (unsigned)a.n_qk / (unsigned)a.n_heads);
    u.slot = a.cache_idx ? __ldg(a.cache_idx + u.s) : u.s;
    int L, row0;
    const int st = draft_span(a.tok.cu, u.s, a.tok.T, a.tok.total, L, row0);
    u.on = u.slot >= 0 && u.slot < a.n_slots && st == 0;
    const long long start = (long long)u.seg * p.seg_len;
    if (u.on && start >= L && u.seg > 0) u.on = false;
    if (u.on && p.state_only && start + p.seg_len >= L) u.on = false;
    if (u.on && !p.state_only && L > p.seg_len && p.ws_left[u.s]) u.on = false;
    u.row0 = row0 + (int)(u.on ? start : 0);
    u.n = u.on ? min(p.seg_len, L - (int)start) : 0;
    u.chunks = (u.n + kChunk - 1) / kChunk;
    u.last = u.on && start + u.n >= L;
    u.cut = u.on && L > p.seg_len;
    u.init = a.has_init ? __ldg(a.has_init + u.s) != 0 : true;
    return u;
}

// The block's n-th unit: -1 none any more, -2 none this time.  Sorted units go out forwards and backwards in
// turn, so a block that got a long one first gets a short one next.  (Packing them into the blocks by their
// lengths, which leaves 4 % between the fullest block and the mean where this leaves 19 %, measured no faster:
// 8 prompts of 1.5k-5.8k tokens, 48 heads, 333 us against 320.)
__device__ __forceinline__ int unit_index(const LinattnChunkParams &p, const ChunkShared *sh, int n) {
    const int G = gridDim.x, b = blockIdx.x;
    const long long idx = (long long)n * G + (p.sort && (n & 1) ? G - 1 - b : b);
    const int units = p.sort ? sh->units : p.units;
    return idx < units ? (int)idx : (long long)n * G < units ? -2 : -1;
}

// The block's bounded waits: polls of one wait, and the flag that one of them has given up.
struct Waits {
    volatile int *dead;
    unsigned polls;
};
// One poll of a barrier's phase, which may suspend the thread for up to 20 us.
__device__ __forceinline__ bool poll(uint64_t *bar, unsigned parity) {
    unsigned done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done != 0;
}
// Whether the phase is over, for the whole warp.
__device__ __forceinline__ bool over(uint64_t *bar, unsigned parity) {
    unsigned done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return __all_sync(0xffffffffu, done != 0);
}
__device__ __noinline__ bool wait_long(uint64_t *bar, unsigned parity, Waits waits) {
#pragma unroll 1
    for (unsigned i = 0; i < waits.polls; ++i) {
        if (__all_sync(0xffffffffu, poll(bar, parity))) return true;
        if (__any_sync(0xffffffffu, *waits.dead)) return false;
    }
    *waits.dead = 1;
    return false;
}
// Bounded wait of a whole warp; false once the block has given up.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, unsigned parity, Waits waits) {
    return over(bar, parity) || wait_long(bar, parity, waits);
}
__device__ __forceinline__ bool wait_one(uint64_t *bar, unsigned parity, Waits waits) {
#pragma unroll 1
    for (unsigned i = 0; i < waits.polls; ++i) {
        if (poll(bar, parity)) return true;
        if (*waits.dead) return false;
    }
    *waits.dead = 1;
    return false;
}
// One arrival for the warp, after all its lanes' earlier work.
__device__ __forceinline__ void arrive_warp(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ float clamp_log2(float g) {
    g *= kLog2e;
    return g < kMinLog2 ? kMinLog2 : g;  // a NaN stays
}

// A box of 64 channels of 128 tokens of one head into shared memory.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int c, int h, int t, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
            dst),
        "l"(map), "r"(c), "r"(h), "r"(t), "r"(smem_u32(bar))
        : "memory");
}

// A NaN or an infinity in v spoils its column for the rows above it in A V (0 * NaN).  This computes 8 columns of
// row i of A V again, over the tokens up to the row itself only, from A in tensor memory: a warp's lanes hold 32 rows of
// v and pass them around (a prompt of 2048 tokens, one head: 52 us, with an infinity in every chunk 60, in every
// column of every chunk 135; with the state mended as well, below, 111 and 263).
__device__ __noinline__ void row_long_way(const LinattnParams &a, long long row0, int rows, int h, uint32_t tp, int i, int c0,
                                          float *o) {
    const uint16_t *const v =
        reinterpret_cast<const uint16_t *>(a.tok.v) + row0 * a.tok.v_tok + (long long)h * a.tok.v_head + c0;
    const int lane = i & 31;
    float sum[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) sum[x] = 0.0f;
#pragma unroll 1
    for (int b = 0; b <= i >> 5; ++b) {
        uint4 mine = make_uint4(0u, 0u, 0u, 0u);
        if (32 * b + lane < rows) mine = __ldg(reinterpret_cast<const uint4 *>(v + (long long)(32 * b + lane) * a.tok.v_tok));
        uint32_t w[16];
        tmem_ld16(w, tp + 16 * b);
        tmem_wait_ld(w);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const uint32_t r[4] = {__shfl_sync(0xffffffffu, mine.x, j), __shfl_sync(0xffffffffu, mine.y, j),
                                   __shfl_sync(0xffffffffu, mine.z, j), __shfl_sync(0xffffffffu, mine.w, j)};
            const float f = __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
            if (32 * b + j <= i) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    sum[2 * x] = fmaf(f, __uint_as_float(r[x] << 16), sum[2 * x]);
                    sum[2 * x + 1] = fmaf(f, __uint_as_float(r[x] & 0xffff0000u), sum[2 * x + 1]);
                }
            }
        }
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) o[x] = sum[x];
}

// Whether one of 8 bf16 values is a NaN or an infinity: its exponent plus one carries into the sign.
__device__ __forceinline__ uint32_t carries(uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; }
__device__ __forceinline__ uint32_t carries(const uint4 &w) { return carries(w.x) | carries(w.y) | carries(w.z) | carries(w.w); }
constexpr uint32_t kCarry = 0x80008000u;

// A bit at `shift` and above for each group of 8 columns in which the warp's rows of a tile of v hold a NaN or inf.
__device__ __noinline__ void note_bad(const unsigned char *vt, int t, int shift, int *apart) {
    int where = 0;
#pragma unroll 1
    for (int x = 0; x < 8; ++x) {
        const uint4 w = *reinterpret_cast<const uint4 *>(vt + swizzled(t, x));
        if (__any_sync(0xffffffffu, carries(w) & kCarry)) where |= 1 << x;
    }
    if ((t & 31) == 0) atomicOr(apart, 2 | where << shift);
}

// An infinity in k, v or the gain leaves a NaN in K'^T V (of two parts of K', or of the zeros past the end of k), where
// the recurrence has an infinity.  Outputs that depend on it are not finite either way.  For the state a
// unit leaves, this goes through its tokens again: an element that is NaN becomes what the
// tokens that are not finite (and those that drop the state) add up to, since no finite one
// changes it.  Piece q of the thread's row, 4 columns from c0 + 4 q on, is at[(q ^ flip) * step].
__device__ __noinline__ void mend_state(const LinattnChunkParams &p, const ChunkShared *sh, int idx, float4 *at, int flip, int step,
                                        int c0, int pieces) {
    const LinattnParams &a = p.a;
    const Unit u = unit_of(p, sh, idx);
    const int r = threadIdx.x & 127, lane = r & 31;
    const float nan = __int_as_float(0x7fffffff);
    unsigned mine[2] = {0u, 0u};  // the columns to mend
    const float *const start = a.state + (long long)u.slot * a.st_slot + (long long)u.h * a.st_head + (long long)r * a.dv;
    const float4 *const cut =
        reinterpret_cast<const float4 *>(p.ws_state) + (((long long)u.s * a.n_heads + u.h) * p.n_segs + u.seg) * (32 * p.dv_pad) + r;
#pragma unroll 1
    for (int q = 0; q < pieces; ++q) {
        const int c = c0 + 4 * q;
        if (r >= a.dk || c >= a.dv) continue;
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);  // the state before the unit
        if (!p.state_only && (u.seg > 0 || u.init)) f = u.cut ? cut[(c >> 2) * 128] : *reinterpret_cast<const float4 *>(start + c);
        float *const x = reinterpret_cast<float *>(at + (q ^ flip) * step);
        const float before[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (isnan(x[e]) && !isnan(before[e])) {
                mine[q >> 3] |= 1u << (4 * (q & 7) + e);
                x[e] = isinf(before[e]) ? before[e] : 0.0f;
            }
    }
    if (!__any_sync(0xffffffffu, mine[0] | mine[1])) return;
    const uint16_t *const k = reinterpret_cast<const uint16_t *>(a.tok.k) + (long long)u.hq * a.tok.k_head;
    const uint16_t *const v = reinterpret_cast<const uint16_t *>(a.tok.v) + (long long)u.h * a.tok.v_head + c0;
#pragma unroll 1
    for (int t = 0; t < u.n; t += 32) {
        const bool in = t + lane < u.n;
        const long long row = (long long)u.row0 + t;
        float decay = 1.0f, gain = 1.0f;
        uint32_t high = 0u;
        if (in) {
            decay = expf(__ldg(a.tok.g + (row + lane) * a.tok.g_tok + u.h));
            if (a.tok.b) gain = __ldg(a.tok.b + (row + lane) * a.tok.b_tok + u.h);
#pragma unroll 4
            for (int x = 0; x < a.dk; x += 8) high |= carries(__ldg(reinterpret_cast<const uint4 *>(k + (row + lane) * a.tok.k_tok + x)));
        }
        const unsigned drop = __ballot_sync(0xffffffffu, !(decay > 0.0f));
        const unsigned all = drop | __ballot_sync(0xffffffffu, (high & kCarry) || !(fabsf(gain) < INFINITY));
#pragma unroll 1
        for (int q = 0; q < pieces && c0 + 4 * q < a.dv; ++q) {
            uint2 w = make_uint2(0u, 0u);
            if (in) w = __ldg(reinterpret_cast<const uint2 *>(v + (row + lane) * a.tok.v_tok + 4 * q));
            unsigned todo = all | __ballot_sync(0xffffffffu, (carries(w.x) | carries(w.y)) & kCarry);
            const unsigned cols = mine[q >> 3] >> (4 * (q & 7)) & 15u;
            float *const x = reinterpret_cast<float *>(at + (q ^ flip) * step);
#pragma unroll 1
            for (; todo; todo &= todo - 1) {
                const int j = __ffs(todo) - 1;
                const uint32_t w0 = __shfl_sync(0xffffffffu, w.x, j), w1 = __shfl_sync(0xffffffffu, w.y, j);
                const float kb = __shfl_sync(0xffffffffu, gain, j) * (r < a.dk ? widen<uint16_t>(__ldg(k + (row + j) * a.tok.k_tok + r)) : 0.0f);
                const float e = __shfl_sync(0xffffffffu, decay, j), f = drop >> j & 1 ? e : 1.0f;
                const float y[4] = {__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xffff0000u), __uint_as_float(w1 << 16),
                                    __uint_as_float(w1 & 0xffff0000u)};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (cols >> i & 1) x[i] = fmaf(f, x[i], kb * y[i]);
            }
        }
    }
#pragma unroll 1
    for (int q = 0; q < pieces; ++q) {  // a NaN of finite tokens (sums past fp32) stays one
        float *const x = reinterpret_cast<float *>(at + (q ^ flip) * step);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if ((mine[q >> 3] >> (4 * (q & 7) + i) & 1) && fabsf(x[i]) < INFINITY) x[i] = nan;
    }
}

// Two elements of k times the weight, as a high and a low bf16 part: off by 2^-17 of a term at most, about 4e-6 of
// the state, which is read for bf16 outputs (2^-9).  A third part would bring it to fp32's own for a sixth product
// and 32 KB of shared memory that are not there.
__device__ __forceinline__ void split(uint32_t k, f2 w2, f2 neg, uint32_t &hi, uint32_t &lo) {
    const f2 f = f2_mul(f2_pack(__uint_as_float(k << 16), __uint_as_float(k & 0xffff0000u)), w2);
    float f0, f1;
    f2_unpack(f, f0, f1);
    hi = pack_bf16(f0, f1);
    f2_unpack(f2_fma(f2_pack(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)), neg, f), f0, f1);
    lo = pack_bf16(f0, f1);
}
// 16 scores of a row times rf * col_j, rounded to bf16 pairs.
template <bool ROW>
__device__ __forceinline__ void weigh(const uint32_t *r, float rf, const float *col, uint32_t *o) {
    const f2 rf2 = f2_pack(rf, rf);
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
        const ulonglong2 c = *reinterpret_cast<const ulonglong2 *>(col + j);
        float f0, f1;
        f2_unpack(f2_mul(f2_pack(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), ROW ? f2_mul(rf2, c.x) : c.x), f0, f1);
        o[j / 2] = pack_bf16(f0, f1);
        f2_unpack(f2_mul(f2_pack(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3])), ROW ? f2_mul(rf2, c.y) : c.y), f0, f1);
        o[j / 2 + 1] = pack_bf16(f0, f1);
    }
}
// The same without a row factor, plus `own` in column `at` (none when it is outside).
__device__ __forceinline__ void weigh_own(const uint32_t *r, const float *col, float own, int at, uint32_t *o) {
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = fmaf(__uint_as_float(r[j]), col[j], j == at ? own : 0.0f);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
}
// Lane i keeps columns up to i - j0 of 16 packed ones (a diagonal block's part right of the diagonal goes).
__device__ __forceinline__ void keep_lower(uint32_t *o, int left) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] &= left > 2 * j ? 0xffffffffu : left == 2 * j ? 0xffffu : 0u;
}
// Row i of A for a chunk that decays by more than 2^80: exponents from the sums between i and j.
template <int DV>
__device__ __noinline__ void scores_strong(const LinattnParams &a, int row0, int rows, int h, const float *Gs, const float *col,
                                           const float *tot, uint32_t tp, int w4, int lane, float skip) {
    const float G = Gs[32 * w4 + lane], t1 = tot[1], t2 = tot[2], scale = a.scale;
    const bool in = 32 * w4 + lane < rows;
    const long long row = row0 + 32 * w4 + lane;
    const float bi = in ? (a.tok.b ? __ldg(a.tok.b + row * a.tok.b_tok + h) : 1.0f) : 0.0f;
    for (int x = 0; x < 8; ++x) {  // 16 columns at a time, ascending: A goes where earlier scores were
        const int J = x >> 1, j0 = 16 * (x & 1);
        uint32_t r[16], o[8];
        if (J > w4) {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = 0u;
        } else {
            tmem_ld16(r, tp + 16 * x);
            tmem_wait_ld(r);
            if (J < w4) {
                const float between = (J < 1 && w4 > 1 ? t1 : 0.0f) + (J < 2 && w4 > 2 ? t2 : 0.0f);
                weigh<true>(r, exp2_fast(G + between) * scale, col + 16 * x, o);
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float Gj = __shfl_sync(0xffffffffu, G, j0 + j), bj = __shfl_sync(0xffffffffu, bi, j0 + j);
                    const float v = __uint_as_float(r[j]) * scale * (exp2_fast(G - Gj) * bj);
                    r[j] = __float_as_uint(j0 + j == lane ? v + skip : v);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = pack_bf16(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
                keep_lower(o, lane - j0);
            }
        }
        tmem_st8(tp + 8 * x, o);
    }
}

template <int DV>
__global__ void __launch_bounds__(kChunkThreads, 1) linattn_chunk(const __grid_constant__ LinattnChunkParams p) {
    constexpr int kTileV = kChunk * DV * 2, kBlock = kChunk * 128;  // a tile's blocks of 64 channels
    constexpr int HALVES = DV / 64;  // of S, by columns
    constexpr uint32_t kColP = 0, kColO = 128, kColS = 128 + 2 * DV, kCols = 512;  // (two buffers of outputs)
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *const k_tile = smem, *const hi_tile = k_tile + kTileQK, *const lo_tile = hi_tile + kTileQK;
    unsigned char *const q_tile = lo_tile + kTileQK, *const v_tile = q_tile + kTileQK;  // v: stage s at + s * its size
    unsigned char *const s_copy = v_tile + 2 * kTileV;
    ChunkShared *const sh = reinterpret_cast<ChunkShared *>(s_copy + kTileV);
    const LinattnParams &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool so = p.state_only;
    // (the skip weight enters A divided by scale, which therefore has to be a number of ordinary size)
    const float strong_at = a.skip && !(fabsf(a.scale) > 1e-4f) ? INFINITY : kStrong;

    // the layout below needs its bytes and the swizzle's alignment
    if (dynamic_smem_bytes() < chunk_smem_bytes<DV>() || (smem_u32(smem) & 1023u) != 0) return;
    if (warp == 23) tmem_alloc(&sh->tmem, kCols);
    if (tid == 0) {
        sh->dead = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->v_full[i], 1);
            mbar_init(&sh->v_empty[i], so ? 1 : 4);
            mbar_init(&sh->out[i], 1);
            mbar_init(&sh->out_free[i], 4);
            mbar_init(&sh->s_done[i], 1);
            mbar_init(&sh->g_full[i], 1);
            mbar_init(&sh->g_empty[i], so ? 4 : 12);
        }
        mbar_init(&sh->key_empty, 8);
        mbar_init(&sh->k_full, 1);
        mbar_init(&sh->k_empty, so ? 8 : 9);
        mbar_init(&sh->q_full, 1);
        mbar_init(&sh->scores, 1);
        mbar_init(&sh->a_ready, 12);
        mbar_init(&sh->keys, 8);
        mbar_init(&sh->q_used, 1);
        mbar_init(&sh->s_init, 4);
        mbar_init(&sh->s_ready, 4);
        mbar_init(&sh->s_used, 4);
        mbar_init(&sh->last, 1);
        mbar_init_fence();
    }
    grid_dep_wait();
    grid_dep_launch();
    if (so)
        for (int s = blockIdx.x * kChunkThreads + tid; s < a.n_seq; s += gridDim.x * kChunkThreads) p.ws_left[s] = 0;
    if (p.sort) {
        // each sequence's full pieces and the length of its rest (-1 none; a sequence without tokens has one of
        // length zero; only pieces with a next one have states of their own)
        int *const fulls = reinterpret_cast<int *>(sh->G), *const rests = reinterpret_cast<int *>(sh->col);
        static_assert(kChunkMaxSorted <= kChunk, "a sequence's counts");
        if (tid < a.n_seq) {
            int L, row0;
            if (draft_span(a.tok.cu, tid, a.tok.T, a.tok.total, L, row0)) L = 0;
            const int f = p.n_segs > 1 ? L / p.seg_len : 0, rest = L - f * p.seg_len;
            fulls[tid] = so && rest == 0 && f > 0 ? f - 1 : f;
            rests[tid] = so || (rest == 0 && L > 0) ? -1 : rest;
        }
        __syncthreads();
        if (tid < a.n_seq) {
            const int rest = rests[tid];
            int before = 0, full = 0, parts = 0, rank = 0;
            for (int i = 0; i < a.n_seq; ++i) {
                const int other = rests[i];
                before += i < tid ? fulls[i] : 0;
                full += fulls[i];
                parts += other >= 0;
                rank += other > rest || (other == rest && i < tid);
            }
            sh->first[tid] = (uint16_t)before;
            if (rest >= 0) sh->order[rank] = (uint8_t)tid;
            if (tid == 0) sh->first[a.n_seq] = (uint16_t)full, sh->full = full, sh->units = (full + parts) * a.n_heads;
        }
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tm = sh->tmem;
    const Waits waits{&sh->dead, a.polls};
    const int role = warp >> 2;
    const int w4 = warp & 3;  // the quarter of tensor memory this warp reaches
    const uint32_t tl = tm + ((uint32_t)(32 * w4) << 16);

    int it = 0;  // chunks of the stream so far
    if (warp == 20) {
        // ---------------------------------------------------------------------------- decays
        bool ok = true;
        for (int n = 0, idx; ok && (idx = unit_index(p, sh, n)) != -1; ++n) {
            if (idx < 0) continue;
            const Unit u = unit_of(p, sh, idx);
            if (a.err && u.h == 0 && u.seg == 0 && lane == 0 && u.slot >= 0) {
                int L, row0;
                const int st = (u.slot >= a.n_slots ? 1 : 0) | draft_span(a.tok.cu, u.s, a.tok.T, a.tok.total, L, row0);
                if (st) atomicOr(a.err + u.s, st);
            }
            for (int c = 0; c < u.chunks; ++c, ++it) {
                const int rows = u.n - c * kChunk;
                const long long row = u.row0 + c * kChunk;
                // four tokens a lane, a block of 32 in 8 lanes
                float g[4], b[4], G[4], after[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int t = 4 * lane + x;
                    g[x] = t < rows ? __ldg(a.tok.g + (row + t) * a.tok.g_tok + u.h) : 0.0f;
                    b[x] = t < rows ? (a.tok.b ? __ldg(a.tok.b + (row + t) * a.tok.b_tok + u.h) : 1.0f) : 0.0f;
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) g[x] = clamp_log2(g[x]);
                G[0] = g[0], G[1] = G[0] + g[1], G[2] = G[1] + g[2], G[3] = G[2] + g[3];
                after[3] = 0.0f, after[2] = g[3], after[1] = g[3] + g[2], after[0] = after[1] + g[1];
                float up = G[3], down = G[3];  // of this lane and those before (after) it in the block
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) {
                    const float x = __shfl_up_sync(0xffffffffu, up, o, 8), y = __shfl_down_sync(0xffffffffu, down, o, 8);
                    if ((lane & 7) >= o) up += x;
                    if ((lane & 7) + o < 8) down += y;
                }
                float before = __shfl_up_sync(0xffffffffu, up, 1, 8), later = __shfl_down_sync(0xffffffffu, down, 1, 8);
                if ((lane & 7) == 0) before = 0.0f;
                if ((lane & 7) == 7) later = 0.0f;
                const float t0 = __shfl_sync(0xffffffffu, up, 7), t1 = __shfl_sync(0xffffffffu, up, 15),
                            t2 = __shfl_sync(0xffffffffu, up, 23), t3 = __shfl_sync(0xffffffffu, up, 31);
                const int block = lane >> 3;
                const bool strong = !((t0 + t1) + (t2 + t3) > strong_at);
                if (!strong) before += (block > 0 ? t0 : 0.0f) + (block > 1 ? t1 : 0.0f) + (block > 2 ? t2 : 0.0f);
                const float ahead = (block < 1 ? t1 : 0.0f) + (block < 2 ? t2 : 0.0f) + (block < 3 ? t3 : 0.0f);
                const bool drops = __any_sync(0xffffffffu, fminf(fminf(g[0], g[1]), fminf(g[2], g[3])) < kDrop);
                const int stage = it & 1;
                if ((it > 1 && !wait_warp(&sh->g_empty[stage], ((it >> 1) & 1) ^ 1, waits)) ||
                    (it > 0 && !wait_warp(&sh->key_empty, (it - 1) & 1, waits))) {
                    ok = false;
                    break;
                }
                float col[4], key[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    G[x] += before;
                    col[x] = exp2_fast(strong ? after[x] + later : -G[x]) * b[x];
                    key[x] = exp2_fast(after[x] + later + ahead) * b[x];
                }
                *reinterpret_cast<float4 *>(sh->G[stage] + 4 * lane) = make_float4(G[0], G[1], G[2], G[3]);
                *reinterpret_cast<float4 *>(sh->col[stage] + 4 * lane) = make_float4(col[0], col[1], col[2], col[3]);
                *reinterpret_cast<float4 *>(sh->key + 4 * lane) = make_float4(key[0], key[1], key[2], key[3]);
                if (lane == 0) {
                    *reinterpret_cast<float4 *>(sh->tot[stage]) = make_float4(t0, t1, t2, t3);
                    sh->apart[stage] = strong | (drops ? 4 : 0);
                }
                arrive_warp(&sh->g_full[stage]);
            }
        }
    } else if (warp == 21 && lane == 0) {
        // ---------------------------------------------------------------------- load: k and q
        bool ok = true;
        int k_sent = 0, q_sent = 0;
        for (int n = 0, idx; ok && (idx = unit_index(p, sh, n)) != -1; ++n) {
            if (idx < 0) continue;
            const Unit u = unit_of(p, sh, idx);
            for (int c = 0; c < u.chunks; ++c, ++it) {
                const int row = u.row0 + c * kChunk;
                if (it >= 1 && !wait_one(&sh->k_empty, (it - 1) & 1, waits)) {
                    ok = false;
                    break;
                }
                const uint32_t k = smem_u32(k_tile);
                mbar_arrive_expect_tx(&sh->k_full, kTileQK);
                tma_load(k, &p.k_map, 0, u.hq, row, &sh->k_full);
                tma_load(k + kBlock, &p.k_map, 64, u.hq, row, &sh->k_full);
                ++k_sent;
                if (!so) {
                    if (it >= 1 && !wait_one(&sh->q_used, (it - 1) & 1, waits)) {
                        ok = false;
                        break;
                    }
                    const uint32_t q = smem_u32(q_tile);
                    mbar_arrive_expect_tx(&sh->q_full, kTileQK);
                    tma_load(q, &p.q_map, 0, u.hq, row, &sh->q_full);
                    tma_load(q + kBlock, &p.q_map, 64, u.hq, row, &sh->q_full);
                    ++q_sent;
                }
            }
        }
        // nothing of the block's is in flight when it returns
        if (k_sent > 0) mbar_wait_bounded(&sh->k_full, (k_sent - 1) & 1, kPolls);
        if (q_sent > 0) mbar_wait_bounded(&sh->q_full, (q_sent - 1) & 1, kPolls);
    } else if (warp == 23 && lane == 0) {
        // --------------------------------------------------------------------------- load: v
        bool ok = true;
        int sent = 0;
        for (int n = 0, idx; ok && (idx = unit_index(p, sh, n)) != -1; ++n) {
            if (idx < 0) continue;
            const Unit u = unit_of(p, sh, idx);
            // the unit's first state, into L2 before the state warps come to it
            if (u.on && !so && (u.seg > 0 || u.init)) {
                const float *const st =
                    u.cut ? p.ws_state + (((long long)u.s * a.n_heads + u.h) * p.n_segs + u.seg) * (kChunk * DV)
                          : a.state + (long long)u.slot * a.st_slot + (long long)u.h * a.st_head;
                bulk_prefetch_l2(st, (unsigned)(u.cut ? kChunk * DV : a.dk * a.dv) * 4);
            }
            for (int c = 0; c < u.chunks; ++c, ++it) {
                const int stage = it & 1, row = u.row0 + c * kChunk;
                if (it >= 2 && !wait_one(&sh->v_empty[stage], ((it >> 1) & 1) ^ 1, waits)) {
                    ok = false;
                    break;
                }
                const uint32_t v = smem_u32(v_tile + stage * kTileV);
                mbar_arrive_expect_tx(&sh->v_full[stage], kTileV);
                tma_load(v, &p.v_map, 0, u.h, row, &sh->v_full[stage]);
                if (DV == 128) tma_load(v + kBlock, &p.v_map, 64, u.h, row, &sh->v_full[stage]);
                ++sent;
            }
        }
        for (int x = max(0, sent - 2); x < sent; ++x) mbar_wait_bounded(&sh->v_full[x & 1], (x >> 1) & 1, kPolls);
    } else if (role == 0 && !so) {
        // ---------------------------------------------------------------------------- scores
        bool ok = true;
        const uint32_t tp = tl + kColP;
        for (int n = 0, idx; ok && (idx = unit_index(p, sh, n)) != -1; ++n) {
            if (idx < 0) continue;
            const Unit u = unit_of(p, sh, idx);
            const float skip = a.skip ? __ldg(a.skip + u.h) : 0.0f;
            for (int c = 0; c < u.chunks; ++c, ++it) {
                const int stage = it & 1;
                if (!wait_warp(&sh->g_full[stage], (it >> 1) & 1, waits) || !wait_warp(&sh->scores, it & 1, waits)) {
                    ok = false;
                    break;
                }
                tmem_fence_after();
                const float4 bt = *reinterpret_cast<const float4 *>(sh->tot[stage]);
                if ((bt.x + bt.y) + (bt.z + bt.w) > strong_at) {
                    // A overlays the scores: 16 columns go where earlier ones were read.  With skip, A_ii holds
                    // skip / (scale exp(G_i)) too.
                    const float own = a.skip ? skip / a.scale * exp2_fast(-sh->G[stage][32 * w4 + lane]) : 0.0f;
                    uint32_t r[16], o[8];
                    int x = 0;
#pragma unroll 1
                    for (; x < 2 * w4 + 2; ++x) {
                        tmem_ld16(r, tp + 16 * x);
                        const int left = 32 * w4 + lane - 16 * x;  // the row's own column among these
                        tmem_wait_ld(r);
                        if (a.skip)
                            weigh_own(r, sh->col[stage] + 16 * x, own, left, o);
                        else
                            weigh<false>(r, 1.0f, sh->col[stage] + 16 * x, o);
                        if (x >= 2 * w4) keep_lower(o, left);
                        tmem_st8(tp + 8 * x, o);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = 0u;
#pragma unroll 1
                    for (; x < 8; ++x) tmem_st8(tp + 8 * x, o);
                } else {
                    scores_strong<DV>(a, u.row0 + c * kChunk, u.n - c * kChunk, u.h, sh->G[stage], sh->col[stage], sh->tot[stage], tp, w4, lane, skip);
                }
                tmem_wait_st();
                tmem_fence_before();
                arrive_warp(&sh->a_ready);
                arrive_warp(&sh->g_empty[stage]);
            }
        }
    } else if (role == 1) {
        // ----------------------------------------------------------------------------- state
        const int r = 32 * w4 + lane;  // the row of S
        const uint32_t ts = tl + kColS;
        // rows of this warp through its quarter of the copy's shared memory, 64 columns at a time
        float4 *const mine = reinterpret_cast<float4 *>(s_copy + w4 * (kTileV / 4));
        constexpr int PW = DV / 8;           // float4 pieces of a row per pass: the quarter holds 32 rows of them
        constexpr int PASSES = DV / 4 / PW;  // 2
        bool ok = true;
        int units = 0;
        for (int n = 0, idx; ok && (idx = unit_index(p, sh, n)) != -1; ++n) {
            if (idx < 0) continue;
            const Unit u = unit_of(p, sh, idx);
            if (!u.on) continue;
            float *const st = a.state + (long long)u.slot * a.st_slot + (long long)u.h * a.st_head;
            const long long wsi = ((long long)u.s * a.n_heads + u.h) * p.n_segs;
            if (u.chunks == 0) {  // an empty prompt: zeros without an initial state
                if (!u.init && r < a.dk)
                    for (int j = 0; j < a.dv; j += 4)
                        *reinterpret_cast<float4 *>(st + (long long)r * a.dv + j) = make_float4(0.f, 0.f, 0.f, 0.f);
                continue;
            }
            // the state before the unit
            const bool zero = so ? true : u.seg == 0 && !u.init;
            if (zero || u.cut) {
                const float4 *src = reinterpret_cast<const float4 *>(p.ws_state) + (wsi + u.seg) * (32 * DV);
#pragma unroll 1
                for (int j = 0; j < DV; j += 16) {
                    uint32_t v[16];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float4 f = zero ? make_float4(0.f, 0.f, 0.f, 0.f) : src[(j / 4 + x) * 128 + r];
                        v[4 * x] = __float_as_uint(f.x), v[4 * x + 1] = __float_as_uint(f.y);
                        v[4 * x + 2] = __float_as_uint(f.z), v[4 * x + 3] = __float_as_uint(f.w);
                    }
                    tmem_st16(ts + j, v);
                }
            } else {
#pragma unroll 1
                for (int h = 0; h < PASSES; ++h) {
                    __syncwarp();
#pragma unroll 4
                    for (int e = lane; e < 32 * PW; e += 32) {
                        const int row = e / PW, q = e % PW, col = (h * PW + q) * 4;
                        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (32 * w4 + row < a.dk && col < a.dv)
                            f = *reinterpret_cast<const float4 *>(st + (long long)(32 * w4 + row) * a.dv + col);
                        mine[row * PW + (q ^ (row & 7))] = f;
                    }
                    __syncwarp();
#pragma unroll 1
                    for (int j = 0; j < PW; j += 4) {
                        uint32_t v[16];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const float4 f = mine[lane * PW + ((j + x) ^ (lane & 7))];
                            v[4 * x] = __float_as_uint(f.x), v[4 * x + 1] = __float_as_uint(f.y);
                            v[4 * x + 2] = __float_as_uint(f.z), v[4 * x + 3] = __float_as_uint(f.w);
                        }
                        tmem_st16(ts + (h * PW + j) * 4, v);
                    }
                }
                __syncwarp();
            }
            tmem_wait_st();
            // the copy's rows go over every warp's quarter: all are through with theirs first
            arrive_warp(&sh->s_init);
            if (!wait_warp(&sh->s_init, units++ & 1, waits)) break;
            float total = 1.0f, tot = 1.0f;  // decays of the unit so far, and of the last chunk
            bool drops = false;              // some token of the unit drops the state
            // 16 columns of S, and of the last chunk's products where there are any
            auto current = [&](uint32_t *x, int j, bool products) {
                tmem_ld16(x, ts + j);
                if (!products) {
                    tmem_wait_ld(x);
                    return;
                }
                uint32_t y[16];
                tmem_ld16(y, tl + kColO + (it & 1) * DV + j);
                tmem_wait_ld(x);
                tmem_tie(y);
                const f2 tot2 = f2_pack(tot, tot);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    float f0, f1;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), tot2,
                                     f2_pack(__uint_as_float(y[e]), __uint_as_float(y[e + 1]))),
                              f0, f1);
                    x[e] = __float_as_uint(f0), x[e + 1] = __float_as_uint(f1);
                }
            };
            for (int c = 0; c < u.chunks; ++c, ++it) {
                const int stage = it & 1;
                if (!wait_warp(&sh->g_full[stage], (it >> 1) & 1, waits)) {
                    ok = false;
                    break;
                }
                const float4 bt = *reinterpret_cast<const float4 *>(sh->tot[stage]);
                if (so) drops |= (*(volatile int *)&sh->apart[stage] & 4) != 0;
                arrive_warp(&sh->g_empty[stage]);
#pragma unroll 1
                for (int h = 0; h < HALVES; ++h) {
                    // the last chunk's products for this half are done, and the one that read its copy (at a
                    // unit's start they were waited for at the end of the one before)
                    if (c > 0 && !wait_warp(&sh->s_done[h], (it - 1) & 1, waits)) {
                        ok = false;
                        break;
                    }
                    tmem_fence_after();
                    if (so && c == 0) continue;  // (from zero, and nothing reads a copy)
#pragma unroll 1
                    for (int j = h * 64; j < h * 64 + 64; j += 16) {
                        uint32_t x[16];
                        current(x, j, c > 0);
                        if (c > 0) tmem_st16(ts + j, x);
                        if (so) continue;
                        unsigned char *const at = s_copy + (j >> 6) * kBlock;
                        *reinterpret_cast<uint4 *>(at + swizzled(r, (j >> 3) & 7)) =
                            make_uint4(pack_bf16(__uint_as_float(x[0]), __uint_as_float(x[1])),
                                       pack_bf16(__uint_as_float(x[2]), __uint_as_float(x[3])),
                                       pack_bf16(__uint_as_float(x[4]), __uint_as_float(x[5])),
                                       pack_bf16(__uint_as_float(x[6]), __uint_as_float(x[7])));
                        *reinterpret_cast<uint4 *>(at + swizzled(r, ((j >> 3) & 7) + 1)) =
                            make_uint4(pack_bf16(__uint_as_float(x[8]), __uint_as_float(x[9])),
                                       pack_bf16(__uint_as_float(x[10]), __uint_as_float(x[11])),
                                       pack_bf16(__uint_as_float(x[12]), __uint_as_float(x[13])),
                                       pack_bf16(__uint_as_float(x[14]), __uint_as_float(x[15])));
                    }
                }
                if (!ok) break;
                tot = exp2_fast((bt.x + bt.y) + (bt.z + bt.w));
                total *= tot;
                tmem_wait_st();
                tmem_fence_before();
                fence_smem_to_async();
                if (c > 0) arrive_warp(&sh->s_used);
                arrive_warp(&sh->s_ready);
            }
            if (!ok || !wait_warp(&sh->s_done[HALVES - 1], (it - 1) & 1, waits)) {
                ok = false;
                break;
            }
            tmem_fence_after();
            // the state after it
            if (so) {
                float4 *dst = reinterpret_cast<float4 *>(p.ws_state) + (wsi + u.seg + 1) * (32 * DV);
                bool nan = false;
#pragma unroll 1
                for (int j = 0; j < DV; j += 16) {
                    uint32_t v[16];
                    current(v, j, true);
#pragma unroll
                    for (int x = 0; x < 16; ++x) nan |= isnan(__uint_as_float(v[x]));
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        dst[(j / 4 + x) * 128 + r] = make_float4(__uint_as_float(v[4 * x]), __uint_as_float(v[4 * x + 1]),
                                                                 __uint_as_float(v[4 * x + 2]), __uint_as_float(v[4 * x + 3]));
                }
                if (__any_sync(0xffffffffu, nan))
#pragma unroll 1
                    for (int h = 0; h < HALVES; ++h) mend_state(p, sh, idx, dst + h * (16 * 128) + r, 0, 128, 64 * h, 16);
                // (an infinity before the piece stays one, however small its decay, unless a token drops it)
                if (r == 0) p.ws_decay[wsi + u.seg] = total == 0.0f && !drops ? __int_as_float(1) : total;
            } else if (u.last) {
#pragma unroll 1
                for (int h = 0; h < PASSES; ++h) {
                    bool nan = false;
                    __syncwarp();
#pragma unroll 1
                    for (int j = 0; j < PW; j += 4) {
                        uint32_t v[16];
                        current(v, (h * PW + j) * 4, true);
#pragma unroll
                        for (int x = 0; x < 16; ++x) nan |= isnan(__uint_as_float(v[x]));
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            mine[lane * PW + ((j + x) ^ (lane & 7))] =
                                make_float4(__uint_as_float(v[4 * x]), __uint_as_float(v[4 * x + 1]),
                                            __uint_as_float(v[4 * x + 2]), __uint_as_float(v[4 * x + 3]));
                    }
                    if (__any_sync(0xffffffffu, nan)) mend_state(p, sh, idx, mine + lane * PW, lane & 7, 1, h * PW * 4, PW);
                    __syncwarp();
#pragma unroll 4
                    for (int e = lane; e < 32 * PW; e += 32) {
                        const int row = e / PW, q = e % PW, col = (h * PW + q) * 4;
                        if (32 * w4 + row < a.dk && col < a.dv)
                            *reinterpret_cast<float4 *>(st + (long long)(32 * w4 + row) * a.dv + col) =
                                mine[row * PW + (q ^ (row & 7))];
                    }
                }
                __syncwarp();
            }
            tmem_fence_before();
            arrive_warp(&sh->s_used);
        }
    } else if (role == 2 && !so) {
        // ---------------------------------------------------------------------------- output
        const int i = 32 * w4 + lane;  // the row of the chunk
        bool ok = true;
        for (int n = 0, idx; ok && (idx = unit_index(p, sh, n)) != -1; ++n) {
            if (idx < 0) continue;
            const Unit u = unit_of(p, sh, idx);
            for (int c = 0; c < u.chunks; ++c, ++it) {
                const int stage = it & 1;
                if (!wait_warp(&sh->g_full[stage], (it >> 1) & 1, waits)) {
                    ok = false;
                    break;
                }
                // out = pre * (Q S + A V), or pre * (Q S) + post * (A V) where they are kept apart
                const float4 bt = *reinterpret_cast<const float4 *>(sh->tot[stage]);
                float G = sh->G[stage][i];
                const bool strong = !((bt.x + bt.y) + (bt.z + bt.w) > strong_at);
                if (strong) G += (w4 > 0 ? bt.x : 0.0f) + (w4 > 1 ? bt.y : 0.0f) + (w4 > 2 ? bt.z : 0.0f);
                const float pre = exp2_fast(G) * a.scale;
                if (!wait_warp(&sh->out[it & 1], (it >> 1) & 1, waits)) {
                    ok = false;
                    break;
                }
                tmem_fence_after();
                const int bad = *(volatile int *)&sh->apart[stage] >> 1;  // v holds a NaN or inf; from bit 7 on, where
                arrive_warp(&sh->g_empty[stage]);
                const int t0 = c * kChunk;
                unsigned char *const vt = v_tile + stage * kTileV;  // v is used up: the rows go through its tile
                const uint32_t to = tl + kColO + (it & 1) * DV, ta = tl + kColO + (~it & 1) * DV;
                if (!strong && !bad) {
                    const f2 pre2 = f2_pack(pre, pre);
#pragma unroll 2
                    for (int j = 0; j < DV; j += 16) {
                        uint32_t x[16], o[8];
                        tmem_ld16(x, to + j);
                        tmem_wait_ld(x);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float f0, f1;
                            f2_unpack(f2_mul(pre2, f2_pack(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]))), f0, f1);
                            o[e] = pack_bf16(f0, f1);
                        }
                        unsigned char *const at = vt + (j >> 6) * kBlock;
                        *reinterpret_cast<uint4 *>(at + swizzled(i, (j >> 3) & 7)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4 *>(at + swizzled(i, ((j >> 3) & 7) + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                } else {
                    // where a NaN or an infinity in v has spoiled columns of A V: the long way
                    const float post = strong ? 1.0f : pre;
#pragma unroll 1
                    for (int j = 0; j < DV; j += 8) {
                        uint32_t x[8], y[8], o[4];
                        float part[8];
                        tmem_ld8x2(x, y, to + j, ta + j);
                        tmem_wait_ld8x2(x, y);
#pragma unroll
                        for (int e = 0; e < 8; ++e) part[e] = __uint_as_float(y[e]);
                        if (bad >> (7 + j / 8) & 1) row_long_way(a, u.row0 + t0, u.n - t0, u.h, tl + kColP, i, j, part);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = pack_bf16(fmaf(pre, __uint_as_float(x[2 * e]), post * part[2 * e]),
                                             fmaf(pre, __uint_as_float(x[2 * e + 1]), post * part[2 * e + 1]));
                        *reinterpret_cast<uint4 *>(vt + (j >> 6) * kBlock + swizzled(i, (j >> 3) & 7)) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                        __syncwarp();
                    }
                }
                __syncwarp();
                tmem_fence_before();
                arrive_warp(&sh->out_free[it & 1]);
                // whole rows from there to memory, DV * 2 contiguous bytes each
                constexpr int PC = DV / 8, RP = 32 / PC;
                const int pc = lane % PC, r0 = 32 * w4 + lane / PC;
                uint16_t *dst = reinterpret_cast<uint16_t *>(a.out) + (long long)(u.row0 + t0 + r0) * a.o_tok +
                                (long long)u.h * a.o_head + pc * 8;
                const int end = pc * 8 < a.dv ? u.n - t0 : 0;
#pragma unroll 4
                for (int r = r0; r < 32 * w4 + 32; r += RP, dst += RP * a.o_tok) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(vt + (pc >> 3) * kBlock + swizzled(r, pc & 7));
                    if (r < end) *reinterpret_cast<uint4 *>(dst) = v;
                }
                fence_smem_to_async();
                arrive_warp(&sh->v_empty[stage]);
            }
        }
    } else if (role == 3 || role == 4) {
        // ------------------------------------------------------------------------------ keys
        const int t = 32 * w4 + lane, half = role - 3;  // the token, and which 64 of its channels
        bool ok = true;
        for (int n = 0, idx; ok && (idx = unit_index(p, sh, n)) != -1; ++n) {
            if (idx < 0) continue;
            const Unit u = unit_of(p, sh, idx);
            for (int c = 0; c < u.chunks; ++c, ++it) {
                const int stage = it & 1;
                if (!wait_warp(&sh->g_full[stage], (it >> 1) & 1, waits)) {
                    ok = false;
                    break;
                }
                const float w = sh->key[t];
                arrive_warp(&sh->key_empty);
                // K' has its place once the last chunk's products are done (and this role never runs two phases
                // ahead of the issuing warp)
                if (!wait_warp(&sh->k_full, it & 1, waits) || (it > 0 && !wait_warp(&sh->s_done[HALVES - 1], (it - 1) & 1, waits))) {
                    ok = false;
                    break;
                }
                const f2 w2 = f2_pack(w, w), neg = f2_pack(-1.0f, -1.0f);
                const int at = half * kBlock;
                const bool in = t < u.n - c * kChunk;
#pragma unroll 1
                for (int x0 = 0; x0 < 8; x0 += 2) {
                    uint4 k[2], hi[2], lo[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) k[x] = *reinterpret_cast<const uint4 *>(k_tile + at + swizzled(t, x0 + x));
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        split(k[x].x, w2, neg, hi[x].x, lo[x].x);
                        split(k[x].y, w2, neg, hi[x].y, lo[x].y);
                        split(k[x].z, w2, neg, hi[x].z, lo[x].z);
                        split(k[x].w, w2, neg, hi[x].w, lo[x].w);
                        // past the end the tile holds whatever follows the sequence there: zeros instead
                        if (!in) hi[x] = lo[x] = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4 *>(hi_tile + at + swizzled(t, x0 + x)) = hi[x];
                        *reinterpret_cast<uint4 *>(lo_tile + at + swizzled(t, x0 + x)) = lo[x];
                    }
                }
                arrive_warp(&sh->k_empty);
                unsigned char *const vt = v_tile + stage * kTileV + half * kBlock;
                if (half * 64 < DV) {
                    if (!wait_warp(&sh->v_full[stage], (it >> 1) & 1, waits)) {
                        ok = false;
                        break;
                    }
                    if (!in)  // in v too
#pragma unroll 1
                        for (int x = 0; x < 8; ++x) *reinterpret_cast<uint4 *>(vt + swizzled(t, x)) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_smem_to_async();
                arrive_warp(&sh->keys);
                if (so) continue;
                if (half * 64 < DV) {  // while the state's products run: is there a NaN or an infinity in v?
                    uint32_t high = 0u;
#pragma unroll 2
                    for (int x = 0; x < 8; ++x) high |= carries(*reinterpret_cast<const uint4 *>(vt + swizzled(t, x)));
                    if (__any_sync(0xffffffffu, high & kCarry)) note_bad(vt, t, 8 + 8 * half, &sh->apart[stage]);
                }
                // (an arrival before the last chunk's phase is over would count there)
                if (it > 0 && !wait_warp(&sh->a_ready, (it - 1) & 1, waits)) {
                    ok = false;
                    break;
                }
                arrive_warp(&sh->a_ready);
            }
        }
    } else if (warp == 22) {
        // ----------------------------------------------------------------------------- issue
        const uint32_t lead = elect_lane();
        const uint32_t q = desc_k(smem_u32(q_tile)), kt = desc_k(smem_u32(k_tile)), sc = desc_mn(smem_u32(s_copy), kBlock),
                       hi = desc_mn(smem_u32(hi_tile), kBlock), lo = desc_mn(smem_u32(lo_tile), kBlock);
        constexpr uint32_t id_qk = mma_desc(128, false, false),
                           id_kv = mma_desc(64, true, true), id_av = mma_desc(DV, false, true);
        bool apart_before = false, bad_before = false;
        bool ok = true;
        for (int n = 0, idx; ok && (idx = unit_index(p, sh, n)) != -1; ++n) {
            if (idx < 0) continue;
            const int chunks = unit_of(p, sh, idx).chunks;
            for (int c = 0; c < chunks; ++c, ++it) {
                const int stage = it & 1;
                const uint32_t v = desc_mn(smem_u32(v_tile + stage * kTileV), kBlock);
                ok = false;
                if (!so) {
                    // the last chunk's A, under the scores, is used up by the products before these, unless the output
                    // warps read it too
                    if (!wait_warp(&sh->k_full, it & 1, waits) || !wait_warp(&sh->q_full, it & 1, waits) ||
                        (bad_before && !wait_warp(&sh->out_free[~it & 1], ((it - 1) >> 1) & 1, waits)))
                        break;
                    tmem_fence_after();
#pragma unroll 1
                    for (int x = 0; x < 8; ++x) {
                        const uint32_t off = ((x >> 2) * kBlock + (x & 3) * 32) >> 4;
                        mma_ss(lead, tm + kColP, q + off, kt + off, id_qk, x > 0);
                    }
                    mma_commit(lead, &sh->scores);
                    mma_commit(lead, &sh->k_empty);
                }
                // Q S and A V add up in one buffer, of two in turn.  K'^T V goes to the other, between the last
                // chunk's outputs there and the next one's.  A chunk that keeps Q S and A V apart has A V there, once
                // K'^T V has been read.
                const uint32_t mine = tm + kColO + (it & 1) * DV, other = tm + kColO + (~it & 1) * DV;
                if (!wait_warp(&sh->s_ready, it & 1, waits)) break;  // (the last K'^T V has been read from `mine`)
                if (!so) {
                    if (apart_before && !wait_warp(&sh->out_free[~it & 1], ((it - 1) >> 1) & 1, waits)) break;
                    tmem_fence_after();
#pragma unroll 1
                    for (int x = 0; x < 8; ++x)
                        mma_ss(lead, mine, q + (((x >> 2) * kBlock + (x & 3) * 32) >> 4), sc + x * 128, id_av, x > 0);
                    mma_commit(lead, &sh->q_used);
                }
                if (!wait_warp(&sh->keys, it & 1, waits) ||  // (these waited for v)
                    (!so && it > 0 && !wait_warp(&sh->out_free[~it & 1], ((it - 1) >> 1) & 1, waits)))
                    break;
                tmem_fence_after();
#pragma unroll 1
                for (int h = 0; h < HALVES; ++h) {
#pragma unroll 1
                    for (int x = 0; x < 8; ++x) {
                        mma_ss(lead, other + h * 64, hi + x * 128, v + h * (kBlock >> 4) + x * 128, id_kv, x > 0);
                        mma_ss(lead, other + h * 64, lo + x * 128, v + h * (kBlock >> 4) + x * 128, id_kv, true);
                    }
                    mma_commit(lead, &sh->s_done[h]);
                }
                if (so) mma_commit(lead, &sh->v_empty[stage]);
                if (!so) {
                    if (!wait_warp(&sh->a_ready, it & 1, waits)) break;
                    const int why = *(volatile int *)&sh->apart[stage];
                    const bool apart = why != 0;
                    if (apart && !wait_warp(&sh->s_used, it & 1, waits)) break;
                    tmem_fence_after();
#pragma unroll 1
                    for (int x = 0; x < 8; ++x)
                        mma_ts(lead, apart ? other : mine, tm + kColP + x * 8, v + x * 128, id_av, !apart || x > 0);
                    mma_commit(lead, &sh->out[it & 1]);
                    apart_before = apart, bad_before = (why & 2) != 0;
                }
                ok = true;
            }
        }
        // nothing of the block's is in flight when it gives tensor memory back
        mma_commit(lead, &sh->last);
        mbar_wait_bounded(&sh->last, 0, kPolls);
    }
    __syncwarp();
    tmem_wait_st();  // (of a role that gave up)
    tmem_fence_before();
    __syncthreads();
    if (*waits.dead && tid == 0)
        for (int n = 0, idx; (idx = unit_index(p, sh, n)) != -1; ++n)
            if (idx >= 0) {
                const Unit u = unit_of(p, sh, idx);
                if (!u.on) continue;
                if (a.err) atomicOr(a.err + u.s, kSeqTimeout);
                if (so) p.ws_decay[((long long)u.s * a.n_heads + u.h) * p.n_segs + u.seg] = kNoDecay;
            }
    if (warp == 23) {
        tmem_fence_after();
        tmem_free(tm, kCols);
    }
}

// S_0 = the initial state; S_{i+1} = decay_i S_i + own_i, written over own_i.  A thread takes 4 columns
// of a row; the pieces are read ahead 8 at a time, since only the sums depend on one another.
__global__ void __launch_bounds__(kJoinThreads) chunk_join(const __grid_constant__ LinattnChunkParams p) {
    grid_dep_wait();
    grid_dep_launch();
    const LinattnParams &a = p.a;
    const int dv_pad = p.dv_pad, parts = dv_pad / 4;  // blocks a head: 128 rows by 4 columns each
    const int part = blockIdx.x % parts, sh = blockIdx.x / parts;
    const int h = sh % a.n_heads, s = sh / a.n_heads, row = threadIdx.x, col = part * 4;
    const int slot = a.cache_idx ? __ldg(a.cache_idx + s) : s;
    int L, row0;
    if (slot < 0 || slot >= a.n_slots || draft_span(a.tok.cu, s, a.tok.T, a.tok.total, L, row0)) return;
    const int n = (L + p.seg_len - 1) / p.seg_len - 1;  // pieces with a next one
    const bool init = a.has_init ? __ldg(a.has_init + s) != 0 : true;
    float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
    if (init && row < a.dk && col < a.dv)
        S = *reinterpret_cast<const float4 *>(a.state + (long long)slot * a.st_slot + (long long)h * a.st_head +
                                              (long long)row * a.dv + col);
    const long long base = ((long long)s * a.n_heads + h) * p.n_segs;
    float4 *const own = reinterpret_cast<float4 *>(p.ws_state) + base * (32 * dv_pad) + part * 128 + row;
    const float *const dec = p.ws_decay + base;
    const long long step = 32LL * dv_pad;
    // The first piece's state too: the last piece writes the sequence's while the first may not have begun.
    if (n > 0) *own = S;
    bool left = false;
    for (int i0 = 0; i0 < n; i0 += 8) {
        float4 f[8];
        float d[8];
#pragma unroll
        for (int x = 0; x < 8; ++x)
            if (i0 + x < n) f[x] = own[(i0 + x + 1) * step], d[x] = dec[i0 + x];
#pragma unroll
        for (int x = 0; x < 8; ++x)
            if (i0 + x < n) {
                left |= d[x] == kNoDecay;
                S.x = fmaf(d[x], S.x, f[x].x), S.y = fmaf(d[x], S.y, f[x].y);
                S.z = fmaf(d[x], S.z, f[x].z), S.w = fmaf(d[x], S.w, f[x].w);
                own[(i0 + x + 1) * step] = S;
            }
    }
    if (left && row == 0) p.ws_left[s] = 1;
}

}  // namespace

ChunkKernel chunk_kernel(int dv) {
    if (dv <= 64) return {linattn_chunk<64>, chunk_smem_bytes<64>()};
    return {linattn_chunk<128>, chunk_smem_bytes<128>()};
}
LinattnChunkKernel chunk_join_kernel() { return chunk_join; }

}  // namespace cvk
