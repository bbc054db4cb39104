// Device parts that the attention kernels share: sequences, the split of the work over blocks, ancestors.
#pragma once

#include "cv_attn.h"
#include "cv_device.cuh"

namespace cvk {

constexpr int kSeqBadSlot = 1, kSeqBadAccept = 4, kSeqBadTree = 32, kSeqBadLength = 64, kSeqBadPage = 128, kSeqBadToken = 256,
              kSeqBadProbs = 512, kSeqNoPages = 1024, kSeqBadPosition = 2048;

struct AttnSeq {
    int slot, L, T, row0;  // row0: the first of its packed rows (cu), 0 without
    int status;
};

// What is known of sequence s without reading its pages; T = 0 where there is nothing to do.
__device__ __forceinline__ AttnSeq attn_seq(const AttnParams &p, int s) {
    AttnSeq q;
    q.slot = p.idx ? __ldg(p.idx + s) : s;
    q.L = __ldg(p.len + s);
    q.T = p.T, q.row0 = 0, q.status = 0;
    if (p.cu) q.status = draft_span(p.cu, s, p.T, p.total, q.T, q.row0);
    if (q.slot >= p.c.n_slots) q.status |= kSeqBadSlot;
    if (!(q.status & kSeqBadSpan) && (q.L < 0 || (long long)q.L + q.T > (long long)p.c.max_pages * p.c.page))
        q.status |= kSeqBadLength;
    if (q.slot < 0) q.status = 0;
    if (q.slot < 0 || q.status) q.T = 0;
    return q;
}
__device__ __forceinline__ int attn_key_tiles(const AttnParams &p, const AttnSeq &q) { return (q.L + q.T - 1) / p.keys + 1; }
__device__ __forceinline__ int attn_row_tiles(const AttnParams &p, const AttnSeq &q) { return (q.T * p.G + p.rows - 1) / p.rows; }
__device__ __forceinline__ long long attn_tiles(const AttnParams &p, const AttnSeq &q) {
    return q.T > 0 ? (long long)attn_key_tiles(p, q) * attn_row_tiles(p, q) * p.c.n_kv : 0;
}

// A block's run of tiles [begin, end), and the sequence it begins in.
struct AttnRange {
    long long begin, end, per, before;  // before: tiles of the sequences before s
    int s;
};

// Every thread of the block calls this.  Sequences' flags that need no page are raised here, each by one block.
__device__ __forceinline__ void attn_range(const AttnParams &p, AttnRange *r, long long *scratch) {
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = nt >> 5;
    long long sum = 0, first = 0;
    for (int s = tid; s < p.n_seq; s += nt) {
        const AttnSeq q = attn_seq(p, s);
        if (p.err && q.status && s % (int)gridDim.x == (int)blockIdx.x) atomicOr(p.err + s, q.status);
        const long long n = attn_tiles(p, q);
        if (s == tid) first = n;
        sum += n;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) scratch[warp] = sum;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < warps; ++w) total += scratch[w];
    const long long per = (total + p.parts - 1) / p.parts;
    const long long begin = per * blockIdx.x, end = begin + per < total ? begin + per : total;
    if (tid == 0) r->begin = begin, r->end = end, r->per = per, r->s = p.n_seq, r->before = 0;
    if (begin < end) {
        long long before = 0;
        for (int base = 0; base < p.n_seq && before <= begin; base += nt) {
            const int s = base + tid;
            const long long mine = base == 0 ? first : s < p.n_seq ? attn_tiles(p, attn_seq(p, s)) : 0;
            long long up = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long x = __shfl_up_sync(0xffffffffu, up, o);
                if (lane >= o) up += x;
            }
            __syncthreads();
            if (lane == 31) scratch[warp] = up;
            __syncthreads();
            long long chunk = 0;
            for (int w = 0; w < warps; ++w) {
                if (w < warp) up += scratch[w];
                chunk += scratch[w];
            }
            if (before + up > begin && before + up - mine <= begin) r->s = s, r->before = before + up - mine;
            before += chunk;
        }
    }
    __syncthreads();
}

// A block's part of one unit.
struct AttnUnit {
    int s, h, row, rows;           // kv head, first row of the unit and their number
    int tile, last;                // key tiles [tile, last) of this block
    int tiles;                     // of the whole unit
    long long first;               // the unit's first tile among all
    AttnSeq q;
};
// The units of a block, one after the other; each role walks them by itself.
struct AttnWalk {
    long long at, end, before;
    int s;
    AttnSeq q;
    __device__ __forceinline__ AttnWalk(const AttnParams &p, const AttnRange &r) : at(r.begin), end(r.end), before(r.before), s(r.s) {
        if (at < end) q = attn_seq(p, s);
    }
    __device__ __forceinline__ bool next(const AttnParams &p, AttnUnit &u) {
        if (at >= end) return false;
        long long n = attn_tiles(p, q);
        while (at - before >= n) {
            before += n;
            q = attn_seq(p, ++s);
            n = attn_tiles(p, q);
        }
        const int kt = attn_key_tiles(p, q), mt = attn_row_tiles(p, q);
        const long long local = at - before;
        const int unit = (int)(local / kt);
        u.s = s, u.q = q, u.tiles = kt;
        u.tile = (int)(local - (long long)unit * kt);
        u.h = unit / mt;
        u.row = (unit - u.h * mt) * p.rows;
        u.rows = min(p.rows, q.T * p.G - u.row);
        u.first = at - u.tile;
        const long long left = end - at;
        u.last = u.tile + (int)(kt - u.tile < left ? kt - u.tile : left);
        at += u.last - u.tile;
        return true;
    }
};

// Where a block leaves what it has of a unit that others have parts of too: slot 0 for one that began before it, 1 for
// one that begins in it and goes on.
__device__ __forceinline__ float *attn_part(const AttnParams &p, int block, int slot) {
    return p.ws + (2LL * block + slot) * part_floats(p.pad, p.dp);
}

// Ancestors-or-selves of the drafts as 128-bit masks, by pointer jumping: after i rounds a mask covers 2^i steps up.
// `sync` joins the threads that call (128 of them or more, draft = their number).  Returns whether a parent is outside [-1, t).
struct AttnTree {
    uint4 mask[2][128];
    int up[2][128];
};
template <typename Sync>
__device__ __forceinline__ bool attn_ancestors(const int *parent, int T, int draft, AttnTree *tree, uint4 *out, Sync sync) {
    uint4 m = make_uint4(0, 0, 0, 0);
    uint32_t *w = &m.x;
    int up = -1;
    bool bad = false;
    if (draft < 128) {
#pragma unroll
        for (int i = 0; i < 4; ++i)  // (a chain: all before it)
            w[i] = parent ? (draft >> 5 == i ? 1u << (draft & 31) : 0u)
                          : draft >= 32 * i + 31 ? 0xffffffffu : draft >= 32 * i ? (2u << (draft & 31)) - 1 : 0u;
        if (parent && draft < T) {
            up = __ldg(parent + draft);
            bad = up < -1 || up >= draft;
            if (bad) up = -1;
        }
        tree->mask[0][draft] = m, tree->up[0][draft] = up;
    }
    sync();
    int from = 0;
    if (parent)
        for (int reach = 1; reach < T; reach *= 2) {
            if (draft < 128) {
                if (up >= 0) {
                    up &= 127;  // (in bounds even where the other threads' part never came)
                    const uint4 o = tree->mask[from][up];
                    m.x |= o.x, m.y |= o.y, m.z |= o.z, m.w |= o.w;
                    up = tree->up[from][up];
                }
                tree->mask[from ^ 1][draft] = m, tree->up[from ^ 1][draft] = up;
            }
            from ^= 1;
            sync();
        }
    if (draft < 128) out[draft] = m;
    return bad;
}

}  // namespace cvk
