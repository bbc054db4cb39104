// Device parts that the attention kernels share: sequences, the split of the work over blocks, ancestors.
#pragma once

#include "cv_attn.h"
#include "cv_device.cuh"

namespace cvk {

constexpr int kSeqBadSlot = 1, kSeqBadAccept = 4, kSeqBadTree = 32, kSeqBadLength = 64, kSeqBadPage = 128, kSeqBadToken = 256,
              kSeqBadProbs = 512, kSeqNoPages = 1024, kSeqBadPosition = 2048, kSeqSharedPage = 4096;

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
__device__ __forceinline__ long long attn_units(const AttnParams &p, const AttnSeq &q) { return (long long)attn_row_tiles(p, q) * p.c.n_kv; }
__device__ __forceinline__ unsigned attn_div(long long a, int b) {  // (a 64-bit division costs 100 instructions)
    return a >> 32 == 0 ? (unsigned)a / (unsigned)b : (unsigned)(a / b);
}

// A block's run of work [begin, end).  A sequence's work is the key tiles of its units, and `cost` more for each unit.
struct AttnRange {
    long long begin, end, per, before;  // before: work of the sequences before s
    int s, cost;                        // the sequence it begins in
    AttnSeq q;
};
struct AttnScratch {
    long long tiles[32], units[32];
};

// Every thread of the block calls this.  Sequences' flags that need no page are raised here, each by one block.
__device__ __forceinline__ void attn_range(const AttnParams &p, AttnRange *r, AttnScratch *sh) {
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = nt >> 5;
    long long tiles = 0, units = 0;      // of this thread's sequences
    AttnSeq mine = {-1, 0, 0, 0, 0};     // its first
    for (int s = tid; s < p.n_seq; s += nt) {
        const AttnSeq q = attn_seq(p, s);
        if (p.err && q.status && s % (int)gridDim.x == (int)blockIdx.x) atomicOr(p.err + s, q.status);
        if (s == tid) mine = q;
        if (q.T > 0) units += attn_units(p, q), tiles += attn_units(p, q) * attn_key_tiles(p, q);
    }
    long long up_t = tiles, up_u = units;  // up to this thread: what comes before its first sequence, where there is one a thread
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, up_t, o), y = __shfl_up_sync(0xffffffffu, up_u, o);
        if (lane >= o) up_t += x, up_u += y;
    }
    if (lane == 31) sh->tiles[warp] = up_t, sh->units[warp] = up_u;
    __syncthreads();
    long long all_t = 0, all_u = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) up_t += sh->tiles[w], up_u += sh->units[w];
        all_t += sh->tiles[w], all_u += sh->units[w];
    }
    // a unit's cost matters where blocks have many tiles; few are better spread evenly
    const long long most = all_t / (4LL * p.parts);
    const int cost = most < p.unit_cost ? (int)most : p.unit_cost;
    const long long total = all_t + cost * all_u;
    const long long per = total + p.parts - 1 < (1LL << 32) ? attn_div(total + p.parts - 1, p.parts) : (total + p.parts - 1) / p.parts;
    const long long begin = per * blockIdx.x, end = begin + per < total ? begin + per : total;
    if (tid == 0) r->begin = begin, r->end = end, r->per = per, r->cost = cost;
    if (p.n_seq <= nt) {
        const long long up = up_t + cost * up_u, before = up - (tiles + cost * units);
        if (begin < end && up > begin && before <= begin) r->s = tid, r->before = before, r->q = mine;
    } else if (begin < end) {
        long long before = 0;
        for (int base = 0; base < p.n_seq && before <= begin; base += nt) {
            const int s = base + tid;
            AttnSeq q = {-1, 0, 0, 0, 0};
            if (s < p.n_seq) q = attn_seq(p, s);
            const long long n = q.T > 0 ? attn_units(p, q) * (attn_key_tiles(p, q) + cost) : 0;
            long long up = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long x = __shfl_up_sync(0xffffffffu, up, o);
                if (lane >= o) up += x;
            }
            __syncthreads();
            if (lane == 31) sh->tiles[warp] = up;
            __syncthreads();
            long long chunk = 0;
            for (int w = 0; w < warps; ++w) {
                if (w < warp) up += sh->tiles[w];
                chunk += sh->tiles[w];
            }
            if (before + up > begin && before + up - n <= begin) r->s = s, r->before = before + up - n, r->q = q;
            before += chunk;
        }
    }
    __syncthreads();
}

// A block's part of one unit.
struct AttnUnit {
    int s, h, row, rows;           // kv head, first row of the unit and their number
    int tile, last;                // key tiles [tile, last) of this block, at least one
    int tiles;                     // of the whole unit
    long long first;               // where the unit's first tile stands among all work
    AttnSeq q;
};
// The units of a block, one after the other.  A unit's work is its cost, then its tiles; a block has the tiles that stand in
// its run.
struct AttnWalk {
    long long at, end, before, n;  // n: work of sequence s
    int s, cost, size, mt;         // size: work of one of its units
    AttnSeq q;
    __device__ __forceinline__ void enter(const AttnParams &p) {
        size = mt = 1, n = 0;
        if (q.T > 0) {
            size = attn_key_tiles(p, q) + cost, mt = attn_row_tiles(p, q);
            n = (long long)size * mt * p.c.n_kv;
        }
    }
    __device__ __forceinline__ AttnWalk(const AttnParams &p, const AttnRange &r)
        : at(r.begin), end(r.end), before(r.before), s(r.s), cost(r.cost), q(r.q) {
        if (at < end) enter(p);
    }
    __device__ __forceinline__ bool next(const AttnParams &p, AttnUnit &u) {
        while (at < end) {
            while (at - before >= n) {
                before += n;
                q = attn_seq(p, ++s);
                enter(p);
            }
            const long long local = at - before;
            const int unit = (int)attn_div(local, size), from = (int)(local - (long long)unit * size);
            const int to = (int)(end - at < size - from ? from + (end - at) : size);
            u.first = at - from + cost;
            at += to - from;
            u.tile = max(from - cost, 0), u.last = max(to - cost, 0);
            if (u.tile >= u.last) continue;
            u.s = s, u.q = q, u.tiles = size - cost;
            u.h = mt > 1 ? unit / mt : unit;
            u.row = (unit - u.h * mt) * p.rows;
            u.rows = min(p.rows, q.T * p.G - u.row);
            return true;
        }
        return false;
    }
};

// Where a block leaves what it has of a unit that others have parts of too: slot 0 for one that began before it, 1 for
// one that begins in it and goes on.
__device__ __forceinline__ float *attn_part(const AttnParams &p, int block, int slot) {
    return p.ws + (2LL * block + slot) * part_floats(p.pad, p.dp);
}

// What a part begins with: whether there is one (0: none), the unit's number of parts, the block of the first, the unit's rows and the
// first of them, sequence, kv head, and the sequence's first packed row.
__device__ __forceinline__ void attn_part_head(float *part, const AttnRange &r, long long first, int tiles, int rows, int row, int s, int h,
                                               int row0) {
    auto block = [&](long long at) { return (int)(at >> 32 == 0 && r.per >> 32 == 0 ? (unsigned)at / (unsigned)r.per : at / r.per); };
    const int c0 = block(first), c1 = block(first + tiles - 1);
    int4 *const to = reinterpret_cast<int4 *>(part);
    to[0] = make_int4(1, c1 - c0 + 1, c0, rows), to[1] = make_int4(row, s, h, row0);
}

// Ancestors-or-selves of the drafts as 128-bit masks, by pointer jumping: after i rounds a mask covers 2^i steps up.  All
// `threads` callers take drafts of their own, threads apart; sync joins them.  Returns whether one of the caller's has a parent
// outside [-1, t).
struct AttnTree {
    uint4 mask[2][128];
    int up[2][128];
};
template <typename Sync>
__device__ __forceinline__ bool attn_ancestors(const int *parent, int T, int thread, int threads, AttnTree *tree, uint4 *out, Sync sync) {
    bool bad = false;
    for (int t = thread; t < 128; t += threads) {
        uint4 m;
        uint32_t *const w = &m.x;
        int up = -1;
#pragma unroll
        for (int i = 0; i < 4; ++i)  // (a chain: all before it)
            w[i] = parent ? (t >> 5 == i ? 1u << (t & 31) : 0u) : t >= 32 * i + 31 ? 0xffffffffu : t >= 32 * i ? (2u << (t & 31)) - 1 : 0u;
        if (parent && t < T) {
            up = __ldg(parent + t);
            if (up < -1 || up >= t) bad = true, up = -1;
        }
        if (!parent) out[t] = m;
        tree->mask[0][t] = m, tree->up[0][t] = up;
    }
    if (!parent) return false;
    sync();
    int from = 0;
    for (int reach = 1; reach < T; reach *= 2, from ^= 1) {
        for (int t = thread; t < T; t += threads) {
            uint4 m = tree->mask[from][t];
            int up = tree->up[from][t];
            if (up >= 0) {
                const uint4 o = tree->mask[from][up];
                m.x |= o.x, m.y |= o.y, m.z |= o.z, m.w |= o.w;
                up = tree->up[from][up];
            }
            tree->mask[from ^ 1][t] = m, tree->up[from ^ 1][t] = up;
        }
        sync();
    }
    // (rows past the drafts see none of them: where rows share a decision, what an earlier call left here would reach the others' bits)
    for (int t = thread; t < 128; t += threads) out[t] = t < T ? tree->mask[from][t] : make_uint4(0, 0, 0, 0);
    return bad;
}

}  // namespace cvk
