// Attention of drafted tokens over a paged cache on the tensor cores (bf16).
//
// Mathematics.  A unit is up to 128 rows (draft, query head of a group) of one kv head of a sequence.  For each tile of
// KT keys, with c = scale log2(e),
//   S = Q K^T,   p = 2^(c S - m),   l += sum p,   O += P V,      out = O / l
// in one pass over K and V.  m is the row's maximum when it was last moved: it moves only when a tile exceeds it by
// more than 2^8, since that costs a pass over O; until then p is at most 2^8, which bf16 and the fp32 sums hold as well as 1.
// P is rounded to bf16 (2^-8 of a term), as the operand of the second product; l sums what was not rounded.
//
// Layout.  A block (one per SM) takes a run of key tiles of the units' tiles in a row, so that all blocks read the same
// number of keys whatever the lengths; a unit that is cut leaves (m, l, O) in the workspace for the join.  All rows of a
// kv head's group share one read of its keys, so HBM bounds it: a tile of 128 keys of 128 channels is 64 KB, 1.4 us of an SM's
// share, and takes 0.7 us of the tensor pipe at any number of rows.  Roles, each a stream of tiles of its own:
//   load     1 warp: units (also for the others, through a queue in shared memory), Q, K and V by TMA, a box for each page
//   issue    1 warp: Q K^T of the next tile, then P V of this one
//   softmax  4 warps, a row a thread: S from tensor memory, P back over it, O's rescaling, and at the end the outputs
// Tensor memory: two buffers of S (and P), O (two for up to 192 channels, so that a unit begins while the last one's rows
// are written).
//
// Masks.  Cached tokens are seen by every row; only the tiles that reach past them look at masks.  There the rows of V past the
// end are zeroed in shared memory (0 * what lies there may be NaN), and so are drafts' rows of V that hold a NaN or an
// infinity, which are added at the end to the rows that see them.
//
// Every wait is bounded; one that gives up ends the block's work, flags the sequences of its run and returns.
#include "cv_attn.cuh"
#include "cv_tcgen05.cuh"

namespace cvk {
namespace {

constexpr float kNone = -INFINITY;
constexpr float kSlack = 8.0f;  // log2 of what a weight may reach before its row's maximum is moved
constexpr unsigned kDrainPolls = 1u << 16;
constexpr int kTcThreads = 192, kQueue = 4;

template <int DP>
struct Tc {
    static constexpr int KT = DP <= 128 ? 128 : 64;     // keys a tile
    static constexpr int BLOCKS = DP / 64;              // blocks of 64 channels
    static constexpr int KV = KT * DP * 2, Q = 128 * DP * 2;
    static constexpr int QBUF = DP <= 192 ? 2 : 1, OBUF = DP <= 192 ? 2 : 1;
    static constexpr int STAGES = DP == 64 ? 8 : DP == 128 ? 4 : DP == 192 ? 5 : 4;
    static constexpr int COL_O = 2 * KT;
    static_assert(COL_O + OBUF * DP <= 512, "tensor memory");
};
constexpr uint32_t kTmemCols = 512;

struct TcUnit {
    int s, h, row, rows, tile, last, tiles, slot, L, T, row0, begins;
    long long first;
};

struct TcShared {
    uint64_t kv_full[8], kv_empty[8], q_full[2], q_empty[2], s_full[2], p_ready[2], o_free[2], unit_full[kQueue], unit_empty[kQueue],
        pv_done, meet, last;
    TcUnit unit[kQueue];
    uint32_t tmem;
    int dead, flags;
    uint32_t bad[2][4];  // drafts whose v holds a NaN or an infinity; of two units in turn
    uint4 see[128];
    AttnTree tree;
    AttnRange range;
    long long scratch[32];
};

template <int DP>
__host__ __device__ constexpr int tc_smem() {
    return Tc<DP>::QBUF * Tc<DP>::Q + Tc<DP>::STAGES * Tc<DP>::KV + (int)sizeof(TcShared) + 1024;
}

struct Waits {
    volatile int *dead;
    unsigned polls;
};
// One poll of up to 20 us.
__device__ __forceinline__ bool poll(uint64_t *bar, unsigned parity) {
    unsigned done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done != 0;
}
// Bounded wait of a whole warp; false once the block has given up.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, unsigned parity, Waits waits) {
#pragma unroll 1
    for (unsigned i = 0; i < waits.polls; ++i) {
        if (__all_sync(0xffffffffu, poll(bar, parity))) return true;
        if (__any_sync(0xffffffffu, *waits.dead)) return false;
    }
    *waits.dead = 1;
    return false;
}
__device__ __forceinline__ void arrive_warp(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void tma_load4(uint32_t dst, const CUtensorMap *map, int c, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(
            dst),
        "l"(map), "r"(c), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// 32 columns of the calling warp's 32 lanes, there after tmem_wait_ld32 on the same array.
#define CV_E8(r, i, m) m((r)[i]), m((r)[i + 1]), m((r)[i + 2]), m((r)[i + 3]), m((r)[i + 4]), m((r)[i + 5]), m((r)[i + 6]), m((r)[i + 7])
#define CV_E32(r, m) CV_E8(r, 0, m), CV_E8(r, 8, m), CV_E8(r, 16, m), CV_E8(r, 24, m)
#define CV_OUT(x) "=r"(x)
#define CV_INOUT(x) "+r"(x)
__device__ __forceinline__ void tmem_ld32(uint32_t *r, uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        : CV_E32(r, CV_OUT)
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld32(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" : CV_E32(r, CV_INOUT)::"memory");
}
__device__ __forceinline__ void tmem_tie32(uint32_t *r) { asm volatile("" : CV_E32(r, CV_INOUT)::"memory"); }
#undef CV_E8
#undef CV_E32
#undef CV_OUT
#undef CV_INOUT

// Whether one of 8 bf16 values is a NaN or an infinity: its exponent plus one carries into the sign.
__device__ __forceinline__ uint32_t carries(uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; }
__device__ __forceinline__ bool not_finite(const uint4 &w) {
    return ((carries(w.x) | carries(w.y) | carries(w.z) | carries(w.w)) & 0x80008000u) != 0;
}

// Drafts whose v is not finite, to the rows that see them: their weights again from q and k, and O in tensor memory plus
// weight times v.
template <int DP>
__device__ __noinline__ void add_bad_drafts(const AttnParams &p, const TcUnit &u, const uint32_t *bad, uint4 see, int r, float m,
                                            uint32_t to) {
    const uint16_t *const q = reinterpret_cast<const uint16_t *>(p.q) + (p.cu ? 0LL : (long long)u.s * p.q_seq) +
                              (long long)(u.row0 + (u.row + r) / p.G) * p.q_tok +
                              (long long)(u.h * p.G + (u.row + r) % p.G) * p.q_head;
    const int *const table = p.c.table + (long long)u.slot * p.c.table_row;
    for (int b = 0; b < u.T; ++b) {
        if (!(bad[b >> 5] >> (b & 31) & 1)) continue;
        const int j = u.L + b;
        if (j < u.tile * Tc<DP>::KT || j >= u.last * Tc<DP>::KT) continue;
        const int pg = __ldg(table + j / p.c.page), in = j % p.c.page;
        const uint16_t *const k = reinterpret_cast<const uint16_t *>(p.c.k) + (long long)pg * p.c.k_page +
                                  (long long)in * p.c.k_row + (long long)u.h * p.c.k_head;
        const uint16_t *const v = reinterpret_cast<const uint16_t *>(p.c.v) + (long long)pg * p.c.v_page +
                                  (long long)in * p.c.v_row + (long long)u.h * p.c.v_head;
        const bool sees = r < u.rows && ((&see.x)[b >> 5] >> (b & 31) & 1);
        float w = 0.f;
        if (sees) {
            for (int c = 0; c < p.c.d; ++c) w = fmaf(widen<uint16_t>(q[c]), widen<uint16_t>(k[c]), w);
            w = exp2_fast(fmaf(w, p.scale, m == kNone ? 0.f : -m));
        }
        __syncwarp();
#pragma unroll 1
        for (int c = 0; c < DP; c += 16) {
            uint32_t x[16];
            tmem_ld16(x, to + c);
            tmem_wait_ld(x);
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (sees && c + e < p.c.d) x[e] = __float_as_uint(fmaf(w, widen<uint16_t>(v[c + e]), __uint_as_float(x[e])));
            tmem_st16(to + c, x);
        }
        tmem_wait_st();
    }
}

template <int DP>
__global__ void __launch_bounds__(kTcThreads, 1) attn_tc(const __grid_constant__ AttnMaps mp) {
    using K = Tc<DP>;
    constexpr int KT = K::KT, STAGES = K::STAGES;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *const smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) / 1024 * 1024);
    unsigned char *const q_tile = smem, *const kv_tile = smem + K::QBUF * K::Q;
    TcShared *const sh = reinterpret_cast<TcShared *>(kv_tile + STAGES * K::KV);
    const AttnParams &p = mp.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (dynamic_smem_bytes() < (unsigned)tc_smem<DP>()) return;
    if (tid == 0) {
        for (int i = 0; i < 8; ++i) mbar_init(&sh->kv_full[i], 1), mbar_init(&sh->kv_empty[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->q_full[i], 1), mbar_init(&sh->q_empty[i], 1), mbar_init(&sh->s_full[i], 1);
            mbar_init(&sh->p_ready[i], 4), mbar_init(&sh->o_free[i], 4);
        }
        for (int i = 0; i < kQueue; ++i) mbar_init(&sh->unit_full[i], 1), mbar_init(&sh->unit_empty[i], 5);
        mbar_init(&sh->pv_done, 1), mbar_init(&sh->meet, 4), mbar_init(&sh->last, 1);
        mbar_init_fence();
        sh->dead = 0, sh->flags = 0;
    }
    if (warp == 5) tmem_alloc(&sh->tmem, kTmemCols);
    if (warp == 4 && lane < 3) {
        const CUtensorMap *const map = lane == 0 ? &mp.q : lane == 1 ? &mp.k : &mp.v;
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(map) : "memory");
    }
    grid_dep_wait();
    grid_dep_launch();
    attn_range(p, &sh->range, sh->scratch);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tm = sh->tmem;
    const Waits waits{&sh->dead, p.polls};
    const AttnRange &range = sh->range;
    const int total = (int)(range.end > range.begin ? range.end - range.begin : 0);

    if (warp == 4) {
        // ------------------------------------------------------------------------------ load
        AttnWalk walk(p, range);
        AttnUnit u, next;
        bool has = walk.next(p, u), has_next = false;
        const int boxes = KT / mp.page_rows;           // of a tile
        const int blk = lane % K::BLOCKS, box = lane / K::BLOCKS;  // this lane's copy
        int pos = 0, units = 0;
        bool ok = true;
        struct Where {
            int page, row, h, n;  // this lane's; n: bytes of the tile's boxes
            bool on;
        };
        auto where = [&](const AttnUnit &a, int tile) {
            Where w;
            const int j = tile * KT + box * mp.page_rows, end = a.q.L + a.q.T;
            w.on = box < boxes && j < end;
            w.page = w.on ? __ldg(p.c.table + (long long)a.q.slot * p.c.table_row + j / p.c.page) : 0;
            w.row = j % p.c.page, w.h = a.h;
            const int left = end - tile * KT;
            w.n = min(boxes, (left + mp.page_rows - 1) / mp.page_rows) * (K::BLOCKS * 128) * mp.page_rows;
            return w;
        };
        auto copy = [&](const CUtensorMap *map, const Where &w) {
            const int stage = pos % STAGES;
            if (pos >= STAGES && !wait_warp(&sh->kv_empty[stage], (pos / STAGES - 1) & 1, waits)) return false;
            if (lane == 0) mbar_arrive_expect_tx(&sh->kv_full[stage], (unsigned)w.n);
            __syncwarp();
            if (w.on)
                tma_load4(smem_u32(kv_tile) + stage * K::KV + blk * (KT * 128) + box * mp.page_rows * 128, map, blk * 64, w.row, w.h,
                          w.page, &sh->kv_full[stage]);
            ++pos;
            return true;
        };
        auto publish = [&](bool end) {
            const int at = units % kQueue;
            if (units >= kQueue && !wait_warp(&sh->unit_empty[at], (units / kQueue - 1) & 1, waits)) return false;
            if (lane == 0) {
                TcUnit &t = sh->unit[at];
                t.s = end ? -1 : u.s, t.h = u.h, t.row = u.row, t.rows = u.rows, t.tile = u.tile, t.last = u.last, t.tiles = u.tiles;
                t.slot = u.q.slot, t.L = u.q.L, t.T = u.q.T, t.row0 = u.q.row0, t.first = u.first, t.begins = u.tile == 0;
                mbar_arrive(&sh->unit_full[at]);
            }
            __syncwarp();
            return true;
        };
        Where cur, before;
        if (has) cur = where(u, u.tile);
        bool pending = false;  // V of the tile before
        int q_sent = 0;
        while (ok && has) {
            if (!(ok = publish(false))) break;
            const int qb = units % K::QBUF;
            if (units >= K::QBUF && !(ok = wait_warp(&sh->q_empty[qb], (units / K::QBUF - 1) & 1, waits))) break;
            if (lane == 0) mbar_arrive_expect_tx(&sh->q_full[qb], (unsigned)(K::BLOCKS * 128 * mp.tok * p.G));
            __syncwarp();
            if (lane < K::BLOCKS)
                tma_load4(smem_u32(q_tile) + qb * K::Q + lane * (128 * 128), &mp.q, lane * 64, u.h * p.G, u.q.row0 + u.row / p.G,
                          p.cu ? 0 : u.s, &sh->q_full[qb]);
            ++units, ++q_sent;
            has_next = walk.next(p, next);
            for (int tile = u.tile; tile < u.last; ++tile) {
                // the next tile's pages are looked up while this one's copies wait for their place
                Where then;
                if (tile + 1 < u.last) then = where(u, tile + 1);
                else if (has_next) then = where(next, next.tile);
                if (!(ok = copy(&mp.k, cur))) break;
                if (pending && !(ok = copy(&mp.v, before))) break;
                before = cur, pending = true;
                cur = then;
            }
            u = next, has = has_next;
        }
        if (ok) ok = publish(true);
        if (ok && pending) copy(&mp.v, before);
        // nothing of the block's is in flight when it returns
        __syncwarp();
        for (int x = max(0, pos - STAGES); x < pos; ++x) mbar_wait_bounded(&sh->kv_full[x % STAGES], (x / STAGES) & 1, kDrainPolls);
        for (int x = max(0, q_sent - K::QBUF); x < q_sent; ++x)
            mbar_wait_bounded(&sh->q_full[x % K::QBUF], (x / K::QBUF) & 1, kDrainPolls);
    } else if (warp == 5) {
        // ----------------------------------------------------------------------------- issue
        const uint32_t lead = elect_lane();
        constexpr uint32_t id_qk = mma_desc(KT, false, false), id_pv = mma_desc(DP, false, true);
        int pos = 0, units = 0, qk_left = 0, n_next = 0, it = 0, pv_unit = 0, pv_left = 0, pv_at = 0;
        auto pop = [&](int &n) {  // tiles of the next unit, 0 after the last one, -1: gave up
            const int at = units % kQueue;
            if (!wait_warp(&sh->unit_full[at], (units / kQueue) & 1, waits)) return false;
            n = sh->unit[at].s < 0 ? 0 : sh->unit[at].last - sh->unit[at].tile;
            arrive_warp(&sh->unit_empty[at]);
            ++units;
            return true;
        };
        auto scores = [&](int i, bool first, bool last) {
            const int qb = (units - 1) % K::QBUF, stage = pos % STAGES;
            if (first && !wait_warp(&sh->q_full[qb], ((units - 1) / K::QBUF) & 1, waits)) return false;
            if (!wait_warp(&sh->kv_full[stage], (pos / STAGES) & 1, waits)) return false;
            tmem_fence_after();
            const uint32_t q = desc_k(smem_u32(q_tile) + qb * K::Q), k = desc_k(smem_u32(kv_tile) + stage * K::KV);
#pragma unroll 4
            for (int x = 0; x < DP / 16; ++x)
                mma_ss(lead, tm + (i & 1) * KT, q + (((x >> 2) * (128 * 128) + (x & 3) * 32) >> 4),
                       k + (((x >> 2) * (KT * 128) + (x & 3) * 32) >> 4), id_qk, x > 0);
            mma_commit(lead, &sh->s_full[i & 1]);
            mma_commit(lead, &sh->kv_empty[stage]);
            if (last) mma_commit(lead, &sh->q_empty[qb]);
            ++pos;
            return true;
        };
        int n = 0;
        bool ok = pop(n) && n > 0;
        if (ok) {
            qk_left = pv_left = n;
            ok = scores(0, true, n == 1);
            --qk_left;
        }
        while (ok) {
            ok = false;
            bool more = qk_left > 0;
            if (more) {
                if (!scores(it + 1, false, qk_left == 1)) break;
                --qk_left;
            } else if (n > 0) {
                if (!pop(n)) break;
                n_next = n;
                if (n > 0) {
                    if (!scores(it + 1, true, n == 1)) break;
                    qk_left = n - 1;
                }
            }
            const int ob = pv_unit % K::OBUF, stage = pos % STAGES;
            if (pv_at == 0 && pv_unit >= K::OBUF && !wait_warp(&sh->o_free[ob], (pv_unit / K::OBUF - 1) & 1, waits)) break;
            if (!wait_warp(&sh->kv_full[stage], (pos / STAGES) & 1, waits) || !wait_warp(&sh->p_ready[it & 1], (it >> 1) & 1, waits))
                break;
            tmem_fence_after();
            const uint32_t v = desc_mn(smem_u32(kv_tile) + stage * K::KV, KT * 128);
#pragma unroll 4
            for (int x = 0; x < KT / 16; ++x)
                mma_ts(lead, tm + K::COL_O + ob * DP, tm + (it & 1) * KT + x * 8, v + x * 128, id_pv, pv_at > 0 || x > 0);
            mma_commit(lead, &sh->kv_empty[stage]);
            mma_commit(lead, &sh->pv_done);
            ++pos, ++it, ++pv_at;
            ok = true;
            if (--pv_left == 0) {
                if (n == 0) break;  // the last unit
                ++pv_unit, pv_at = 0, pv_left = n_next;
            }
        }
        // nothing of the block's is in flight when it gives tensor memory back
        mma_commit(lead, &sh->last);
        mbar_wait_bounded(&sh->last, 0, kDrainPolls);
    } else {
        // --------------------------------------------------------------------------- softmax
        const int r = tid;  // the row
        const uint32_t tl = tm + ((uint32_t)(32 * warp) << 16);
        int it = 0, s_before = -1;
        uint4 see = make_uint4(0, 0, 0, 0);
        bool ok = true;
        unsigned met = 0;
        auto meet = [&] {  // the softmax warps; bounded as every wait
            arrive_warp(&sh->meet);
            return wait_warp(&sh->meet, met++ & 1, waits);
        };
        for (int units = 0; ok; ++units) {
            const int at = units % kQueue, ob = units % K::OBUF;
            if (!wait_warp(&sh->unit_full[at], (units / kQueue) & 1, waits)) break;
            const TcUnit u = sh->unit[at];
            arrive_warp(&sh->unit_empty[at]);
            if (u.s < 0) break;
            const int end = u.L + u.T;
            uint32_t *const bad = sh->bad[units & 1];
            if (r < 4) bad[r] = 0;
            if (u.s != s_before) {
                // ancestors, and a look at every page and parent of the sequence
                s_before = u.s;
                if (r == 0) sh->flags = 0;
                const int *parent = p.parent ? p.parent + (p.cu ? (long long)u.row0 : (long long)u.s * p.T) : nullptr;
                int st = attn_ancestors(parent, u.T, r, &sh->tree, sh->see, [&] { ok = ok && meet(); }) ? kSeqBadTree : 0;
                if (!ok) break;
                const int *const table = p.c.table + (long long)u.slot * p.c.table_row;
                for (int i = r; i <= (end - 1) / p.c.page; i += 128) {
                    const int g = __ldg(table + i);
                    if (g < 0 || g >= p.c.n_pages) st |= kSeqBadPage;
                }
                if (st) {
                    if (p.err) atomicOr(p.err + u.s, st);
                    atomicOr(&sh->flags, st);
                }
            }
            if (!(ok = meet())) break;
            const bool bad_unit = sh->flags != 0;
            const bool active = 32 * warp < u.rows;
            see = sh->see[min((u.row + r) / p.G, 127)];
            float m = kNone, l = 0.f;
            bool looked = false;
            for (int tile = u.tile; tile < u.last; ++tile, ++it) {
                const int j0 = tile * KT, ahead = j0 + KT - u.L;  // keys of the tile that are no cached tokens
                if (ahead > 0) {
                    // rows of V past the end, and drafts' that are not finite
                    looked = true;
                    const int pos = it + 1 < total ? 2 * it + 2 : 2 * it + 1, stage = pos % STAGES;
                    if (!(ok = wait_warp(&sh->kv_full[stage], (pos / STAGES) & 1, waits))) break;
                    const int j = j0 + r;
                    if (r < KT && j >= u.L) {
                        unsigned char *const row = kv_tile + stage * K::KV + r * 128;
                        bool clear = j >= end;
                        if (!clear) {
#pragma unroll 4
                            for (int x = 0; x < DP / 8; ++x)
                                clear |= not_finite(*reinterpret_cast<const uint4 *>(row + (x >> 3) * (KT * 128) + (x & 7) * 16));
                            if (clear) atomicOr(&bad[(j - u.L) >> 5], 1u << ((j - u.L) & 31));
                        }
                        if (clear)
#pragma unroll 4
                            for (int x = 0; x < DP / 8; ++x)
                                *reinterpret_cast<uint4 *>(row + (x >> 3) * (KT * 128) + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_smem_to_async();
                }
                if (!(ok = wait_warp(&sh->s_full[it & 1], (it >> 1) & 1, waits))) break;
                tmem_fence_after();
                if (active) {
                    uint32_t s[KT];
                    const uint32_t ts = tl + (it & 1) * KT;
#pragma unroll
                    for (int x = 0; x < KT; x += 32) tmem_ld32(s + x, ts + x);
                    tmem_wait_ld32(s);
#pragma unroll
                    for (int x = 32; x < KT; x += 32) tmem_tie32(s + x);
                    if (ahead > 0) {
                        // bit i of the mask: whether the row sees key j0 + i
                        const int off = u.L - j0;  // of draft 0 in the tile; below 0 it lies before the tile
#pragma unroll
                        for (int w = 0; w < KT / 32; ++w) {
                            const int lo = 32 * w - off;  // draft of the word's first key
                            uint32_t bits;
                            if (lo <= -32) {
                                bits = 0xffffffffu;
                            } else if (lo < 0) {
                                bits = (1u << -lo) - 1 | see.x << -lo;
                            } else {
                                const int word = lo >> 5;
                                const uint32_t a = word == 0 ? see.x : word == 1 ? see.y : word == 2 ? see.z : word == 3 ? see.w : 0u;
                                const uint32_t b = word == 0 ? see.y : word == 1 ? see.z : word == 2 ? see.w : 0u;
                                bits = __funnelshift_r(a, b, lo & 31);
                            }
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                if (!(bits >> x & 1)) s[32 * w + x] = __float_as_uint(kNone);
                        }
                    }
                    float top[4] = {kNone, kNone, kNone, kNone};
#pragma unroll
                    for (int x = 0; x < KT; x += 4)
#pragma unroll
                        for (int e = 0; e < 4; ++e) top[e] = fmaxf(top[e], __uint_as_float(s[x + e]));
                    const float t = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale;
                    if (tile == u.tile) {
                        m = t;
                    } else if (__any_sync(0xffffffffu, t > m + kSlack)) {
                        const float f = t > m + kSlack ? exp2_fast(m - t) : 1.0f;
                        if (t > m + kSlack) m = t, l *= f;
                        if (!(ok = wait_warp(&sh->pv_done, (it - 1) & 1, waits))) break;
                        tmem_fence_after();
                        const uint32_t to = tl + K::COL_O + ob * DP;
#pragma unroll 1
                        for (int x = 0; x < DP; x += 16) {
                            uint32_t o[16];
                            tmem_ld16(o, to + x);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16(to + x, o);
                        }
                    }
                    const float base = m == kNone ? 0.f : -m;
                    const f2 c2 = f2_pack(p.scale, p.scale), b2 = f2_pack(base, base);
                    f2 sum[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
                    for (int x = 0; x < KT; x += 32) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float a, b;
                            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[x + 2 * e]), __uint_as_float(s[x + 2 * e + 1])), c2, b2), a, b);
                            a = exp2_fast(a), b = exp2_fast(b);
                            sum[e & 1] = f2_add(sum[e & 1], f2_pack(a, b));
                            w[e] = pack_bf16(a, b);
                        }
                        tmem_st16(ts + x / 2, w);
                    }
                    float a, b;
                    f2_unpack(f2_add(sum[0], sum[1]), a, b);
                    l += a + b;
                    tmem_wait_st();
                    tmem_fence_before();
                }
                arrive_warp(&sh->p_ready[it & 1]);
            }
            if (!ok || !(ok = wait_warp(&sh->pv_done, (it - 1) & 1, waits))) break;
            tmem_fence_after();
            const uint32_t to = tl + K::COL_O + ob * DP;
            const bool cut = u.last - u.tile < u.tiles;
            if (looked && !(ok = meet())) break;  // (all notes of drafts are there)
            if (active && !bad_unit) {
                if (looked && (bad[0] | bad[1] | bad[2] | bad[3])) add_bad_drafts<DP>(p, u, bad, see, r, m, to);
                const float inv = cut ? 1.0f : 1.0f / l;
                float *const part = cut ? attn_part(p, blockIdx.x, u.begins) : nullptr;
                if (cut && r < u.rows) part[kPartHead + r] = m, part[kPartHead + p.pad + r] = l;
                uint16_t *const out = reinterpret_cast<uint16_t *>(p.out) + (p.cu ? 0LL : (long long)u.s * p.o_seq) +
                                      (long long)(u.row0 + (u.row + r) / p.G) * p.o_tok +
                                      (long long)(u.h * p.G + (u.row + r) % p.G) * p.o_head;
#pragma unroll 1
                for (int x = 0; x < DP; x += 32) {
                    uint32_t o[32];
                    tmem_ld32(o, to + x);
                    tmem_wait_ld32(o);
                    if (r < u.rows && cut) {
                        float4 *const dst = reinterpret_cast<float4 *>(part + kPartHead + 2 * p.pad + (long long)r * DP + x);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]),
                                                 __uint_as_float(o[4 * e + 3]));
                    } else if (r < u.rows) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (x + 8 * e >= p.c.d) break;  // (d is a multiple of 8)
                            uint32_t w[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                w[y] = pack_bf16(__uint_as_float(o[8 * e + 2 * y]) * inv, __uint_as_float(o[8 * e + 2 * y + 1]) * inv);
                            if (mp.o_vec) {
                                *reinterpret_cast<uint4 *>(out + x + 8 * e) = make_uint4(w[0], w[1], w[2], w[3]);
                            } else {
#pragma unroll
                                for (int y = 0; y < 4; ++y) {
                                    out[x + 8 * e + 2 * y] = (uint16_t)w[y];
                                    out[x + 8 * e + 2 * y + 1] = (uint16_t)(w[y] >> 16);
                                }
                            }
                        }
                    }
                    __syncwarp();
                }
            }
            if (cut && r == 0) {
                int *const head = reinterpret_cast<int *>(attn_part(p, blockIdx.x, u.begins));
                head[0] = u.begins && !bad_unit, head[1] = (int)((u.first + u.tiles - 1) / range.per) - (int)blockIdx.x + 1;
                head[2] = u.s, head[3] = u.h, head[4] = u.row, head[5] = 1;
            }
            if (r == 0 && p.ws && !(cut && u.begins)) *reinterpret_cast<int *>(attn_part(p, blockIdx.x, 1)) = 0;
            tmem_fence_before();
            arrive_warp(&sh->o_free[ob]);
        }
    }
    __syncwarp();
    tmem_wait_st();  // (of a role that gave up)
    tmem_fence_before();
    __syncthreads();
    if (tid == 0) {
        if (sh->dead) {
            AttnWalk walk(p, range);
            AttnUnit u;
            while (walk.next(p, u))
                if (p.err) atomicOr(p.err + u.s, kSeqTimeout);
            if (p.ws) reinterpret_cast<int *>(attn_part(p, blockIdx.x, 0))[5] = 0;
        }
        if (p.ws && (sh->dead || total == 0)) *reinterpret_cast<int *>(attn_part(p, blockIdx.x, 1)) = 0;
    }
    if (warp == 5) {
        tmem_fence_after();
        tmem_free(tm, kTmemCols);
    }
}

template <int DP>
AttnTc tc() {
    return {attn_tc<DP>, tc_smem<DP>(), Tc<DP>::KT, kTcThreads};
}

}  // namespace

AttnTc attn_tc_kernel(int dp) { return dp == 64 ? tc<64>() : dp == 128 ? tc<128>() : dp == 192 ? tc<192>() : tc<256>(); }

}  // namespace cvk
