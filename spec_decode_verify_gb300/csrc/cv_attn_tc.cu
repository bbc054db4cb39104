// Attention of drafted tokens over a paged cache on the tensor cores (bf16).
//
// Mathematics.  A unit is up to 128 rows (draft, query head of a group) of one kv head of a sequence.  For each tile of
// KT keys, with c = scale log2(e),
//   S = Q K^T,   p = 2^(c S - m),   l += sum p,   O += P V,      out = O / l
// in one pass over K and V.  m is the row's maximum when it was last moved: it moves only when a tile exceeds it by
// more than 2^8, since that costs a pass over O; until then p is at most 2^8, which bf16 and the fp32 sums hold as well as 1.
// P is rounded to bf16 (2^-8 of a term), as the operand of the second product; l sums what was not rounded.  The outputs are off by
// 2.1e-3 to 2.4e-3 in the mean square for it, 1.65e-3 of them their own rounding.  P in two bf16 parts, a second product with the same V,
// leaves that 1.65e-3 alone and takes longer: 128 x 8 drafts over 8k 206 us against 201, 64 tokens of 32/8 heads of 128 over 2k-4k 157
// against 148, of heads of 64 152 against 125, 17 drafts of 64/8 heads over 100k 131 against 110.
//
// Layout.  A block (one per SM) takes an equal run of the units' work: their key tiles in a row, and for each unit about what
// its beginning and end take, so that all blocks read for the same time whatever the lengths; a unit that is cut leaves (m, l, O) in the workspace
// for the join.  All rows of a kv head's group share one read of its keys, so HBM bounds it: a tile of 128 keys of 128
// channels is 64 KB, 1.4 us of an SM's share, and takes 0.7 us of the tensor pipe at any number of rows.  Two row tiles a unit
// are a chain instead: each group has one buffer of S, so that its next scores wait for its softmax (1650 cycles), its P V and the
// next Q K^T behind the other group's, about 2.2 us a tile (17 drafts of 64/8 heads over 100k 107 us, tensor pipe 47 %, HBM 49 %).
// Roles, each a stream of its own:
//   load K   1 warp: the units (also for the others, through a queue in shared memory), Q and K by TMA, a box for each page
//   load V   1 warp: V (one warp for both took 45 cycles a box, 64 boxes a tile for pages of 16 tokens: slower than HBM)
//   issue    1 warp: Q K^T of the next tile, then P V of this one
//   scout    1 warp: of each sequence the drafts' ancestors, and a look at every page and parent
//   softmax  4 warps, a row a thread: S from tensor memory, P back over it, O's rescaling; or two groups of 4,
//            which write their own rows (see Tc)
//   output   4 warps, a row a thread: O / l, or (m, l, O), to memory, while the next unit runs (beside one group)
// Tensor memory: two buffers of S (and P), O (two for up to 192 channels).
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
constexpr int kTcThreads = 384, kQueue = 4;

// GROUPS: groups of 4 softmax warps.  One takes every tile, and 4 more warps write the outputs while the next unit runs.  Two, in units of
// two row tiles, take a row tile each of every tile of keys, which then serves up to 256 rows, and write their own rows.
template <int DP, int GROUPS>
struct Tc {
    static constexpr int KT = DP <= 128 ? 128 : 64;     // keys a tile
    static constexpr int BLOCKS = DP / 64;              // blocks of 64 channels
    static constexpr int KV = KT * DP * 2, Q = 128 * DP * 2;
    static constexpr int QTILES = DP <= 128 ? 2 : 1;    // of two units in turn, or of the two row tiles
    static constexpr int OBUF = GROUPS * DP <= 192 ? 2 : 1;
    static constexpr int KS = DP == 64 ? 4 : DP == 192 ? 3 : 2, VS = KS;  // stages of K and of V
    static constexpr int COL_O = 2 * KT;
    static_assert(COL_O + OBUF * GROUPS * DP <= 512, "tensor memory");
};
constexpr uint32_t kTmemCols = 512;

struct TcUnit {
    int s, h, row, rows, tile, last, tiles, slot, L, T, row0, begins;
    long long first;
};

struct TcShared {
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4], q_full[2], q_empty[2], s_full[2], p_ready[2], pv_done[2], o_full[2], o_free[2],
        ml_full[2], ml_free[2], see_full[2], see_empty[2], unit_full[kQueue], unit_empty[kQueue], last;
    TcUnit unit[kQueue];
    int unit_pages[kQueue][32];  // the pages of its first tiles
    uint32_t tmem;
    int dead;
    int flags[2];            // of a sequence, and its drafts' ancestors; two in turn
    uint4 see[2][128];
    uint32_t bad[2][8][4];   // drafts whose v holds a NaN or an infinity, as each softmax warp saw them; of two units in turn
    float m[2][128], l[2][128];  // of two units in turn
    AttnTree tree;
    AttnRange range;
    AttnScratch scratch;
};

template <int DP, int GROUPS>
__host__ __device__ constexpr int tc_smem() {
    using K = Tc<DP, GROUPS>;
    return K::QTILES * K::Q + (K::KS + K::VS) * K::KV + (int)sizeof(TcShared) + 1024;
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

// Drafts whose v is not finite, to the rows that see them: their weights again from q and k, and 32 channels of O plus weight
// times v.
__device__ __noinline__ void add_bad_drafts(const AttnParams &p, const TcUnit &u, const uint32_t *bad, uint4 see, int row, int first,
                                            int last, float m, int c0, uint32_t *o) {
    const uint16_t *const q = reinterpret_cast<const uint16_t *>(p.q) + (p.cu ? 0LL : (long long)u.s * p.q_seq) +
                              (long long)(u.row0 + row / p.G) * p.q_tok + (long long)(u.h * p.G + row % p.G) * p.q_head;
    const int *const table = p.c.table + (long long)u.slot * p.c.table_row;
    for (int b = 0; b < u.T; ++b) {
        const int j = u.L + b;
        if (!(bad[b >> 5] >> (b & 31) & 1) || !((&see.x)[b >> 5] >> (b & 31) & 1) || j < first || j >= last) continue;
        const int pg = __ldg(table + j / p.c.page), in = j % p.c.page;
        const uint16_t *const k = reinterpret_cast<const uint16_t *>(p.c.k) + (long long)pg * p.c.k_page +
                                  (long long)in * p.c.k_row + (long long)u.h * p.c.k_head;
        const uint16_t *const v = reinterpret_cast<const uint16_t *>(p.c.v) + (long long)pg * p.c.v_page +
                                  (long long)in * p.c.v_row + (long long)u.h * p.c.v_head;
        float w = 0.f;
        for (int c = 0; c < p.c.d; ++c) w = fmaf(widen<uint16_t>(q[c]), widen<uint16_t>(k[c]), w);
        w = exp2_fast(fmaf(w, p.scale, m == kNone ? 0.f : -m));
        for (int e = 0; e < 32; ++e)
            if (c0 + e < p.c.d) o[e] = __float_as_uint(fmaf(w, widen<uint16_t>(v[c0 + e]), __uint_as_float(o[e])));
    }
}

template <int DP, int GROUPS>
__global__ void __launch_bounds__(kTcThreads, 1) attn_tc(const __grid_constant__ AttnMaps mp) {
    using K = Tc<DP, GROUPS>;
    constexpr int KT = K::KT, KS = K::KS, VS = K::VS;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *const smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) / 1024 * 1024);
    unsigned char *const q_tile = smem, *const k_tile = smem + K::QTILES * K::Q, *const v_tile = k_tile + KS * K::KV;
    TcShared *const sh = reinterpret_cast<TcShared *>(v_tile + VS * K::KV);
    const AttnParams &p = mp.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (dynamic_smem_bytes() < (unsigned)tc_smem<DP, GROUPS>()) return;
    if (tid == 0) {
        for (int i = 0; i < 4; ++i)
            mbar_init(&sh->k_full[i], 1), mbar_init(&sh->k_empty[i], 1), mbar_init(&sh->v_full[i], 1), mbar_init(&sh->v_empty[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->q_full[i], 1), mbar_init(&sh->q_empty[i], 1), mbar_init(&sh->s_full[i], 1), mbar_init(&sh->p_ready[i], 4);
            mbar_init(&sh->o_full[i], 1), mbar_init(&sh->o_free[i], 4 * GROUPS), mbar_init(&sh->ml_full[i], 4 * GROUPS), mbar_init(&sh->ml_free[i], 4);
            mbar_init(&sh->see_full[i], 1), mbar_init(&sh->see_empty[i], 8), mbar_init(&sh->pv_done[i], 1);
        }
        for (int i = 0; i < kQueue; ++i) mbar_init(&sh->unit_full[i], 1), mbar_init(&sh->unit_empty[i], 11);
        mbar_init(&sh->last, 1);
        mbar_init_fence();
        sh->dead = 0;
    }
    if (warp == 5) tmem_alloc(&sh->tmem, kTmemCols);
    if (warp == 4 && lane < 3) {
        const CUtensorMap *const map = lane == 0 ? &mp.q : lane == 1 ? &mp.k : &mp.v;
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(map) : "memory");
    }
    grid_dep_wait();
    grid_dep_launch();
    attn_range(p, &sh->range, &sh->scratch);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tm = sh->tmem;
    const Waits waits{&sh->dead, p.polls};
    const AttnRange &range = sh->range;
    // A step is a tile, or a row tile of one: steps take turns at the two buffers of S, and at the groups.
    constexpr bool pair = GROUPS == 2;
    const int half = mp.tok * p.G;                    // rows of a row tile
    constexpr int q_bufs = pair || K::QTILES == 1 ? 1 : 2;  // units' queries that have a place
    // The next unit of the queue for the calling warp; s < 0 after the last one.
    auto pop = [&](TcUnit &u, int units) {
        const int at = units % kQueue;
        if (!wait_warp(&sh->unit_full[at], (units / kQueue) & 1, waits)) return false;
        u = sh->unit[at];
        arrive_warp(&sh->unit_empty[at]);
        return true;
    };
    // Copies of a tile: a lane takes one block of 64 channels of one page's rows.
    const int boxes = KT / mp.page_rows, tiles_page = p.c.page > KT ? p.c.page / KT : 1;
    const int blk = lane % K::BLOCKS, box = lane / K::BLOCKS;
    // A table row's entries, 32 at a time a lane each, the next 32 on their way (a look-up for each tile held every
    // copy up by its latency: 2850 cycles a tile of 128 x 128, 2.9 us for each stage of shared memory to come round).
    struct Pages {
        const int *row;
        int n, base, cur, next;
        __device__ __forceinline__ int fetch(int at, int lane) const { return at + lane < n ? __ldg(row + at + lane) : 0; }
    };
    Pages pages = {nullptr, 0, 0, 0, 0};
    auto pages_at = [&](int slot, int end, int tile) {
        Pages g;
        g.row = p.c.table + (long long)slot * p.c.table_row, g.n = (end - 1) / p.c.page + 1;
        g.base = tiles_page > 1 ? tile / tiles_page : tile * boxes;
        g.cur = g.next = 0;
        return g;
    };
    auto copy = [&](const CUtensorMap *map, unsigned char *dst, uint64_t *bar, int h, int end, int tile) {
        const int j0 = tile * KT, first = tiles_page > 1 ? tile / tiles_page : tile * boxes;  // (32 is a multiple of boxes)
        if (first - pages.base >= 32) {
            pages.cur = pages.next, pages.base += 32;
            pages.next = pages.fetch(pages.base + 32, lane);
        }
        const int page = __shfl_sync(0xffffffffu, pages.cur, first - pages.base + box);
        const int n = min(boxes, (end - j0 + mp.page_rows - 1) / mp.page_rows);
        if (lane == 0) mbar_arrive_expect_tx(bar, (unsigned)(n * (K::BLOCKS * 128) * mp.page_rows));
        __syncwarp();
        if (box < n)
            tma_load4(smem_u32(dst) + blk * (KT * 128) + box * mp.page_rows * 128, map, blk * 64, (tile % tiles_page) * KT, h, page, bar);
    };

    // A row tile's outputs, or its part of them, from tensor memory: row r of the tile a thread, with its maximum and sum; b: which notes
    // of drafts, q: which sequence's masks.
    bool goes_on = false, came = false;  // parts left in slots 1 and 0
    auto leave = [&](const TcUnit &u, int y, uint32_t to, int r, float m, float l, int b, int q) {
        const bool bad_unit = sh->flags[q] != 0, cut = u.last - u.tile < u.tiles;
        goes_on = cut && u.begins && !bad_unit;
        came |= cut && !u.begins && !bad_unit;
        const int row = y * half + r;  // of the unit
        const bool on = r < half && row < u.rows;
        if (bad_unit || !__any_sync(0xffffffffu, on)) return;
        uint32_t bad[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            bad[i] = 0;
#pragma unroll
            for (int w = 0; w < 4 * GROUPS; ++w) bad[i] |= sh->bad[b][w][i];
        }
        const float inv = cut ? 1.0f : 1.0f / l;
        float *const part = cut ? attn_part(p, blockIdx.x, u.begins) : nullptr;
        if (cut && on) part[kPartHead + row] = m, part[kPartHead + p.pad + row] = l;
        if (cut && row == 0) attn_part_head(part, range, u.first, u.tiles, u.rows, u.row, u.s, u.h, u.row0);
        uint16_t *const out = reinterpret_cast<uint16_t *>(p.out) + (p.cu ? 0LL : (long long)u.s * p.o_seq) +
                              (long long)(u.row0 + (u.row + row) / p.G) * p.o_tok +
                              (long long)(u.h * p.G + (u.row + row) % p.G) * p.o_head;
#pragma unroll 1
        for (int x = 0; x < DP; x += 32) {
            uint32_t o[32];
            tmem_ld32(o, to + x);
            tmem_wait_ld32(o);
            if (on && (bad[0] | bad[1] | bad[2] | bad[3])) {
                uint32_t c[32];  // (o itself stays in registers)
#pragma unroll
                for (int e = 0; e < 32; ++e) c[e] = o[e];
                add_bad_drafts(p, u, bad, sh->see[q][(u.row + row) / p.G], u.row + row, u.tile * KT, u.last * KT, m, x, c);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = c[e];
            }
            if (on && cut) {
                float4 *const dst = reinterpret_cast<float4 *>(part + kPartHead + 2 * p.pad + (long long)row * DP + x);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dst[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]),
                                         __uint_as_float(o[4 * e + 3]));
            } else if (on) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (x + 8 * e >= p.c.d) break;  // (d is a multiple of 8)
                    uint32_t w[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        w[z] = pack_bf16(__uint_as_float(o[8 * e + 2 * z]) * inv, __uint_as_float(o[8 * e + 2 * z + 1]) * inv);
                    if (mp.o_vec) {
                        *reinterpret_cast<uint4 *>(out + x + 8 * e) = make_uint4(w[0], w[1], w[2], w[3]);
                    } else {
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            out[x + 8 * e + 2 * z] = (uint16_t)w[z];
                            out[x + 8 * e + 2 * z + 1] = (uint16_t)(w[z] >> 16);
                        }
                    }
                }
            }
            __syncwarp();
        }
    };
    // The join reads both slots of every block: what is not there, after the last unit (the caller's first thread).
    auto left_out = [&] {
        if (p.ws && !goes_on) *reinterpret_cast<int *>(attn_part(p, blockIdx.x, 1)) = 0;
        if (p.ws && !came) *reinterpret_cast<int *>(attn_part(p, blockIdx.x, 0)) = 0;
    };

    if (warp == 4) {
        // ------------------------------------------------------------------- load: units, Q, K
        AttnWalk walk(p, range);
        AttnUnit u, next;
        bool has = walk.next(p, u), ok = true;
        int units = 0, it = 0;
        auto publish = [&](bool end) {
            const int at = units % kQueue;
            if (units >= kQueue && !wait_warp(&sh->unit_empty[at], (units / kQueue - 1) & 1, waits)) return false;
            if (lane == 0) {
                TcUnit &t = sh->unit[at];
                t.s = end ? -1 : u.s, t.h = u.h, t.row = u.row, t.rows = u.rows, t.tile = u.tile, t.last = u.last, t.tiles = u.tiles;
                t.slot = u.q.slot, t.L = u.q.L, t.T = u.q.T, t.row0 = u.q.row0, t.first = u.first, t.begins = u.tile == 0;
            }
            sh->unit_pages[at][lane] = pages.cur;
            arrive_warp(&sh->unit_full[at]);
            return true;
        };
        // a unit ahead of its copies: the next one's lengths and first pages are looked up while this one's keys are copied
        Pages ahead = pages;
        auto look = [&](const AttnUnit &a) {
            ahead = pages_at(a.q.slot, a.q.L + a.q.T, a.tile);
            ahead.cur = ahead.fetch(ahead.base, lane), ahead.next = ahead.fetch(ahead.base + 32, lane);
        };
        if (has) look(u);
        while (ok && has) {
            pages = ahead;
            if (!(ok = publish(false))) break;
            const int qb = q_bufs == 2 ? units & 1 : 0, end = u.q.L + u.q.T, tiles_q = pair ? 2 : 1;
            if (units >= q_bufs && !(ok = wait_warp(&sh->q_empty[qb], (units / q_bufs - 1) & 1, waits))) break;
            if (lane == 0) mbar_arrive_expect_tx(&sh->q_full[qb], (unsigned)(tiles_q * K::BLOCKS * 128 * half));
            __syncwarp();
            if (lane < K::BLOCKS * tiles_q) {
                const int x = lane % K::BLOCKS, y = lane / K::BLOCKS;  // (rows past the tensor's end are zeros)
                tma_load4(smem_u32(q_tile) + (qb + y) * K::Q + x * (128 * 128), &mp.q, x * 64, u.h * p.G,
                          u.q.row0 + u.row / p.G + y * mp.tok, p.cu ? 0 : u.s, &sh->q_full[qb]);
            }
            ++units;
            bool has_next = false;
            for (int tile = u.tile; tile < u.last; ++tile, ++it) {
                const int stage = it % KS;
                if (it >= KS && !(ok = wait_warp(&sh->k_empty[stage], (it / KS - 1) & 1, waits))) break;
                copy(&mp.k, k_tile + stage * K::KV, &sh->k_full[stage], u.h, end, tile);
                if (tile == u.tile) {
                    has_next = walk.next(p, next);
                    if (has_next) look(next);
                }
            }
            u = next, has = has_next;
        }
        if (ok) publish(true);
        // nothing of the block's is in flight when it returns
        __syncwarp();
        for (int x = max(0, it - KS); x < it; ++x) mbar_wait_bounded(&sh->k_full[x % KS], (x / KS) & 1, kDrainPolls);
        for (int x = max(0, units - q_bufs); x < units; ++x) mbar_wait_bounded(&sh->q_full[x % q_bufs], (x / q_bufs) & 1, kDrainPolls);
    } else if (warp == 7) {
        // --------------------------------------------------------------------------- load: V
        int it = 0;
        bool ok = true;
        TcUnit u;
        for (int units = 0; ok; ++units) {
            const int at = units % kQueue;
            if (!(ok = wait_warp(&sh->unit_full[at], (units / kQueue) & 1, waits))) break;
            u = sh->unit[at];
            const int first = sh->unit_pages[at][lane];
            arrive_warp(&sh->unit_empty[at]);
            if (u.s < 0) break;
            const int end = u.L + u.T;
            pages = pages_at(u.slot, end, u.tile);
            pages.cur = first, pages.next = pages.fetch(pages.base + 32, lane);
            for (int tile = u.tile; tile < u.last; ++tile, ++it) {
                const int stage = it % VS;
                if (it >= VS && !(ok = wait_warp(&sh->v_empty[stage], (it / VS - 1) & 1, waits))) break;
                copy(&mp.v, v_tile + stage * K::KV, &sh->v_full[stage], u.h, end, tile);
            }
        }
        __syncwarp();
        for (int x = max(0, it - VS); x < it; ++x) mbar_wait_bounded(&sh->v_full[x % VS], (x / VS) & 1, kDrainPolls);
    } else if (warp == 6) {
        // ----------------------------------------------------------------------------- scout
        int seqs = 0, s_before = -1;
        TcUnit u;
        for (int units = 0; pop(u, units) && u.s >= 0; ++units) {
            if (u.s == s_before) continue;
            s_before = u.s;
            const int b = seqs & 1;
            if (seqs >= 2 && !wait_warp(&sh->see_empty[b], ((seqs >> 1) - 1) & 1, waits)) break;
            ++seqs;
            const int *const parent = p.parent ? p.parent + (p.cu ? (long long)u.row0 : (long long)u.s * p.T) : nullptr;
            int st = attn_ancestors(parent, u.T, lane, 32, &sh->tree, sh->see[b], [] { __syncwarp(); }) ? kSeqBadTree : 0;
            const int *const table = p.c.table + (long long)u.slot * p.c.table_row;
            const int pages = (u.L + u.T - 1) / p.c.page + 1;
#pragma unroll 8
            for (int i = lane; i < pages; i += 32) {
                const int g = __ldg(table + i);
                if (g < 0 || g >= p.c.n_pages) st |= kSeqBadPage;
            }
            st = __reduce_or_sync(0xffffffffu, (unsigned)st);
            if (lane == 0) {
                if (st && p.err) atomicOr(p.err + u.s, st);
                sh->flags[b] = st;
            }
            arrive_warp(&sh->see_full[b]);
        }
    } else if (warp == 5) {
        // ----------------------------------------------------------------------------- issue
        const uint32_t lead = elect_lane();
        constexpr uint32_t id_qk = mma_desc(KT, false, false), id_pv = mma_desc(DP, false, true);
        int units = 0, qk_left = 0, n_next = 0, it = 0, pv_unit = 0, pv_left = 0, pv_at = 0;  // it: steps
        auto steps = [&](int &n) {  // of the next unit; 0 after the last one
            const int at = units % kQueue;
            if (!wait_warp(&sh->unit_full[at], (units / kQueue) & 1, waits)) return false;
            n = sh->unit[at].s < 0 ? 0 : (sh->unit[at].last - sh->unit[at].tile) * (pair ? 2 : 1);
            arrive_warp(&sh->unit_empty[at]);
            ++units;
            return true;
        };
        auto scores = [&](int i, bool first, bool last) {
            const int qb = (units - 1) % q_bufs, tile = pair ? i >> 1 : i, stage = tile % KS;
            if (first && !wait_warp(&sh->q_full[qb], ((units - 1) / q_bufs) & 1, waits)) return false;
            if (!wait_warp(&sh->k_full[stage], (tile / KS) & 1, waits)) return false;
            tmem_fence_after();
            const uint32_t q = desc_k(smem_u32(q_tile) + (pair ? i & 1 : qb) * K::Q), k = desc_k(smem_u32(k_tile) + stage * K::KV);
#pragma unroll 4
            for (int x = 0; x < DP / 16; ++x)
                mma_ss(lead, tm + (i & 1) * KT, q + (((x >> 2) * (128 * 128) + (x & 3) * 32) >> 4),
                       k + (((x >> 2) * (KT * 128) + (x & 3) * 32) >> 4), id_qk, x > 0);
            mma_commit(lead, &sh->s_full[i & 1]);
            if (!pair || (i & 1)) mma_commit(lead, &sh->k_empty[stage]);
            if (last) mma_commit(lead, &sh->q_empty[qb]);
            return true;
        };
        int n = 0;
        bool ok = steps(n) && n > 0;
        if (ok) {
            qk_left = pv_left = n;
            ok = scores(0, true, n == 1);
            --qk_left;
        }
        while (ok) {
            ok = false;
            if (qk_left > 0) {
                if (!scores(it + 1, false, qk_left == 1)) break;
                --qk_left;
            } else if (n > 0) {
                if (!steps(n)) break;
                n_next = n;
                if (n > 0) {
                    if (!scores(it + 1, true, n == 1)) break;
                    qk_left = n - 1;
                }
            }
            const int ob = pv_unit % K::OBUF, tile = pair ? it >> 1 : it, stage = tile % VS, g = GROUPS == 2 ? it & 1 : 0;
            if (pv_at == 0 && pv_unit >= K::OBUF && !wait_warp(&sh->o_free[ob], (pv_unit / K::OBUF - 1) & 1, waits)) break;
            if (!wait_warp(&sh->v_full[stage], (tile / VS) & 1, waits) || !wait_warp(&sh->p_ready[it & 1], (it >> 1) & 1, waits)) break;
            tmem_fence_after();
            const uint32_t v = desc_mn(smem_u32(v_tile) + stage * K::KV, KT * 128);
#pragma unroll 4
            for (int x = 0; x < KT / 16; ++x)
                mma_ts(lead, tm + K::COL_O + (ob * GROUPS + g) * DP, tm + (it & 1) * KT + x * 8, v + x * 128, id_pv,
                       pv_at >= GROUPS || x > 0);
            if (!pair || (it & 1)) mma_commit(lead, &sh->v_empty[stage]);
            mma_commit(lead, &sh->pv_done[g]);
            ++it, ++pv_at;
            ok = true;
            if (--pv_left == 0) {
                mma_commit(lead, &sh->o_full[ob]);
                if (n == 0) break;  // the last unit
                ++pv_unit, pv_at = 0, pv_left = n_next;
            }
        }
        // nothing of the block's is in flight when it gives tensor memory back
        mma_commit(lead, &sh->last);
        mbar_wait_bounded(&sh->last, 0, kDrainPolls);
    } else if (warp < 4 || GROUPS == 2) {
        // --------------------------------------------------------------------------- softmax
        const int g = warp >= 8, w4 = warp & 3, r = 32 * w4 + lane;  // the group, and the row of its row tile
        const uint32_t tl = tm + ((uint32_t)(32 * w4) << 16);
        int it = 0, s_before = -1, seqs = 0;  // seqs: sequences begun
        uint4 see = make_uint4(0, 0, 0, 0);
        bool ok = true;
        TcUnit u;
        for (int units = 0; ok && (ok = pop(u, units)) && u.s >= 0; ++units) {
            const int ob = units % K::OBUF, b = units & 1;
            // the unit two before has left its place (and its sequence's masks: no warp is two sequences ahead of another)
            if (!pair && units >= 2 && !(ok = wait_warp(&sh->ml_free[b], ((units >> 1) - 1) & 1, waits))) break;
            if (u.s != s_before) {
                if (seqs > 0) arrive_warp(&sh->see_empty[(seqs - 1) & 1]);
                s_before = u.s, ++seqs;
            }
            if (lane < 4) sh->bad[b][4 * g + w4][lane] = 0;
            __syncwarp();
            const int end = u.L + u.T;
            const bool active = 32 * w4 < (pair ? min(u.rows - g * half, half) : u.rows);
            float m = kNone, l = 0.f;
            bool sees = false, begun = false;
            const int to_do = (u.last - u.tile) * (pair ? 2 : 1);
            for (int step = 0; step < to_do; ++step, ++it) {
                if (GROUPS == 2 && (it & 1) != g) continue;
                const int tile = u.tile + (pair ? step >> 1 : step), key_tile = pair ? it >> 1 : it;
                const int j0 = tile * KT, ahead = j0 + KT - u.L;  // keys of the tile that are no cached tokens
                if (ahead > 0) {
                    if (!sees) {
                        if (!(ok = wait_warp(&sh->see_full[(seqs - 1) & 1], ((seqs - 1) >> 1) & 1, waits))) break;
                        see = sh->see[(seqs - 1) & 1][min((u.row + (pair ? g * half : 0) + r) / p.G, 127)];
                        sees = true;
                    }
                    // Rows of V past the end, and drafts' that are not finite.  A stage is not touched before the tile that it held
                    // before has been read: it has once this step's scores are there, whose product was issued after that
                    // one's.  (V's barrier alone does not tell: two phases back looks like this one.)
                    const int stage = key_tile % VS;
                    if (key_tile >= VS && !(ok = wait_warp(&sh->s_full[it & 1], (it >> 1) & 1, waits))) break;
                    if (!(ok = wait_warp(&sh->v_full[stage], (key_tile / VS) & 1, waits))) break;
                    const int j = j0 + r;
                    if (r < KT && j >= u.L) {
                        unsigned char *const row = v_tile + stage * K::KV + r * 128;
                        bool clear = j >= end;
                        if (!clear) {
#pragma unroll 4
                            for (int x = 0; x < DP / 8; ++x)
                                clear |= not_finite(*reinterpret_cast<const uint4 *>(row + (x >> 3) * (KT * 128) + (x & 7) * 16));
                            if (clear) atomicOr(&sh->bad[b][4 * g + w4][(j - u.L) >> 5], 1u << ((j - u.L) & 31));
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
                    const uint32_t ts = tl + (it & 1) * KT;
                    // Word w of the mask: whether the row sees keys j0 + 32 w and on.
                    auto seen = [&](int w) {
                        const int lo = 32 * w - (u.L - j0);  // draft of the word's first key
                        if (lo <= -32) return 0xffffffffu;
                        if (lo < 0) return ((1u << -lo) - 1) | see.x << -lo;
                        const int word = lo >> 5;
                        const uint32_t a = word == 0 ? see.x : word == 1 ? see.y : word == 2 ? see.z : word == 3 ? see.w : 0u;
                        const uint32_t c = word == 0 ? see.y : word == 1 ? see.z : word == 2 ? see.w : 0u;
                        return __funnelshift_r(a, c, lo & 31);
                    };
                    auto mask = [&](uint32_t *s, int w) {
                        const uint32_t bits = seen(w);
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (!(bits >> x & 1)) s[x] = __float_as_uint(kNone);
                    };
                    float top[4] = {kNone, kNone, kNone, kNone};
                    auto most = [&](const uint32_t *s) {
#pragma unroll
                        for (int x = 0; x < 32; ++x) top[x & 3] = fmaxf(top[x & 3], __uint_as_float(s[x]));
                    };
                    uint32_t s[KT];
#pragma unroll
                    for (int x = 0; x < KT; x += 32) tmem_ld32(s + x, ts + x);
                    tmem_wait_ld32(s);
#pragma unroll
                    for (int x = 32; x < KT; x += 32) tmem_tie32(s + x);
#pragma unroll
                    for (int x = 0; x < KT; x += 32) {
                        if (ahead > 0) mask(s + x, x / 32);
                        most(s + x);
                    }
                    const float t = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale;
                    if (!begun) {
                        m = t;
                    } else if (__any_sync(0xffffffffu, t > m + kSlack)) {
                        const float f = t > m + kSlack ? exp2_fast(m - t) : 1.0f;
                        if (t > m + kSlack) m = t, l *= f;
                        // (this group's last step: the one before, or the one before that)
                        if (!(ok = GROUPS == 1 ? wait_warp(&sh->pv_done[0], (it - 1) & 1, waits)
                                               : wait_warp(&sh->pv_done[g], ((it >> 1) - 1) & 1, waits)))
                            break;
                        tmem_fence_after();
                        const uint32_t to = tl + K::COL_O + (ob * GROUPS + g) * DP;
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
                            float a, c;
                            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[x + 2 * e]), __uint_as_float(s[x + 2 * e + 1])), c2, b2), a, c);
                            a = exp2_fast(a), c = exp2_fast(c);
                            sum[e & 1] = f2_add(sum[e & 1], f2_pack(a, c));
                            w[e] = pack_bf16(a, c);
                        }
                        tmem_st16(ts + x / 2, w);
                    }
                    float a, c;
                    f2_unpack(f2_add(sum[0], sum[1]), a, c);
                    l += a + c;
                    tmem_wait_st();
                    tmem_fence_before();
                }
                begun = true;
                arrive_warp(&sh->p_ready[it & 1]);
            }
            if (!ok) break;
            if (!pair) {
                sh->m[b][r] = m, sh->l[b][r] = l;
                arrive_warp(&sh->ml_full[b]);
                continue;
            }
            // its own rows, once both groups' notes of drafts are there (one may have cleared a row before the other looked)
            arrive_warp(&sh->ml_full[b]);
            if (!(ok = wait_warp(&sh->see_full[(seqs - 1) & 1], ((seqs - 1) >> 1) & 1, waits)) ||
                !(ok = wait_warp(&sh->ml_full[b], (units >> 1) & 1, waits)) || !(ok = wait_warp(&sh->o_full[ob], (units / K::OBUF) & 1, waits)))
                break;
            tmem_fence_after();
            leave(u, g, tl + K::COL_O + (ob * GROUPS + g) * DP, r, m, l, b, (seqs - 1) & 1);
            tmem_fence_before();
            arrive_warp(&sh->o_free[ob]);
        }
        if (pair && g == 0 && r == 0) left_out();
    } else {
        // ---------------------------------------------------------------------------- output
        const int w4 = warp - 8, r = 32 * w4 + lane;  // the row
        const uint32_t tl = tm + ((uint32_t)(32 * w4) << 16);
        int s_before = -1, seqs = 0;
        bool ok = true;
        TcUnit u;
        for (int units = 0; ok && (ok = pop(u, units)) && u.s >= 0; ++units) {
            const int ob = units % K::OBUF, b = units & 1;
            if (u.s != s_before) {
                if (seqs > 0) arrive_warp(&sh->see_empty[(seqs - 1) & 1]);
                s_before = u.s, ++seqs;
            }
            if (!(ok = wait_warp(&sh->see_full[(seqs - 1) & 1], ((seqs - 1) >> 1) & 1, waits)) ||
                !(ok = wait_warp(&sh->ml_full[b], (units >> 1) & 1, waits)) ||
                !(ok = wait_warp(&sh->o_full[ob], (units / K::OBUF) & 1, waits)))
                break;
            tmem_fence_after();
            leave(u, 0, tl + K::COL_O + ob * DP, r, sh->m[b][r], sh->l[b][r], b, (seqs - 1) & 1);
            tmem_fence_before();
            arrive_warp(&sh->o_free[ob]);
            arrive_warp(&sh->ml_free[b]);
        }
        if (r == 0) left_out();
    }
    __syncwarp();
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");  // (of a role that gave up)
    tmem_wait_st();
    tmem_fence_before();
    __syncthreads();
    if (tid == 0 && sh->dead) {
        AttnWalk walk(p, range);
        AttnUnit u;
        while (walk.next(p, u))
            if (p.err) atomicOr(p.err + u.s, kSeqTimeout);
        if (p.ws) {
            *reinterpret_cast<int *>(attn_part(p, blockIdx.x, 0)) = 0;
            *reinterpret_cast<int *>(attn_part(p, blockIdx.x, 1)) = 0;
        }
    }
    if (warp == 5) {
        tmem_fence_after();
        tmem_free(tm, kTmemCols);
    }
}

template <int DP, int GROUPS>
AttnTc tc() {
    return {attn_tc<DP, GROUPS>, tc_smem<DP, GROUPS>(), Tc<DP, GROUPS>::KT, kTcThreads};
}

}  // namespace

AttnTc attn_tc_kernel(int dp, bool two) {
    if (dp == 64) return two ? tc<64, 2>() : tc<64, 1>();
    if (dp == 128) return two ? tc<128, 2>() : tc<128, 1>();
    return dp == 192 ? tc<192, 1>() : tc<256, 1>();
}

}  // namespace cvk
