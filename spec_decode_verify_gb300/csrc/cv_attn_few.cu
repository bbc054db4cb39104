// Attention of few rows over a paged cache in fp32 products: units of at most 8 rows (draft, query head) of a kv head, where the
// rows of the cache are whole 16-byte pieces.  Single tokens in fp32, and bf16 ones over pages that the tensor-core kernel does not take.
//
// Mathematics, with c = scale log2(e):  p = 2^(c q.k - m),  l += sum p,  O += p V,  out = O / l.  m moves only when a
// score exceeds it by more than 8, since that costs a pass over O; fp32 holds a weight of 2^8 as well as 1.
//
// Layout.  Nothing of K and V is used twice by few rows, so they go from memory to registers and not through shared
// memory: a warp takes 8 keys of every 64, a lane 4 channels of a key (8 of 256; 64 channels are half a warp's), with
// the rows of O that it needs of them in registers (those of Q as well spilled: 75 us against 67 for 13 tokens of 64/8 heads of 128
// over 3k).  The 16 sums of R rows and NK keys are added up over the lanes by halves that are exchanged, 16 shuffles (15 for heads of 64), after
// which a lane has the score of one row and one key, and one exponential.  (Four keys a lane: 69 us.)  The warps have
// maxima, sums and outputs of their own, which are joined at a unit's end.
//
// HBM bounds one row a head: 16 tokens of 8 heads of 256 over 4k take 151 us, 5.9 TB/s; 13 tokens of 32/8 heads of 128 over 6k take 80, 4.9
// TB/s.  With 8 rows instructions (half of the issue slots) and the loads' latency share the time, which 128 registers do not
// hide better: 13 tokens of 64/8 heads over 20k take 330 us, 3.9 TB/s, and 338 with the loads two steps ahead, which spill.
#include "cv_attn.cuh"

namespace cvk {
namespace {

constexpr float kNone = -INFINITY;
constexpr float kSlack = 8.0f;
constexpr int kWarps = kFewThreads / 32, kRun = kFewKeys / kWarps;  // keys of a tile that a warp takes

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <typename B>
struct Raw4 {
    uint32_t w[sizeof(B)];  // 4 channels as they lie in memory
};
template <typename B>
__device__ __forceinline__ Raw4<B> load4(const B *p, bool on) {
    Raw4<B> r;
    if (sizeof(B) == 4) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (on) x = __ldg(reinterpret_cast<const uint4 *>(p));
        r.w[0] = x.x, r.w[1] = x.y, r.w[sizeof(B) / 2] = x.z, r.w[sizeof(B) - 1] = x.w;
    } else {
        uint2 x = make_uint2(0, 0);
        if (on) x = __ldg(reinterpret_cast<const uint2 *>(p));
        r.w[0] = x.x, r.w[1] = x.y;
    }
    return r;
}
template <typename B>
__device__ __forceinline__ float4 wide4(const Raw4<B> &r) {
    if (sizeof(B) == 4)
        return make_float4(__uint_as_float(r.w[0]), __uint_as_float(r.w[1]), __uint_as_float(r.w[sizeof(B) / 2]),
                           __uint_as_float(r.w[sizeof(B) - 1]));
    return make_float4(__uint_as_float(r.w[0] << 16), __uint_as_float(r.w[0] & 0xffff0000u), __uint_as_float(r.w[1] << 16),
                       __uint_as_float(r.w[1] & 0xffff0000u));
}

// Sums over 2 * OFF lanes of N values: the lane with bit OFF set goes on with the upper half of them.
template <int N, int OFF>
__device__ __forceinline__ void exchange(float *s, int lane) {
    if constexpr (N > 1) {
        const bool up = lane & OFF;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float keep = up ? s[i + N / 2] : s[i], give = up ? s[i] : s[i + N / 2];
            s[i] = keep + __shfl_xor_sync(0xffffffffu, give, OFF);
        }
    } else {
        s[0] += __shfl_xor_sync(0xffffffffu, s[0], OFF);
    }
    if constexpr (OFF > 1) exchange<(N > 1 ? N / 2 : 1), OFF / 2>(s, lane);
}

template <int DP, int R>
struct Few {
    static constexpr int NV = DP > 128 ? 2 : 1;                // pieces of 4 channels of a lane
    static constexpr int LANES = DP / (4 * NV), SIDES = 32 / LANES;  // lanes of a key; keys side by side in a warp
    static constexpr int NK = 16 / R;                          // keys that a lane has at a time
    static constexpr int GROUP = NK * SIDES, VALS = R * NK, SAME = LANES / VALS;  // SAME: lanes that end up with the same score
    static_assert(kRun % GROUP == 0 && VALS * SAME == LANES, "a warp's keys of a tile are whole groups");
};
template <int DP, int R>
struct FewShared {
    float q[R][DP], o[kWarps][R][DP], p[kWarps][2][Few<DP, R>::GROUP][R];
    float m[kWarps][R], l[kWarps][R];
    long long k_at[kWarps][2][32], v_at[kWarps][2][32];  // where the warp's keys stand, -1: none; two batches of 32 in turn
    AttnTree tree;
    uint4 see[128];
    AttnRange range;
    AttnScratch scratch;
};

template <typename B, int DP, int R>
__global__ void __launch_bounds__(kFewThreads, DP <= 128 ? 2 : 1) attn_few(const __grid_constant__ AttnParams p) {
    using F = Few<DP, R>;
    constexpr int NV = F::NV, LANES = F::LANES, NK = F::NK, GROUP = F::GROUP, VALS = F::VALS, SAME = F::SAME, C4 = DP / 4;
    constexpr int BATCH = 32 / GROUP;  // groups of a batch
    extern __shared__ __align__(16) unsigned char smem[];
    FewShared<DP, R> *sh = reinterpret_cast<FewShared<DP, R> *>(smem);
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, d = p.c.d;
    const int side = lane / LANES, at = lane % LANES, mine = at / SAME, row = mine / NK, key = side * NK + mine % NK;
    attn_range(p, &sh->range, &sh->scratch);
    AttnWalk walk(p, sh->range);
    AttnUnit u;
    int s_before = -1;
    bool bad = false, goes_on = false, came = false;  // parts left in slots 1 and 0
    while (walk.next(p, u)) {
        const B *const K = reinterpret_cast<const B *>(p.c.k) + (long long)u.h * p.c.k_head + 4 * at;
        const B *const V = reinterpret_cast<const B *>(p.c.v) + (long long)u.h * p.c.v_head + 4 * at;
        const int *const table = p.c.table + (long long)u.q.slot * p.c.table_row;
        const int L = u.q.L, T = u.q.T, end = L + T;
        __syncthreads();
        if (u.s != s_before) {
            s_before = u.s;
            const int *parent = p.parent ? p.parent + (p.cu ? (long long)u.q.row0 : (long long)u.s * p.T) : nullptr;
            int st = attn_ancestors(parent, T, tid, kFewThreads, &sh->tree, sh->see, [] { __syncthreads(); }) ? kSeqBadTree : 0;
            for (int i = tid; i <= (end - 1) / p.c.page; i += kFewThreads) {
                const int g = __ldg(table + i);
                if (g < 0 || g >= p.c.n_pages) st |= kSeqBadPage;
            }
            if (st && p.err) atomicOr(p.err + u.s, st);
            bad = __syncthreads_or(st) != 0;
        }
        const bool cut = u.last - u.tile < u.tiles, begins = u.tile == 0;
        goes_on = cut && begins && !bad;
        came |= cut && !begins && !bad;
        if (bad) continue;
        for (int i = tid; i < R * C4; i += kFewThreads) {
            const int r = i / C4, c = i % C4 * 4, t = (u.row + r) / p.G, g = (u.row + r) % p.G;
            const B *const from = reinterpret_cast<const B *>(p.q) + (p.cu ? 0LL : (long long)u.s * p.q_seq) +
                                  (long long)(u.q.row0 + t) * p.q_tok + (long long)(u.h * p.G + g) * p.q_head + c;
            *reinterpret_cast<float4 *>(&sh->q[r][c]) = wide4<B>(load4<B>(from, r < u.rows && c < d));
        }
        float4 o[R][NV];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int v = 0; v < NV; ++v) o[r][v] = make_float4(0.f, 0.f, 0.f, 0.f);
        // the warp's keys, n = 0, 1, ...: kRun of each tile
        const int n_keys = (u.last - u.tile) * kRun, groups = n_keys / GROUP;
        auto key_at = [&](int n) { return (u.tile + n / kRun) * kFewKeys + warp * kRun + n % kRun; };
        // (looked up two batches ahead: a key past the run's, which may be past 2^31 too, is never made)
        auto page_of = [&](int batch) {
            const int n = 32 * batch + lane;
            if (n >= n_keys) return -1;
            const int j = key_at(n);
            return j < end ? __ldg(table + j / p.c.page) : -1;
        };
        auto place = [&](int batch, int page) {
            long long k_at = -1, v_at = -1;
            if (page >= 0) {
                const int in = key_at(32 * batch + lane) % p.c.page;
                k_at = (long long)page * p.c.k_page + (long long)in * p.c.k_row;
                v_at = (long long)page * p.c.v_page + (long long)in * p.c.v_row;
            }
            sh->k_at[warp][batch & 1][lane] = k_at, sh->v_at[warp][batch & 1][lane] = v_at;
        };
        auto load = [&](Raw4<B> (&x)[NK][NV], const B *base, const long long (&places)[2][32], int g) {
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                const long long to = places[g / BATCH & 1][g % BATCH * GROUP + side * NK + k];
#pragma unroll
                for (int v = 0; v < NV; ++v) x[k][v] = load4<B>(base + to + 128 * v, to >= 0 && 4 * at + 128 * v < d);
            }
        };
        float m = kNone, l = 0.f;  // of this lane's row; l: its keys' part
        const int t_mine = min((u.row + row) / p.G, 127);
        Raw4<B> k_raw[NK][NV], v_raw[NK][NV];
        place(0, page_of(0));
        int page = page_of(1);
        __syncthreads();
        load(k_raw, K, sh->k_at[warp], 0);
        load(v_raw, V, sh->v_at[warp], 0);
#pragma unroll 1
        for (int g = 0; g < groups; ++g) {
            if (g % BATCH == 0) {
                place(g / BATCH + 1, page);
                page = page_of(g / BATCH + 2);
                __syncwarp();
            }
            float s[VALS];  // [row][key]
#pragma unroll
            for (int v = 0; v < NV; ++v) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float4 b = *reinterpret_cast<const float4 *>(&sh->q[r][4 * at + 128 * v]);
#pragma unroll
                    for (int k = 0; k < NK; ++k) {
                        const float4 a = wide4<B>(k_raw[k][v]);
                        const float first = v == 0 ? a.x * b.x : fmaf(a.x, b.x, s[r * NK + k]);
                        s[r * NK + k] = fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, first)));
                    }
                }
            }
            if (g + 1 < groups) load(k_raw, K, sh->k_at[warp], g + 1);
            exchange<VALS, LANES / 2>(s, lane);
            float x = s[0] * p.scale;
            const int j0 = key_at(g * GROUP);
            const bool masked = j0 + GROUP > L;
            if (masked) {
                const int back = j0 + key - L;
                if (back >= 0 && (back >= T || !((&sh->see[t_mine].x)[back >> 5] >> (back & 31) & 1))) x = kNone;
            }
            if (__any_sync(0xffffffffu, x > m + kSlack)) {
                float top = fmaxf(m, x);
#pragma unroll
                for (int off = NK * SAME / 2; off >= SAME; off /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                if (LANES == 16) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                const float down = top == kNone ? 1.f : ex2(m - top);
                l *= down, m = top;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float f = __shfl_sync(0xffffffffu, down, r * NK * SAME);
#pragma unroll
                    for (int v = 0; v < NV; ++v) o[r][v].x *= f, o[r][v].y *= f, o[r][v].z *= f, o[r][v].w *= f;
                }
            }
            const float e = ex2(x - (m == kNone ? 0.f : m));
            l += e;
            if (at % SAME == 0) sh->p[warp][g & 1][key][row] = e;
            __syncwarp();
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                float w[R];
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(&sh->p[warp][g & 1][side * NK + k][r]);
                    w[r] = f.x, w[r + 1] = f.y, w[r + 2] = f.z, w[r + 3] = f.w;
                }
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const float4 a = wide4<B>(v_raw[k][v]);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        // (a key that a row does not see has weight 0, and 0 times a NaN or an infinity is left out)
                        if (masked && w[r] == 0.f) continue;
                        o[r][v].x = fmaf(w[r], a.x, o[r][v].x), o[r][v].y = fmaf(w[r], a.y, o[r][v].y);
                        o[r][v].z = fmaf(w[r], a.z, o[r][v].z), o[r][v].w = fmaf(w[r], a.w, o[r][v].w);
                    }
                }
            }
            if (g + 1 < groups) load(v_raw, V, sh->v_at[warp], g + 1);
        }
#pragma unroll
        for (int off = NK * SAME / 2; off >= SAME; off /= 2) l += __shfl_xor_sync(0xffffffffu, l, off);
        if (LANES == 16) l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (side == 0 && at % (NK * SAME) == 0) sh->m[warp][row] = m, sh->l[warp][row] = l;
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float4 f = o[r][v];
                if (LANES == 16) {
                    f.x += __shfl_xor_sync(0xffffffffu, f.x, 16), f.y += __shfl_xor_sync(0xffffffffu, f.y, 16);
                    f.z += __shfl_xor_sync(0xffffffffu, f.z, 16), f.w += __shfl_xor_sync(0xffffffffu, f.w, 16);
                }
                if (side == 0) *reinterpret_cast<float4 *>(&sh->o[warp][r][4 * at + 128 * v]) = f;
            }
        }
        __syncthreads();
        float *const part = cut ? attn_part(p, blockIdx.x, begins) : nullptr;
        if (cut && tid == 0) attn_part_head(part, sh->range, u.first, u.tiles, u.rows, u.row, u.s, u.h, u.q.row0);
        for (int i = tid; i < u.rows * C4; i += kFewThreads) {
            const int r = i / C4, c = i % C4 * 4;
            float top = kNone, sum = 0.f;
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh->m[w][r]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                // (a warp whose keys the row does not see, or of scores of minus infinity alone; its sum may be a NaN, which stays)
                if (sh->m[w][r] == kNone && sh->l[w][r] == 0.f) continue;
                const float by = sh->m[w][r] == kNone ? 1.f : ex2(sh->m[w][r] - top);
                const float4 x = *reinterpret_cast<const float4 *>(&sh->o[w][r][c]);
                sum = fmaf(by, sh->l[w][r], sum);
                f.x = fmaf(by, x.x, f.x), f.y = fmaf(by, x.y, f.y), f.z = fmaf(by, x.z, f.z), f.w = fmaf(by, x.w, f.w);
            }
            if (cut) {
                if (c == 0) part[kPartHead + r] = top, part[kPartHead + R + r] = sum;
                reinterpret_cast<float4 *>(part + kPartHead + 2 * R)[i] = f;
                continue;
            }
            const int t = (u.row + r) / p.G, g = (u.row + r) % p.G;
            const float inv = 1.0f / sum;
            B *const out = reinterpret_cast<B *>(p.out) + (p.cu ? 0LL : (long long)u.s * p.o_seq) + (long long)(u.q.row0 + t) * p.o_tok +
                           (long long)(u.h * p.G + g) * p.o_head;
            const float y[4] = {f.x * inv, f.y * inv, f.z * inv, f.w * inv};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < d) out[c + e] = narrow<B>(y[e]);
        }
    }
    // the join reads both slots of every block
    if (p.ws && tid == 0 && !goes_on) *reinterpret_cast<int *>(attn_part(p, blockIdx.x, 1)) = 0;
    if (p.ws && tid == 0 && !came) *reinterpret_cast<int *>(attn_part(p, blockIdx.x, 0)) = 0;
}

template <typename B, int DP, int R>
AttnSimt few() {
    return {attn_few<B, DP, R>, (int)sizeof(FewShared<DP, R>), kFewKeys};
}
template <typename B>
AttnSimt few(int dp, int rows) {
    if (rows == 4) return dp == 64 ? few<B, 64, 4>() : dp == 128 ? few<B, 128, 4>() : few<B, 256, 4>();
    return dp == 64 ? few<B, 64, 8>() : dp == 128 ? few<B, 128, 8>() : few<B, 256, 8>();
}

}  // namespace

AttnSimt attn_few_kernel(bool bf16, int dp, int rows) { return bf16 ? few<uint16_t>(dp, rows) : few<uint32_t>(dp, rows); }

}  // namespace cvk
