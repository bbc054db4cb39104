// Attention of drafted tokens over a paged cache in fp32 products: fp32 calls, and bf16 calls whose rows, pages or head
// size the tensor-core kernel does not take; with more than 8 rows a kv head, or rows that are no whole 16-byte pieces.  Also the
// join of units that were cut.
//
// Mathematics.  A unit is up to 32 rows (draft, query head) of a kv head.  For each tile of keys, with the scores
// s = scale q.k and the running maximum m and sum l of its row,
//   m' = max(m, s),  p = exp(s - m'),  l' = l exp(m - m') + sum p,  O' = O exp(m - m') + p V,
// and out = O / l at the end: one pass over K and V.  A unit that is cut leaves (m, l, O); the join adds the parts
// with weights exp(m_i - max m).
//
// A block takes a tile of keys to shared memory, where 32 rows share it; the reads of shared memory (6 of 16 bytes for 32 multiply-adds of
// the scores) bound it: 16 sequences of 8 drafts of 32/4 heads over up to 2k take 164 us, 21 TFLOP/s.  (Copies ahead of
// their tile: 115 us against 118 for 13 tokens of 64/8 heads over 3k, but 460 against 374 with heads of 256.)
#include "cv_attn.cuh"

namespace cvk {
namespace {

constexpr float kNone = -INFINITY;

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <int DP>
__host__ __device__ constexpr int simt_keys() { return DP <= 128 ? 64 : 32; }
template <int DP>
struct SimtShared {
    static constexpr int KT = simt_keys<DP>();
    float q[kSimtRows][DP + 4], k[KT][DP + 4], v[KT][DP], p[KT][kSimtRows + 4];
    float scale[kSimtRows], m[kSimtRows], l[kSimtRows];
    AttnTree tree;
    uint4 see[128];
    AttnRange range;
    AttnScratch scratch;
};

// 4 channels from c on of a row (zeros past d).
template <typename B, bool VEC>
__device__ __forceinline__ float4 row4(const B *row, int c, int d) {
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (VEC) {
        if (c < d) {
            if (sizeof(B) == 4) {
                f = *reinterpret_cast<const float4 *>(row + c);
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(row + c);
                f = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                                __uint_as_float(w.y & 0xffff0000u));
            }
        }
    } else {
        if (c < d) f.x = widen<B>(row[c]);
        if (c + 1 < d) f.y = widen<B>(row[c + 1]);
        if (c + 2 < d) f.z = widen<B>(row[c + 2]);
        if (c + 3 < d) f.w = widen<B>(row[c + 3]);
    }
    return f;
}

template <typename B, int DP, bool VEC>
__global__ void __launch_bounds__(kSimtThreads) attn_simt(const __grid_constant__ AttnParams p) {
    constexpr int KT = simt_keys<DP>(), KPT = KT / 16, RPT = DP / 32, C4 = DP / 4;
    extern __shared__ __align__(16) unsigned char smem[];
    SimtShared<DP> *sh = reinterpret_cast<SimtShared<DP> *>(smem);
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, d = p.c.d;
    attn_range(p, &sh->range, &sh->scratch);
    const int rg = tid / 16, kg = tid % 16;   // scores: rows 2 rg and 2 rg + 1, keys kg + 16 i
    const int c4 = tid % C4, og = tid / C4;   // outputs: channels 4 c4 .., rows og * RPT ..
    AttnWalk walk(p, sh->range);
    AttnUnit u;
    int s_before = -1;
    bool bad = false, goes_on = false, came = false;  // parts left in slots 1 and 0
    while (walk.next(p, u)) {
        const B *const K = reinterpret_cast<const B *>(p.c.k) + (long long)u.h * p.c.k_head;
        const B *const V = reinterpret_cast<const B *>(p.c.v) + (long long)u.h * p.c.v_head;
        const int *const table = p.c.table + (long long)u.q.slot * p.c.table_row;
        const int end = u.q.L + u.q.T;
        __syncthreads();
        if (u.s != s_before) {
            s_before = u.s;
            const int *parent = p.parent ? p.parent + (p.cu ? (long long)u.q.row0 : (long long)u.s * p.T) : nullptr;
            int st = attn_ancestors(parent, u.q.T, tid, kSimtThreads, &sh->tree, sh->see, [] { __syncthreads(); }) ? kSeqBadTree : 0;
            for (int i = tid; i <= (end - 1) / p.c.page; i += kSimtThreads) {
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
        for (int i = tid; i < kSimtRows * C4; i += kSimtThreads) {
            const int r = i / C4, c = i % C4 * 4, t = (u.row + r) / p.G, g = (u.row + r) % p.G;
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < u.rows)
                f = row4<B, VEC>(reinterpret_cast<const B *>(p.q) + (p.cu ? 0LL : (long long)u.s * p.q_seq) +
                                     (long long)(u.q.row0 + t) * p.q_tok + (long long)(u.h * p.G + g) * p.q_head,
                                 c, d);
            *reinterpret_cast<float4 *>(&sh->q[r][c]) = f;
        }
        const bool scores = tid / 32 * 4 < u.rows;  // whether this warp's rows are the unit's
        float m[2] = {kNone, kNone}, l[2] = {0.f, 0.f};
        float4 o[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int tile = u.tile; tile < u.last; ++tile) {
            const int j0 = tile * KT;
            __syncthreads();
#pragma unroll 4
            for (int i = tid; i < KT * C4; i += kSimtThreads) {
                const int r = i / C4, c = i % C4 * 4, j = j0 + r;
                float4 fk = make_float4(0.f, 0.f, 0.f, 0.f), fv = fk;
                if (j < end) {
                    const int pg = __ldg(table + j / p.c.page), in = j % p.c.page;
                    fk = row4<B, VEC>(K + (long long)pg * p.c.k_page + (long long)in * p.c.k_row, c, d);
                    fv = row4<B, VEC>(V + (long long)pg * p.c.v_page + (long long)in * p.c.v_row, c, d);
                }
                *reinterpret_cast<float4 *>(&sh->k[r][c]) = fk;
                *reinterpret_cast<float4 *>(&sh->v[r][c]) = fv;
            }
            __syncthreads();
            float s[2][KPT];
#pragma unroll
            for (int i = 0; i < KPT; ++i) s[0][i] = s[1][i] = 0.f;
            const int span = scores ? DP : 0;
#pragma unroll 4
            for (int c = 0; c < span; c += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(&sh->q[2 * rg][c]);
                const float4 b = *reinterpret_cast<const float4 *>(&sh->q[2 * rg + 1][c]);
#pragma unroll
                for (int i = 0; i < KPT; ++i) {
                    const float4 k = *reinterpret_cast<const float4 *>(&sh->k[kg + 16 * i][c]);
                    s[0][i] = fmaf(a.x, k.x, fmaf(a.y, k.y, fmaf(a.z, k.z, fmaf(a.w, k.w, s[0][i]))));
                    s[1][i] = fmaf(b.x, k.x, fmaf(b.y, k.y, fmaf(b.z, k.z, fmaf(b.w, k.w, s[1][i]))));
                }
            }
            const bool drafts = j0 + KT > u.q.L;
            if (scores) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = 2 * rg + x, t = min((u.row + r) / p.G, 127);
                    float top = m[x];
#pragma unroll
                    for (int i = 0; i < KPT; ++i) {
                        s[x][i] *= p.scale;
                        if (drafts) {
                            const int back = j0 + kg + 16 * i - u.q.L;
                            if (back >= 0 && (back >= u.q.T || !((&sh->see[t].x)[back >> 5] >> (back & 31) & 1))) s[x][i] = kNone;
                        }
                        top = fmaxf(top, s[x][i]);
                    }
#pragma unroll
                    for (int b = 8; b > 0; b >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, b));
                    const float base = top == kNone ? 0.f : top, down = ex2(m[x] - base);
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < KPT; ++i) {
                        const float e = ex2(s[x][i] - base);
                        sum += e;
                        sh->p[kg + 16 * i][r] = e;
                    }
                    l[x] = fmaf(l[x], down, sum);
                    m[x] = top;
                    if (kg == 0) sh->scale[r] = down;
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float f = sh->scale[og * RPT + i];
                o[i].x *= f, o[i].y *= f, o[i].z *= f, o[i].w *= f;
            }
            // (a key that a row does not see has weight 0, and 0 times a NaN or an infinity is left out)
            const int steps = og * RPT < u.rows ? KT : 0;
#pragma unroll 4
            for (int j = 0; j < steps; ++j) {
                const float4 v = *reinterpret_cast<const float4 *>(&sh->v[j][4 * c4]);
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const float w = sh->p[j][og * RPT + i];
                    if (!drafts || w != 0.f) {
                        o[i].x = fmaf(w, v.x, o[i].x), o[i].y = fmaf(w, v.y, o[i].y);
                        o[i].z = fmaf(w, v.z, o[i].z), o[i].w = fmaf(w, v.w, o[i].w);
                    }
                }
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int b = 8; b > 0; b >>= 1) l[x] += __shfl_xor_sync(0xffffffffu, l[x], b);
            if (kg == 0) sh->m[2 * rg + x] = m[x], sh->l[2 * rg + x] = l[x];
        }
        __syncthreads();
        if (!cut) {
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const int r = og * RPT + i, t = (u.row + r) / p.G, g = (u.row + r) % p.G;
                if (r >= u.rows) break;
                const float inv = 1.0f / sh->l[r];
                B *const out = reinterpret_cast<B *>(p.out) + (p.cu ? 0LL : (long long)u.s * p.o_seq) +
                               (long long)(u.q.row0 + t) * p.o_tok + (long long)(u.h * p.G + g) * p.o_head;
                const float f[4] = {o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * c4 + e < d) out[4 * c4 + e] = narrow<B>(f[e]);
            }
        } else {
            float *const part = attn_part(p, blockIdx.x, begins);
            if (tid == 0) attn_part_head(part, sh->range, u.first, u.tiles, u.rows, u.row, u.s, u.h, u.q.row0);
            if (tid < kSimtRows) part[kPartHead + tid] = sh->m[tid], part[kPartHead + kSimtRows + tid] = sh->l[tid];
            float4 *const to = reinterpret_cast<float4 *>(part + kPartHead + 2 * kSimtRows);
#pragma unroll
            for (int i = 0; i < RPT; ++i) to[(og * RPT + i) * C4 + c4] = o[i];
        }
    }
    // the join reads both slots of every block
    if (p.ws && tid == 0 && !goes_on) *reinterpret_cast<int *>(attn_part(p, blockIdx.x, 1)) = 0;
    if (p.ws && tid == 0 && !came) *reinterpret_cast<int *>(attn_part(p, blockIdx.x, 0)) = 0;
}

// The units that were cut.  A unit of n parts is spread over the blocks of its n parts, kAttnJoinY each; a row takes one warp, or
// several where there are few rows for them, each with every so many parts: eight parts' flags, maxima, sums and rows on their
// way at once, added up under a running maximum.
template <typename B, int E>  // E: 128 channels each that a warp holds
__global__ void __launch_bounds__(kAttnJoinThreads, 4 - E) attn_join(const __grid_constant__ AttnParams p) {
    constexpr int WARPS = kAttnJoinThreads / 32, N = 8 / E;
    __shared__ float4 sum[WARPS][32 * E];
    __shared__ float sum_l[WARPS], sum_m[WARPS];
    __shared__ int left_out[WARPS];
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int4 *const mine_at = reinterpret_cast<const int4 *>(attn_part(p, blockIdx.x, blockIdx.z));
    const int4 h0 = mine_at[0], h1 = mine_at[1];  // (see attn_part_head)
    if (h0.x == 0) return;
    const int n = h0.y, c0 = h0.z, rows = h0.w, row0 = h1.x, s = h1.y, h = h1.z, packed = h1.w;
    const float *const first = attn_part(p, c0, 1);
    const long long step = part_floats(p.pad, p.dp);
    const int share = ((int)blockIdx.x - c0) * kAttnJoinY + blockIdx.y, shares = n * kAttnJoinY;
    int each = 1;  // warps a row
    while (each < WARPS && each * 2 * rows <= shares * WARPS) each *= 2;
    const int at_once = WARPS / each, mine = warp % each;
    for (int base = share * at_once; base < rows; base += shares * at_once) {
        const int r = base + warp / each;
        const bool on = r < rows;
        float4 o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f, top = kNone;
        int gone = 0;  // (a block that gave up leaves no part)
        if (on) {
            for (int i0 = mine; i0 < n; i0 += N * each) {
                float4 v[N][E];
                float m[N], w[N];
                int flag[N];
#pragma unroll
                for (int x = 0; x < N; ++x) {
                    const int i = i0 + x * each;
                    m[x] = kNone, w[x] = 0.f, flag[x] = 1;
                    if (i < n) {
                        const float *const a = first + (i == 0 ? 0 : 2 * i - 1) * step;  // i > 0: slot 0 of block c0 + i
                        flag[x] = *reinterpret_cast<const int *>(a);
                        m[x] = a[kPartHead + r], w[x] = a[kPartHead + p.pad + r];
                        const float4 *const row = reinterpret_cast<const float4 *>(a + kPartHead + 2 * p.pad + (long long)r * p.dp);
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            if (4 * (lane + 32 * e) < p.dp) v[x][e] = row[lane + 32 * e];
                    }
                }
                float now = top;
#pragma unroll
                for (int x = 0; x < N; ++x) now = fmaxf(now, m[x]);
                const float down = now == kNone ? 1.f : ex2(top - now);
                top = now, l *= down;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e].x *= down, o[e].y *= down, o[e].z *= down, o[e].w *= down;
#pragma unroll
                for (int x = 0; x < N; ++x) {
                    gone |= flag[x] == 0;
                    // (a part in which the row sees nothing, or minus infinity alone; its sum may be a NaN, which stays)
                    if (m[x] == kNone && w[x] == 0.f) continue;
                    const float f = m[x] == kNone ? 1.f : ex2(m[x] - top);
                    l = fmaf(f, w[x], l);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        o[e].x = fmaf(f, v[x][e].x, o[e].x), o[e].y = fmaf(f, v[x][e].y, o[e].y);
                        o[e].z = fmaf(f, v[x][e].z, o[e].z), o[e].w = fmaf(f, v[x][e].w, o[e].w);
                    }
                }
            }
        }
        if (each > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < E; ++e) sum[warp][lane + 32 * e] = o[e];
            if (lane == 0) sum_l[warp] = l, sum_m[warp] = top, left_out[warp] = gone;
            __syncthreads();
            if (mine == 0) {
                float now = top;
                for (int w = warp + 1; w < warp + each; ++w) now = fmaxf(now, sum_m[w]), gone |= left_out[w];
                const float down = now == kNone ? 1.f : ex2(top - now);
                l *= down;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e].x *= down, o[e].y *= down, o[e].z *= down, o[e].w *= down;
                for (int w = warp + 1; w < warp + each; ++w) {
                    const float m = sum_m[w];
                    if (m == kNone && sum_l[w] == 0.f) continue;
                    const float f = m == kNone ? 1.f : ex2(m - now);
                    l = fmaf(f, sum_l[w], l);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float4 x = sum[w][lane + 32 * e];
                        o[e].x = fmaf(f, x.x, o[e].x), o[e].y = fmaf(f, x.y, o[e].y);
                        o[e].z = fmaf(f, x.z, o[e].z), o[e].w = fmaf(f, x.w, o[e].w);
                    }
                }
            }
        }
        if (!on || mine != 0 || gone) continue;
        const float inv = 1.0f / l;
        const int t = (row0 + r) / p.G, g = (row0 + r) % p.G;
        B *const out = reinterpret_cast<B *>(p.out) + (p.cu ? 0LL : (long long)s * p.o_seq) + (long long)(packed + t) * p.o_tok +
                       (long long)(h * p.G + g) * p.o_head;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float f[4] = {o[e].x * inv, o[e].y * inv, o[e].z * inv, o[e].w * inv};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int c = 4 * (lane + 32 * e) + x;
                if (c < p.c.d) out[c] = narrow<B>(f[x]);
            }
        }
    }
}

template <typename B, int DP>
AttnSimt simt(bool vec) {
    return {vec ? attn_simt<B, DP, true> : attn_simt<B, DP, false>, (int)sizeof(SimtShared<DP>), simt_keys<DP>()};
}

}  // namespace

AttnSimt attn_simt_kernel(bool bf16, int dp, bool vec) {
    if (bf16) return dp <= 64 ? simt<uint16_t, 64>(vec) : dp <= 128 ? simt<uint16_t, 128>(vec) : simt<uint16_t, 256>(vec);
    return dp <= 64 ? simt<uint32_t, 64>(vec) : dp <= 128 ? simt<uint32_t, 128>(vec) : simt<uint32_t, 256>(vec);
}
AttnKernel attn_join_kernel(bool bf16, int dp) {
    if (dp <= 128) return bf16 ? attn_join<uint16_t, 1> : attn_join<uint32_t, 1>;
    return bf16 ? attn_join<uint16_t, 2> : attn_join<uint32_t, 2>;
}

}  // namespace cvk
