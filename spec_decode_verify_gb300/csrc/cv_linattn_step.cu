// Linear attention with a decay for each head, recurrent form: decoding, the verify of draft tokens
// with the deferred commit of the previous ones, and prompts that the chunked kernel does not take.
//
// Mathematics.  For a group of n tokens with a_u = exp(g_u) and the state S before them,
//   out_t = scale * ( (prod_{u<=t} a_u) S^T q_t + sum_{t'<=t} (prod_{t'<u<=t} a_u) b_t' (q_t.k_t') v_t' )
//           + skip v_t
//   S'    = (prod_u a_u) S + sum_t (prod_{u>t} a_u) b_t k_t v_t^T
// so the tile of S is read from registers once for all outputs of a group and once for its update,
// one fused multiply-add per state element and token each.  The decays enter as products of
// exponentials, never as differences of sums: a decay of zero (g = -inf) stays exact.
//
// Layout.  A block of 256 threads owns VS columns (of dv) of one sequence's head.  Its tile of the
// state lives in registers: each thread holds R rows x 4 columns, a row's VS columns spread over
// VS/4 neighbouring lanes (16-byte accesses, whole 128-byte lines), the rows over the row groups.
// q and k are staged in shared memory as [row][token], so a thread reads the TG tokens of a row as
// one or two broadcast vectors; the row groups' partial outputs are summed through shared memory in
// a fixed order.  The state is the traffic (64 KB a head at 128 x 128 against a few hundred bytes
// per token): the kernel is bound by HBM when there are many heads and by latency when there are few.
#include "cv_device.cuh"
#include "cv_linattn.h"

namespace cvk {
namespace {

// Four consecutive elements i..i+3 of a row of n (zero past its end).
__device__ __forceinline__ float4 load4(const void *base, long long row, int i, int n, int bf16, int vec) {
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i >= n) return r;
    if (bf16) {
        const uint16_t *p = reinterpret_cast<const uint16_t *>(base) + row + i;
        if (vec) {
            const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p));
            r.x = __uint_as_float(w.x << 16), r.y = __uint_as_float(w.x & 0xffff0000u);
            r.z = __uint_as_float(w.y << 16), r.w = __uint_as_float(w.y & 0xffff0000u);
        } else {
            r.x = widen<uint16_t>(__ldg(p));
            if (i + 1 < n) r.y = widen<uint16_t>(__ldg(p + 1));
            if (i + 2 < n) r.z = widen<uint16_t>(__ldg(p + 2));
            if (i + 3 < n) r.w = widen<uint16_t>(__ldg(p + 3));
        }
    } else {
        const float *p = reinterpret_cast<const float *>(base) + row + i;
        if (vec) {
            r = __ldg(reinterpret_cast<const float4 *>(p));
        } else {
            r.x = __ldg(p);
            if (i + 1 < n) r.y = __ldg(p + 1);
            if (i + 2 < n) r.z = __ldg(p + 2);
            if (i + 3 < n) r.w = __ldg(p + 3);
        }
    }
    return r;
}

// TG consecutive floats of shared memory, aligned to their size (at most 16 bytes).
template <int TG>
__device__ __forceinline__ void load_group(float *r, const float *p) {
    if constexpr (TG == 1) {
        r[0] = *p;
    } else {
#pragma unroll
        for (int j = 0; j < TG; j += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(p + j);
            r[j] = v.x, r[j + 1] = v.y, r[j + 2] = v.z, r[j + 3] = v.w;
        }
    }
}

template <int VS, int R, int TG>
__global__ void __launch_bounds__(kStepThreads, 2) linattn_step(const __grid_constant__ LinattnParams p) {
    constexpr int LANES = VS / 4;               // threads along a row
    constexpr int RG = kStepThreads / LANES;    // row groups: rows i*RG + rg
    constexpr int DKP = R * RG;
    extern __shared__ __align__(16) float sm[];
    float *const qs = sm;                       // [DKP][TG]
    float *const ks = qs + DKP * TG;            // [DKP][TG]
    float *const vs = ks + DKP * TG;            // [TG][VS]
    float *const red = vs + TG * VS;            // [RG][TG][VS]
    float *const pt = red + RG * TG * VS;       // [TG][TG]
    float *const as = pt + TG * TG;             // [TG] decays
    float *const bs = as + TG;                  // [TG] gains

    grid_dep_wait();
    grid_dep_launch();
    if (dynamic_smem_bytes() < step_smem_floats(VS, R, TG) * 4) return;

    const int tid = threadIdx.x;
    const int slice = blockIdx.x % p.slices;
    const int unit = blockIdx.x / p.slices;
    const int h = unit % p.n_heads, s = unit / p.n_heads;
    const int hq = (int)((long long)h * p.n_qk / p.n_heads);
    const int c0 = slice * VS;

    const int slot = p.cache_idx ? __ldg(p.cache_idx + s) : s;
    int status = 0, n_tok = p.tok.T, n_prev = p.prev.T, row0 = 0, prow0 = 0;
    if (slot >= p.n_slots) status |= 1;
    if (slot >= 0 && p.tok.cu) status |= draft_span(p.tok.cu, s, p.tok.T, p.tok.total, n_tok, row0);
    if (slot >= 0 && p.prev.T > 0) {
        if (p.prev.cu) status |= draft_span(p.prev.cu, s, p.prev.T, p.prev.total, n_prev, prow0);
        const int a = __ldg(p.accept + s);
        if (a < 0 || a > n_prev) status |= 4;
        n_prev = a;
    }
    if (p.err && h == 0 && slice == 0 && tid == 0) p.err[s] = slot < 0 ? 0 : status;
    if (slot < 0 || status) return;
    const bool init = p.has_init ? __ldg(p.has_init + s) != 0 : true;

    // this thread's part of the state tile
    const int rg = tid / LANES;
    const int c = c0 + (tid % LANES) * 4;
    float *const st = p.state + (long long)slot * p.st_slot + (long long)h * p.st_head + c;
    float S[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int row = i * RG + rg;
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
        if (init && row < p.dk) {
            const float *src = st + (long long)row * p.dv;
            if (p.st_vec) {
                if (c < p.dv) w = *reinterpret_cast<const float4 *>(src);
            } else {
                if (c < p.dv) w.x = src[0];
                if (c + 1 < p.dv) w.y = src[1];
                if (c + 2 < p.dv) w.z = src[2];
                if (c + 3 < p.dv) w.w = src[3];
            }
        }
        S[i][0] = w.x, S[i][1] = w.y, S[i][2] = w.z, S[i][3] = w.w;
    }
    auto store_state = [&]() {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int row = i * RG + rg;
            if (row >= p.dk) continue;
            float *dst = st + (long long)row * p.dv;
            if (p.st_vec) {
                if (c < p.dv) *reinterpret_cast<float4 *>(dst) = make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c + j < p.dv) dst[j] = S[i][j];
            }
        }
    };

    // tokens t0 .. t0+n-1 (n <= TG) of a run into shared memory, zeros past n
    auto stage = [&](const LinattnRun &run, int first_row, int t0, int n, bool with_q) {
        const long long sq = run.cu ? 0 : s;
        for (int idx = tid; idx < TG * (DKP / 4); idx += kStepThreads) {
            const int t = idx % TG, i = (idx / TG) * 4;
            float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), qv = kv;
            if (t < n) {
                const long long row = (long long)first_row + t0 + t;
                kv = load4(run.k, sq * run.k_seq + row * run.k_tok + hq * run.k_head, i, p.dk, p.bf16, run.vec);
                if (with_q)
                    qv = load4(run.q, sq * run.q_seq + row * run.q_tok + hq * run.q_head, i, p.dk, p.bf16, run.vec);
            }
            ks[i * TG + t] = kv.x, ks[(i + 1) * TG + t] = kv.y, ks[(i + 2) * TG + t] = kv.z, ks[(i + 3) * TG + t] = kv.w;
            if (with_q)
                qs[i * TG + t] = qv.x, qs[(i + 1) * TG + t] = qv.y, qs[(i + 2) * TG + t] = qv.z,
                qs[(i + 3) * TG + t] = qv.w;
        }
        for (int idx = tid; idx < TG * LANES; idx += kStepThreads) {
            const int t = idx / LANES, i = (idx % LANES) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t < n)
                v = load4(run.v, sq * run.v_seq + ((long long)first_row + t0 + t) * run.v_tok + (long long)h * run.v_head,
                          c0 + i, p.dv, p.bf16, run.vec);
            *reinterpret_cast<float4 *>(vs + t * VS + i) = v;
        }
        if (tid < TG) {
            const long long row = (long long)first_row + t0 + tid;
            as[tid] = tid < n ? expf(__ldg(run.g + sq * run.g_seq + row * run.g_tok + h)) : 1.0f;
            bs[tid] = tid < n ? (run.b ? __ldg(run.b + sq * run.b_seq + row * run.b_tok + h) : 1.0f) : 0.0f;
        }
    };

    // S <- S advanced over the n staged tokens
    auto advance = [&](int n) {
        float vw[TG][4], tail = 1.0f;
#pragma unroll
        for (int t = TG - 1; t >= 0; --t) {
            const float4 v = *reinterpret_cast<const float4 *>(vs + t * VS + (tid % LANES) * 4);
            const float w = tail * bs[t];
            vw[t][0] = w * v.x, vw[t][1] = w * v.y, vw[t][2] = w * v.z, vw[t][3] = w * v.w;
            if (t < n) tail *= as[t];
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float kr[TG];
            load_group<TG>(kr, ks + (i * RG + rg) * TG);
#pragma unroll
            for (int j = 0; j < 4; ++j) S[i][j] *= tail;
#pragma unroll
            for (int t = 0; t < TG; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) S[i][j] = fmaf(kr[t], vw[t][j], S[i][j]);
        }
    };

    if (p.prev.T > 0) {
        for (int t0 = 0; t0 < n_prev; t0 += TG) {
            const int n = min(TG, n_prev - t0);
            stage(p.prev, prow0, t0, n, false);
            __syncthreads();
            advance(n);
            __syncthreads();
        }
        if (n_prev > 0 || !init) store_state();
    }

    const float sk = p.skip ? __ldg(p.skip + h) : 0.0f;
    for (int t0 = 0; t0 < n_tok; t0 += TG) {
        const int n = min(TG, n_tok - t0);
        stage(p.tok, row0, t0, n, true);
        __syncthreads();

        // products of the group's tokens, (q_t . k_u) for u <= t < n: LP lanes per pair
        constexpr int PPW = TG * TG / 8 > 0 ? TG * TG / 8 : 1;
        constexpr int LP = 32 / PPW;
        const int pair = (tid / 32) * PPW + (tid % 32) / LP;
        if (tid / 32 < (TG * TG + PPW - 1) / PPW) {
            const int t = pair / TG, u = pair % TG;
            float acc = 0.0f;
            for (int r = tid % LP; r < DKP; r += LP) acc = fmaf(qs[r * TG + t], ks[r * TG + u], acc);
#pragma unroll
            for (int o = LP / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
            if (u <= t && t < n) {
                float w = bs[u];
                for (int x = u + 1; x <= t; ++x) w *= as[x];
                if (tid % LP == 0) pt[t * TG + u] = acc * w;
            }
        }
        // the row groups' parts of S^T q
        {
            float acc[TG][4];
#pragma unroll
            for (int t = 0; t < TG; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.0f;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float qr[TG];
                load_group<TG>(qr, qs + (i * RG + rg) * TG);
#pragma unroll
                for (int t = 0; t < TG; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[t][j] = fmaf(qr[t], S[i][j], acc[t][j]);
            }
#pragma unroll
            for (int t = 0; t < TG; ++t)
                *reinterpret_cast<float4 *>(red + (rg * TG + t) * VS + (tid % LANES) * 4) =
                    make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
        }
        if (p.update || t0 + TG < n_tok) advance(n);
        __syncthreads();
        for (int idx = tid; idx < n * VS; idx += kStepThreads) {
            const int t = idx / VS, j = idx % VS;
            if (c0 + j >= p.dv) continue;
            float o = 0.0f, a = 1.0f;
            for (int w = 0; w < RG; ++w) o += red[(w * TG + t) * VS + j];
            for (int u = 0; u <= t; ++u) a *= as[u];
            o *= a;
            for (int u = 0; u <= t; ++u) o = fmaf(pt[t * TG + u], vs[u * VS + j], o);
            o *= p.scale;
            if (p.skip) o = fmaf(sk, vs[t * VS + j], o);
            const long long at = (p.tok.cu ? 0 : s * p.o_seq) + ((long long)row0 + t0 + t) * p.o_tok +
                                 (long long)h * p.o_head + c0 + j;
            if (p.bf16)
                reinterpret_cast<uint16_t *>(p.out)[at] = narrow<uint16_t>(o);
            else
                reinterpret_cast<float *>(p.out)[at] = o;
        }
        if (t0 + TG < n_tok) __syncthreads();
    }
    if (p.update && (n_tok > 0 || !init)) store_state();
}

template <int VS, int R>
StepKernel pick(int tg) {
    constexpr int rows = R * (kStepThreads / (VS / 4));
    if (tg == 1) return {linattn_step<VS, R, 1>, rows, step_smem_floats(VS, R, 1) * 4};
    if (tg == 4) return {linattn_step<VS, R, 4>, rows, step_smem_floats(VS, R, 4) * 4};
    return {linattn_step<VS, R, 8>, rows, step_smem_floats(VS, R, 8) * 4};
}

}  // namespace

StepKernel step_kernel(int vs, int dk, int tg) {
    if (vs == 128) return dk <= 64 ? pick<128, 8>(tg) : pick<128, 16>(tg);
    if (vs == 64) return dk <= 64 ? pick<64, 4>(tg) : dk <= 128 ? pick<64, 8>(tg) : pick<64, 16>(tg);
    return dk <= 64 ? pick<32, 2>(tg) : dk <= 128 ? pick<32, 4>(tg) : pick<32, 8>(tg);
}

}  // namespace cvk
