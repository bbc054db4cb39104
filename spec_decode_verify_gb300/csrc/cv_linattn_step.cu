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

// The same for aligned rows, with everything loaded ahead.  Blocks stay (16 warps per SM) and walk the units
// (sequence, head, 16 columns a warp); while one unit is computed from registers, the next one's state tile
// and the next group's rows are on their way into shared memory by cp.async.
//
// A warp owns 16 columns of all rows: lane = 4 * (row group) + (column quad), a row group being R
// consecutive rows, held in registers as pairs of rows (S[m][j] = rows 2m, 2m + 1 of column j).  A token's
// q or k, as it lies in memory, is then read as R * 2 (bf16) consecutive bytes per lane and multiplies
// pairs of rows by paired fp32 instructions; the sum over the row groups stays inside the warp.  Only the
// products q_t . k_u are shared by the block's warps.
//
// Measured: 128 x 8 drafts with the commit of the previous ones (48 heads of 128 x 128, 13 padded) 172 us,
// 4.4 TB/s, half the issue slots busy: the paired multiply-adds, the reads of q and k and a group's two barriers
// share the time with HBM (rows spread over the warps and fp32 copies of q and k took 239 us).  64 single fp32
// tokens of 32 heads of 64 x 128: 22 us, 6.0 TB/s, bound by HBM; 1 token of 48 heads of 128 x 128: 5 us, bound
// by latency.
constexpr int kTileWords = 4;  // columns a lane

// N consecutive pairs of rows of a token's q or k.
template <int N, bool BF>
__device__ __forceinline__ void load_rows(f2 *r, const unsigned char *at) {
    if constexpr (BF) {
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const uint4 w = *reinterpret_cast<const uint4 *>(at + j * 4);
            r[j] = f2_pack(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u));
            r[j + 1] = f2_pack(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
            r[j + 2] = f2_pack(__uint_as_float(w.z << 16), __uint_as_float(w.z & 0xffff0000u));
            r[j + 3] = f2_pack(__uint_as_float(w.w << 16), __uint_as_float(w.w & 0xffff0000u));
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(at + j * 8);
            r[j] = w.x, r[j + 1] = w.y;
        }
    }
}
// Four consecutive elements.
template <bool BF>
__device__ __forceinline__ float4 load_four(const unsigned char *at) {
    if constexpr (!BF) return *reinterpret_cast<const float4 *>(at);
    const uint2 w = *reinterpret_cast<const uint2 *>(at);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, bool on) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(on ? 16u : 0u) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(dst), "l"(src), "n"(BYTES), "r"(on ? BYTES : 0)
                     : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// R rows a lane (8 row groups: dk <= 8 R), groups of TG tokens.
template <int R, int TG, bool BF>
__global__ void __launch_bounds__(kStepThreads, 2) linattn_stream(const __grid_constant__ LinattnParams p) {
    constexpr int RP = R / 2, DKP = 8 * R, ES = BF ? 2 : 4;
    constexpr int PITCH = StreamLayout::row_bytes(DKP, BF);
    constexpr int KSH = (R == 16 ? 4 : 3) + (BF ? 0 : 1);  // log2 of a row's 16-byte pieces
    extern __shared__ __align__(16) unsigned char smem[];
    const int warps = blockDim.x >> 5, nt = blockDim.x, VS = 16 * warps;
    const StreamLayout lay(warps, R, TG, BF);
    const int pitch_v = StreamLayout::row_bytes(VS, BF), vsh = 31 - __clz(VS * ES / 16);
    float4 *const tile = reinterpret_cast<float4 *>(smem);              // [R][threads]
    float *const pt = reinterpret_cast<float *>(smem + lay.products);   // [TG][TG]
    StepUnit *const ring = reinterpret_cast<StepUnit *>(smem + lay.ring);  // unit n at n % 4
    if (dynamic_smem_bytes() < (unsigned)lay.bytes) return;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rg = lane >> 2, quad = lane & 3, vc = warp * 16 + quad * 4;  // vc: column within the unit
    const unsigned total = (unsigned)p.n_seq * (unsigned)(p.pieces * p.n_heads * p.slices);
    grid_dep_wait();
    grid_dep_launch();

    auto unit_of = [&](unsigned idx) {
        StepUnit u;
        u.on = idx < total;
        u.n_tok = u.n_prev = u.row0 = u.prow0 = u.status = u.s = u.h = u.slice = u.piece = 0;
        u.init = true, u.update = p.update;
        u.from = u.to = p.state;
        if (!u.on) return u;
        u.slice = (int)(idx % (unsigned)p.slices);
        unsigned unit = idx / (unsigned)p.slices;
        u.h = (int)(unit % (unsigned)p.n_heads);
        unit /= (unsigned)p.n_heads;
        u.piece = (int)(unit % (unsigned)p.pieces), u.s = (int)(unit / (unsigned)p.pieces);
        if (p.pieces > 1 && p.n_seq <= kStepMaxCounted) {
            // only the pieces that there are (of a sequence's own states: those with a next one)
            const LinattnRun &run = p.own_states ? p.prev : p.tok;
            u.on = false;
            for (int s = 0; s < p.n_seq; ++s) {
                int L, row0;
                if (draft_span(run.cu, s, run.T, run.total, L, row0)) L = 0;
                const int some = (L + p.piece_len - 1) / p.piece_len;
                const unsigned n = (unsigned)(p.own_states ? max(some - 1, 0) : max(some, 1));
                if (unit < n) {
                    u.s = s, u.piece = (int)unit, u.on = true;
                    break;
                }
                unit -= n;
            }
            if (!u.on) {
                u.s = 0, u.piece = 1;  // (a first piece would report the sequence's status)
                return u;
            }
        }
        const int slot = p.cache_idx ? __ldg(p.cache_idx + u.s) : u.s;
        u.n_tok = p.tok.T, u.n_prev = p.prev.T;
        if (slot >= p.n_slots) u.status |= 1;
        if (p.tok.cu) u.status |= draft_span(p.tok.cu, u.s, p.tok.T, p.tok.total, u.n_tok, u.row0);
        if (p.prev.T > 0) {
            if (p.prev.cu) u.status |= draft_span(p.prev.cu, u.s, p.prev.T, p.prev.total, u.n_prev, u.prow0);
            if (p.accept) {
                const int a = __ldg(p.accept + u.s);
                if (a < 0 || a > u.n_prev) u.status |= 4;
                u.n_prev = a;
            }
        }
        if (p.has_init) u.init = __ldg(p.has_init + u.s) != 0;
        if (slot < 0) u.status = 0;
        u.on = slot >= 0 && u.status == 0;
        if (!u.on) return u;
        u.from = u.to = p.state + (long long)slot * p.st_slot + (long long)u.h * p.st_head;
        if (p.pieces > 1) {
            // in a launch for the pieces' own states the tokens are the run `prev`, from zero
            int &n = p.own_states ? u.n_prev : u.n_tok, &row = p.own_states ? u.prow0 : u.row0;
            const long long start = (long long)u.piece * p.piece_len;
            const bool last = start + p.piece_len >= n;
            u.on = u.piece == 0 || start < n;
            if (p.own_states && last) u.on = false;
            const bool cut = n > p.piece_len;
            float *const ws = p.ws_state + (((long long)u.s * p.n_heads + u.h) * p.pieces + u.piece) * p.dk * p.dv;
            n = u.on ? min(p.piece_len, n - (int)start) : 0;
            row += u.on ? (int)start : 0;
            if (p.own_states) u.init = false, u.to = ws + (long long)p.dk * p.dv;
            else if (cut) u.init = u.init || u.piece > 0, u.from = ws;
            if (!last) u.update = p.own_states;
        }
        return u;
    };
    auto groups_of = [](const StepUnit &u) {
        return u.on ? (u.n_prev + TG - 1) / TG + (u.n_tok + TG - 1) / TG : 0;
    };
    // from a head's state to this lane's first word of it (row rg * R)
    auto lane_of = [&](const StepUnit &u) { return u.slice * VS + vc + rg * R * p.dv; };
    auto fetch_state = [&](const StepUnit &u) {
        const float *st = u.from + lane_of(u);
        const bool col = u.init && u.slice * VS + vc < p.dv;
        const uint32_t dst = smem_u32(tile + tid);
#pragma unroll
        for (int i = 0; i < R; ++i, st += p.dv) {
            const bool in = col && rg * R + i < p.dk;
            copy_async<16>(dst + i * nt * 16, in ? st : p.state, in);
        }
    };
    // group g of the unit -> raw rows in buffer b (previous drafts first), zeros past the tokens
    auto fetch_group = [&](const StepUnit &u, int g, int b) {
        const int gp = (u.n_prev + TG - 1) / TG;
        const bool old = g < gp;
        const LinattnRun &run = old ? p.prev : p.tok;
        const int t0 = (old ? g : g - gp) * TG, n = min(TG, (old ? u.n_prev : u.n_tok) - t0);
        const long long sq = run.cu ? 0 : u.s, first = (long long)(old ? u.prow0 : u.row0) + t0;
        const int hq = (int)((unsigned)u.h * (unsigned)p.n_qk / (unsigned)p.n_heads);
        const uint32_t base = smem_u32(smem + lay.raw + b * lay.raw_bytes);
        auto rows = [&](uint32_t dst, int pitch, int sh, const void *src, long long at, long long tok, int width) {
            const unsigned char *const s0 = reinterpret_cast<const unsigned char *>(src) + at * ES;
            for (int e = tid; e < TG << sh; e += nt) {
                const int t = e >> sh, c = (e & ((1 << sh) - 1)) * 16;
                const bool in = t < n && c < width * ES;
                copy_async<16>(dst + t * pitch + c, in ? s0 + t * tok * ES + c : s0, in);
            }
        };
        rows(base, PITCH, KSH, run.k, sq * run.k_seq + first * run.k_tok + hq * run.k_head, run.k_tok, p.dk);
        if (!old)
            rows(base + TG * PITCH, PITCH, KSH, run.q, sq * run.q_seq + first * run.q_tok + hq * run.q_head, run.q_tok, p.dk);
        rows(base + 2 * TG * PITCH, pitch_v, vsh, run.v,
             sq * run.v_seq + first * run.v_tok + (long long)u.h * run.v_head + u.slice * VS, run.v_tok,
             min(VS, p.dv - u.slice * VS));
        if (tid < TG) {
            const bool in = tid < n;
            const uint32_t at = base + 2 * TG * PITCH + TG * pitch_v + tid * 4;
            copy_async<4>(at, in ? run.g + sq * run.g_seq + (first + tid) * run.g_tok + u.h : run.g, in);
            if (run.b) copy_async<4>(at + TG * 4, in ? run.b + sq * run.b_seq + (first + tid) * run.b_tok + u.h : run.b, in);
        }
    };

    if (tid < 2) ring[tid] = unit_of(blockIdx.x + tid * gridDim.x);
    __syncthreads();
    if (groups_of(ring[0]) > 0) fetch_group(ring[0], 0, 0);
    if (ring[0].on) fetch_state(ring[0]);
    copies_commit();
    int buf = 0;  // buffer of the group to compute next

    int turn = 0;
    for (unsigned idx = blockIdx.x; idx < total; idx += gridDim.x, ++turn) {
        copies_wait<0>();  // the tile and the first group
        __syncthreads();
        const StepUnit &cur = ring[turn & 3], &nxt = ring[(turn + 1) & 3];
        if (tid == nt - 1) ring[(turn + 2) & 3] = unit_of(idx + 2 * gridDim.x);
        if (p.err && cur.h == 0 && cur.slice == 0 && cur.piece == 0 && !p.own_states && tid == 0) p.err[cur.s] = cur.status;
        f2 S[RP][kTileWords];
        const int gp = (cur.n_prev + TG - 1) / TG, ng = groups_of(cur);
        const bool col = cur.slice * VS + vc < p.dv;
        auto store_state = [&]() {
            float *st = cur.to + lane_of(cur);
#pragma unroll
            for (int m = 0; m < RP; ++m) {
                float4 w[2];
                f2_unpack(S[m][0], w[0].x, w[1].x);
                f2_unpack(S[m][1], w[0].y, w[1].y);
                f2_unpack(S[m][2], w[0].z, w[1].z);
                f2_unpack(S[m][3], w[0].w, w[1].w);
#pragma unroll
                for (int b = 0; b < 2; ++b, st += p.dv)
                    if (rg * R + 2 * m + b < p.dk && col) *reinterpret_cast<float4 *>(st) = w[b];
            }
        };
        if (cur.on) {
#pragma unroll
            for (int m = 0; m < RP; ++m) {
                const float4 w = tile[2 * m * nt + tid], x = tile[(2 * m + 1) * nt + tid];
                S[m][0] = f2_pack(w.x, x.x), S[m][1] = f2_pack(w.y, x.y);
                S[m][2] = f2_pack(w.z, x.z), S[m][3] = f2_pack(w.w, x.w);
            }
            // a new sequence without accepted drafts: its zeros, unless its tokens' state is written below
            if (gp == 0 && !cur.init && (cur.update ? cur.n_tok == 0 : p.prev.T > 0)) store_state();
        }
        bool state_pending = false;  // the next unit's tile was committed after the next group's rows
        float decay = 1.0f;          // of the previous drafts
        for (int g = 0; g < ng; ++g) {
            if (g > 0) {
                if (state_pending)
                    copies_wait<1>();
                else
                    copies_wait<0>();
                __syncthreads();  // the rows are there, the last group's products are used up
            }
            state_pending = false;
            const bool old = g < gp;
            const int t0 = (old ? g : g - gp) * TG, n = min(TG, (old ? cur.n_prev : cur.n_tok) - t0);
            const unsigned char *const raw = smem + lay.raw + buf * lay.raw_bytes;
            const unsigned char *const raw_v = raw + 2 * TG * PITCH;
            // what comes next sets out now
            buf ^= 1;
            if (g + 1 < ng)
                fetch_group(cur, g + 1, buf);
            else if (groups_of(nxt) > 0)
                fetch_group(nxt, 0, buf);
            copies_commit();
            if (g == 0 && nxt.on) {
                fetch_state(nxt);
                copies_commit();
                state_pending = true;
            }
            // lane t of every TG: the token's decay a and gain b, the product of the decays up to it, and its
            // weight in the state after the group
            const float *const gb = reinterpret_cast<const float *>(raw_v + TG * pitch_v);
            const int lt = lane % TG;
            const float a = lt < n ? expf(gb[lt]) : 1.0f;
            const float b = lt < n ? ((old ? p.prev.b : p.tok.b) ? gb[TG + lt] : 1.0f) : 0.0f;
            float upto = a, after = __shfl_down_sync(0xffffffffu, a, 1, TG);
            if (lt == TG - 1) after = 1.0f;
#pragma unroll
            for (int o = 1; o < TG; o <<= 1) {
                const float x = __shfl_up_sync(0xffffffffu, upto, o, TG), y = __shfl_down_sync(0xffffffffu, after, o, TG);
                if (lt >= o) upto *= x;
                if (lt + o < TG) after *= y;
            }
            const float weight = after * b;

            auto advance = [&]() {
                const float all = __shfl_sync(0xffffffffu, upto, TG - 1, TG);
                const f2 all2 = f2_pack(all, all);
#pragma unroll
                for (int m = 0; m < RP; ++m)
#pragma unroll
                    for (int j = 0; j < kTileWords; ++j) S[m][j] = f2_mul(S[m][j], all2);
#pragma unroll
                for (int t = 0; t < TG; ++t) {
                    if (t >= n) break;
                    const float w = __shfl_sync(0xffffffffu, weight, t, TG);
                    const float4 v = load_four<BF>(raw_v + t * pitch_v + vc * ES);
                    f2 k2[RP];
                    load_rows<RP, BF>(k2, raw + t * PITCH + rg * R * ES);
                    const f2 x = f2_pack(w * v.x, w * v.x), y = f2_pack(w * v.y, w * v.y), z = f2_pack(w * v.z, w * v.z),
                             q = f2_pack(w * v.w, w * v.w);
#pragma unroll
                    for (int m = 0; m < RP; ++m) {
                        S[m][0] = f2_fma(k2[m], x, S[m][0]);
                        S[m][1] = f2_fma(k2[m], y, S[m][1]);
                        S[m][2] = f2_fma(k2[m], z, S[m][2]);
                        S[m][3] = f2_fma(k2[m], q, S[m][3]);
                    }
                }
            };
            if (old) {
                advance();
                decay *= __shfl_sync(0xffffffffu, upto, TG - 1, TG);
                if (g + 1 == gp && !(cur.update && cur.n_tok > 0)) store_state();
                continue;
            }
            const unsigned char *const raw_q = raw + TG * PITCH;
            // The block's products: pair (t, u) with u <= t < n, 4 lanes a pair, weighted by the gain of u and the
            // decays after it up to t.
            for (int e = warp * 8; e < TG * TG; e += warps * 8) {
                const int pair = e + (lane >> 2), t = pair / TG, u = pair % TG;
                float acc = 0.0f;
                if (pair < TG * TG && u <= t && t < n) {
                    f2 a2 = f2_pack(0.0f, 0.0f);
#pragma unroll
                    for (int x = 0; x < DKP / 4; x += 8) {  // pieces of 8 elements, the 4 lanes side by side
                        f2 q2[4], k2[4];
                        load_rows<4, BF>(q2, raw_q + t * PITCH + (x * 4 + quad * 8) * ES);
                        load_rows<4, BF>(k2, raw + u * PITCH + (x * 4 + quad * 8) * ES);
#pragma unroll
                        for (int y = 0; y < 4; ++y) a2 = f2_fma(q2[y], k2[y], a2);
                    }
                    float odd;
                    f2_unpack(a2, acc, odd);
                    acc += odd;
                }
                acc += __shfl_xor_sync(0xffffffffu, acc, 1);
                acc += __shfl_xor_sync(0xffffffffu, acc, 2);
                float w = __shfl_sync(0xffffffffu, b, u, TG);
#pragma unroll
                for (int x = 1; x < TG; ++x) {
                    const float ax = __shfl_sync(0xffffffffu, a, x, TG);
                    if (x > u && x <= t) w *= ax;
                }
                if (pair < TG * TG && quad == 0) pt[pair] = acc * w;
            }
            // S^T q: this lane's rows for every token
            float o[TG][4];
#pragma unroll
            for (int t = 0; t < TG; ++t) {
                o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.0f;
                if (t < n) {
                    f2 q2[RP], acc[4];
                    load_rows<RP, BF>(q2, raw_q + t * PITCH + rg * R * ES);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        acc[j] = f2_mul(q2[0], S[0][j]);
#pragma unroll
                        for (int m = 1; m < RP; ++m) acc[j] = f2_fma(q2[m], S[m][j], acc[j]);
                        float lo, hi;
                        f2_unpack(acc[j], lo, hi);
                        o[t][j] = lo + hi;
                    }
                }
            }
            // over the row groups; with 8 tokens each lane ends up with the token of its row group's number
            if constexpr (TG == 8) {
#pragma unroll
                for (int h = 4; h > 0; h >>= 1) {  // keep the half of the tokens whose bit is this lane's
                    const bool up = rg & h;
#pragma unroll
                    for (int t = 0; t < h; ++t)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float give = up ? o[t][j] : o[t + h][j], keep = up ? o[t + h][j] : o[t][j];
                            o[t][j] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * h);
                        }
                }
            } else {
#pragma unroll
                for (int h = 4; h < 32; h <<= 1)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[0][j] += __shfl_xor_sync(0xffffffffu, o[0][j], h);
            }
            __syncthreads();  // the products are there
            const int t = TG == 8 ? rg : 0;
            const float pre = __shfl_sync(0xffffffffu, upto, t, TG);
            if ((TG == 8 || rg == 0) && t < n && col) {
                float4 x = make_float4(pre * o[0][0], pre * o[0][1], pre * o[0][2], pre * o[0][3]), v;
#pragma unroll
                for (int u = 0; u < TG; ++u) {
                    if (u > t) break;
                    v = load_four<BF>(raw_v + u * pitch_v + vc * ES);
                    const float w = pt[t * TG + u];
                    x.x = fmaf(w, v.x, x.x), x.y = fmaf(w, v.y, x.y), x.z = fmaf(w, v.z, x.z), x.w = fmaf(w, v.w, x.w);
                }
                x.x *= p.scale, x.y *= p.scale, x.z *= p.scale, x.w *= p.scale;
                if (p.skip) {  // v is the token's own by now
                    const float sk = __ldg(p.skip + cur.h);
                    x.x = fmaf(sk, v.x, x.x), x.y = fmaf(sk, v.y, x.y), x.z = fmaf(sk, v.z, x.z), x.w = fmaf(sk, v.w, x.w);
                }
                const long long at = (p.tok.cu ? 0 : cur.s * p.o_seq) + ((long long)cur.row0 + t0 + t) * p.o_tok +
                                     (long long)cur.h * p.o_head + cur.slice * VS + vc;
                if (!p.o_vec) {
                    const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if constexpr (BF)
                            reinterpret_cast<uint16_t *>(p.out)[at + j] = narrow<uint16_t>(y[j]);
                        else
                            reinterpret_cast<float *>(p.out)[at + j] = y[j];
                } else if constexpr (BF) {
                    *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(p.out) + at) =
                        make_uint2(pack_halves(narrow<uint16_t>(x.x), narrow<uint16_t>(x.y)),
                                   pack_halves(narrow<uint16_t>(x.z), narrow<uint16_t>(x.w)));
                } else {
                    *reinterpret_cast<float4 *>(reinterpret_cast<float *>(p.out) + at) = x;
                }
            }
            if (g + 1 < ng || cur.update) advance();
            if (g + 1 == ng && cur.update) store_state();
        }
        if (p.own_states && cur.on && cur.slice == 0 && tid == 0)
            p.ws_decay[((long long)cur.s * p.n_heads + cur.h) * p.pieces + cur.piece] = decay;
        if (ng == 0) {  // no group: the next unit's loads set out here
            if (groups_of(nxt) > 0) fetch_group(nxt, 0, buf);
            if (nxt.on) fetch_state(nxt);
            copies_commit();
        }
    }
    copies_wait<0>();
}

// S_0 = the initial state; S_{i+1} = decay_i S_i + own_i, written over own_i.  One word a thread; the pieces
// are read ahead 8 at a time, since only the sums depend on one another.
__global__ void __launch_bounds__(kStateJoinThreads) state_join(const __grid_constant__ LinattnParams p) {
    grid_dep_wait();
    grid_dep_launch();
    const int words = p.dk * p.dv, parts = (words + kStateJoinThreads - 1) / kStateJoinThreads;
    const int e = (int)(blockIdx.x % (unsigned)parts) * kStateJoinThreads + threadIdx.x;
    const int sh = (int)(blockIdx.x / (unsigned)parts), h = sh % p.n_heads, s = sh / p.n_heads;
    const int slot = p.cache_idx ? __ldg(p.cache_idx + s) : s;
    int L, row0;
    if (slot < 0 || slot >= p.n_slots || draft_span(p.tok.cu, s, p.tok.T, p.tok.total, L, row0) || e >= words) return;
    const int n = (L + p.piece_len - 1) / p.piece_len - 1;  // pieces with a next one
    const bool init = p.has_init ? __ldg(p.has_init + s) != 0 : true;
    float S = init && n > 0 ? p.state[(long long)slot * p.st_slot + (long long)h * p.st_head + e] : 0.0f;
    const long long base = (long long)sh * p.pieces;
    float *const own = p.ws_state + base * words + e;
    const float *const dec = p.ws_decay + base;
    // The first piece's state too: the last piece writes the sequence's while the first may not have begun.
    if (n > 0) *own = S;
    for (int i0 = 0; i0 < n; i0 += 8) {
        float f[8], d[8];
#pragma unroll
        for (int x = 0; x < 8; ++x)
            if (i0 + x < n) f[x] = own[(long long)(i0 + x + 1) * words], d[x] = dec[i0 + x];
#pragma unroll
        for (int x = 0; x < 8; ++x)
            if (i0 + x < n) own[(long long)(i0 + x + 1) * words] = S = fmaf(d[x], S, f[x]);
    }
}

template <int VS, int R>
StepKernel pick(int tg) {
    if (tg == 1) return {linattn_step<VS, R, 1>, step_smem_floats(VS, R, 1) * 4};
    return {linattn_step<VS, R, kStepMaxGroup>, step_smem_floats(VS, R, kStepMaxGroup) * 4};
}
template <int R, int TG>
StepKernel pick_stream(int warps, bool bf16) {
    return {bf16 ? linattn_stream<R, TG, true> : linattn_stream<R, TG, false>, StreamLayout(warps, R, TG, bf16).bytes};
}

}  // namespace

StepKernel step_kernel(int vs, int dk, int tg) {
    if (vs == 64) return dk <= 64 ? pick<64, 4>(tg) : dk <= 128 ? pick<64, 8>(tg) : pick<64, 16>(tg);
    return dk <= 64 ? pick<32, 2>(tg) : dk <= 128 ? pick<32, 4>(tg) : pick<32, 8>(tg);
}
LinattnKernel state_join_kernel() { return state_join; }
StepKernel stream_kernel(int warps, int dk, int tg, bool bf16) {
    if (dk <= 64) return tg == 1 ? pick_stream<8, 1>(warps, bf16) : pick_stream<8, kStepMaxGroup>(warps, bf16);
    return tg == 1 ? pick_stream<16, 1>(warps, bf16) : pick_stream<16, kStepMaxGroup>(warps, bf16);
}

}  // namespace cvk
