// The RMS norms around a block, fused with its gate and its scaled residual.
//
// Per row:  a = y [* act(z)];  a *= rsqrt(mean_group a^2 + eps) * w_post;  a [*= act(z)];
//           r = res + scale * cs * a;  out = r * rsqrt(mean_row r^2 + eps) * w_pre.
// Sums are fp32 in a fixed order (per thread, a shuffle tree, then the warps in order): a row's bits do
// not depend on the other rows' values (their number may choose another split of the row).  r enters the second
// norm unrounded.  Every tensor is read and written once: the kernels are bound by HBM (large calls) or by
// latency (a few rows).
//   norm_groups  no residual, narrow groups (a norm for each head): a group's elements sit in up to
//                32 lanes of one warp, 16 bytes a lane, so no shared memory and no barrier (30822 x 6144
//                gated, groups of 128, bf16: 202 us, 5.6 TB/s)
//   norm_row     a block a row, the row's values in registers between the two norms (1023 x 4096, fp32
//                residual: 12.9 us, 127 registers hold 608 rows on the card, so 1.7 waves; 14648 x 4096: 125 us,
//                6.7 TB/s)
//   norm_any     a block a row, values read again (from L1/L2) for each pass, one element an access: rows too wide
//                for registers and residual rows with several groups (30000 x 4096 gated, groups of 128, fp32
//                residual: 1155 us, 4.5 times its floor)
#include "cv_device.cuh"
#include "cv_norm.h"

namespace cvk {
namespace {

// V consecutive elements as raw words: 16 or 32 bytes in 16-byte accesses, or V = 2 in one access of 4 or
// 8 bytes, or V = 1.
template <typename B, int V>
struct Run {
    static constexpr int W = V == 1 ? 1 : V * (int)sizeof(B) / 4;
    uint32_t w[W];
    __device__ __forceinline__ void load(const void *base, long long i) {
        const B *p = reinterpret_cast<const B *>(base) + i;
        if constexpr (V == 1)
            w[0] = *p;
        else if constexpr (W == 1)
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        else
            ldv<W == 2 ? 8 : 16, W>(w, p);
    }
    __device__ __forceinline__ float operator[](int j) const {
        if constexpr (V == 1)
            return widen<B>((B)w[0]);
        else
            return elem_f<B>(w, j);
    }
};
template <typename B, int V>
__device__ __forceinline__ void load_run(float *r, const void *base, long long i) {
    Run<B, V> t;
    t.load(base, i);
#pragma unroll
    for (int j = 0; j < V; ++j) r[j] = t[j];
}
template <typename B, int V>
__device__ __forceinline__ void store_run(void *base, long long i, const float *r) {
    B *p = reinterpret_cast<B *>(base) + i;
    if constexpr (V == 1) {
        *p = narrow<B>(r[0]);
    } else {
        constexpr int W = V * (int)sizeof(B) / 4;
        uint32_t w[W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            if constexpr (sizeof(B) == 2)
                w[j] = pack_halves(narrow<uint16_t>(r[2 * j]), narrow<uint16_t>(r[2 * j + 1]));
            else
                w[j] = __float_as_uint(r[j]);
        }
        if constexpr (W == 1)
            *reinterpret_cast<uint32_t *>(p) = w[0];
        else
            stv<W == 2 ? 8 : 16, W>(p, w);
    }
}

// act(z) for n values: silu as the conv computes it, or the sigmoid by the same fast instructions, with
// the exact forms below -80, where those flush.
__device__ __forceinline__ float sigmoid_fast(float z) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}
template <int N>
__device__ __forceinline__ void gate_run(const float *z, float *g, int act) {
    if (act == 0) {
        silu_run<N>(z, g);
    } else {
        float lo = z[0];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            g[i] = sigmoid_fast(z[i]);
            lo = fminf(lo, z[i]);
        }
        if (lo < -80.0f) {
#pragma unroll
            for (int i = 0; i < N; ++i) g[i] = z[i] < -80.0f ? 1.0f / (1.0f + expf(-z[i])) : g[i];
        }
    }
}
__device__ __forceinline__ float gate_of(float z, int act) {
    float g;
    gate_run<1>(&z, &g, act);
    return g;
}

// U groups a thread at once, so that U loads of each tensor are in flight.
template <typename B, int V, int NV, int U>
__global__ void __launch_bounds__(kNormGroupThreads) norm_groups(const __grid_constant__ NormParams p) {
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x % p.lanes;  // within the group
    const int per_block = kNormGroupThreads / p.lanes;
    const int per_row = p.flat ? 1 : p.dim / p.group;
    const long long total = p.rows * (p.dim / p.group);
    const long long step = (long long)gridDim.x * per_block * U;
    const long long first = (long long)blockIdx.x * per_block * U;
    // whole warps walk the groups together, so the shuffles below always have all lanes
    for (long long base = first; base < total; base += step) {
        Run<B, V> y[U][NV], z[U][NV];
        long long row[U];
        int c0[U];
        bool on[U];
#pragma unroll
        for (int x = 0; x < U; ++x) {
            const long long gi = base + x * per_block + threadIdx.x / p.lanes;
            on[x] = gi < total;
            // rows one after the other (flat): a group is a row of its own
            if (p.flat)
                row[x] = gi, c0[x] = 0;
            else if (total <= 0x7fffffff)
                row[x] = (unsigned)gi / (unsigned)per_row, c0[x] = (int)((unsigned)gi % (unsigned)per_row) * p.group;
            else
                row[x] = gi / per_row, c0[x] = (int)(gi % per_row) * p.group;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * p.lanes + lane) * V;
#pragma unroll
                for (int j = 0; j < Run<B, V>::W; ++j) y[x][i].w[j] = z[x][i].w[j] = 0u;
                if (on[x] && c < p.group) {
                    y[x][i].load(p.y, row[x] * p.y_row + c0[x] + c);
                    if (p.gate) z[x][i].load(p.gate, row[x] * p.gate_row + c0[x] + c);
                }
            }
        }
#pragma unroll
        for (int x = 0; x < U; ++x) {
            float a[NV][V], g[NV][V], sum = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
#pragma unroll
                for (int j = 0; j < V; ++j) a[i][j] = y[x][i][j];
                if (p.gate) {
                    float t[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) t[j] = z[x][i][j];
                    gate_run<V>(t, g[i], p.gate_act);
                    if (p.gate_first)
#pragma unroll
                        for (int j = 0; j < V; ++j) a[i][j] *= g[i][j];
                }
#pragma unroll
                for (int j = 0; j < V; ++j) sum = fmaf(a[i][j], a[i][j], sum);
            }
            for (int o = p.lanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float inv = rsqrtf(sum / (float)p.group + p.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * p.lanes + lane) * V;
                if (!on[x] || c >= p.group) continue;
                Run<B, V> w;
                if (p.post) w.load(p.post, c);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float u = a[i][j] * inv;
                    if (p.post) u *= w[j];
                    if (p.gate && !p.gate_first) u *= g[i][j];
                    a[i][j] = u;
                }
                store_run<B, V>(p.out, row[x] * p.out_row + c0[x] + c, a[i]);
            }
        }
    }
}

// Asks for `bytes` bytes (a multiple of 16, from a 16-byte boundary) in L2.
__device__ __forceinline__ void prefetch_l2(const void *p, int bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Sum over the block, the same for every thread (warps added in order).
__device__ __forceinline__ float block_sum(float v, float *sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int nw = (blockDim.x + 31) / 32;
    if (nw == 1) return v;
    __syncthreads();  // the last use of sh is over
    if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.0f;
    for (int i = 0; i < nw; ++i) v += sh[i];
    return v;
}

// blockDim.x threads a row; rows of one warp each share a block (blockDim.y of them).  Every choice that is
// the call's (a gate, a weight, a residual) is made outside the loops over a thread's elements: with
// one-element accesses (odd widths) the kernel is bound by its instructions (30000 gated residual rows of 1023,
// bf16: 222 -> 155 us).
template <typename B, typename RB, int V, int NV>
__global__ void __launch_bounds__(kNormRowThreads, V * NV <= 8 ? 2 : 1) norm_row(const __grid_constant__ NormParams p) {
    __shared__ float sh[kNormRowThreads / 32];
    constexpr int CH = V >= 8 ? 1 : NV < 8 / V ? NV : 8 / V;  // accesses a thread handles at once after the first sum
    // the weights too are loaded before the first sum while registers allow it
    constexpr bool kEarly = V > 1 && CH == NV && Run<B, V>::W * NV <= 8;
    const int nt = blockDim.x;
    grid_dep_wait();
    grid_dep_launch();
    for (long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y; row < p.rows; row += (long long)gridDim.x * blockDim.y) {
        auto at = [&](int i) { return (i * nt + (int)threadIdx.x) * V; };
        // n accesses from the i0-th on (zeros outside of the row)
        auto fetch = [&](auto *t, int n, const void *base, long long off, int i0) {
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const int c = at(i0 + i);
#pragma unroll
                for (int j = 0; j < (int)(sizeof t[0] / 4); ++j) t[i].w[j] = 0u;
                if (c < p.dim) t[i].load(base, off + c);
            }
        };
        Run<B, V> y[NV], z[NV], w[CH], cs[CH], w2[CH];
        Run<RB, V> r[NV];
        // Rows of 16-byte accesses: the row that a later block will read is asked for in L2, since a block
        // loads nothing while it sums and stores.  One row an SM ahead (14648 rows of 4096, bf16: 93 -> 81 us,
        // f32 133 -> 111; two or four rows an SM are no faster and push wide fp32 rows out again;
        // up to 16 rows an SM, where few later blocks are left to read it, it costs 4 %);
        // not for rows that share a block (of 64: 17.6 us with it, 15.5 without).
        if constexpr (V > 2) {
            const long long next = row + p.ahead;
            if (threadIdx.x == 0 && blockDim.y == 1 && next < p.rows) {
                prefetch_l2(reinterpret_cast<const B *>(p.y) + next * p.y_row, p.dim * (int)sizeof(B));
                if (p.gate) prefetch_l2(reinterpret_cast<const B *>(p.gate) + next * p.gate_row, p.dim * (int)sizeof(B));
                if (p.res) prefetch_l2(reinterpret_cast<const RB *>(p.res) + next * p.res_row, p.dim * (int)sizeof(RB));
            }
        }
        fetch(y, NV, p.y, row * p.y_row, 0);
        if (p.gate) fetch(z, NV, p.gate, row * p.gate_row, 0);
        if (p.res) fetch(r, NV, p.res, row * p.res_row, 0);
        if constexpr (kEarly) {
            if (p.post) fetch(w, CH, p.post, 0, 0);
            if (p.cs) fetch(cs, CH, p.cs, 0, 0);
            if (p.pre) fetch(w2, CH, p.pre, 0, 0);
        }
        float a[NV * V], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) a[i * V + j] = y[i][j];
        if (p.gate && p.gate_first) {
#pragma unroll
            for (int i0 = 0; i0 < NV; i0 += CH) {
                float t[CH * V], g[CH * V];
#pragma unroll
                for (int k = 0; k < CH * V; ++k) t[k] = z[i0 + k / V][k % V];
                gate_run<CH * V>(t, g, p.gate_act);
#pragma unroll
                for (int k = 0; k < CH * V; ++k) a[i0 * V + k] *= g[k];
            }
        }
#pragma unroll
        for (int k = 0; k < NV * V; ++k) sum = fmaf(a[k], a[k], sum);
        const float inv = p.group > 0 ? rsqrtf(block_sum(sum, sh) / (float)p.dim + p.eps) : 1.0f;
        sum = 0.0f;
#pragma unroll
        for (int i0 = 0; i0 < NV; i0 += CH) {
            if (V * NV > 8 && at(i0) >= p.dim) break;
            float *u = a + i0 * V;
            if constexpr (!kEarly) {
                if (p.post) fetch(w, CH, p.post, 0, i0);
                if (p.cs) fetch(cs, CH, p.cs, 0, i0);
            }
#pragma unroll
            for (int k = 0; k < CH * V; ++k) u[k] *= inv;
            if (p.post)
#pragma unroll
                for (int k = 0; k < CH * V; ++k) u[k] *= w[k / V][k % V];
            if (p.gate && !p.gate_first) {
                float t[CH * V], g[CH * V];
#pragma unroll
                for (int k = 0; k < CH * V; ++k) t[k] = z[i0 + k / V][k % V];
                gate_run<CH * V>(t, g, p.gate_act);
#pragma unroll
                for (int k = 0; k < CH * V; ++k) u[k] *= g[k];
            }
            if (p.res) {
                if (p.cs)
#pragma unroll
                    for (int k = 0; k < CH * V; ++k) u[k] = fmaf(p.scale * cs[k / V][k % V], u[k], r[i0 + k / V][k % V]);
                else
#pragma unroll
                    for (int k = 0; k < CH * V; ++k) u[k] = fmaf(p.scale, u[k], r[i0 + k / V][k % V]);
#pragma unroll
                for (int i = 0; i < CH; ++i)
                    if (at(i0 + i) < p.dim) {
#pragma unroll
                        for (int j = 0; j < V; ++j) sum = fmaf(u[i * V + j], u[i * V + j], sum);
                        store_run<RB, V>(p.res_out, row * p.res_out_row + at(i0 + i), u + i * V);
                    }
            } else {
#pragma unroll
                for (int i = 0; i < CH; ++i)
                    if (at(i0 + i) < p.dim) store_run<B, V>(p.out, row * p.out_row + at(i0 + i), u + i * V);
            }
        }
        if (p.res && p.out) {
            const float inv2 = rsqrtf(block_sum(sum, sh) / (float)p.dim + p.eps);
#pragma unroll
            for (int i0 = 0; i0 < NV; i0 += CH) {
                if (V * NV > 8 && at(i0) >= p.dim) break;
                float *u = a + i0 * V;
                if constexpr (!kEarly) {
                    if (p.pre) fetch(w2, CH, p.pre, 0, i0);
                }
#pragma unroll
                for (int k = 0; k < CH * V; ++k) u[k] *= inv2;
                if (p.pre)
#pragma unroll
                    for (int k = 0; k < CH * V; ++k) u[k] *= w2[k / V][k % V];
#pragma unroll
                for (int i = 0; i < CH; ++i)
                    if (at(i0 + i) < p.dim) store_run<B, V>(p.out, row * p.out_row + at(i0 + i), u + i * V);
            }
        }
    }
}

template <typename B, typename RB>
__global__ void __launch_bounds__(kNormAnyThreads) norm_any(const __grid_constant__ NormParams p) {
    extern __shared__ float sh[];  // the warps' sums, then one factor per group
    float *const inv = sh + kNormAnyThreads / 32;
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, lane = tid % 32;
    const int n_groups = p.group > 0 ? p.dim / p.group : 0;
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        auto gate = [&](int c) {
            float z;
            load_run<B, 1>(&z, p.gate, row * p.gate_row + c);
            return gate_of(z, p.gate_act);
        };
        auto value = [&](int c) {  // the first norm's input
            float v;
            load_run<B, 1>(&v, p.y, row * p.y_row + c);
            return p.gate && p.gate_first ? v * gate(c) : v;
        };
        // narrow groups: a warp each; a few wide ones: the whole block on each
        if (n_groups >= kNormAnyThreads / 32) {
            for (int g = tid / 32; g < n_groups; g += kNormAnyThreads / 32) {
                float sum = 0.0f;
                for (int c = lane; c < p.group; c += 32) {
                    const float v = value(g * p.group + c);
                    sum = fmaf(v, v, sum);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (lane == 0) inv[g] = rsqrtf(sum / (float)p.group + p.eps);
            }
        } else {
            for (int g = 0; g < n_groups; ++g) {
                float sum = 0.0f;
                for (int c = tid; c < p.group; c += kNormAnyThreads) {
                    const float v = value(g * p.group + c);
                    sum = fmaf(v, v, sum);
                }
                sum = block_sum(sum, sh);
                if (tid == 0) inv[g] = rsqrtf(sum / (float)p.group + p.eps);
            }
        }
        __syncthreads();
        auto first = [&](int c) {  // after the first norm and the gate
            float u = value(c), w;
            if (p.group > 0) u *= inv[c / p.group];
            if (p.post) {
                load_run<B, 1>(&w, p.post, c % p.group);
                u *= w;
            }
            return p.gate && !p.gate_first ? u * gate(c) : u;
        };
        auto resid = [&](int c) {
            float r, f;
            load_run<RB, 1>(&r, p.res, row * p.res_row + c);
            if (p.cs) load_run<B, 1>(&f, p.cs, c);
            return fmaf(p.cs ? p.scale * f : p.scale, first(c), r);
        };
        if (!p.res) {
            for (int c = tid; c < p.dim; c += kNormAnyThreads) {
                const float u = first(c);
                store_run<B, 1>(p.out, row * p.out_row + c, &u);
            }
        } else {
            float sum = 0.0f, inv2 = 1.0f;
            if (p.out) {
                for (int c = tid; c < p.dim; c += kNormAnyThreads) {
                    const float r = resid(c);
                    sum = fmaf(r, r, sum);
                }
                inv2 = rsqrtf(block_sum(sum, sh) / (float)p.dim + p.eps);
            }
            // each thread reads its channel once more before it writes it: in-place calls are safe
            for (int c = tid; c < p.dim; c += kNormAnyThreads) {
                const float r = resid(c);
                store_run<RB, 1>(p.res_out, row * p.res_out_row + c, &r);
                if (p.out) {
                    float x = r * inv2, w;
                    if (p.pre) {
                        load_run<B, 1>(&w, p.pre, c);
                        x *= w;
                    }
                    store_run<B, 1>(p.out, row * p.out_row + c, &x);
                }
            }
        }
        __syncthreads();  // inv and sh are free for the next row
    }
}

template <typename B, typename RB, int V>
NormKernel pick_row(int elems) {
    if (elems == 8) return norm_row<B, RB, V, 8 / V>;
    if constexpr (V > 2) {
        if (elems == 32) return norm_row<B, RB, V, 32 / V>;
    }
    return norm_row<B, RB, V, 16 / V>;
}

}  // namespace

NormKernel norm_groups_kernel(bool bf16, bool vec, int nv, int unroll) {
    if (bf16) {
        if (vec && nv == 1) return unroll > 1 ? norm_groups<uint16_t, 8, 1, kNormUnroll> : norm_groups<uint16_t, 8, 1, 1>;
        if (vec) return norm_groups<uint16_t, 8, 2, 1>;
        return norm_groups<uint16_t, 1, 4, 1>;
    }
    if (vec && nv == 1) return unroll > 1 ? norm_groups<uint32_t, 4, 1, kNormUnroll> : norm_groups<uint32_t, 4, 1, 1>;
    if (vec) return norm_groups<uint32_t, 4, 2, 1>;
    return norm_groups<uint32_t, 1, 4, 1>;
}

NormKernel norm_row_kernel(bool bf16, bool res_f32, int v, int elems) {
    if (bf16) {
        if (res_f32)
            return v == 8   ? pick_row<uint16_t, uint32_t, 8>(elems)
                   : v == 2 ? pick_row<uint16_t, uint32_t, 2>(elems)
                            : pick_row<uint16_t, uint32_t, 1>(elems);
        return v == 8   ? pick_row<uint16_t, uint16_t, 8>(elems)
               : v == 2 ? pick_row<uint16_t, uint16_t, 2>(elems)
                        : pick_row<uint16_t, uint16_t, 1>(elems);
    }
    return v == 4   ? pick_row<uint32_t, uint32_t, 4>(elems)
           : v == 2 ? pick_row<uint32_t, uint32_t, 2>(elems)
                    : pick_row<uint32_t, uint32_t, 1>(elems);
}

NormKernel norm_any_kernel(bool bf16, bool res_f32) {
    if (!bf16) return norm_any<uint32_t, uint32_t>;
    return res_f32 ? norm_any<uint16_t, uint32_t> : norm_any<uint16_t, uint16_t>;
}

}  // namespace cvk
