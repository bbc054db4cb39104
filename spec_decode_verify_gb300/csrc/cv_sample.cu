// Verification of drafted tokens: which of them stand, and the token sampled after them.
//
// A cluster of 8 blocks takes a sequence.  Each block walks the drafts by itself (a gather of two probabilities a
// draft, then one pass over the drafts, since a child comes after its parent), which says what row to sample from.  The
// row's weights are summed by 128 warps, a run of tokens each; the 128 sums go to all blocks through distributed
// shared memory, and the block whose run holds the token reads that run once more and finds it.
//
// Weights are summed as integers in units of 2^-60, so a sum has one value whatever the order, and the same
// one in both passes.  HBM bounds it at many sequences; one sequence is bound by latency: a gather, a row's part, a
// cluster barrier, and a run again.
#include "cv_attn.cuh"

namespace cvk {
namespace {

using u64 = unsigned long long;
constexpr int kRuns = kSampleCluster * (kSampleThreads / 32);
constexpr int kMaxDrafts = 128;
constexpr int kMaxSum = 4;  // weights that add up to as much are refused: their integers would not fit

// x in units of 2^-60, cut off; what is not above 0 is 0, and 2 and more is just below 2.
__device__ __forceinline__ u64 units(float x) {
    if (!(x > 0.f)) return 0;
    const uint32_t b = min(__float_as_uint(x), 0x3fffffffu);
    const int shift = (int)(b >> 23) - (127 + 23 - 60);
    const uint32_t m = (b & 0x7fffffu) | 0x800000u;  // (a subnormal is below a unit)
    return shift >= 0 ? (u64)m << shift : shift > -24 ? m >> -shift : 0u;
}

enum { kRow = 0, kDiff = 1, kLeft = 2 };

struct SampleShared {
    double mass[kMaxDrafts], draft[kMaxDrafts];
    int tok[kMaxDrafts], up[kMaxDrafts], tried[kMaxDrafts], path[kMaxDrafts];
    int n_tried, accept, end, mode, child, T, row0, status;
    u64 sum[kRuns], plain[kRuns];  // of the weights, and of the target's row alone
    float size[kRuns];
    u64 before, target;            // of the run found: weights before it, and what to exceed
    int run, use_plain;
    u64 warp_sum[kSampleThreads / 32];
};

template <typename B>
__device__ __forceinline__ float prob(const void *base, long long at) {
    return widen<B>(__ldg(reinterpret_cast<const B *>(base) + at));
}

__device__ __forceinline__ u64 shfl_up64(u64 v, int o) { return __shfl_up_sync(0xffffffffu, v, o); }

// 16 bytes of a row from token j on as fp32, zeros before token 0 and from V on; wide: j is on a 16-byte boundary.
template <typename B, int N>
__device__ __forceinline__ void load_probs(float *f, const B *row, int j, int V, bool wide) {
    if (wide && j >= 0 && j + N <= V) {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(row + j));
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = elem_f<B>(x, i);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = j + i >= 0 && j + i < V ? widen<B>(__ldg(row + j + i)) : 0.f;
    }
}

template <typename B>
__global__ void __cluster_dims__(kSampleCluster, 1, 1) __launch_bounds__(kSampleThreads)
    draft_sample(const __grid_constant__ SampleParams p) {
    constexpr int N = 16 / (int)sizeof(B);
    __shared__ SampleShared sh;
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int s = blockIdx.x / kSampleCluster, rank = blockIdx.x % kSampleCluster;
    const bool on = !p.idx || __ldg(p.idx + s) >= 0;
    int T = p.T, row0 = 0, status = 0;
    if (on && p.cu) {
        status = draft_span(p.cu, s, p.T, p.total, T, row0);
        if (!status && T == 0) status = kSeqBadSpan;
    }
    const bool walks = on && !status;
    const long long pbase = p.cu ? (long long)row0 * p.p_tok : (long long)s * p.p_seq;
    const long long qbase = p.cu ? (long long)row0 * p.q_tok : (long long)s * p.q_seq;
    if (walks) {
        const long long at = p.cu ? (long long)row0 : (long long)s * p.T;
        int bad = 0;
        if (tid < T) {
            const int tok = __ldg(p.tok + at + tid);
            int up = p.parent ? __ldg(p.parent + at + tid) : tid - 1;
            if (up < -1 || up >= tid) bad |= kSeqBadTree, up = -1;
            double mass = 0., draft = 0.;
            if (tid > 0) {
                if (tok < 0 || tok >= p.vocab) bad |= kSeqBadToken;
                else if (up >= 0) {
                    mass = (double)prob<B>(p.p, pbase + (long long)up * p.p_tok + tok);
                    if (p.q) draft = (double)prob<B>(p.q, qbase + (long long)tid * p.q_tok + tok);
                }
            }
            sh.tok[tid] = tok, sh.up[tid] = up, sh.mass[tid] = mass, sh.draft[tid] = draft;
        }
        if (tid == 0) sh.status = 0;
        __syncthreads();
        if (bad) atomicOr(&sh.status, bad);
        __syncthreads();
        status = sh.status;
        if (!status && tid == 0) {
            const float *const u = p.u + (long long)s * (p.T + 1);
            int end = 0, n = 1, tried = 0;
            float draw = __ldg(u);
            double sum = 0.;
            sh.path[0] = 0;
            for (int t = 1; t < T; ++t) {
                if (sh.up[t] != end) continue;
                const int tok = sh.tok[t];
                bool twin = false;
                for (int i = 0; i < tried; ++i) twin |= sh.tried[i] == tok;
                if (twin) continue;
                const double d = draw > 0.f ? fmin((double)draw, 0x1.fffffep-1) : 0.;
                sum += sh.mass[t];
                if (p.q ? d * sh.draft[t] < sh.mass[t] : d < sum) {
                    sh.path[n++] = t;
                    end = t, tried = 0, sum = 0.;
                    draw = __ldg(u + t);
                } else {
                    sh.tried[tried++] = tok;
                    sh.child = t;
                }
            }
            sh.accept = n, sh.end = end, sh.n_tried = tried;
            sh.mode = tried == 0 ? kRow : p.q ? kDiff : kLeft;
        }
        __syncthreads();
    }
    const bool sums = walks && !status;
    const int V = p.vocab, mode = sums ? sh.mode : kRow;
    const B *const row = reinterpret_cast<const B *>(p.p) + pbase + (sums ? (long long)sh.end * p.p_tok : 0);
    const B *const minus = mode == kDiff ? reinterpret_cast<const B *>(p.q) + qbase + (long long)sh.child * p.q_tok : nullptr;
    // runs of whole accesses of a warp that begin on 16-byte boundaries, the first one up to N - 1 tokens before token 0
    const int shift = (int)(reinterpret_cast<uintptr_t>(row) % 16) / (int)sizeof(B);
    const bool wide = (reinterpret_cast<uintptr_t>(minus) % 16) / sizeof(B) == (unsigned)shift;
    const int len = (V + shift + kRuns * 32 * N - 1) / (kRuns * 32 * N) * (32 * N);
    const int run = rank * (kSampleThreads / 32) + warp;
    if (sums) {
        const int lo = min(V, run * len - shift), hi = min(V, lo + len);
        u64 sum = 0, plain = 0;
        float size = 0.f;
        if (mode == kDiff) {
#pragma unroll 4
            for (int j = lo + lane * N; j < hi; j += 32 * N) {
                float a[N], b[N];
                load_probs<B, N>(a, row, j, V, true);
                load_probs<B, N>(b, minus, j, V, wide);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const u64 x = units(a[i]), y = units(b[i]);
                    plain += x;
                    sum += x > y ? x - y : 0;
                    size += a[i] > 0.f ? fminf(a[i], 2.f) : 0.f;
                }
            }
        } else {
#pragma unroll 4
            for (int j = lo + lane * N; j < hi; j += 32 * N) {
                float a[N];
                load_probs<B, N>(a, row, j, V, true);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    plain += units(a[i]);
                    size += a[i] > 0.f ? fminf(a[i], 2.f) : 0.f;
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            plain += __shfl_xor_sync(0xffffffffu, plain, o);
            size += __shfl_xor_sync(0xffffffffu, size, o);
        }
        if (mode == kRow) sum = plain;
        if (mode == kLeft) {  // the children's tokens again, to leave them out
            u64 out = 0;
            for (int i = lane; i < sh.n_tried; i += 32)
                if (sh.tried[i] >= lo && sh.tried[i] < hi) out += units(widen<B>(__ldg(row + sh.tried[i])));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) out += __shfl_xor_sync(0xffffffffu, out, o);
            sum = plain - out;
        }
        // to every block of the cluster, a lane each (all of them have begun)
        asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
        if (lane < kSampleCluster) {
            auto to = [&](const void *mine) {
                uint32_t a;
                asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(smem_u32(mine)), "r"(lane));
                return a;
            };
            asm volatile("st.shared::cluster.b64 [%0], %1;\n" ::"r"(to(&sh.sum[run])), "l"(sum) : "memory");
            asm volatile("st.shared::cluster.b64 [%0], %1;\n" ::"r"(to(&sh.plain[run])), "l"(plain) : "memory");
            asm volatile("st.shared::cluster.b32 [%0], %1;\n" ::"r"(to(&sh.size[run])), "f"(size) : "memory");
        }
    } else {
        asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
    if (!on) return;
    if (sums) {
        if (warp == 0) {  // 4 runs a lane
            u64 a[4], b[4], ta = 0, tb = 0;
            float size = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = sh.sum[4 * lane + i], b[i] = sh.plain[4 * lane + i];
                ta += a[i], tb += b[i], size += sh.size[4 * lane + i];
            }
            u64 all = ta, all_plain = tb;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                all += __shfl_xor_sync(0xffffffffu, all, o);
                all_plain += __shfl_xor_sync(0xffffffffu, all_plain, o);
                size += __shfl_xor_sync(0xffffffffu, size, o);
            }
            const bool use_plain = all == 0;
            if (use_plain) {
                all = all_plain, ta = tb;
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = b[i];
            }
            if (lane == 0) sh.use_plain = use_plain, sh.run = -1;
            if (all == 0 || !(size < (float)kMaxSum)) {
                status = kSeqBadProbs;
            } else {
                const float draw = __ldg(p.u + (long long)s * (p.T + 1) + p.T);
                const double d = draw > 0.f ? fmin((double)draw, 0x1.fffffep-1) : 0.;
                const u64 target = __umul64hi((u64)(d * 0x1p64), all);  // the token's sum exceeds it
                u64 up = ta;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const u64 x = shfl_up64(up, o);
                    if (lane >= o) up += x;
                }
                u64 before = up - ta;
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (before <= target && target < before + a[i]) sh.run = 4 * lane + i, sh.before = before, sh.target = target;
                    before += a[i];
                }
            }
            if (lane == 0) sh.status = status;
        }
        __syncthreads();
        status = sh.status;
    }
    if (status) {
        if (rank == 0 && tid == 0 && p.err) p.err[s] = status;
        return;
    }
    const int n = sh.accept;
    if (rank == 0) {
        if (tid == 0) {
            p.accept[s] = n;
            if (p.node) p.node[s] = sh.end + 1;
            if (p.err) p.err[s] = 0;
        }
        for (int t = tid; t < p.T; t += kSampleThreads) {
            if (p.path) p.path[(long long)s * p.T + t] = t < n ? sh.path[t] : -1;
            if (t != n - 1) p.out[(long long)s * p.T + t] = t + 1 < n ? sh.tok[sh.path[t + 1]] : -1;
        }
    }
    if (sh.run / (kSampleThreads / 32) != rank) return;
    // the run again, each thread a few tokens in a row
    const int lo = sh.run * len - shift, hi = min(V, lo + len);
    const int each = (len + kSampleThreads - 1) / kSampleThreads, to = min(hi, lo + (tid + 1) * each), from = max(0, lo + tid * each);
    const bool plain = sh.use_plain != 0;
    auto weight = [&](int j) {
        const u64 x = units(widen<B>(__ldg(row + j)));
        if (plain || mode == kRow) return x;
        if (mode == kDiff) {
            const u64 y = units(widen<B>(__ldg(minus + j)));
            return x > y ? x - y : 0;
        }
        for (int i = 0; i < sh.n_tried; ++i)
            if (sh.tried[i] == j) return (u64)0;
        return x;
    };
    u64 mine = 0;
#pragma unroll 4
    for (int j = from; j < to; ++j) mine += weight(j);
    u64 up = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 x = shfl_up64(up, o);
        if (lane >= o) up += x;
    }
    if (lane == 31) sh.warp_sum[warp] = up;
    __syncthreads();
    u64 before = sh.before + up - mine;
    for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
    if (before <= sh.target && sh.target < before + mine)
        for (int j = from; j < to; ++j) {
            before += weight(j);
            if (sh.target < before) {
                p.out[(long long)s * p.T + n - 1] = j;
                break;
            }
        }
}

}  // namespace

SampleKernel sample_kernel(bool bf16) { return bf16 ? draft_sample<uint16_t> : draft_sample<uint32_t>; }

}  // namespace cvk
