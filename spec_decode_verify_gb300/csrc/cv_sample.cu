// Verification of drafted tokens: which of them stand, and the token sampled after them.
//
// A cluster of 8 blocks takes a sequence (fewer where there are sequences for every SM).  Each block finds the end of
// the walk by itself: a thread a draft gathers its probabilities; a chain then has its end where the first draft falls, a tree is
// walked by one warp, which sees a node's children by a ballot.  That says what row to sample from.  The row's weights are summed
// by all warps of the cluster, a run of tokens each; the runs' sums go to all blocks through distributed shared memory, and the block
// whose run holds the token reads that run once more and finds it.
//
// Weights are summed as integers in units of 2^-60, so a sum has one value whatever the order, and the same one in both
// passes.  HBM bounds it at many sequences: 115 sequences over 128,000 fp32 tokens, a row each and for most of them a second one, take
// 38 us, of which the rows take about 20.  One sequence is bound by latency: tokens, their probabilities, the row, a cluster barrier, and a run again.
#include "cv_attn.cuh"

namespace cvk {
namespace {

using u64 = unsigned long long;
constexpr int kWarps = kSampleThreads / 32, kRuns = kSampleCluster * kWarps;
constexpr int kMaxDrafts = 128;
constexpr float kMaxSum = 4.0f * 0x1p28f;  // weights that add up to 4 and more are refused: their integers would not fit

// x in units of 2^-60, cut off; what is not above 0 (NaN too) is 0, and 2 and more is just below 2.  `whole`: the units of 2^-28.
// (With 64-bit shifts of the mantissa instead of conversions 115 rows of 128,000 took 47 us, 38 with these.)
__device__ __forceinline__ u64 units(float x, float &whole) {
    x = x > 0x1.fffffep0f ? 0x1.fffffep0f : x;
    const float t = x * 0x1p28f;
    const uint32_t hi = __float2uint_rz(t);  // (at most 24 bits are set, so it is a float again)
    whole = __uint2float_rn(hi);
    return (u64)hi << 32 | __float2uint_rz((t - whole) * 0x1p32f);
}
__device__ __forceinline__ u64 units(float x) {
    float whole;
    return units(x, whole);
}

enum { kRow = 0, kDiff = 1, kLeft = 2 };

struct SampleShared {
    double mass[kMaxDrafts];
    float u[kMaxDrafts + 1];
    int tok[kMaxDrafts], tried[kMaxDrafts], path[kMaxDrafts], fell[kMaxDrafts / 32];
    int n_tried, accept, end, mode, child, status;
    u64 sum[kRuns], plain[kRuns];  // of the weights, and of the target's row alone
    float size[kRuns];
    u64 before, target;            // of the run found: weights before it, and what to exceed
    int run, use_plain;
    u64 warp_sum[kWarps];
};

template <typename B>
__device__ __forceinline__ double prob(const void *base, long long at) {
    return (double)widen<B>(__ldg(reinterpret_cast<const B *>(base) + at));
}
// A uniform within [0, 1).
__device__ __forceinline__ double within(float u) { return u > 0.f ? (double)fminf(u, 0x1.fffffep-1f) : 0.; }

// What a warp has of its run: the sum of the weights, that of the target's row, and the latter in units of 2^-28.
struct RunSum {
    u64 sum, plain;
    float size;
};
// The weights of the tokens [lo, hi) of a row, of which 16-byte boundaries are at lo, lo + N, ...; U of a lane's accesses are on
// their way at once, without a branch between them.  DIFF: less those of the row `minus`, whose boundaries are the same with WIDE.
template <typename B, bool DIFF, bool WIDE>
__device__ __forceinline__ RunSum run_sum(const B *row, const B *minus, int lo, int hi, int V) {
    constexpr int N = 16 / (int)sizeof(B), U = DIFF ? 2 : 4;
    const int lane = threadIdx.x & 31;
    RunSum r{0, 0, 0.f};
    auto add = [&](float x, float y) {
        float whole;
        const u64 a = units(x, whole);
        r.plain += a, r.size += whole;
        if (DIFF) {
            const u64 b = units(y);
            r.sum += a > b ? a - b : 0;
        }
    };
    for (int j = lo + lane * N; j < hi; j += U * 32 * N) {
        uint4 a[U], b[U];
        float y[WIDE ? 1 : U][N];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = j + u * 32 * N;
            const bool in = at < hi && at >= 0 && at + N <= V;
            a[u] = b[u] = make_uint4(0, 0, 0, 0);
            if (in) a[u] = __ldg(reinterpret_cast<const uint4 *>(row + at));
            if (DIFF && WIDE && in) b[u] = __ldg(reinterpret_cast<const uint4 *>(minus + at));
            if (DIFF && !WIDE)
#pragma unroll
                for (int i = 0; i < N; ++i) y[WIDE ? 0 : u][i] = in ? widen<B>(__ldg(minus + at + i)) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t x[4] = {a[u].x, a[u].y, a[u].z, a[u].w}, z[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
#pragma unroll
            for (int i = 0; i < N; ++i) add(elem_f<B>(x, i), !DIFF ? 0.f : WIDE ? elem_f<B>(z, i) : y[WIDE ? 0 : u][i]);
        }
    }
    // the accesses that reach over an end of the row, token by token
    const int head = lo < 0 ? min(lo + N, V) : 0, tail = V - (V - lo) % N;
    if (lo < 0 && lane < head) add(widen<B>(__ldg(row + lane)), DIFF ? widen<B>(__ldg(minus + lane)) : 0.f);
    if (tail < V && tail >= max(lo, head) && tail < hi && tail + lane < V)
        add(widen<B>(__ldg(row + tail + lane)), DIFF ? widen<B>(__ldg(minus + tail + lane)) : 0.f);
    return r;
}

template <typename B>
__global__ void __launch_bounds__(kSampleThreads, kSampleBlocks) draft_sample(const __grid_constant__ SampleParams p) {
    constexpr int N = 16 / (int)sizeof(B);
    __shared__ SampleShared sh;
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int s = blockIdx.x / p.cluster, rank = blockIdx.x - s * p.cluster;
    const bool on = !p.idx || __ldg(p.idx + s) >= 0;
    int T = p.T, row0 = 0, status = 0;
    if (p.cu) {
        status = draft_span(p.cu, s, p.T, p.total, T, row0);
        if (!status && T == 0) status = kSeqBadSpan;
    }
    const bool walks = on && !status;
    const long long pbase = p.cu ? (long long)row0 * p.p_tok : (long long)s * p.p_seq;
    const long long qbase = p.cu ? (long long)row0 * p.q_tok : (long long)s * p.q_seq;
    if (walks) {
        const long long at = p.cu ? (long long)row0 : (long long)s * p.T;
        int up = -1, bad = 0;
        if (tid <= kMaxDrafts && tid <= p.T) sh.u[tid] = __ldg(p.u + (long long)s * (p.T + 1) + tid);
        if (tid < kMaxDrafts) {
            bool fell = false;
            if (tid < T) {
                const int tok = __ldg(p.tok + at + tid);
                up = p.parent ? __ldg(p.parent + at + tid) : tid - 1;
                if (up < -1 || up >= tid) bad |= kSeqBadTree, up = -1;
                double mass = 0.;
                if (tid > 0) {
                    if (tok < 0 || tok >= p.vocab) bad |= kSeqBadToken;
                    else if (up >= 0) {
                        mass = prob<B>(p.p, pbase + (long long)up * p.p_tok + tok);
                        if (!p.parent) {  // a chain: every draft's own test
                            const double draw = within(__ldg(p.u + (long long)s * (p.T + 1) + up));
                            fell = !(p.q ? draw * prob<B>(p.q, qbase + (long long)tid * p.q_tok + tok) < mass : draw < mass);
                        }
                    }
                }
                sh.tok[tid] = tok, sh.mass[tid] = mass, sh.path[tid] = tid;
            }
            const unsigned vote = __ballot_sync(0xffffffffu, fell);
            if (lane == 0) sh.fell[warp] = vote;
        }
        if (tid == 0) sh.status = 0;
        __syncthreads();
        if (bad) atomicOr(&sh.status, bad);
        if (!p.parent && tid == 0) {
            int n = T;
#pragma unroll
            for (int w = kMaxDrafts / 32 - 1; w >= 0; --w)
                if (sh.fell[w]) n = 32 * w + __ffs(sh.fell[w]) - 1;
            sh.accept = n, sh.end = n - 1, sh.n_tried = n < T, sh.child = n;
            if (n < T) sh.tried[0] = sh.tok[n];
            sh.mode = n == T ? kRow : p.q ? kDiff : kLeft;
        } else if (p.parent && warp == 0) {
            // lanes hold the parents of every 32nd draft
            int ups[kMaxDrafts / 32];
#pragma unroll
            for (int w = 0; w < kMaxDrafts / 32; ++w) {
                const int t = 32 * w + lane;
                ups[w] = t > 0 && t < T ? __ldg(p.parent + at + t) : -2;
            }
            int end = 0, n = 1, tried = 0;
            for (bool more = true; more;) {
                more = false, tried = 0;
                const double draw = within(sh.u[end]);
                double sum = 0.;
#pragma unroll
                for (int w = 0; w < kMaxDrafts / 32; ++w) {
                    unsigned kids = __ballot_sync(0xffffffffu, ups[w] == end);
                    for (; kids && !more; kids &= kids - 1) {
                        const int t = 32 * w + __ffs(kids) - 1, tok = sh.tok[t];
                        bool twin = false;
                        for (int i = lane; i < tried; i += 32) twin |= sh.tried[i] == tok;
                        if (__any_sync(0xffffffffu, twin)) continue;
                        sum += sh.mass[t];
                        if (draw < sum) {
                            more = true, end = t;
                            if (lane == 0) sh.path[n] = t;
                            ++n;
                        } else {
                            if (lane == 0) sh.tried[tried] = tok;
                            ++tried;
                            __syncwarp();
                        }
                    }
                    if (more) break;
                }
            }
            if (lane == 0) sh.accept = n, sh.end = end, sh.n_tried = tried, sh.child = 0, sh.mode = tried ? kLeft : kRow;
        }
        __syncthreads();
        status = sh.status;
    }
    const bool sums = walks && !status;
    const int V = p.vocab, mode = sums ? sh.mode : kRow;
    const B *const row = reinterpret_cast<const B *>(p.p) + pbase + (sums ? (long long)sh.end * p.p_tok : 0);
    const B *const minus = mode == kDiff ? reinterpret_cast<const B *>(p.q) + qbase + (long long)sh.child * p.q_tok : nullptr;
    // runs of whole accesses of a warp that begin on 16-byte boundaries, the first one up to N - 1 tokens before token 0
    const int shift = (int)(reinterpret_cast<uintptr_t>(row) % 16) / (int)sizeof(B), runs = p.cluster * kWarps;
    const bool wide = (reinterpret_cast<uintptr_t>(minus) % 16) / sizeof(B) == (unsigned)shift;
    const int len = (V + shift + runs * 32 * N - 1) / (runs * 32 * N) * (32 * N);
    const int run = rank * kWarps + warp;
    if (sums) {
        const int lo = run * len - shift, hi = min(V, lo + len);
        const RunSum r = lo >= hi ? RunSum{0, 0, 0.f} : mode != kDiff ? run_sum<B, false, true>(row, nullptr, lo, hi, V)
                         : wide ? run_sum<B, true, true>(row, minus, lo, hi, V) : run_sum<B, true, false>(row, minus, lo, hi, V);
        u64 sum = r.sum, plain = r.plain;
        float size = r.size;
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
        if (lane < p.cluster) {
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
        if (warp == 0) {  // a few runs a lane
            constexpr int EACH = kRuns / 32;
            u64 a[EACH], b[EACH], ta = 0, tb = 0;
            float size = 0.f;
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                const int r = EACH * lane + i;
                a[i] = r < runs ? sh.sum[r] : 0, b[i] = r < runs ? sh.plain[r] : 0;
                ta += a[i], tb += b[i], size += r < runs ? sh.size[r] : 0.f;
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
                for (int i = 0; i < EACH; ++i) a[i] = b[i];
            }
            if (lane == 0) sh.use_plain = use_plain, sh.run = -1;
            if (all == 0 || !(size < kMaxSum)) {
                status = kSeqBadProbs;
            } else {
                const u64 target = __umul64hi((u64)(within(sh.u[p.T]) * 0x1p64), all);  // the token's sum exceeds it
                u64 up = ta;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const u64 x = __shfl_up_sync(0xffffffffu, up, o);
                    if (lane >= o) up += x;
                }
                u64 before = up - ta;
                __syncwarp();
#pragma unroll
                for (int i = 0; i < EACH; ++i) {
                    if (before <= target && target < before + a[i]) sh.run = EACH * lane + i, sh.before = before, sh.target = target;
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
    if (sh.run / kWarps != rank) return;
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
        const u64 x = __shfl_up_sync(0xffffffffu, up, o);
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
