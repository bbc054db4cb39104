// RMS norms of query and key heads and the rotation by position, with K and V written into the cache's pages.
//
// A head's row goes through registers once: read, its mean square over the lanes that share it, scale, rotate, round,
// write.  A lane owns two pieces of 8 channels chosen so that both partners of a rotated pair are its own: piece i
// of each half of the rotated channels, or neighbours where pairs are neighbours.  HBM bounds it; nothing is read twice but the
// angles, which all heads of a token share in L1.
#include "cv_attn.cuh"

namespace cvk {
namespace {

struct TokenAt {
    long long q, qo, k, ko, v, kc, vc;  // offsets of the token's rows; kc, vc: in the cache
    int pos, on;                        // on: 0 = left out
};

template <typename B>
__device__ __forceinline__ void load8(float *f, const B *p) {
    if (sizeof(B) == 2) {
        const uint4 w = ld16(p);
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = elem_f<B>(x, i);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 w = *reinterpret_cast<const float4 *>(p + 4 * h);
            f[4 * h] = w.x, f[4 * h + 1] = w.y, f[4 * h + 2] = w.z, f[4 * h + 3] = w.w;
        }
    }
}
template <typename B>
__device__ __forceinline__ void store8(B *p, const float *f) {
    if (sizeof(B) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_halves(narrow<uint16_t>(f[2 * i]), narrow<uint16_t>(f[2 * i + 1]));
        st16(p, make_uint4(w[0], w[1], w[2], w[3]));
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            *reinterpret_cast<float4 *>(p + 4 * h) = make_float4(f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]);
    }
}

// 8 channels with their own bits.
template <typename B>
__device__ __forceinline__ void copy8(B *to, const B *from) {
#pragma unroll
    for (int h = 0; h < (int)sizeof(B) / 2; ++h) st16(to + 4 * h, ld16(from + 4 * h));
}

// Where token `tok` (of all) reads and writes.
__device__ __forceinline__ TokenAt token_at(const RopeParams &p, long long tok) {
    TokenAt a;
    a.on = 0;
    int s, t, n = p.T, row0 = 0, status = 0;
    if (p.cu) {
        if (tok < __ldg(p.cu) || tok >= __ldg(p.cu + p.n_seq)) return a;  // (a row of no sequence)
        int lo = 0, hi = p.n_seq - 1;
        while (lo < hi) {  // the last sequence that begins at or before it
            const int mid = (lo + hi + 1) >> 1;
            if (__ldg(p.cu + mid) <= tok) lo = mid;
            else hi = mid - 1;
        }
        s = lo;
        status = draft_span(p.cu, s, p.T, p.total, n, row0);
        t = (int)(tok - row0);
        if (status) n = 0;
        else if (t < 0 || t >= n) return a;
    } else {
        s = (int)(tok / p.T), t = (int)(tok - (long long)s * p.T);
    }
    const int slot = p.idx ? __ldg(p.idx + s) : s;
    if (slot < 0) return a;
    const int L = p.len ? __ldg(p.len + s) : 0;
    if (p.paged) {
        if (slot >= p.c.n_slots) status |= kSeqBadSlot;
        if (L < 0 || (long long)L + n > (long long)p.c.max_pages * p.c.page) status |= kSeqBadLength;
    } else if (L < 0) {
        status |= kSeqBadLength;
    }
    if (!status) {
        a.pos = p.pos ? __ldg(p.pos + tok) : (int)((unsigned)L + (unsigned)t);
        if (p.rot > 0 && (a.pos < 0 || a.pos >= p.n_pos)) status |= kSeqBadPosition;
        if (p.paged) {
            const int at = L + t, pg = __ldg(p.c.table + (long long)slot * p.c.table_row + at / p.c.page);
            if (pg < 0 || pg >= p.c.n_pages) status |= kSeqBadPage;
            else {
                a.kc = (long long)pg * p.c.k_page + (long long)(at % p.c.page) * p.c.k_row;
                a.vc = (long long)pg * p.c.v_page + (long long)(at % p.c.page) * p.c.v_row;
            }
        }
    }
    if (status) {
        if (p.err) atomicOr(p.err + s, status);
        return a;
    }
    const long long row = p.cu ? tok : t, seq = p.cu ? 0 : s;
    a.q = seq * p.q_seq + row * p.q_tok, a.qo = seq * p.qo_seq + row * p.qo_tok;
    a.k = seq * p.k_seq + row * p.k_tok, a.ko = seq * p.ko_seq + row * p.ko_tok;
    a.v = seq * p.v_seq + row * p.v_tok;
    a.on = 1;
    return a;
}

// A head's row: what it is read from and written to (a key may go to two places).
template <typename B>
struct HeadRow {
    const B *from, *w;
    B *to, *to2;
    bool norm, turn;
};
template <typename B>
__device__ __forceinline__ HeadRow<B> head_row(const RopeParams &p, const TokenAt &a, int h) {
    HeadRow<B> r;
    r.to2 = nullptr;
    if (h < p.n_heads) {
        r.from = reinterpret_cast<const B *>(p.q) + a.q + (long long)h * p.q_head;
        r.to = reinterpret_cast<B *>(p.q_out) + a.qo + (long long)h * p.qo_head;
        r.w = reinterpret_cast<const B *>(p.wq), r.norm = p.norm != 0, r.turn = p.rot > 0;
        return r;
    }
    h -= p.n_heads;
    if (h < p.n_kv) {
        r.from = reinterpret_cast<const B *>(p.k) + a.k + (long long)h * p.k_head;
        B *const out = p.k_out ? reinterpret_cast<B *>(p.k_out) + a.ko + (long long)h * p.ko_head : nullptr;
        B *const in = p.paged ? reinterpret_cast<B *>(p.c.k) + a.kc + (long long)h * p.c.k_head : nullptr;
        r.to = out ? out : in, r.to2 = out ? in : nullptr;
        r.w = reinterpret_cast<const B *>(p.wk), r.norm = p.norm != 0, r.turn = p.rot > 0;
        return r;
    }
    h -= p.n_kv;
    r.from = reinterpret_cast<const B *>(p.v) + a.v + (long long)h * p.v_head;
    r.to = reinterpret_cast<B *>(p.c.v) + a.vc + (long long)h * p.c.v_head;
    r.w = nullptr, r.norm = r.turn = false;
    return r;
}

// Rows of 16-byte pieces: p.lanes lanes a head, each two pieces of 8 channels.
template <typename B>
__global__ void __launch_bounds__(kRopeThreads) norm_rope(const __grid_constant__ RopeParams p) {
    __shared__ TokenAt at[kRopeTokens];
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x;
    const long long tok0 = (long long)blockIdx.x * p.block_tokens;
    const int toks = (int)(p.tokens - tok0 < p.block_tokens ? p.tokens - tok0 : p.block_tokens);
    if (tid < toks) at[tid] = token_at(p, tok0 + tid);
    __syncthreads();
    const int heads = p.n_heads + p.n_kv + (p.v ? p.n_kv : 0);
    const int i = tid % p.lanes, per = kRopeThreads / p.lanes, half = p.rot / 2;
    // the channels of this lane's two pieces
    const bool has = 16 * i < p.d, turned = 16 * i < p.rot;
    const int c0 = turned && !p.pairs ? 8 * i : 16 * i, c1 = turned && !p.pairs ? half + 8 * i : 16 * i + 8;
    const int items = toks * heads, rounds = (items + per - 1) / per;
    for (int n = 0; n < rounds; ++n) {
        const int item = n * per + tid / p.lanes;
        const int tk = item / heads;
        const bool on = item < items && has && at[tk < toks ? tk : 0].on;
        float x[16];
        HeadRow<B> r;
        float sq = 0.f;
        if (on) {
            r = head_row<B>(p, at[tk], item - tk * heads);
            load8<B>(x, r.from + c0);
            load8<B>(x + 8, r.from + c1);
#pragma unroll
            for (int e = 0; e < 16; ++e) sq = fmaf(x[e], x[e], sq);
        }
        for (int o = p.lanes / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
        if (!on) continue;
        if (r.norm) {
            const float inv = 1.0f / sqrtf(sq / (float)p.d + p.eps);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] *= inv;
            if (r.w) {
                float w[16];
                load8<B>(w, r.w + c0);
                load8<B>(w + 8, r.w + c1);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] *= w[e];
            }
        }
        if (r.turn && turned) {
            const float *const cs = p.cs + (long long)at[tk].pos * p.cs_row + 8 * i;
            float co[8], si[8];
            load8<uint32_t>(co, reinterpret_cast<const uint32_t *>(cs));
            load8<uint32_t>(si, reinterpret_cast<const uint32_t *>(cs + half));
            if (!p.pairs) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a = x[e], b = x[e + 8];
                    x[e] = a * co[e] - b * si[e], x[e + 8] = b * co[e] + a * si[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a = x[2 * e], b = x[2 * e + 1];
                    x[2 * e] = a * co[e] - b * si[e], x[2 * e + 1] = b * co[e] + a * si[e];
                }
            }
        }
        if (r.norm || r.turn) {
            store8<B>(r.to + c0, x);
            store8<B>(r.to + c1, x + 8);
            if (r.to2) {
                store8<B>(r.to2 + c0, x);
                store8<B>(r.to2 + c1, x + 8);
            }
        } else {  // raw bits
            copy8<B>(r.to + c0, r.from + c0);
            copy8<B>(r.to + c1, r.from + c1);
            if (r.to2) {
                copy8<B>(r.to2 + c0, r.from + c0);
                copy8<B>(r.to2 + c1, r.from + c1);
            }
        }
    }
}

// Any rows: a warp a head, its channels read twice.
template <typename B>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_any(const __grid_constant__ RopeParams p) {
    __shared__ TokenAt at[kRopeTokens];
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, lane = tid & 31;
    const long long tok0 = (long long)blockIdx.x * p.block_tokens;
    const int toks = (int)(p.tokens - tok0 < p.block_tokens ? p.tokens - tok0 : p.block_tokens);
    if (tid < toks) at[tid] = token_at(p, tok0 + tid);
    __syncthreads();
    const int heads = p.n_heads + p.n_kv + (p.v ? p.n_kv : 0), half = p.rot / 2;
    for (int item = tid >> 5; item < toks * heads; item += kRopeThreads / 32) {
        const int tk = item / heads;
        if (!at[tk].on) continue;
        const HeadRow<B> r = head_row<B>(p, at[tk], item - tk * heads);
        float inv = 1.0f;
        if (r.norm) {
            float sq = 0.f;
            for (int c = lane; c < p.d; c += 32) {
                const float x = widen<B>(r.from[c]);
                sq = fmaf(x, x, sq);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
            inv = 1.0f / sqrtf(sq / (float)p.d + p.eps);
        }
        __syncwarp();
        auto value = [&](int c) {
            float x = widen<B>(r.from[c]);
            if (r.norm) x = r.w ? x * inv * widen<B>(__ldg(r.w + c)) : x * inv;
            return x;
        };
        const int turned = r.turn ? half : 0;
        for (int n = lane; n < turned + (p.d - 2 * turned); n += 32) {  // a pair, or a channel that stays
            if (n < turned) {
                const int a = p.pairs ? 2 * n : n, b = p.pairs ? 2 * n + 1 : n + half;
                const float *const cs = p.cs + (long long)at[tk].pos * p.cs_row;
                const float co = __ldg(cs + n), si = __ldg(cs + half + n), x = value(a), y = value(b);
                const B lo = narrow<B>(x * co - y * si), hi = narrow<B>(y * co + x * si);
                r.to[a] = lo, r.to[b] = hi;
                if (r.to2) r.to2[a] = lo, r.to2[b] = hi;
            } else {
                const int c = n + turned;
                const B x = r.norm ? narrow<B>(value(c)) : r.from[c];
                r.to[c] = x;
                if (r.to2) r.to2[c] = x;
            }
        }
    }
}

}  // namespace

RopeKernel rope_kernel(bool bf16, bool vec) {
    if (bf16) return vec ? norm_rope<uint16_t> : norm_rope_any<uint16_t>;
    return vec ? norm_rope<uint32_t> : norm_rope_any<uint32_t>;
}

}  // namespace cvk
