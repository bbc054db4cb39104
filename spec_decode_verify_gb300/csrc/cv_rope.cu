// RMS norms of query and key heads and the rotation by position, with K and V written into the cache's pages.
//
// A head's row goes through registers once: read, its mean square over the lanes that share it, scale, rotate, round,
// write.  A lane owns two pieces of 8 channels chosen so that both partners of a rotated pair are its own: piece i
// of each half of the rotated channels, or neighbours where pairs are neighbours.  A group of lanes takes one token and
// every so many of its heads, so that the token's angles and the weights are loaded once.  HBM bounds it: nothing is read twice.
#include "cv_attn.cuh"

namespace cvk {
namespace {

// Heads that a thread of norm_rope has on their way.
template <typename B>
__host__ __device__ constexpr int rope_ring() { return sizeof(B) == 2 ? 8 : 4; }

struct TokenAt {
    long long q, qo, k, ko, v, kc, vc;  // offsets of the token's rows; kc, vc: in the cache
    int pos, on;                        // on: 0 = left out
};

// 8 channels as they lie in memory.
template <typename B>
struct Raw8 {
    uint4 w[sizeof(B) / 2];
};
template <typename B>
__device__ __forceinline__ Raw8<B> load8(const B *p) {
    Raw8<B> r;
#pragma unroll
    for (int h = 0; h < (int)sizeof(B) / 2; ++h) r.w[h] = ld16(p + 8 / (sizeof(B) / 2) * h);
    return r;
}
template <typename B>
__device__ __forceinline__ void store8(B *p, const Raw8<B> &r) {
#pragma unroll
    for (int h = 0; h < (int)sizeof(B) / 2; ++h) st16(p + 8 / (sizeof(B) / 2) * h, r.w[h]);
}
// What is known of sequence s without its tokens.
struct SeqAt {
    int slot, L, n, row0, status;  // n, row0: its tokens and the first one's row with cu
};
__device__ __forceinline__ SeqAt seq_at(const RopeParams &p, int s) {
    SeqAt q;
    q.slot = p.idx ? __ldg(p.idx + s) : s;
    q.L = p.len ? __ldg(p.len + s) : 0;
    q.n = p.T, q.row0 = 0, q.status = 0;
    if (p.cu) q.status = draft_span(p.cu, s, p.T, p.total, q.n, q.row0);
    if (q.status) q.n = 0;
    if (p.paged) {
        if (q.slot >= p.c.n_slots) q.status |= kSeqBadSlot;
        if (q.L < 0 || (long long)q.L + q.n > (long long)p.c.max_pages * p.c.page) q.status |= kSeqBadLength;
    } else if (q.L < 0) {
        q.status |= kSeqBadLength;
    }
    if (q.slot < 0) q.status = 0;
    return q;
}
// The flags of sequences that no token may tell of (of packed rows, or none), each raised by one block; and whether counts fall
// anywhere: then a row may belong to several sequences.  Every thread of the block calls this.
__device__ __forceinline__ bool check_sequences(const RopeParams &p) {
    bool falls = false;
    for (int s = threadIdx.x; s < p.n_seq; s += kRopeThreads) {
        if (p.cu) falls |= __ldg(p.cu + s + 1) < __ldg(p.cu + s);
        if (p.err && s % (int)gridDim.x == (int)blockIdx.x) {
            const SeqAt q = seq_at(p, s);
            if (q.status) atomicOr(p.err + s, q.status);
        }
    }
    return __syncthreads_or(falls);
}
// Where sequence s reads and writes token `tok` (of all).
__device__ __forceinline__ TokenAt token_of(const RopeParams &p, int s, long long tok) {
    TokenAt a;
    a.on = 0;
    const SeqAt q = seq_at(p, s);
    const int t = p.cu ? (int)(tok - q.row0) : (int)(tok - (long long)s * p.T);
    if (q.slot < 0) return a;
    int status = q.status;
    if (!status) {
        if (t < 0 || t >= q.n) return a;
        a.pos = p.pos ? __ldg(p.pos + tok) : (int)((unsigned)q.L + (unsigned)t);
        if (p.rot > 0 && (a.pos < 0 || a.pos >= p.n_pos)) status |= kSeqBadPosition;
        if (p.paged) {
            const int at = q.L + t, pg = __ldg(p.c.table + (long long)q.slot * p.c.table_row + at / p.c.page);
            if (pg < 0 || pg >= p.c.n_pages) status |= kSeqBadPage;
            else {
                if (p.c.refs && __ldg(p.c.refs + pg) > 1) status |= kSeqSharedPage;
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
// The same of the sequence that the token belongs to, where counts do not fall.
__device__ __forceinline__ TokenAt token_at(const RopeParams &p, long long tok) {
    if (!p.cu) return token_of(p, (int)(tok / p.T), tok);
    TokenAt none;
    none.on = 0;
    if (tok < __ldg(p.cu) || tok >= __ldg(p.cu + p.n_seq)) return none;  // (a row of no sequence)
    int lo = 0, hi = p.n_seq - 1;
    while (lo < hi) {  // the last sequence that begins at or before it
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(p.cu + mid) <= tok) lo = mid;
        else hi = mid - 1;
    }
    return token_of(p, lo, tok);
}

// A head's row: what it is read from and written to (a key may go to two places, or with outs = false to the cache alone).
template <typename B>
struct HeadRow {
    const B *from, *w;
    B *to, *to2;
    bool norm, turn;
};
template <typename B>
__device__ __forceinline__ HeadRow<B> head_row(const RopeParams &p, const TokenAt &a, int h, bool outs) {
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
        B *const out = p.k_out && outs ? reinterpret_cast<B *>(p.k_out) + a.ko + (long long)h * p.ko_head : nullptr;
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

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
// 8 channels as pairs of fp32, and back with one rounding.
template <typename B>
__device__ __forceinline__ void pairs8(f2 *f, const Raw8<B> &r) {
    const uint32_t *const w = reinterpret_cast<const uint32_t *>(r.w);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2_pack(elem_f<B>(w, 2 * i), elem_f<B>(w, 2 * i + 1));
}
template <typename B>
__device__ __forceinline__ Raw8<B> round8(const f2 *f) {
    Raw8<B> r;
    uint32_t *const w = reinterpret_cast<uint32_t *>(r.w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        f2_unpack(f[i], lo, hi);
        if (sizeof(B) == 2) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(hi), "f"(lo));
        else w[2 * i] = __float_as_uint(lo), w[2 * i + 1] = __float_as_uint(hi);
    }
    return r;
}

// One head by a warp, its channels read twice.
template <typename B>
__device__ __forceinline__ void one_head(const RopeParams &p, const TokenAt &at, const HeadRow<B> &r) {
    const int lane = threadIdx.x & 31, half = p.rot / 2;
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
            const float *const cs = p.cs + (long long)at.pos * p.cs_row;
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

// Packed rows of counts that fall somewhere, of which several sequences may own one: a warp a row, for each of its sequences in turn.  Every one's
// cache gets it, q_out and k_out that of the last: they may be q and k, so nothing is read after they are written.
template <typename B>
__device__ __noinline__ void falling_rows(const RopeParams &p) {
    const long long warps = (long long)gridDim.x * (kRopeThreads / 32);
    const int heads = p.n_heads + p.n_kv + (p.v ? p.n_kv : 0);
    for (long long tok = (long long)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5); tok < p.tokens; tok += warps) {
        auto owners = [&](int base) {  // of 32 sequences
            const int s = base + (threadIdx.x & 31);
            return __ballot_sync(0xffffffffu, s < p.n_seq && __ldg(p.cu + s) <= tok && tok < __ldg(p.cu + s + 1));
        };
        int last = -1;
        for (int base = (p.n_seq - 1) & ~31; base >= 0 && last < 0; base -= 32)
            for (unsigned of = owners(base); of && last < 0;) {
                const int s = 31 - __clz(of);
                if (token_of(p, base + s, tok).on) last = base + s;
                of ^= 1u << s;
            }
        for (int base = 0; base <= last; base += 32)
            for (unsigned of = owners(base); of; of &= of - 1) {
                const int s = base + __ffs(of) - 1;
                if (s > last || (s < last && !p.paged)) continue;
                const TokenAt at = token_of(p, s, tok);
                if (!at.on) continue;
                for (int h = s < last ? p.n_heads : 0; h < heads; ++h) one_head<B>(p, at, head_row<B>(p, at, h, s == last));
            }
    }
}
// What a kernel does before its tokens: the sequences that no token may tell of.  Whether the rows are done already.
template <typename B>
__device__ __forceinline__ bool packed_falls(const RopeParams &p) {
    if (!p.cu && p.tokens > 0) return false;  // (every sequence has tokens)
    if (!check_sequences(p)) return false;
    falling_rows<B>(p);
    return true;
}

// Rows of 16-byte pieces: p.lanes lanes a group, which takes a token and every p.groups-th of its heads.  A thread's next heads
// are on their way to places of its own in shared memory (30,822 tokens of 48 heads: 162 us with them in registers, which
// left 16 warps an SM; 143 so, with products of two channels an instruction).
template <typename B>
__global__ void __launch_bounds__(kRopeThreads, 2) norm_rope(const __grid_constant__ RopeParams p) {
    constexpr int R = rope_ring<B>(), P = 2 * (int)sizeof(B) / 2;  // heads on their way; 16-byte pieces of each
    extern __shared__ __align__(16) uint4 ring[];
    grid_dep_wait();
    grid_dep_launch();
    if (packed_falls<B>(p)) return;
    const int tid = threadIdx.x, i = tid % p.lanes, half = p.rot / 2;
    const long long group = (long long)blockIdx.x * (kRopeThreads / p.lanes) + tid / p.lanes;
    const long long tok = group / p.groups;
    const int part = (int)(group - tok * p.groups);
    if (tok >= p.tokens) return;
    const TokenAt at = token_at(p, tok);
    if (!at.on) return;
    const unsigned mask = ((1u << p.lanes) - 1) << (tid & 31 & ~(p.lanes - 1));  // this group (16 lanes at most)
    // the channels of this lane's two pieces of 8; a lane past the last ones reads the first ones, adds nothing and writes nothing
    const bool has = 16 * i < p.d, turned = 16 * i < p.rot;
    const int c0 = !has ? 0 : turned && !p.pairs ? 8 * i : 16 * i, c1 = !has ? 0 : turned && !p.pairs ? half + 8 * i : 16 * i + 8;
    // This group's heads are part, part + groups, ... of the queries, keys and values in a row: n_q, n_k and n_v of them.
    auto upto = [&](int n) { return n > part ? (n - part + p.groups - 1) / p.groups : 0; };
    const int n_q = upto(p.n_heads), n_k = upto(p.n_heads + p.n_kv) - n_q, n_v = p.v ? upto(p.n_heads + 2 * p.n_kv) - n_q - n_k : 0;
    const int k0 = part + n_q * p.groups - p.n_heads, v0 = part + (n_q + n_k) * p.groups - p.n_heads - p.n_kv;

    const B *next = reinterpret_cast<const B *>(p.q) + at.q + (long long)part * p.q_head;
    long long step = p.groups * p.q_head;
    int left = n_q, stage = 0, put = 0, get = 0;  // of the heads to fetch: left in this tensor, which tensor; places in the ring
    auto fetch = [&] {
        while (left == 0 && stage < 2) {
            ++stage;
            left = stage == 1 ? n_k : n_v;
            next = stage == 1 ? reinterpret_cast<const B *>(p.k) + at.k + (long long)k0 * p.k_head
                              : reinterpret_cast<const B *>(p.v) + at.v + (long long)v0 * p.v_head;
            step = p.groups * (stage == 1 ? p.k_head : p.v_head);
        }
        if (left > 0) {
            uint4 *const to = ring + put * (P * kRopeThreads) + tid;
#pragma unroll
            for (int x = 0; x < P / 2; ++x) {
                cp_async16(to + x * kRopeThreads, next + c0 + x * (16 / (int)sizeof(B)));
                cp_async16(to + (P / 2 + x) * kRopeThreads, next + c1 + x * (16 / (int)sizeof(B)));
            }
            next += step, --left;
        }
        cp_async_commit();
        put = put + 1 == R ? 0 : put + 1;
    };
    auto take = [&](Raw8<B> &a, Raw8<B> &b) {
        cp_async_wait<R - 1>();
        const uint4 *const from = ring + get * (P * kRopeThreads) + tid;
#pragma unroll
        for (int x = 0; x < P / 2; ++x) a.w[x] = from[x * kRopeThreads], b.w[x] = from[(P / 2 + x) * kRopeThreads];
        get = get + 1 == R ? 0 : get + 1;
        fetch();
    };
#pragma unroll
    for (int n = 0; n < R; ++n) fetch();
    f2 co[4], si[4], ni[4];  // cosines, sines and the sines' negatives
    if (turned) {
        const uint32_t *const cs = reinterpret_cast<const uint32_t *>(p.cs + (long long)at.pos * p.cs_row + 8 * i);
        pairs8<uint32_t>(co, load8<uint32_t>(cs));
        pairs8<uint32_t>(si, load8<uint32_t>(cs + half));
        const f2 minus = f2_pack(-1.f, -1.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) ni[e] = f2_mul(si[e], minus);
    }
    auto heads = [&](int n, B *to, long long to_step, B *to2, long long to2_step, const B *weight) {
        f2 w[8];
        const bool scaled = p.norm && weight;
        if (scaled && n > 0) pairs8<B>(w, load8<B>(weight + c0)), pairs8<B>(w + 4, load8<B>(weight + c1));
        for (; n > 0; --n) {
            Raw8<B> a, b;
            take(a, b);
            if (p.norm || turned) {
                f2 x[8];
                pairs8<B>(x, a), pairs8<B>(x + 4, b);
                if (p.norm) {
                    f2 s2[2] = {f2_mul(x[0], x[0]), f2_mul(x[4], x[4])};
#pragma unroll
                    for (int e = 1; e < 4; ++e) s2[0] = f2_fma(x[e], x[e], s2[0]), s2[1] = f2_fma(x[4 + e], x[4 + e], s2[1]);
                    float lo, hi;
                    f2_unpack(f2_add(s2[0], s2[1]), lo, hi);
                    float sq = has ? lo + hi : 0.f;
                    for (int o = p.lanes / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(mask, sq, o);
                    const float inv = rsqrtf(sq / (float)p.d + p.eps);
                    const f2 inv2 = f2_pack(inv, inv);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = f2_mul(x[e], inv2);
                    if (scaled)
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = f2_mul(x[e], w[e]);
                }
                if (turned && p.pairs) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float c[2], s[2], f, g;
                        f2_unpack(co[e / 2], c[0], c[1]), f2_unpack(si[e / 2], s[0], s[1]), f2_unpack(x[e], f, g);
                        x[e] = f2_fma(f2_pack(g, f), f2_pack(-s[e & 1], s[e & 1]), f2_mul(x[e], f2_pack(c[e & 1], c[e & 1])));
                    }
                } else if (turned) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f2 y = x[e], z = x[4 + e];
                        x[e] = f2_fma(z, ni[e], f2_mul(y, co[e])), x[4 + e] = f2_fma(y, si[e], f2_mul(z, co[e]));
                    }
                }
                a = round8<B>(x), b = round8<B>(x + 4);
            }
            if (has) store8<B>(to + c0, a), store8<B>(to + c1, b);
            to += to_step;
            if (to2) {
                if (has) store8<B>(to2 + c0, a), store8<B>(to2 + c1, b);
                to2 += to2_step;
            }
        }
    };
    heads(n_q, reinterpret_cast<B *>(p.q_out) + at.qo + (long long)part * p.qo_head, p.groups * p.qo_head, nullptr, 0,
          reinterpret_cast<const B *>(p.wq));
    if (n_k > 0) {
        B *const in = p.paged ? reinterpret_cast<B *>(p.c.k) + at.kc + (long long)k0 * p.c.k_head : nullptr;
        B *const out = p.k_out ? reinterpret_cast<B *>(p.k_out) + at.ko + (long long)k0 * p.ko_head : nullptr;
        heads(n_k, out ? out : in, p.groups * (out ? p.ko_head : p.c.k_head), out ? in : nullptr, p.groups * p.c.k_head,
              reinterpret_cast<const B *>(p.wk));
    }
    if (n_v > 0) {
        B *to = reinterpret_cast<B *>(p.c.v) + at.vc + (long long)v0 * p.c.v_head;
        for (int n = n_v; n > 0; --n, to += p.groups * p.c.v_head) {
            Raw8<B> a, b;
            take(a, b);
            if (has) store8<B>(to + c0, a), store8<B>(to + c1, b);
        }
    }
    cp_async_wait<0>();
}

// Any rows: a warp a head.
template <typename B>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_any(const __grid_constant__ RopeParams p) {
    __shared__ TokenAt at[kRopeTokens];
    grid_dep_wait();
    grid_dep_launch();
    if (packed_falls<B>(p)) return;
    const int tid = threadIdx.x;
    const long long tok0 = (long long)blockIdx.x * p.block_tokens;
    const int toks = (int)(p.tokens - tok0 < p.block_tokens ? p.tokens - tok0 : p.block_tokens);
    if (tid < toks) at[tid] = token_at(p, tok0 + tid);
    __syncthreads();
    const int heads = p.n_heads + p.n_kv + (p.v ? p.n_kv : 0);
    for (int item = tid >> 5; item < toks * heads; item += kRopeThreads / 32) {
        const int tk = item / heads;
        if (at[tk].on) one_head<B>(p, at[tk], head_row<B>(p, at[tk], item - tk * heads, true));
    }
}

}  // namespace

int rope_smem(bool bf16) { return bf16 ? rope_ring<uint16_t>() * 2 * kRopeThreads * 16 : rope_ring<uint32_t>() * 4 * kRopeThreads * 16; }
RopeKernel rope_kernel(bool bf16, bool vec) {
    if (bf16) return vec ? norm_rope<uint16_t> : norm_rope_any<uint16_t>;
    return vec ? norm_rope<uint32_t> : norm_rope_any<uint32_t>;
}

}  // namespace cvk
