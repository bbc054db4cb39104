// The pages of a cache: new pages for growing and forked sequences, shared pages and copies of them, released pages, and the
// accepted path of a tree of drafts moved to its place.
//
// A page is free while its reference count is 0, and the free pages with the lowest numbers are given out in the order of the
// call's sequences; so the only state is the table, the counts and the slots' numbers of pages, and results do not depend
// on the order in which threads come.  One block finds the free pages (8 counts a thread at a time, a scan over the
// block), since their order is one of all pages: 70,000 counts are 280 KB, and it stops once it has enough.  Sharing
// and copying take a cluster a sequence, releasing a block a sequence, compacting one for each part of the layers.
#include "cv_attn.cuh"

namespace cvk {
namespace {

// Pages that hold n tokens.
__device__ __forceinline__ int pages_for(int n, int page) { return n <= 0 ? 0 : (n - 1) / page + 1; }

// Sum over a block of 1024 threads, and the sum of the threads before this one.
__device__ __forceinline__ long long block_scan(long long v, long long &before, long long *scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long up = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += x;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = up;
    __syncthreads();
    const long long mine = scratch[lane];
    long long sums = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, sums, o);
        if (lane >= o) sums += x;
    }
    before = __shfl_sync(0xffffffffu, sums - mine, warp) + up - v;
    return __shfl_sync(0xffffffffu, sums, 31);
}

constexpr int kCheckPages = 128;  // pages of a fork's source that a warp looks at in one go
constexpr int kScanEach = 8, kScanPages = kTakeThreads * kScanEach;  // counts a thread, and the block, looks at in one go
static_assert(kScanPages >= 2 * kMaxPageSeqs, "a fork's notes fit into the list");

// OP: kPages*.  (A kernel for each: the code that a call does not need, on its way from memory, is a good part of the time of a block
// that runs alone.  64 forks and then 64 slots that grow: 22.6 us with one kernel for all, 20.7 with three.)
template <int OP>
__global__ void __launch_bounds__(kTakeThreads) pages_take(const __grid_constant__ PagesParams p) {
    extern __shared__ __align__(8) long long smem[];
    long long *const scratch = smem, *const pre = smem + 32;  // pre: pages of the sequences before
    int *const slots = reinterpret_cast<int *>(pre + p.n_seq), *const flagged = slots + p.n_seq, *const first = flagged + p.n_seq,
        *const src = first + p.n_seq, *const list = src + p.n_seq;  // list: free pages in order
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x;
    constexpr bool fork = OP == kPagesFork, own = OP == kPagesOwn;
    const CacheView &c = p.c;
    // Of a fork: whether a page of the source is not there, and its tokens (the list's places are not used before the scan).
    int *const gone = list, *const tokens = list + kMaxPageSeqs;
    int most = 0;  // pages of a fork, in kCheckPages
    for (int i = tid; i < p.n_seq; i += kTakeThreads) {
        int slot = p.idx ? __ldg(p.idx + i) : i;
        const int from = fork ? __ldg(p.src + i) : 0;
        if (fork) {
            int n = __ldg(p.n_tok + i);
            if (slot < 0 || from < 0 || from >= c.n_slots || n > (long long)c.max_pages * c.page) n = 0;
            gone[i] = 0, tokens[i] = n;
            most = max(most, (pages_for(n, c.page) + kCheckPages - 1) / kCheckPages);
        }
        if (from < 0) slot = -1;
        slots[i] = slot, src[i] = slot < 0 ? -1 : from;
    }
    if (fork) {
        most = __reduce_max_sync(0xffffffffu, most);
        if ((tid & 31) == 0) scratch[tid >> 5] = most;
    }
    __syncthreads();
    if (fork) most = __reduce_max_sync(0xffffffffu, (int)scratch[tid & 31]);
    // Pages each sequence needs; -1 - bits where it is flagged.
    auto needs = [&](int i) {
        const int slot = slots[i];
        first[i] = 0;
        if (slot < 0) return 0;
        if (slot >= c.n_slots) return -1 - kSeqBadSlot;
        const int n = __ldg(p.n_tok + i), held = c.held[slot];
        int st = 0, need = 0;
        if (p.idx)
#pragma unroll 8
            for (int j = 0; j < i; ++j) st |= slots[j] == slot;
        if (fork) {
#pragma unroll 8
            for (int j = 0; j < p.n_seq; ++j) st |= src[j] == slot;
            if (src[i] >= c.n_slots || held != 0) st = 1;
            if (!st) {
                const int have = c.held[src[i]];
                if (n < 0 || have < 0 || have > c.max_pages || n > (long long)have * c.page) return -1 - kSeqBadLength;
            }
            need = n % c.page != 0;
            first[i] = n / c.page;
        } else {
            if (!st && (n < 0 || n > (long long)c.max_pages * c.page || held < 0 || held > c.max_pages)) return -1 - kSeqBadLength;
            need = max(0, pages_for(n, c.page) - held);
            first[i] = held;
            if (own && !st) {  // and one for each shared page that is to be written
                const int L = __ldg(p.len + i);
                if (L < 0 || L > (long long)held * c.page) return -1 - kSeqBadLength;
                const int *const row = c.table + (long long)slot * c.table_row;
                for (int x = L / c.page; x < (L < n ? min(held, pages_for(n, c.page)) : 0); ++x) {
                    const int g = row[x];
                    if (g < 0 || g >= c.n_pages) return -1 - kSeqBadPage;
                    if (c.refs[g] > 1) ++need, --first[i];
                }
            }
        }
        return st ? -1 - kSeqBadSlot : need;
    };
    // A fork's sources' pages, in runs of kCheckPages, by the warps that have no sequence to look at, if there are such: a fork that cannot be
    // made takes no page from the others.
    const int warp = tid >> 5, busy = p.n_seq <= kTakeThreads / 2 ? (p.n_seq + 31) / 32 : 0;
    const long long checks = (long long)p.n_seq * most;
    for (long long q = warp < busy ? checks : warp - busy; q < checks; q += kTakeThreads / 32 - busy) {
        const int of = (int)attn_div(q, p.n_seq), i = (int)(q - (long long)of * p.n_seq);
        const long long left = pages_for(tokens[i], c.page) - (long long)of * kCheckPages;
        const int *const from = c.table + (long long)src[i] * c.table_row + (long long)of * kCheckPages;
        bool bad = false;
#pragma unroll 4
        for (int x = tid & 31; x < kCheckPages; x += 32) {
            const int g = x < left ? from[x] : 0;
            bad |= g < 0 || g >= c.n_pages;
        }
        if (bad) gone[i] = 1;
    }
    long long total = 0;
    for (int base = 0; base < p.n_seq; base += kTakeThreads) {
        const int i = base + tid;
        int need = i < p.n_seq ? needs(i) : 0;
        if (fork && base == 0) __syncthreads();  // (the checks)
        if (fork && i < p.n_seq && need >= 0 && gone[i]) need = -1 - kSeqBadPage;
        long long before;
        const long long sum = block_scan(max(need, 0), before, scratch);
        if (i < p.n_seq) {
            pre[i] = total + before;
            flagged[i] = need < 0;
            if (p.err) p.err[i] = need < 0 ? -1 - need : 0;
        }
        total += sum;
    }
    __syncthreads();
    auto ends = [&](int i) { return i + 1 < p.n_seq ? pre[i + 1] : total; };
    // The free pages among counts [base, base + kScanPages) into the list; how many.
    const bool wide = reinterpret_cast<uintptr_t>(c.refs) % 16 == 0;
    auto gather = [&](long long base, bool keep) {
        const long long at = base + (long long)tid * kScanEach;
        uint32_t free = 0;
        if (wide && at + kScanEach <= c.n_pages) {
#pragma unroll
            for (int x = 0; x < kScanEach; x += 4) {
                const int4 r = *reinterpret_cast<const int4 *>(c.refs + at + x);
                free |= (r.x == 0 ? 1u : 0u) << x | (r.y == 0 ? 2u : 0u) << x | (r.z == 0 ? 4u : 0u) << x | (r.w == 0 ? 8u : 0u) << x;
            }
        } else {
#pragma unroll
            for (int x = 0; x < kScanEach; ++x)
                if (at + x < c.n_pages && c.refs[at + x] == 0) free |= 1u << x;
        }
        long long before;
        const int sum = (int)block_scan(__popc(free), before, scratch);
        if (keep)
            for (int rank = (int)before; free; free &= free - 1, ++rank) list[rank] = (int)at + __ffs(free) - 1;
        __syncthreads();
        return sum;
    };
    // Pages `found` .. of those there are, in the list, to the sequences, as far as `limit`.
    auto give = [&](long long found, int n, long long limit) {
        for (int k = tid; k < n && found + k < limit; k += kTakeThreads) {
            const long long rank = found + k;
            int lo = 0, hi = p.n_seq - 1;  // the last sequence whose pages begin at or before this one
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (pre[mid] <= rank) lo = mid;
                else hi = mid - 1;
            }
            int *const row = c.table + (long long)slots[lo] * c.table_row;
            const int at = first[lo] + (int)(rank - pre[lo]);
            if (!own || at >= c.held[slots[lo]]) {
                row[at] = list[k];
                c.refs[list[k]] = 1;
            } else if (k == 0 || rank == pre[lo]) {
                // Pages instead of shared ones, all of the sequence's in the list by one thread, in order: a page's count says which one it
                // replaces, until the next kernel has copied.
                const int end = min(c.held[slots[lo]], pages_for(__ldg(p.n_tok + lo), c.page));
                long long left = min(limit, min((long long)n + found, pre[lo] + c.held[slots[lo]] - first[lo])) - rank;
                for (int x = __ldg(p.len + lo) / c.page, y = k; x < end && left > 0; ++x) {
                    const int g = row[x];
                    if (c.refs[g] <= 1) continue;
                    c.refs[list[y]] = -1 - g, row[x] = list[y];
                    ++y, --left;
                }
            }
        }
        __syncthreads();
    };
    long long found = 0;  // free pages, as far as they are needed
    if (total > 0) {
        const int n = gather(0, true);
        if (n >= total) {
            found = total;
            give(0, n, total);
        } else {
            // first count, since a sequence gets all of its pages or none: those are served whose pages end within what there is
            found = n;
            for (long long base = kScanPages; base < c.n_pages && found < total; base += kScanPages) found += gather(base, false);
            found = min(found, total);
            long long limit = 0;
            for (int i = tid; i < p.n_seq; i += kTakeThreads)
                if (ends(i) <= found) limit = max(limit, ends(i));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) limit = max(limit, __shfl_xor_sync(0xffffffffu, limit, o));
            __syncthreads();
            if ((tid & 31) == 0) scratch[tid >> 5] = limit;
            __syncthreads();
            for (int w = 0; w < 32; ++w) limit = max(limit, scratch[w]);
            __syncthreads();
            long long given = 0;
            for (long long base = 0; given < limit && base < c.n_pages; base += kScanPages) {
                const int m = gather(base, true);
                give(given, m, limit);
                given += m;
            }
        }
    }
    for (int i = tid; i < p.n_seq; i += kTakeThreads) {
        const int slot = slots[i];
        if (slot < 0 || flagged[i]) continue;
        const long long need = ends(i) - pre[i];
        if (need > 0 && ends(i) > found) {
            if (p.err) p.err[i] = kSeqNoPages;
        } else if (fork) {
            c.held[slot] = -1 - i;  // until the next kernel has shared and copied: this sequence, and no other, is on
        } else if (need > 0) {
            c.held[slot] = first[i] + (int)need;
        }
    }
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// An access of BYTES bytes.
template <int BYTES> struct Piece;
template <> struct Piece<16> { using T = uint4; };
template <> struct Piece<4> { using T = uint32_t; };
template <> struct Piece<2> { using T = uint16_t; };

// The head rows of a copy: item = ((layer * 2 + which) * heads + head) * pieces + piece.  Gives the address of the
// layer's head in K or V, and that one's strides of pages and rows, in elements of the access.
template <int BYTES>
struct CopyItem {
    typename Piece<BYTES>::T *base;
    long long page, row;
    __device__ __forceinline__ CopyItem(const PagesParams &p, unsigned item) {
        const CacheView &c = p.c;
        const unsigned row_ = item / (unsigned)p.chunks, piece = item - row_ * p.chunks, lw = row_ / (unsigned)c.n_kv, h = row_ - lw * c.n_kv;
        const bool v = lw & 1;
        const long long layer = lw >> 1;
        const int per = BYTES / p.esize, by = per == 8 ? 3 : per == 4 ? 2 : 0;
        page = (v ? c.v_page : c.k_page) >> by, row = (v ? c.v_row : c.k_row) >> by;
        base = reinterpret_cast<typename Piece<BYTES>::T *>(v ? c.v : c.k) +
               ((layer * (v ? c.v_layer : c.k_layer) + (long long)h * (v ? c.v_head : c.k_head)) >> by) + piece;
    }
};
__device__ __forceinline__ unsigned copy_items(const PagesParams &p) { return 2u * p.c.n_layers * p.c.n_kv * p.chunks; }



// The first `rest` rows of a page to another, in every layer, by the blocks of a cluster: a piece of a head in one row of a layer is an
// item; a thread takes 4 of its rows at a time.
template <int BYTES>
__device__ __forceinline__ void copy_page(const PagesParams &p, int old_page, int new_page, int rest, int rank) {
    const unsigned items = copy_items(p);
    const int quarters = (rest + 3) / 4;
    for (unsigned long long x = rank * kPagesThreads + threadIdx.x; x < (unsigned long long)items * quarters; x += kForkCluster * kPagesThreads) {
        const unsigned q = (unsigned)(x / items), item = (unsigned)(x - (unsigned long long)q * items);
        const CopyItem<BYTES> m(p, item);
        typename Piece<BYTES>::T w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if ((int)(4 * q) + r < rest) w[r] = m.base[old_page * m.page + (4 * q + r) * m.row];
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if ((int)(4 * q) + r < rest) m.base[new_page * m.page + (4 * q + r) * m.row] = w[r];
    }
}

// A cluster a sequence: its first block shares the source's full pages and closes the slot's entry, all copy the rest of the last one.
template <int BYTES>
__global__ void __cluster_dims__(kForkCluster, 1, 1) __launch_bounds__(kPagesThreads)
    pages_fork(const __grid_constant__ PagesParams p) {
    grid_dep_wait();
    grid_dep_launch();
    const CacheView &c = p.c;
    const int tid = threadIdx.x, i = blockIdx.x / kForkCluster, rank = blockIdx.x % kForkCluster;
    const int slot = p.idx ? __ldg(p.idx + i) : i, src = __ldg(p.src + i);
    const int n = __ldg(p.n_tok + i), full = n / c.page, rest = n % c.page;
    // (bounds once more, of what the pages were taken for: a count that was negative before the call may look like its mark)
    const bool named = slot >= 0 && slot < c.n_slots && src >= 0 && src < c.n_slots && n >= 0 && n <= (long long)c.max_pages * c.page;
    int *const to = c.table + (long long)(named ? slot : 0) * c.table_row;
    const int *const from = c.table + (long long)(named ? src : 0) * c.table_row;
    const bool on = named && c.held[slot] == -1 - i;
    const int first = named && tid < full ? from[tid] : -1, old_page = named && rest ? from[full] : -1, new_page = named && rest ? to[full] : -1;
    auto there = [&](int page) { return page >= 0 && page < c.n_pages; };
    cluster_sync();  // every block has read the entry that the first one changes
    if (!on) return;
    if (rank == 0) {
        for (int x = tid; x < full; x += kPagesThreads) {
            const int g = x == tid ? first : from[x];
            to[x] = g;
            if (there(g)) atomicAdd(c.refs + g, 1);
        }
        if (tid == 0) c.held[slot] = full + (rest > 0);
    }
    if (there(old_page) && there(new_page)) copy_page<BYTES>(p, old_page, new_page, rest, rank);
}

// A cluster a sequence that grows (reserve with lengths): the rows of its last token's page to the page that replaces it, then the
// counts of the new and the replaced pages.
template <int BYTES>
__global__ void __cluster_dims__(kForkCluster, 1, 1) __launch_bounds__(kPagesThreads)
    pages_own(const __grid_constant__ PagesParams p) {
    grid_dep_wait();
    grid_dep_launch();
    const CacheView &c = p.c;
    const int tid = threadIdx.x, i = blockIdx.x / kForkCluster, rank = blockIdx.x % kForkCluster;
    const int slot = p.idx ? __ldg(p.idx + i) : i, n = __ldg(p.n_tok + i), L = __ldg(p.len + i);
    bool on = slot >= 0 && slot < c.n_slots && L >= 0 && L < n && n <= (long long)c.max_pages * c.page;
    bool named = false;  // by an earlier sequence, whose pages they are
    if (p.idx && on)
        for (int j = tid; j < i; j += kPagesThreads) named |= __ldg(p.idx + j) == slot;
    on &= !__syncthreads_or(named);
    int *const row = c.table + (long long)(on ? slot : 0) * c.table_row;
    const int begin = L / c.page, end = on ? min(c.held[slot], pages_for(n, c.page)) : 0;
    int old_page = -1, new_page = -1;
    if (on && begin < end && L % c.page) {
        new_page = row[begin];
        if (new_page >= 0 && new_page < c.n_pages) old_page = -1 - c.refs[new_page];
    }
    cluster_sync();  // every block has read the count that the first one changes
    if (rank == 0)
        for (int x = begin + tid; x < end; x += kPagesThreads) {
            const int g = row[x], of = g >= 0 && g < c.n_pages ? -1 - c.refs[g] : -1;
            if (of < 0) continue;
            c.refs[g] = 1;
            atomicSub(c.refs + of, 1);
        }
    if (old_page >= 0) copy_page<BYTES>(p, old_page, new_page, L % c.page, rank);
}

// A block a sequence.
__global__ void __launch_bounds__(kPagesThreads) pages_free(const __grid_constant__ PagesParams p) {
    grid_dep_wait();
    grid_dep_launch();
    const CacheView &c = p.c;
    const int tid = threadIdx.x, i = blockIdx.x;
    const int slot = p.idx ? __ldg(p.idx + i) : i;
    if (slot < 0) {
        if (tid == 0 && p.err) p.err[i] = 0;
        return;
    }
    int st = slot >= c.n_slots ? kSeqBadSlot : 0;
    if (p.idx)
        for (int j = tid; j < i; j += kPagesThreads)
            if (__ldg(p.idx + j) == slot) st |= kSeqBadSlot;
    st = __syncthreads_or(st) ? kSeqBadSlot : 0;
    int held = 0, keep = 0;
    int *const row = c.table + (long long)(st ? 0 : slot) * c.table_row;
    if (!st) {
        const int n = p.n_tok ? __ldg(p.n_tok + i) : 0;
        held = c.held[slot], keep = pages_for(n, c.page);
        if (n < 0 || held < 0 || held > c.max_pages) st = kSeqBadLength;
        int bad = 0;
        if (!st)
            for (int x = keep + tid; x < held; x += kPagesThreads) {
                const int g = row[x];
                bad |= g < 0 || g >= c.n_pages;
            }
        if (__syncthreads_or(bad)) st = kSeqBadPage;
    }
    if (tid == 0 && p.err) p.err[i] = st;
    if (st || keep >= held) return;
    for (int x = keep + tid; x < held; x += kPagesThreads) {
        const int g = row[x];
        if (atomicSub(c.refs + g, 1) <= 0) atomicAdd(c.refs + g, 1);  // (was free: stays so)
        row[x] = -1;
    }
    if (tid == 0) c.held[slot] = keep;
}

constexpr int kMaxPath = 128, kMoveRows = 8;

// Blocks (x) of a sequence (y) share its layers' heads.  A thread moves one piece of each row of the path in order, 8 rows
// read before they are written: the path rises, so a row is written only after every row at or past it was read.
template <int BYTES>
__global__ void __launch_bounds__(kPagesThreads) pages_compact(const __grid_constant__ PagesParams p) {
    __shared__ int src_page[kMaxPath], src_row[kMaxPath], dst_page[kMaxPath], dst_row[kMaxPath];
    __shared__ int first, flags;
    grid_dep_wait();
    grid_dep_launch();
    const CacheView &c = p.c;
    const int tid = threadIdx.x, s = blockIdx.y;
    const int slot = p.idx ? __ldg(p.idx + s) : s;
    const bool head = blockIdx.x == 0 && tid == 0;
    if (slot < 0) {
        if (head && p.err) p.err[s] = 0;
        return;
    }
    int st = slot >= c.n_slots ? kSeqBadSlot : 0;
    const int a = __ldg(p.accept + s), L = __ldg(p.len + s);
    if (a < 0 || a > p.T) st |= kSeqBadAccept;
    if (L < 0) st |= kSeqBadLength;
    if (tid == 0) first = p.T, flags = 0;
    __syncthreads();
    if (!st && tid < a) {
        const int at = __ldg(p.path + (long long)s * p.T + tid);
        const int before = tid > 0 ? __ldg(p.path + (long long)s * p.T + tid - 1) : -1;
        if (at <= before || at < tid || at >= p.T) st |= kSeqBadTree;
        else if ((long long)L + at >= (long long)c.max_pages * c.page) st |= kSeqBadLength;
        else if (at != tid) {
            const int from = L + at, to = L + tid;
            const int *const row = c.table + (long long)slot * c.table_row;
            const int g = __ldg(row + from / c.page), h = __ldg(row + to / c.page);
            if (g < 0 || g >= c.n_pages || h < 0 || h >= c.n_pages) st |= kSeqBadPage;
            else if (c.refs && __ldg(c.refs + h) > 1) st |= kSeqSharedPage;
            src_page[tid] = g, src_row[tid] = from % c.page;
            dst_page[tid] = h, dst_row[tid] = to % c.page;
            atomicMin(&first, tid);
        }
    }
    if (st) atomicOr(&flags, st);
    __syncthreads();
    const int all = flags;
    if (head && p.err) p.err[s] = all;
    if (all) return;
    if (head && p.new_len) p.new_len[s] = L + a;
    const int from = first;  // a rising path that has left its place stays ahead of it
    const unsigned items = copy_items(p);
    for (unsigned x = blockIdx.x * kPagesThreads + tid; x < items; x += gridDim.x * kPagesThreads) {
        const CopyItem<BYTES> m(p, x);
        for (int r0 = from; r0 < a; r0 += kMoveRows) {
            typename Piece<BYTES>::T w[kMoveRows];
#pragma unroll
            for (int r = 0; r < kMoveRows; ++r)
                if (r0 + r < a) w[r] = m.base[src_page[r0 + r] * m.page + src_row[r0 + r] * m.row];
#pragma unroll
            for (int r = 0; r < kMoveRows; ++r)
                if (r0 + r < a) m.base[dst_page[r0 + r] * m.page + dst_row[r0 + r] * m.row] = w[r];
        }
    }
}

}  // namespace

PagesKernel pages_take_kernel(int op) {
    return op == kPagesReserve ? pages_take<kPagesReserve> : op == kPagesOwn ? pages_take<kPagesOwn> : pages_take<kPagesFork>;
}
int pages_take_smem(int n_seq) { return 256 + n_seq * 24 + kScanPages * 4; }
PagesKernel pages_fork_kernel(int bytes) { return bytes == 16 ? pages_fork<16> : bytes == 4 ? pages_fork<4> : pages_fork<2>; }
PagesKernel pages_own_kernel(int bytes) { return bytes == 16 ? pages_own<16> : bytes == 4 ? pages_own<4> : pages_own<2>; }
PagesKernel pages_free_kernel() { return pages_free; }
PagesKernel pages_compact_kernel(int bytes) {
    return bytes == 16 ? pages_compact<16> : bytes == 4 ? pages_compact<4> : pages_compact<2>;
}

}  // namespace cvk
