// skv_pages.cu -- pages of a paged cache shared, moved and copied: fork, compact, copy, move.
//
// fork and compact plan on block tables alone: one cluster of CTAs walks the tables with a bit per page of the
// pool. A page comes free iff its bit, set for every page that some row held, is not cleared for the
// rows that go on; no count per page is kept between calls that could drift from the tables.
// Everything comes out in a fixed order: prefix sums over rows and over the words of bits.
// Pools of up to 32,768 pages keep the bits in shared memory: every CTA marks its share of the rows, reads the
// others' bits after a barrier and works the rest out for itself (a second barrier keeps all CTAs there until
// everybody has read). Larger ones (or more than 1,024 rows) keep them in the workspace, with a barrier of a
// cluster of 16 (half a microsecond, where a launch costs two) after each step.
//
// On the device 6.0 us for a fork of 8 rows (one CTA), 10.0 for one of 700 rows, 90 of them live, of up to 48 pages (a cluster of 8, two barriers), 9.8
// for a compaction of 200 rows of up to 47: latency, some 2.5 us of it the launch and as much the cluster's. In the workspace 16 for a compaction of
// 200 rows of up to 188 pages in a pool of 63,120, 23 for a fork of 4,000 rows, 600 of them live, of up to 189. A warp takes two rows at a time, two pieces of 32 entries of
// each on their way; with a warp per row and its lengths looked up anew for each piece these two took 30 and 73.
//
// copy and move bring the K and V: 16 bytes per thread and step. Copies are bound by HBM: 2,422 pages of 64 x 8 x 128 codes, K and V, in 99 us
// (6.4 TB/s, 0.94 of a copy; 97 with the status written by one of the blocks). Moves are five dependent loads: 3.5 us for 8
// paths of 4; 256 of 13 of 60 nodes take 7.4, 2.6 of them for the block that looks through all entries and 1.9 for the second eight of a path.
#include <cooperative_groups.h>

#include "skv_rows.cuh"

namespace skv {

namespace cg = cooperative_groups;

constexpr uint32_t kPlanThreads = 512, kPlanWarps = kPlanThreads / 32u, kPlanCluster = 8;      // pools whose bits fit shared memory
constexpr uint32_t kLargeThreads = 1024, kLargeWarps = kLargeThreads / 32u, kLargeCluster = 16;

struct PlanArgs {
    FastDiv page;
    uint32_t pool_pages, n_requests, max_pages, free_capacity, trim, capacity;
    const int32_t *parents, *ctx_len, *table, *n_in, *free_in;
    uint64_t table_stride, out_stride;
    int32_t *table_out, *n_out, *ctx_out, *free_pages, *free_out, *src, *dst, *count, *status;
    uint32_t *bits, *now;               // workspace: a bit per page, twice
    uint32_t *words;                    // fork: each row's heir, old row and entries of it; compact: rank of a far page, then the holes
};

// What the CTAs of the cluster tell each other: two numbers each, in every CTA's shared memory.
struct Told {
    uint2 word[2][kLargeCluster];
};

struct Team {
    uint32_t C, rank, parity;
    Told *told;

    // The sums of the CTAs' two numbers (thread 0's), and those of the CTAs before this one. Every thread calls; all writes of
    // the cluster before it, to global memory too, are seen after it (release and acquire of the cluster's barrier).
    __device__ __forceinline__ uint2 sum(uint32_t x, uint32_t y, uint2 *before) {
        cg::cluster_group cluster = cg::this_cluster();
        if (threadIdx.x < C) *cluster.map_shared_rank(&told->word[parity][rank], threadIdx.x) = make_uint2(x, y);
        cluster.sync();
        uint2 all = make_uint2(0u, 0u);
        for (uint32_t j = 0; j < C; ++j) {
            const uint2 w = told->word[parity][j];
            if (j == rank) *before = all;
            all.x += w.x;
            all.y += w.y;
        }
        parity ^= 1u;
        return all;
    }
    __device__ __forceinline__ uint32_t sum(uint32_t x, uint32_t *before) {
        uint2 b;
        const uint32_t all = sum(x, 0u, &b).x;
        *before = b.x;
        return all;
    }
    __device__ __forceinline__ bool any(bool x) {
        uint32_t b;
        return sum(x, &b) != 0u;
    }
    __device__ __forceinline__ void meet() { cg::this_cluster().sync(); }
};

// Exclusive prefix sum over a block of WARPS warps, and the total. part: a word per warp.
template <uint32_t WARPS>
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t *total, uint32_t *part) {
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, in = x;
#pragma unroll
    for (uint32_t d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(~0u, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) part[warp] = x;
    __syncthreads();
    const uint32_t p = lane < WARPS ? part[lane] : 0u;
    *total = __reduce_add_sync(~0u, p);
    return x - in + __reduce_add_sync(~0u, lane < warp ? p : 0u);
}

__device__ __forceinline__ void set_bit(uint32_t *bits, uint32_t page) { atomicOr(bits + (page >> 5), 1u << (page & 31u)); }

// What a walk over the table needs of a row: how many entries, of which row of the old table, and a number of the caller's.
struct Head {
    uint32_t len, from, extra;
};

// f(row, its head, column, g(page)) of every entry: two rows to a warp at a time, two pieces of 32 entries of each on their way.
template <uint32_t WARPS, typename HeadOf, typename G, typename F>
__device__ __forceinline__ void each_entry(const PlanArgs &a, const Team &t, HeadOf head_of, G g, F f) {
    const uint32_t lane = threadIdx.x & 31u, warps = WARPS * t.C;
#pragma unroll 1
    for (uint64_t r0 = (threadIdx.x >> 5) * t.C + t.rank; r0 < a.n_requests; r0 += 2u * warps) {
        Head h[2];
        uint32_t most = 0;
#pragma unroll
        for (uint32_t k = 0; k < 2; ++k) {
            h[k] = r0 + k * warps < a.n_requests ? head_of((uint32_t)r0 + k * warps) : Head{0u, 0u, 0u};
            most = max(most, h[k].len);
        }
#pragma unroll 1
        for (uint32_t j0 = 0; j0 < most; j0 += 64u) {
            int32_t page[2][2];
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) {
                const uint32_t j = j0 + 32u * (k & 1u) + lane;
                const Head &x = h[k >> 1];
                page[k >> 1][k & 1u] = j < x.len ? __ldg(a.table + (uint64_t)x.from * a.table_stride + j) : 0;
            }
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k)
                if (j0 + 32u * (k & 1u) + lane < h[k >> 1].len) page[k >> 1][k & 1u] = g(page[k >> 1][k & 1u]);
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) {
                const uint32_t j = j0 + 32u * (k & 1u) + lane;
                const Head &x = h[k >> 1];
                if (j < x.len) f((uint32_t)r0 + (k >> 1) * warps, x, j, page[k >> 1][k & 1u]);
            }
        }
    }
}

struct AsItIs {
    __device__ __forceinline__ int32_t operator()(int32_t p) const { return p; }
};

// Words of bits of this CTA and, in them, of this thread: runs in order.
__device__ __forceinline__ void run_of(const PlanArgs &a, const Team &t, uint32_t *from, uint32_t *to) {
    const uint32_t n = (a.pool_pages + 31u) >> 5, per_cta = (n + t.C - 1u) / t.C, each = (per_cta + blockDim.x - 1u) / blockDim.x;
    const uint32_t end = min((t.rank + 1u) * per_cta, n);
    *from = min(t.rank * per_cta + threadIdx.x * each, end);
    *to = min(*from + each, end);
}

__device__ __forceinline__ bool ring_bad(const PlanArgs &a, int32_t head, int32_t count) {
    return count < 0 || (uint32_t)count > a.free_capacity || head < 0 ||
           ((uint32_t)head >= a.free_capacity && (head != 0 || a.free_capacity != 0));
}

// The tables handed on as they were, after an error (page counts clamped to the rows).
__device__ __forceinline__ void hand_on(const PlanArgs &a, const Team &t, int32_t err) {
    const uint32_t lane = threadIdx.x & 31u;
    for (uint32_t r = t.rank * (blockDim.x >> 5) + (threadIdx.x >> 5); r < a.n_requests; r += t.C * (blockDim.x >> 5)) {
        const uint32_t n = min((uint32_t)max(__ldg(a.n_in + r), 0), a.max_pages);
        for (uint32_t j = lane; j < n; j += 32u)
            a.table_out[(uint64_t)r * a.out_stride + j] = __ldg(a.table + (uint64_t)r * a.table_stride + j);
        if (lane == 0 && a.n_out) {
            a.n_out[r] = __ldg(a.n_in + r);
            a.ctx_out[r] = __ldg(a.ctx_len + r);
        }
    }
    for (uint32_t i = t.rank * blockDim.x + threadIdx.x; i < a.capacity; i += t.C * blockDim.x) {
        a.src[i] = a.dst[i] = -1;
        if (a.count) a.count[i] = 0;
    }
    if (t.rank == 0 && threadIdx.x == 0) {
        a.free_out[0] = __ldg(a.free_in);
        a.free_out[1] = __ldg(a.free_in + 1);
        *a.status = err;
    }
}

// ---- fork

// The row that row s goes on from, or ~0 (errors are found before).
__device__ __forceinline__ uint32_t parent_row(const PlanArgs &a, uint32_t s) {
    const int32_t p = a.parents ? __ldg(a.parents + s) : (int32_t)s;
    return p < 0 || __ldg(a.ctx_len + p) < 0 ? ~0u : (uint32_t)p;
}

__device__ __forceinline__ uint32_t pages_of(const PlanArgs &a, uint32_t tokens) {
    const uint32_t whole = div_by(tokens, a.page);
    return whole + (tokens != whole * a.page.d);
}

struct Fork {
    uint32_t from;       // ~0: empty
    uint32_t keep;       // entries of the old row
    uint32_t copies;     // 1: one more page, a copy of the old row's next
    uint32_t part;       // tokens of it
    bool heir;
};

__device__ __forceinline__ Fork fork_of(const PlanArgs &a, uint32_t s) {
    Fork f{parent_row(a, s), 0u, 0u, 0u, false};
    if (f.from == ~0u) return f;
    const uint32_t c = (uint32_t)__ldg(a.ctx_len + f.from), whole = div_by(c, a.page), part = c - whole * a.page.d;
    // the workspace holds s + 1 of the lowest row that goes on, 0 for the row itself
    f.heir = __ldcg(a.words + f.from) == (f.from == s ? 0u : s + 1u);
    if (f.heir) {
        f.keep = a.trim ? whole + (part != 0u) : (uint32_t)__ldg(a.n_in + f.from);
    } else {
        f.keep = whole;
        f.copies = part != 0u;
        f.part = part;
    }
    return f;
}

__global__ void __launch_bounds__(kLargeThreads) fork_pages_kernel(const PlanArgs a) {
    __shared__ Told told;
    __shared__ uint32_t part[kLargeWarps];
    cg::cluster_group cluster = cg::this_cluster();
    Team t{cluster.num_blocks(), cluster.block_rank(), 0u, &told};
    const uint32_t tid = threadIdx.x, all_threads = t.C * kLargeThreads, mine_of_all = t.rank * kLargeThreads + tid;
    const int32_t head = __ldg(a.free_in), count = __ldg(a.free_in + 1);
    if (t.rank == 0 && tid == 0) *a.status = SKV_OK;
    cluster.sync();                                       // every CTA has started

    // Errors of the lengths; the workspace is made ready.
    bool bad = ring_bad(a, head, count);
    for (uint32_t r = mine_of_all; r < a.n_requests; r += all_threads) {
        const int32_t p = a.parents ? __ldg(a.parents + r) : (int32_t)r, c = __ldg(a.ctx_len + r), h = __ldg(a.n_in + r);
        bad |= p < -1 || p >= (int32_t)a.n_requests || h < 0 || (uint32_t)h > a.max_pages || (int64_t)c > (int64_t)h * a.page.d;
        a.words[r] = ~0u;
    }
    for (uint32_t i = mine_of_all; i < (a.pool_pages + 31u) >> 5; i += all_threads) a.bits[i] = a.now[i] = 0u;
    if (t.any(__syncthreads_or(bad) != 0)) {
        hand_on(a, t, SKV_ERR_INVALID_ARG);
        return;
    }
    for (uint32_t s = mine_of_all; s < a.n_requests; s += all_threads) {
        const uint32_t p = parent_row(a, s);
        if (p != ~0u) atomicMin(a.words + p, p == s ? 0u : s + 1u);
    }
    t.meet();
    // Pages that rows held, and those that their heirs go on with (all others' are among them).
    bool corrupt = false;
    each_entry<kLargeWarps>(a, t, [&](uint32_t r) {
        const uint32_t n = (uint32_t)__ldg(a.n_in + r), heir = __ldcg(a.words + r);
        const int32_t c = __ldg(a.ctx_len + r);
        return Head{n, r, heir == ~0u ? 0u : a.trim ? pages_of(a, (uint32_t)c) : n};
    }, AsItIs{}, [&](uint32_t, const Head &h, uint32_t j, int32_t p) {
        if ((uint32_t)p >= a.pool_pages) {
            corrupt = true;
            return;
        }
        set_bit(a.bits, (uint32_t)p);
        if (j < h.extra) set_bit(a.now, (uint32_t)p);
    });
    // Copies ranked in order of rows, a stretch of them to a CTA; their pages come off the ring.
    const uint32_t stretch = a.n_requests / t.C + 1u;
    const uint32_t s0 = (uint32_t)min((uint64_t)t.rank * stretch, (uint64_t)a.n_requests), s1 = (uint32_t)min((uint64_t)s0 + stretch, (uint64_t)a.n_requests);
    uint32_t mine = 0, here, before;
    for (uint32_t s = s0 + tid; s < s1; s += kLargeThreads) mine += fork_of(a, s).copies;
    block_scan<kLargeWarps>(mine, &here, part);
    const uint32_t took = t.sum(here, &before);
    if (took > (uint32_t)count) {
        hand_on(a, t, SKV_ERR_CAPACITY);
        return;
    }
    uint32_t k0 = before, *const from_of = a.words + a.n_requests, *const keep_of = from_of + a.n_requests;
#pragma unroll 1
    for (uint32_t base = s0; base < s1; base += kLargeThreads) {
        const uint32_t s = base + tid;
        Fork f{~0u, 0u, 0u, 0u, false};
        if (s < s1) f = fork_of(a, s);
        const uint32_t k = k0 + block_scan<kLargeWarps>(f.copies, &here, part);
        k0 += here;
        if (s >= s1) continue;
        from_of[s] = f.from;
        keep_of[s] = f.keep;
        int32_t from = -1, to = -1;
        if (f.copies) {
            uint64_t e = (uint64_t)head + k;
            if (e >= a.free_capacity) e -= a.free_capacity;
            from = __ldg(a.table + (uint64_t)f.from * a.table_stride + f.keep);
            to = __ldg(a.free_pages + e);
            if ((uint32_t)to < a.pool_pages) set_bit(a.now, (uint32_t)to);
        }
        // both as they are until the rows are written; a pair outside the pool is left out then
        a.src[s] = from;
        a.dst[s] = to;
        a.count[s] = (int32_t)f.part;
        a.n_out[s] = (int32_t)(f.keep + f.copies);
        a.ctx_out[s] = f.from == ~0u ? -1 : __ldg(a.ctx_len + f.from);
    }
    t.meet();
    // Freed pages, counted.
    uint32_t from, to;
    run_of(a, t, &from, &to);
    mine = 0;
    for (uint32_t i = from; i < to; ++i) mine += __popc(__ldcg(a.bits + i) & ~__ldcg(a.now + i));
    uint32_t at = block_scan<kLargeWarps>(mine, &here, part);
    const uint32_t freed = t.sum(here, &before);
    at += before;
    if ((uint64_t)count - took + freed > a.free_capacity) {
        hand_on(a, t, SKV_ERR_CAPACITY);
        return;
    }
    // Into the ring behind its end, the rows, the counts.
    for (uint32_t i = from; i < to; ++i) {
        for (uint32_t w = __ldcg(a.bits + i) & ~__ldcg(a.now + i); w; w &= w - 1u) {
            uint64_t e = (uint64_t)head + (uint32_t)count + at++;
            while (e >= a.free_capacity) e -= a.free_capacity;
            a.free_pages[e] = (int32_t)(32u * i + __ffs(w) - 1u);
        }
    }
    each_entry<kLargeWarps>(a, t, [&](uint32_t s) { return Head{__ldcg(keep_of + s), __ldcg(from_of + s), 0u}; }, AsItIs{},
                            [&](uint32_t s, const Head &, uint32_t j, int32_t p) { a.table_out[(uint64_t)s * a.out_stride + j] = p; });
    for (uint32_t s = s0 + tid; s < s1; s += kLargeThreads) {
        if (a.count[s] == 0) continue;
        const int32_t x = a.src[s], y = a.dst[s];
        a.table_out[(uint64_t)s * a.out_stride + keep_of[s]] = y;
        if ((uint32_t)x >= a.pool_pages || (uint32_t)y >= a.pool_pages) {
            corrupt = true;
            a.src[s] = a.dst[s] = -1;
            a.count[s] = 0;
        }
    }
    if (t.rank == 0 && tid == 0) {
        uint64_t e = (uint64_t)head + took;
        const uint32_t cap = max(a.free_capacity, 1u);
        if (e >= cap) e -= cap;
        a.free_out[0] = (int32_t)e;
        a.free_out[1] = (int32_t)((uint32_t)count - took + freed);
    }
    if (corrupt) set_first(a.status, SKV_ERR_CORRUPT);    // (the first CTA's OK came barriers ago)
}

// ---- compact

// Bits of word i that lie below page `limit`.
__device__ __forceinline__ uint32_t below(uint32_t i, uint32_t limit) {
    const uint32_t first = 32u * i;
    return limit <= first ? 0u : limit - first >= 32u ? ~0u : (1u << (limit - first)) - 1u;
}

__global__ void __launch_bounds__(kLargeThreads, 1) compact_pages_kernel(const PlanArgs a) {
    __shared__ Told told;
    __shared__ uint32_t part[kLargeWarps];
    cg::cluster_group cluster = cg::this_cluster();
    Team t{cluster.num_blocks(), cluster.block_rank(), 0u, &told};
    const uint32_t tid = threadIdx.x, all_threads = t.C * kLargeThreads, mine_of_all = t.rank * kLargeThreads + tid;
    if (t.rank == 0 && tid == 0) *a.status = SKV_OK;
    cluster.sync();                                       // every CTA has started
    bool bad = false, corrupt = false;
    for (uint32_t r = mine_of_all; r < a.n_requests; r += all_threads) {
        const int32_t h = __ldg(a.n_in + r);
        bad |= h < 0 || (uint32_t)h > a.max_pages;
    }
    for (uint32_t i = mine_of_all; i < (a.pool_pages + 31u) >> 5; i += all_threads) a.bits[i] = 0u;
    if (t.any(__syncthreads_or(bad) != 0)) {
        hand_on(a, t, SKV_ERR_INVALID_ARG);
        return;
    }
    const auto row_head = [&](uint32_t r) { return Head{(uint32_t)__ldg(a.n_in + r), r, 0u}; };
    each_entry<kLargeWarps>(a, t, row_head, AsItIs{}, [&](uint32_t, const Head &, uint32_t, int32_t p) {
        if ((uint32_t)p < a.pool_pages) set_bit(a.bits, (uint32_t)p);
        else corrupt = true;
    });
    t.meet();
    // Held pages in all, then holes below that number and held pages from it on.
    uint32_t from, to, mine = 0, here, before;
    run_of(a, t, &from, &to);
    for (uint32_t i = from; i < to; ++i) mine += __popc(__ldcg(a.bits + i));
    block_scan<kLargeWarps>(mine, &here, part);
    const uint32_t live = t.sum(here, &before);
    uint32_t holes = 0, far = 0;
    for (uint32_t i = from; i < to; ++i) {
        const uint32_t w = __ldcg(a.bits + i), low = below(i, live);
        holes += __popc(~w & low);
        far += __popc(w & ~low);
    }
    uint32_t here_holes, here_far;
    uint2 others;
    holes = block_scan<kLargeWarps>(holes, &here_holes, part);
    far = block_scan<kLargeWarps>(far, &here_far, part);
    const uint32_t moves = t.sum(here_holes, here_far, &others).y;
    holes += others.x;
    far += others.y;
    if (moves > a.capacity || a.pool_pages - live > a.free_capacity) {
        hand_on(a, t, SKV_ERR_CAPACITY);
        return;
    }
    uint32_t *rank_of = a.words, *hole = a.words + a.pool_pages;
    for (uint32_t i = from; i < to; ++i) {
        const uint32_t w = __ldcg(a.bits + i), low = below(i, live);
        for (uint32_t m = ~w & low; m; m &= m - 1u) {
            const uint32_t p = 32u * i + __ffs(m) - 1u;
            hole[holes] = p;
            a.dst[holes++] = (int32_t)p;
        }
        for (uint32_t m = w & ~low; m; m &= m - 1u) {
            const uint32_t p = 32u * i + __ffs(m) - 1u;
            rank_of[p] = far;
            a.src[far++] = (int32_t)p;
        }
    }
    for (uint32_t i = moves + mine_of_all; i < a.capacity; i += all_threads) a.src[i] = a.dst[i] = -1;
    for (uint32_t i = mine_of_all; i < a.pool_pages - live; i += all_threads) a.free_pages[i] = (int32_t)(live + i);
    t.meet();
    each_entry<kLargeWarps>(a, t, row_head, [&](int32_t p) {
        return (uint32_t)p >= live && (uint32_t)p < a.pool_pages ? (int32_t)__ldcg(hole + __ldcg(rank_of + p)) : p;
    }, [&](uint32_t r, const Head &, uint32_t j, int32_t p) { a.table_out[(uint64_t)r * a.out_stride + j] = p; });
    if (t.rank == 0 && tid == 0) {
        a.free_out[0] = 0;
        a.free_out[1] = (int32_t)(a.pool_pages - live);
    }
    if (corrupt) set_first(a.status, SKV_ERR_CORRUPT);
}

// ---- both, for pools whose bits fit shared memory

constexpr uint32_t kSmallPool = 32768, kSmallWords = kSmallPool / 32u, kSmallRows = 1024;
static_assert(kSmallWords == 2u * kPlanThreads && kSmallRows == 2u * kPlanThreads, "two words and two rows to a thread");

// Word i of the union of the CTAs' bits (every CTA's, after a barrier).
__device__ __forceinline__ uint32_t union_of(uint32_t *bits, uint32_t i, uint32_t C) {
    cg::cluster_group cluster = cg::this_cluster();
    uint32_t w = 0;
#pragma unroll 8
    for (uint32_t j = 0; j < C; ++j) w |= cluster.map_shared_rank(bits, j)[i];
    return w;
}

// The last of a kernel that reads other CTAs' shared memory: nobody leaves before everybody has read.
__device__ __forceinline__ void leave_together(uint32_t C) {
    if (C > 1u) cg::this_cluster().sync();
}

__global__ void __launch_bounds__(kPlanThreads) fork_small_kernel(const PlanArgs a) {
    __shared__ uint32_t was[kSmallWords], now[kSmallWords];
    __shared__ int32_t parent[kSmallRows], ctx[kSmallRows], have[kSmallRows];
    __shared__ uint32_t heir[kSmallRows], from[kSmallRows], keep[kSmallRows], part[kPlanWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const Team t{cluster.num_blocks(), cluster.block_rank(), 0u, nullptr};
    const uint32_t tid = threadIdx.x, n = a.n_requests;
    const int32_t head = __ldg(a.free_in), count = __ldg(a.free_in + 1);
    bool bad = ring_bad(a, head, count), corrupt = false;
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k) {
        const uint32_t r = k * kPlanThreads + tid;
        was[r] = now[r] = 0u;
        heir[r] = ~0u;
        if (r >= n) continue;
        const int32_t p = a.parents ? __ldg(a.parents + r) : (int32_t)r, c = __ldg(a.ctx_len + r), h = __ldg(a.n_in + r);
        parent[r] = p, ctx[r] = c, have[r] = h;
        bad |= p < -1 || p >= (int32_t)n || h < 0 || (uint32_t)h > a.max_pages || (int64_t)c > (int64_t)h * a.page.d;
    }
    if (t.rank == 0 && tid == 0) *a.status = SKV_OK;
    if (__syncthreads_or(bad)) {                          // the same in every CTA
        cluster.sync();                                   // and every CTA has seen it, before anything is written
        hand_on(a, t, SKV_ERR_INVALID_ARG);
        return;
    }
    const auto from_of = [&](uint32_t s) -> uint32_t { return parent[s] < 0 || ctx[parent[s]] < 0 ? ~0u : (uint32_t)parent[s]; };
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k) {
        const uint32_t s = k * kPlanThreads + tid;
        if (s >= n) continue;
        const uint32_t f = from_of(s);
        if (f != ~0u) atomicMin(heir + f, f == s ? 0u : s + 1u);
    }
    __syncthreads();
    // Entries that an heir of row r keeps, and what row s has.
    const auto kept_of = [&](uint32_t r) -> uint32_t { return a.trim ? pages_of(a, (uint32_t)ctx[r]) : (uint32_t)have[r]; };
    const auto row_of = [&](uint32_t s) {
        Fork f{from_of(s), 0u, 0u, 0u, false};
        if (f.from == ~0u) return f;
        const uint32_t c = (uint32_t)ctx[f.from], whole = div_by(c, a.page);
        f.heir = heir[f.from] == (f.from == s ? 0u : s + 1u);
        f.part = f.heir ? 0u : c - whole * a.page.d;
        f.copies = f.part != 0u;
        f.keep = f.heir ? kept_of(f.from) : whole;
        return f;
    };
    // Copies ranked in order of rows, two rows to a thread; a CTA takes the pages of its share of them.
    Fork mine[2];
    uint32_t took, k0;
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k) {
        mine[k] = 2u * tid + k < n ? row_of(2u * tid + k) : Fork{~0u, 0u, 0u, 0u, false};
        from[2u * tid + k] = mine[k].from;
        keep[2u * tid + k] = mine[k].keep;
    }
    k0 = block_scan<kPlanWarps>(mine[0].copies + mine[1].copies, &took, part);
    if (took > (uint32_t)count) {
        cluster.sync();
        hand_on(a, t, SKV_ERR_CAPACITY);
        return;
    }
    int32_t src[2], dst[2], fresh[2];
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k) {
        const uint32_t s = 2u * tid + k;
        src[k] = dst[k] = -1;
        if (s < n && s % t.C == t.rank && mine[k].copies) {
            uint64_t e = (uint64_t)head + k0 + (k ? mine[0].copies : 0u);
            if (e >= a.free_capacity) e -= a.free_capacity;
            src[k] = __ldg(a.table + (uint64_t)mine[k].from * a.table_stride + mine[k].keep);
            fresh[k] = dst[k] = __ldg(a.free_pages + e);
            if ((uint32_t)dst[k] < a.pool_pages) atomicOr(now + ((uint32_t)dst[k] >> 5), 1u << (dst[k] & 31));
            if ((uint32_t)src[k] >= a.pool_pages || (uint32_t)dst[k] >= a.pool_pages) {
                corrupt = true;
                src[k] = dst[k] = -1;
                mine[k].part = 0u;
            }
        }
    }
    // Pages that rows held, and those that their heirs go on with (all others' are among them).
    each_entry<kPlanWarps>(a, t, [&](uint32_t r) { return Head{(uint32_t)have[r], r, heir[r] == ~0u ? 0u : kept_of(r)}; }, AsItIs{},
                           [&](uint32_t, const Head &h, uint32_t j, int32_t p) {
        if ((uint32_t)p < a.pool_pages) {
            set_bit(was, (uint32_t)p);
            if (j < h.extra) set_bit(now, (uint32_t)p);
        } else {
            corrupt = true;
        }
    });
    cluster.sync();
    uint32_t w[2];
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k) w[k] = union_of(was, 2u * tid + k, t.C) & ~union_of(now, 2u * tid + k, t.C);
    uint32_t freed;
    const uint32_t at0 = block_scan<kPlanWarps>(__popc(w[0]) + __popc(w[1]), &freed, part);
    if ((uint64_t)count - took + freed > a.free_capacity) {
        hand_on(a, t, SKV_ERR_CAPACITY);
        leave_together(t.C);
        return;
    }
    if (tid % t.C == t.rank) {
        uint32_t at = at0;
#pragma unroll
        for (uint32_t k = 0; k < 2; ++k) {
            for (uint32_t m = w[k]; m; m &= m - 1u) {
                uint64_t e = (uint64_t)head + (uint32_t)count + at++;
                while (e >= a.free_capacity) e -= a.free_capacity;
                a.free_pages[e] = (int32_t)(32u * (2u * tid + k) + __ffs(m) - 1u);
            }
        }
    }
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k) {
        const uint32_t s = 2u * tid + k;
        if (s < n && s % t.C == t.rank) {
            a.src[s] = src[k], a.dst[s] = dst[k], a.count[s] = (int32_t)mine[k].part;
            a.n_out[s] = (int32_t)(mine[k].keep + mine[k].copies);
            a.ctx_out[s] = mine[k].from == ~0u ? -1 : ctx[mine[k].from];
            if (mine[k].copies) a.table_out[(uint64_t)s * a.out_stride + mine[k].keep] = fresh[k];
        }
    }
    each_entry<kPlanWarps>(a, t, [&](uint32_t s) { return Head{keep[s], from[s], 0u}; }, AsItIs{},
                           [&](uint32_t s, const Head &, uint32_t j, int32_t p) { a.table_out[(uint64_t)s * a.out_stride + j] = p; });
    if (t.rank == 0 && tid == 0) {
        uint64_t e = (uint64_t)head + took;
        const uint32_t cap = max(a.free_capacity, 1u);
        if (e >= cap) e -= cap;
        a.free_out[0] = (int32_t)e;
        a.free_out[1] = (int32_t)((uint32_t)count - took + freed);
    }
    if (corrupt) set_first(a.status, SKV_ERR_CORRUPT);    // (after the barrier that the first CTA's OK came before)
    leave_together(t.C);
}

__global__ void __launch_bounds__(kPlanThreads) compact_small_kernel(const PlanArgs a) {
    __shared__ uint32_t bits[kSmallWords], held[kSmallWords], part[kPlanWarps];
    __shared__ uint16_t far_before[kSmallWords], hole[kSmallPool / 2u];
    __shared__ int32_t have[kSmallRows];
    cg::cluster_group cluster = cg::this_cluster();
    const Team t{cluster.num_blocks(), cluster.block_rank(), 0u, nullptr};
    const uint32_t tid = threadIdx.x;
    bits[tid] = bits[kPlanThreads + tid] = 0u;
    bool bad = false, corrupt = false;
    for (uint32_t r = tid; r < a.n_requests; r += kPlanThreads) {
        const int32_t h = __ldg(a.n_in + r);
        bad |= h < 0 || (uint32_t)h > a.max_pages;
        have[r] = h;
    }
    if (t.rank == 0 && tid == 0) *a.status = SKV_OK;
    if (__syncthreads_or(bad)) {                          // the same in every CTA
        cluster.sync();                                   // and every CTA has seen it, before anything is written
        hand_on(a, t, SKV_ERR_INVALID_ARG);
        return;
    }
    const auto row_head = [&](uint32_t r) { return Head{(uint32_t)have[r], r, 0u}; };
    each_entry<kPlanWarps>(a, t, row_head, AsItIs{}, [&](uint32_t, const Head &, uint32_t, int32_t p) {
        if ((uint32_t)p < a.pool_pages) set_bit(bits, (uint32_t)p);
        else corrupt = true;
    });
    cluster.sync();
    uint32_t w[2], live, all;
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k) held[2u * tid + k] = w[k] = union_of(bits, 2u * tid + k, t.C);
    block_scan<kPlanWarps>(__popc(w[0]) + __popc(w[1]), &live, part);
    // holes below `live` and held pages from it on, counted together (2^15 of either at most)
    uint32_t low[2], x = 0;
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k) {
        low[k] = below(2u * tid + k, live);
        x += (uint32_t)__popc(~w[k] & low[k]) << 16 | (uint32_t)__popc(w[k] & ~low[k]);
    }
    x = block_scan<kPlanWarps>(x, &all, part);
    const uint32_t moves = all & 0xFFFFu;
    if (moves > a.capacity || a.pool_pages - live > a.free_capacity) {
        hand_on(a, t, SKV_ERR_CAPACITY);
        leave_together(t.C);
        return;
    }
    uint32_t holes = x >> 16, far = x & 0xFFFFu;
    const bool tells = tid % t.C == t.rank;
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k) {
        const uint32_t first = 32u * (2u * tid + k);
        far_before[2u * tid + k] = (uint16_t)far;
        for (uint32_t m = ~w[k] & low[k]; m; m &= m - 1u) {
            const uint32_t p = first + __ffs(m) - 1u;
            hole[holes] = (uint16_t)p;
            if (tells) a.dst[holes] = (int32_t)p;
            ++holes;
        }
        for (uint32_t m = w[k] & ~low[k]; m; m &= m - 1u, ++far)
            if (tells) a.src[far] = (int32_t)(first + __ffs(m) - 1u);
    }
    __syncthreads();
    for (uint32_t i = moves + t.rank * kPlanThreads + tid; i < a.capacity; i += t.C * kPlanThreads) a.src[i] = a.dst[i] = -1;
    for (uint32_t i = t.rank * kPlanThreads + tid; i < a.pool_pages - live; i += t.C * kPlanThreads) a.free_pages[i] = (int32_t)(live + i);
    each_entry<kPlanWarps>(a, t, row_head, [&](int32_t p) -> int32_t {
        if ((uint32_t)p < live || (uint32_t)p >= a.pool_pages) return p;
        const uint32_t i = (uint32_t)p >> 5, under = held[i] & ~below(i, live) & ((1u << (p & 31)) - 1u);
        return hole[far_before[i] + __popc(under)];
    }, [&](uint32_t r, const Head &, uint32_t j, int32_t p) { a.table_out[(uint64_t)r * a.out_stride + j] = p; });
    if (t.rank == 0 && tid == 0) {
        a.free_out[0] = 0;
        a.free_out[1] = (int32_t)(a.pool_pages - live);
    }
    if (corrupt) set_first(a.status, SKV_ERR_CORRUPT);
    leave_together(t.C);
}

// ---- copies of pages

struct CopyArgs {
    uint8_t *k, *v;
    uint64_t page_stride, token_stride, head_stride;      // bytes
    uint32_t page_tokens, n_pages, n, chunks;             // chunks of a page, of kCopyUnits units of 16 bytes
    FastDiv by_chunks, per_token, per_head;               // units of a token and of a head
    const int32_t *src, *dst, *tokens;
    int32_t *status;
    uint32_t checked;                                     // 1: block 0 reports the errors, 2: and does nothing else
};

constexpr uint32_t kCopyThreads = 256, kCopyDeep = 2, kCopyUnits = kCopyThreads * kCopyDeep;

// A pair's pages and how many tokens of them; false: nothing to copy (bad: not as it should be).
__device__ __forceinline__ bool pair_of(const CopyArgs &a, uint32_t i, int32_t *src, int32_t *dst, uint32_t *n, bool *bad) {
    *src = __ldg(a.src + i);
    *dst = __ldg(a.dst + i);
    *n = a.tokens ? (uint32_t)__ldg(a.tokens + i) : a.page_tokens;
    if (*src < 0) return false;
    const bool ok = (uint32_t)*src < a.n_pages && (uint32_t)*dst < a.n_pages && *n <= a.page_tokens;
    *bad |= !ok;
    return ok && *n != 0u;
}

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const CopyArgs a) {
    const uint32_t lane = threadIdx.x & 31u;
    bool bad = false;
    int32_t src, dst;
    uint32_t n;
    if (a.checked && blockIdx.x == 0) {
#pragma unroll 8
        for (uint32_t i = threadIdx.x; i < a.n; i += kCopyThreads) pair_of(a, i, &src, &dst, &n, &bad);
        bad = __syncthreads_or(bad);
        if (threadIdx.x == 0) *a.status = bad ? SKV_ERR_INVALID_ARG : SKV_OK;
        if (a.checked == 2u) return;
        bad = false;
    }
    const uint32_t first = a.checked == 2u ? blockIdx.x - 1u : blockIdx.x, blocks = a.checked == 2u ? gridDim.x - 1u : gridDim.x;
    // Chunks are dealt to the CTAs in turn. A warp looks 32 of its chunks up at once, so that pairs without a copy
    // cost little; all warps of a CTA find the same.
    const uint64_t items = (uint64_t)a.n * a.chunks;
#pragma unroll 1
    for (uint64_t m0 = first; m0 < items; m0 += 32ull * blocks) {
        const uint64_t m = m0 + (uint64_t)lane * blocks;
        bool live = false;
        uint32_t chunk = 0;
        src = dst = 0;
        n = 0;
        if (m < items) {
            const uint32_t i = m >> 31 ? (uint32_t)(m / a.chunks) : div_by((uint32_t)m, a.by_chunks);
            chunk = (uint32_t)(m - (uint64_t)i * a.chunks);
            live = pair_of(a, i, &src, &dst, &n, &bad) && (uint64_t)chunk * kCopyUnits < (uint64_t)n * a.per_token.d;
        }
        uint32_t todo = __ballot_sync(~0u, live);
#pragma unroll 1
        while (todo) {
            const uint32_t l = __ffs(todo) - 1u;
            todo &= todo - 1u;
            const uint64_t from = (uint64_t)__shfl_sync(~0u, src, l) * a.page_stride, to = (uint64_t)__shfl_sync(~0u, dst, l) * a.page_stride;
            const uint32_t u0 = __shfl_sync(~0u, chunk, l) * kCopyUnits, end = __shfl_sync(~0u, n, l) * a.per_token.d;
            uint4 x[kCopyDeep], y[kCopyDeep];
            uint64_t at[kCopyDeep];
#pragma unroll
            for (uint32_t j = 0; j < kCopyDeep; ++j) {
                const uint32_t u = u0 + j * kCopyThreads + threadIdx.x;
                const uint32_t token = div_by(u, a.per_token), rest = u - token * a.per_token.d;
                const uint32_t h = div_by(rest, a.per_head);
                at[j] = token * a.token_stride + h * a.head_stride + 16u * (uint64_t)(rest - h * a.per_head.d);
                if (u < end) {
                    x[j] = *reinterpret_cast<const uint4 *>(a.k + from + at[j]);
                    y[j] = *reinterpret_cast<const uint4 *>(a.v + from + at[j]);
                }
            }
#pragma unroll
            for (uint32_t j = 0; j < kCopyDeep; ++j) {
                if (u0 + j * kCopyThreads + threadIdx.x < end) {
                    *reinterpret_cast<uint4 *>(a.k + to + at[j]) = x[j];
                    *reinterpret_cast<uint4 *>(a.v + to + at[j]) = y[j];
                }
            }
        }
    }
    if (bad && !a.checked) set_first(a.status, SKV_ERR_INVALID_ARG);
}

// ---- moves of tokens

struct MoveArgs {
    uint8_t *k, *v;
    uint64_t page_stride, token_stride, head_stride;      // bytes
    FastDiv page, per_head;                               // units of 16 bytes per head
    uint64_t pool_tokens;
    uint32_t n_requests, n_rows, units, threads, per_request;      // units of a token; threads of a team, teams of a request
    const int32_t *cu, *rows;
    const int64_t *slots, *kept;
    int32_t *status;
    uint32_t checked;                                     // 1: one more block, the first, reports the errors
};

constexpr uint32_t kMoveThreads = 512, kMoveTeam = 256, kMoveDeep = 8;

// Entry i's places; false: nothing to move (bad: not as it should be).
__device__ __forceinline__ bool move_of(const MoveArgs &a, uint32_t i, int64_t *from, int64_t *to, bool *bad) {
    *to = __ldg(a.kept + i);
    const uint32_t row = (uint32_t)__ldg(a.rows + i);
    *from = -1;
    if (*to < 0) return false;
    if (row < a.n_rows) *from = __ldg(a.slots + row);
    const bool ok = (uint64_t)*to < a.pool_tokens && (uint64_t)*from < a.pool_tokens;
    *bad |= !ok;
    return ok && *from != *to;
}

__device__ __forceinline__ uint64_t byte_of(const MoveArgs &a, int64_t slot) {
    const uint64_t p = a.pool_tokens >> 31 ? (uint64_t)slot / a.page.d : div_by((uint32_t)slot, a.page);
    return p * a.page_stride + ((uint64_t)slot - p * a.page.d) * a.token_stride;
}

__device__ __forceinline__ bool move_rows_of(const MoveArgs &a, uint32_t r, uint32_t *lo, uint32_t *hi) {
    const int32_t x = __ldg(a.cu + r), y = __ldg(a.cu + r + 1);
    *lo = (uint32_t)x;
    *hi = (uint32_t)y;
    if (x >= 0 && y >= x && (uint32_t)y <= a.n_rows) return true;
    *lo = *hi = 0u;
    return false;
}

// A thread keeps one 16-byte column of K or V of a request's tokens and moves them in order, so that
// a place that is read before it is written over needs no barrier.
__global__ void __launch_bounds__(kMoveThreads) move_tokens_kernel(const MoveArgs a) {
    const uint32_t lane = threadIdx.x & 31u;
    bool bad = false;
    int64_t from, to;
    uint32_t lo, hi;
    if (a.checked && blockIdx.x == 0) {                       // the errors of every request, row by row
#pragma unroll 4
        for (uint32_t r = threadIdx.x; r < a.n_requests; r += kMoveThreads) bad |= !move_rows_of(a, r, &lo, &hi);
        bad = __syncthreads_or(bad);
        const uint32_t end = bad ? 0u : (uint32_t)__ldg(a.cu + a.n_requests);
#pragma unroll 1
        for (uint32_t i0 = (uint32_t)__ldg(a.cu) + threadIdx.x; i0 < end; i0 += 8u * kMoveThreads) {
            // loads of eight rounds in flight at once
            int64_t to_[8], from_[8];
            uint32_t row[8];
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) {
                const uint32_t i = i0 + k * kMoveThreads;
                to_[k] = i < end ? __ldg(a.kept + i) : -1;
                row[k] = i < end ? (uint32_t)__ldg(a.rows + i) : 0u;
            }
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) from_[k] = to_[k] >= 0 && row[k] < a.n_rows ? __ldg(a.slots + row[k]) : -1;
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) bad |= to_[k] >= 0 && ((uint64_t)to_[k] >= a.pool_tokens || (uint64_t)from_[k] >= a.pool_tokens);
        }
        bad = __syncthreads_or(bad);
        if (threadIdx.x == 0) *a.status = bad ? SKV_ERR_INVALID_ARG : SKV_OK;
        return;
    }
    const uint32_t in_block = threadIdx.x / a.threads, team = (blockIdx.x - a.checked) * (kMoveThreads / a.threads) + in_block;
    const uint32_t r = team / a.per_request;
    const uint32_t column = (team - r * a.per_request) * a.threads + threadIdx.x - in_block * a.threads;
    if (in_block >= kMoveThreads / a.threads || r >= a.n_requests) return;
    bad |= !move_rows_of(a, r, &lo, &hi);
    const bool on = column < 2u * a.units;
    const uint32_t u = column < a.units ? column : column - a.units, h = div_by(u, a.per_head);
    uint8_t *pool = (column < a.units ? a.k : a.v) + h * a.head_stride + 16u * (uint64_t)(u - h * a.per_head.d);
#pragma unroll 1
    for (uint32_t i0 = lo; i0 < hi; i0 += 32u) {
        const uint32_t i = i0 + lane;
        from = to = -1;
        const bool live = i < hi && move_of(a, i, &from, &to, &bad);
        uint32_t todo = __ballot_sync(~0u, live);
#pragma unroll 1
        while (todo) {
            // up to eight entries whose places are all read before any is written; fewer where one reads
            // what an entry before it writes
            uint64_t src[kMoveDeep], dst[kMoveDeep];
            int64_t wrote[kMoveDeep];
            uint32_t n = 0;
#pragma unroll
            for (uint32_t j = 0; j < kMoveDeep; ++j) {
                wrote[j] = -1;
                src[j] = dst[j] = 0;
                if (!todo || n < j) continue;
                const uint32_t l = __ffs(todo) - 1u;
                const int64_t x = __shfl_sync(~0u, from, l), y = __shfl_sync(~0u, to, l);
                bool after = false;
#pragma unroll
                for (uint32_t e = 0; e < j; ++e) after |= wrote[e] == x;
                if (after) continue;
                todo &= todo - 1u;
                wrote[j] = y;
                src[j] = byte_of(a, x);
                dst[j] = byte_of(a, y);
                n = j + 1u;
            }
            uint4 x[kMoveDeep];
#pragma unroll
            for (uint32_t j = 0; j < kMoveDeep; ++j)
                if (on && j < n) x[j] = *reinterpret_cast<const uint4 *>(pool + src[j]);
#pragma unroll
            for (uint32_t j = 0; j < kMoveDeep; ++j)
                if (on && j < n) *reinterpret_cast<uint4 *>(pool + dst[j]) = x[j];
        }
    }
    if (bad && !a.checked) set_first(a.status, SKV_ERR_INVALID_ARG);
}

template <void (*KERNEL)(PlanArgs), bool SMALL>
static bool launch_plan(const PlanArgs &a, cudaStream_t st) {
    // One CTA where a small table leaves little for more: a barrier of several costs more (8 rows of 17 pages 6.2 us with one,
    // 9.7 with 8; 700 rows of 48 27 and 11.5, before two rows went at a time).
    const uint64_t entries = (uint64_t)a.n_requests * a.max_pages;
    const uint32_t cluster = !SMALL ? kLargeCluster : entries <= 2048u ? 1u : kPlanCluster;
    static std::atomic<uint64_t> ready{0};
    if (!SMALL && !allow_cluster(reinterpret_cast<const void *>(KERNEL), ready)) return false;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(SMALL ? kPlanThreads : kLargeThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, KERNEL, a) == cudaSuccess;
}

static bool fits_small(uint32_t pool_pages, uint32_t n_requests, uint32_t max_pages) {
    return pool_pages <= kSmallPool && n_requests <= kSmallRows && max_pages <= (1u << 20);
}

static uint64_t bits_bytes(uint32_t pool_pages) { return ((uint64_t)pool_pages + 511u) / 512u * 64u; }

static uint64_t workspace_bytes(uint32_t n_requests, uint32_t pool_pages) {
    const uint64_t fork = 12ull * n_requests, compact = 8ull * pool_pages;
    return (2u * bits_bytes(pool_pages) + (fork > compact ? fork : compact) + 255u) & ~uint64_t(255);
}

static bool bad_sizes(uint32_t pool_pages, uint32_t n_requests, uint32_t max_pages, uint64_t stride, uint64_t out_stride,
                      uint32_t free_capacity) {
    return pool_pages == 0 || pool_pages > 0x7FFFFFFFu || n_requests > 0x7FFFFFFFu || max_pages > 0x7FFFFFFFu ||
           free_capacity > 0x7FFFFFFFu || (n_requests > 1 && (stride < max_pages || out_stride < max_pages));
}

}  // namespace skv

using namespace skv;

extern "C" int32_t skv_page_workspace_bytes(uint32_t n_requests, uint32_t pool_pages, uint64_t *bytes) {
    if (!bytes || pool_pages == 0 || pool_pages > 0x7FFFFFFFu || n_requests > 0x7FFFFFFFu) return SKV_ERR_INVALID_ARG;
    *bytes = workspace_bytes(n_requests, pool_pages);
    return SKV_OK;
}

extern "C" int32_t skv_page_fork(uint32_t page_tokens, uint32_t pool_pages, uint32_t n_requests, const int32_t *parents,
                                 const int32_t *ctx_len, const int32_t *block_table, uint64_t table_stride, uint32_t max_pages,
                                 const int32_t *n_pages_in, uint32_t trim, int32_t *table_out, uint64_t table_out_stride,
                                 int32_t *n_pages_out, int32_t *ctx_out, int32_t *free_pages, uint32_t free_capacity,
                                 const int32_t *free_in, int32_t *free_out, int32_t *copy_src, int32_t *copy_dst,
                                 int32_t *copy_tokens, int32_t *status, void *workspace, uint64_t ws_bytes, void *stream) {
    if (page_tokens == 0 || page_tokens > (1u << 20) || trim > 1u ||
        bad_sizes(pool_pages, n_requests, max_pages, table_stride, table_out_stride, free_capacity))
        return SKV_ERR_INVALID_ARG;
    if (!free_in || !free_out || !status || !workspace || (free_capacity && !free_pages) ||
        (n_requests && (!ctx_len || !block_table || !n_pages_in || !table_out || !n_pages_out || !ctx_out || !copy_src || !copy_dst ||
                        !copy_tokens)))
        return SKV_ERR_INVALID_ARG;
    const void *words[] = {parents, ctx_len, block_table, n_pages_in, table_out, n_pages_out, ctx_out, free_pages, free_in, free_out,
                           copy_src, copy_dst, copy_tokens, status};
    for (const void *p : words)
        if (!aligned(p, 4)) return SKV_ERR_INVALID_ARG;
    if (!aligned(workspace, 16) || ws_bytes < workspace_bytes(n_requests, pool_pages) || free_in == free_out ||
        (n_requests && (block_table == table_out || n_pages_in == n_pages_out || ctx_len == ctx_out)))
        return SKV_ERR_INVALID_ARG;
    // the lengths written over others than their own are the mistake at hand (every CTA reads them all)
    for (const int32_t *in : {parents, ctx_len, n_pages_in})
        if (in && n_requests && (in == n_pages_out || in == ctx_out)) return SKV_ERR_INVALID_ARG;
    PlanArgs a{};
    a.page = fast_div(page_tokens), a.pool_pages = pool_pages, a.n_requests = n_requests, a.max_pages = max_pages;
    a.free_capacity = free_capacity, a.trim = trim, a.capacity = n_requests;
    a.parents = parents, a.ctx_len = ctx_len, a.table = block_table, a.n_in = n_pages_in, a.free_in = free_in;
    a.table_stride = table_stride, a.out_stride = table_out_stride;
    a.table_out = table_out, a.n_out = n_pages_out, a.ctx_out = ctx_out, a.free_pages = free_pages, a.free_out = free_out;
    a.src = copy_src, a.dst = copy_dst, a.count = copy_tokens, a.status = status;
    a.bits = static_cast<uint32_t *>(workspace);
    a.now = a.bits + bits_bytes(pool_pages) / 4u;
    a.words = a.now + bits_bytes(pool_pages) / 4u;
    const bool small = fits_small(pool_pages, n_requests, max_pages);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return (small ? launch_plan<fork_small_kernel, true>(a, st) : launch_plan<fork_pages_kernel, false>(a, st)) ? SKV_OK : SKV_ERR_CUDA;
}

extern "C" int32_t skv_page_compact(uint32_t pool_pages, uint32_t n_requests, const int32_t *block_table, uint64_t table_stride,
                                    uint32_t max_pages, const int32_t *n_pages, int32_t *table_out, uint64_t table_out_stride,
                                    int32_t *free_pages, uint32_t free_capacity, const int32_t *free_in, int32_t *free_out,
                                    int32_t *copy_src, int32_t *copy_dst, uint32_t copy_capacity, int32_t *status, void *workspace,
                                    uint64_t ws_bytes, void *stream) {
    if (bad_sizes(pool_pages, n_requests, max_pages, table_stride, table_out_stride, free_capacity) || copy_capacity > 0x7FFFFFFFu)
        return SKV_ERR_INVALID_ARG;
    if (!free_in || !free_out || !status || !workspace || (free_capacity && !free_pages) || (copy_capacity && (!copy_src || !copy_dst)) ||
        (n_requests && (!block_table || !n_pages || !table_out)))
        return SKV_ERR_INVALID_ARG;
    const void *words[] = {block_table, n_pages, table_out, free_pages, free_in, free_out, copy_src, copy_dst, status};
    for (const void *p : words)
        if (!aligned(p, 4)) return SKV_ERR_INVALID_ARG;
    if (!aligned(workspace, 16) || ws_bytes < workspace_bytes(n_requests, pool_pages) || free_in == free_out ||
        (n_requests && block_table == table_out))
        return SKV_ERR_INVALID_ARG;
    PlanArgs a{};
    a.pool_pages = pool_pages, a.n_requests = n_requests, a.max_pages = max_pages;
    a.free_capacity = free_capacity, a.capacity = copy_capacity;
    a.table = block_table, a.n_in = n_pages, a.free_in = free_in;
    a.table_stride = table_stride, a.out_stride = table_out_stride;
    a.table_out = table_out, a.free_pages = free_pages, a.free_out = free_out, a.src = copy_src, a.dst = copy_dst, a.status = status;
    a.bits = static_cast<uint32_t *>(workspace);
    a.now = a.bits + bits_bytes(pool_pages) / 4u;
    a.words = a.now + bits_bytes(pool_pages) / 4u;
    const bool small = fits_small(pool_pages, n_requests, max_pages);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return (small ? launch_plan<compact_small_kernel, true>(a, st) : launch_plan<compact_pages_kernel, false>(a, st)) ? SKV_OK : SKV_ERR_CUDA;
}

extern "C" int32_t skv_cache_copy(const skv_paged *cache, const int32_t *src, const int32_t *dst, const int32_t *tokens, uint32_t n,
                                  int32_t *status, void *stream) {
    const int32_t rc = skv_paged_check(cache);
    if (rc != SKV_OK) return rc;
    if (!status || !aligned(status, 4) || n > 0x7FFFFFFFu || (n && (!src || !dst)) || !aligned(src, 4) || !aligned(dst, 4) ||
        !aligned(tokens, 4))
        return SKV_ERR_INVALID_ARG;
    const PagedView c = paged_view(*cache);
    const uint32_t per_head = cache->head_dim / (c.e4m3 ? 16u : 8u);
    const uint64_t per_page = (uint64_t)cache->page_tokens * cache->n_heads * per_head;
    if (per_page > 0x7FFFFFFFu - kCopyUnits) return SKV_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (n == 0) return cudaMemsetAsync(status, 0, sizeof(int32_t), st) == cudaSuccess ? SKV_OK : SKV_ERR_CUDA;
    uint32_t sms = 0;
    if (!device_sms(&sms)) return SKV_ERR_CUDA;
    CopyArgs a{static_cast<uint8_t *>(cache->k_pages), static_cast<uint8_t *>(cache->v_pages), c.page_stride, c.token_stride, c.head_stride,
               cache->page_tokens, cache->n_pages, n, (uint32_t)((per_page + kCopyUnits - 1) / kCopyUnits), {}, fast_div(cache->n_heads * per_head),
               fast_div(per_head), src, dst, tokens, status, 0u};
    // One block reports the errors (it writes the status once; clearing it first is a launch of its own): beside its copies up to 512
    // pairs, as all it does up to 16,384. Pairs of which none, or half, are copied (pages of 4 KB), with the launch and so: 2,000 pairs 6.3 and 3.4,
    // 8.3 and 4.8 us; 16,000 6.8 and 5.7, 28.7 and 24.6; but 32,000 7.4 and 7.9, 65,536 8.4 and 12.4 where none is.
    a.checked = n <= 512u ? 1u : n <= 16384u ? 2u : 0u;
    a.by_chunks = fast_div(a.chunks);
    if (!a.checked && cudaMemsetAsync(status, 0, sizeof(int32_t), st) != cudaSuccess) return SKV_ERR_CUDA;
    const uint64_t items = (uint64_t)n * a.chunks + (a.checked == 2u);
    const unsigned grid = (unsigned)(items < 16u * sms ? items : 16u * sms);
    copy_pages_kernel<<<grid, kCopyThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? SKV_OK : SKV_ERR_CUDA;
}

extern "C" int32_t skv_cache_move(const skv_paged *cache, uint32_t n_requests, const int32_t *cu_new, uint32_t n_rows,
                                  const int32_t *rows, const int64_t *slots, const int64_t *kept, int32_t *status, void *stream) {
    const int32_t rc = skv_paged_check(cache);
    if (rc != SKV_OK) return rc;
    if (!status || !aligned(status, 4) || n_rows > 0x7FFFFFFFu || (n_requests && !cu_new) || !aligned(cu_new, 4) || !aligned(rows, 4) ||
        !aligned(slots, 8) || !aligned(kept, 8) || (n_rows && (!rows || !slots || !kept)))
        return SKV_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (n_requests == 0) return cudaMemsetAsync(status, 0, sizeof(int32_t), st) == cudaSuccess ? SKV_OK : SKV_ERR_CUDA;
    const PagedView c = paged_view(*cache);
    const uint32_t per_head = cache->head_dim / (c.e4m3 ? 16u : 8u), units = cache->n_heads * per_head;
    const uint32_t threads = 2u * units < kMoveTeam ? (2u * units + 31u) & ~31u : kMoveTeam;
    const uint32_t per_request = (2u * units + threads - 1u) / threads;
    if ((uint64_t)n_requests * per_request >= 0x7FFFFFFFu) return SKV_ERR_INVALID_ARG;
    MoveArgs a{static_cast<uint8_t *>(cache->k_pages), static_cast<uint8_t *>(cache->v_pages), c.page_stride, c.token_stride, c.head_stride,
               c.page, fast_div(per_head), (uint64_t)cache->n_pages * cache->page_tokens, n_requests, n_rows, units, threads, per_request, cu_new, rows,
               slots, kept, status, n_rows <= 16384u && n_requests <= 16384u};
    // (One block looks through up to 16,384 entries for errors; beyond, a launch clears the status. With the launch and with the
    // block: 8 requests of 16 nodes 6.3 and 3.9 us, 256 of 60 10.5 and 7.7, 1,000 of 16 6.4 and 6.4, 1,000 of 30 6.8 and 9.8, 1,000 of 60 7.2 and 15.3.)
    if (!a.checked && cudaMemsetAsync(status, 0, sizeof(int32_t), st) != cudaSuccess) return SKV_ERR_CUDA;
    const uint32_t teams = kMoveThreads / threads, blocks = (n_requests * per_request + teams - 1u) / teams;
    move_tokens_kernel<<<blocks + a.checked, kMoveThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? SKV_OK : SKV_ERR_CUDA;
}
