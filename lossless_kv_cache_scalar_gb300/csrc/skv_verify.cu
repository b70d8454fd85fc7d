// skv_verify.cu -- verification of drafted trees.
//
// A cluster of CTAs takes a request. Every warp walks the tree for itself, from the same few scalars (the
// probabilities of the drafted tokens, all gathered at once before the walk): nothing has to be
// passed on. Only a sum over the vocabulary is shared: each warp sums its range of the row as whole numbers of
// 2^-44, so that no order of adding matters, and hands the sum to every CTA through distributed
// shared memory. The warp in whose range the drawn number falls finds the token.
//
// Rows come by asynchronous copies into shared memory, all that it holds of a CTA's part on its way at once: a further sum over
// the same node, after another rejection, reads only what did not fit.
//
// Bound by latency: a chain of 5 nodes over 151,936 tokens takes 7.3 us on the device (launch and end 2.5, then scalars, tests, row, sum,
// the cluster's barrier and the token's search, 0.5 to 1 us each), 24 trees of 27 nodes over 50,257 tokens without draft probabilities 9.4;
// 64 trees of up to 60 nodes over 151,936 tokens 55: a request takes 2.7 sums on average, 6 at most, one after the other, with 8 CTAs to each,
// whose parts of the two rows (152 KB) fit shared memory by a third (HBM would bring the rows in 11.5).
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <atomic>

#include "skv_rows.cuh"

namespace skv {

namespace cg = cooperative_groups;

bool raise_smem(const void *kernel, uint32_t bytes, std::atomic<uint64_t> &ready);      // skv_attend.cu

constexpr uint32_t kNodes = 256;                 // nodes of a request that are gathered at once
constexpr uint32_t kGone = 4096;                 // nodes of a request without draft probabilities
constexpr uint32_t kVerifyCluster = 16;
// Threads of a CTA, 1,024 of an SM's: many requests with draft probabilities wait for the sums of the longest chains, and those
// end sooner on more SMs (64 requests of 30 nodes over 151,936 tokens: 38 us with 256, 46 with 512); without draft
// probabilities more of the only row is under way in larger ones (40 requests over 151,936 tokens: 16 us with 512, 18 with 256).
template <bool DRAFT>
constexpr uint32_t kThreads = DRAFT ? 256u : 512u;
template <bool DRAFT>
constexpr uint32_t kRowBytes = (DRAFT ? 46u : 80u) * 1024u;      // shared memory for rows
constexpr uint32_t kPieces = 16;                 // of a CTA's part without draft probabilities
constexpr uint32_t most_part(uint32_t threads) { return 512u * threads; }      // elements: 512 to a lane

struct VerifyArgs {
    const void *probs, *draft;
    uint64_t probs_stride, draft_stride;         // elements
    uint32_t vocab, distinct, n_rows, n_requests;
    const int32_t *cu, *tokens, *parents;
    const float *uniform;
    const int64_t *slots;
    const int32_t *ctx_len;
    int32_t *accepted, *rows;
    int64_t *kept;
    int32_t *ctx_out, *next, *status;
    uint32_t checked;                            // 1: a cluster behind the requests' reports the errors
    uint32_t per_cta, per_held, per_warp, per_warp_far;      // elements: of a CTA's part, of what it holds of it, of a warp's
                                                             // run of that and of the rest
};

// A probability as it counts: the nearer end outside [0, 1], NaN as 0 (what saturation does).
__device__ __forceinline__ float prob(float x) { return __saturatef(x); }
__device__ __forceinline__ float prob(uint16_t x) { return __saturatef(__uint_as_float((uint32_t)x << 16)); }

// Elements [e0, e0 + m) of a row of `vocab` into dst, by the CTA: whole 16-byte units, asynchronously, from the one that e0 lies
// in on (so that it comes to lie at dst[place_in_unit]); the row's first and last unit element by element where they
// are not all the row's.
template <typename T>
__device__ __forceinline__ uint32_t place_in_unit(const T *p) { return (uint32_t)((uintptr_t)p & 15u) / (uint32_t)sizeof(T); }
template <typename T>
__device__ __forceinline__ void fetch_run(T *dst, const T *row, uint32_t vocab, uint32_t e0, uint32_t m) {
    constexpr uint32_t V = 16u / sizeof(T);
    const uint32_t at = place_in_unit(row + e0), units = m ? (at + m + V - 1u) / V : 0u;
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
    for (uint32_t i = threadIdx.x; i < units; i += blockDim.x) {
        const int32_t e = (int32_t)(e0 + i * V) - (int32_t)at;
        if (e >= 0 && (uint32_t)e + V <= vocab) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 16u * i), "l"(row + e) : "memory");
        } else {
            for (int32_t j = 0; j < (int32_t)V; ++j)
                if (e + j >= 0 && (uint32_t)(e + j) < vocab) dst[i * V + j] = __ldg(row + e + j);
        }
    }
}

// R(y) = max(p - c q, 0), in [0, 1] like p.
__device__ __forceinline__ float rest_of(float p, float q, float c) {
    float r;
    asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(-c), "f"(q), "f"(p));
    return r;
}

// Sums of numbers of [0, 1] in units of 2^-44, each rounded to one, ties to even, without a conversion (a quarter
// of the rate of an addition at best): r + 3 is r rounded to 2^-22, in the low bits of its word; what that
// leaves, at most 2^-23 and exact, added to 1.5 2^-21 is rounded to 2^-44. The two words are summed by
// themselves, modulo 2^32: up to 512 numbers, of at most 2^22 and 2^21 units beyond the constants, leave no doubt.
constexpr uint32_t kHigh = 0x40400000u, kLow = 0x35400000u;          // 3 and 1.5 2^-21
struct Units {
    uint32_t high, low;
};
__device__ __forceinline__ void add_units(Units &u, float r) {
    const float t = r + __uint_as_float(kHigh), rest = r - (t - __uint_as_float(kHigh));
    u.high += __float_as_uint(t) - kHigh;
    u.low += __float_as_uint(rest + __uint_as_float(kLow)) - kLow;
}
__device__ __forceinline__ unsigned long long total_of(uint64_t high, int64_t low) { return (high << 22) + (unsigned long long)low; }
__device__ __forceinline__ unsigned long long units_of_prob(float r) {
    Units u{0u, 0u};
    add_units(u, r);
    return total_of(u.high, (int32_t)u.low);
}
// The warp's sum of up to 512 numbers per lane (high below 2^31, low of either sign): in pieces that
// a 32-bit reduction holds.
__device__ __forceinline__ unsigned long long warp_total(const Units &u) {
    const uint32_t a = __reduce_add_sync(~0u, u.high >> 16), b = __reduce_add_sync(~0u, u.high & 0xFFFFu);
    const int32_t c = __reduce_add_sync(~0u, (int32_t)u.low >> 16);
    const uint32_t d = __reduce_add_sync(~0u, u.low & 0xFFFFu);
    return total_of(((uint64_t)a << 16) + b, ((int64_t)c << 16) + d);
}

// In pieces of 24 bits, which 32-bit reductions hold.
__device__ __forceinline__ unsigned long long sum_of_warp(unsigned long long x) {
    const uint32_t lo = __reduce_add_sync(~0u, (uint32_t)x & 0xFFFFFFu), mid = __reduce_add_sync(~0u, (uint32_t)(x >> 24) & 0xFFFFFFu);
    const uint32_t hi = __reduce_add_sync(~0u, (uint32_t)(x >> 48));
    return lo + ((unsigned long long)mid << 24) + ((unsigned long long)hi << 48);
}
__device__ __forceinline__ unsigned long long prefix_of_warp(unsigned long long x) {
#pragma unroll
    for (uint32_t d = 1; d < 32; d <<= 1) {
        const unsigned long long y = __shfl_up_sync(~0u, x, d);
        if ((threadIdx.x & 31u) >= d) x += y;
    }
    return x;
}

// A node's token, its u, and the token's probabilities at the parent. The sign of u tells whether the token is
// accepted as the first of its siblings to be tried.
struct __align__(16) Node {
    int32_t token;
    float u, p, q;
};

// Whether a request's lengths are in order; its rows.
__device__ __forceinline__ bool rows_of(const VerifyArgs &a, uint32_t r, uint32_t *row0, uint32_t *n) {
    const int32_t lo = __ldg(a.cu + r), hi = __ldg(a.cu + r + 1);
    *row0 = (uint32_t)lo;
    *n = 0;
    if (lo < 0 || hi < lo || (uint32_t)hi > a.n_rows) return false;
    *n = (uint32_t)(hi - lo);
    return a.draft || *n <= kGone;
}

__device__ __forceinline__ int32_t parent_of(const VerifyArgs &a, uint32_t row0, uint32_t i) {
    return a.parents ? __ldg(a.parents + row0 + i) : (int32_t)i - 1;
}

// Node i > 0 of a request has a token and a parent in their ranges.
__device__ __forceinline__ bool node_ok(const VerifyArgs &a, int32_t parent, int32_t token, uint32_t i) {
    return (uint32_t)token < a.vocab && (uint32_t)parent < i;
}

// u q Z < r s, with Z in units of 2^-44 and the products in binary64. Those take a warp most of a microsecond a test, so
// binary32 decides where it can: each of its products is off by 2^-21 at most where it is not tiny.
__device__ __forceinline__ int decided(float left, float right) {
    if (fmaxf(left, right) > 0x1p-90f) {
        if (left < right * (1.0f - 0x1p-20f)) return 1;
        if (left * (1.0f - 0x1p-20f) > right) return 0;
    }
    return -1;
}
// `whole`: s is 1.
__device__ __forceinline__ bool below(float u, float q, unsigned long long Z, float r, bool whole, double s) {
    const int d = decided(u * q * (__ull2float_rn(Z) * 0x1p-44f), whole ? r : r * (float)s);
    return d >= 0 ? d : (double)u * (double)q * ((double)Z * 0x1p-44) < (double)r * s;
}
// u Z < r
__device__ __forceinline__ bool below(float u, double Z, float r) {
    const int d = decided(u * (float)Z, r);
    return d >= 0 ? d : (double)u * Z < (double)r;
}

template <typename T, bool DRAFT>
__global__ void __launch_bounds__(kThreads<DRAFT>, 1024u / kThreads<DRAFT>) verify_kernel(const VerifyArgs a) {
    constexpr uint32_t kVerifyThreads = kThreads<DRAFT>, kVerifyWarps = kVerifyThreads / 32u;
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t C = cluster.num_blocks(), rank = cluster.block_rank();
    const uint32_t request = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    __shared__ Node node[kNodes];
    __shared__ int32_t parent[kNodes];
    extern __shared__ uint4 row_memory[];
    __shared__ unsigned long long sums[2][kVerifyCluster * kVerifyWarps];      // of every warp of the cluster
    __shared__ unsigned long long run_sum[(DRAFT ? 2u : kPieces) * kVerifyWarps];      // of this CTA's runs, in order
    __shared__ int32_t gone[DRAFT ? 1 : kGone];  // rejected tokens of the node (no draft probabilities)
    __shared__ struct {
        uint32_t cur, taken, n_gone;
    } walk;

    if (request == a.n_requests) {               // the errors of every request, row by row
        if (rank) return;
        int32_t *cu = reinterpret_cast<int32_t *>(node);
        for (uint32_t r = tid; r <= a.n_requests; r += kVerifyThreads) cu[r] = __ldg(a.cu + r);
        __syncthreads();
        bool bad = false;
        for (uint32_t r = tid; r < a.n_requests; r += kVerifyThreads) {
            const int32_t lo = cu[r], hi = cu[r + 1u];
            bad |= lo < 0 || hi < lo || (uint32_t)hi > a.n_rows || (!DRAFT && (uint32_t)(hi - lo) > kGone);
        }
        bad = __syncthreads_or(bad);
        const uint32_t end = bad ? 0u : (uint32_t)cu[a.n_requests];
        for (uint32_t i = (uint32_t)cu[0] + tid; i < end; i += kVerifyThreads) {
            uint32_t r = 0, m = a.n_requests;                             // last request with cu <= i
            while (m > 1u) {
                const uint32_t h = m >> 1;
                if ((uint32_t)cu[r + h] <= i) r += h;
                m -= h;
            }
            const uint32_t row = (uint32_t)cu[r], j = i - row;
            if (j) bad |= !node_ok(a, parent_of(a, row, j), __ldg(a.tokens + i), j);
        }
        bad = __syncthreads_or(bad);
        if (tid == 0) *a.status = bad ? SKV_ERR_INVALID_ARG : SKV_OK;
        return;
    }
    uint32_t row0, n;
    const bool in_order = rows_of(a, request, &row0, &n);
    bool bad = !in_order;
    const T *P = static_cast<const T *>(a.probs) + (uint64_t)row0 * a.probs_stride;
    const T *Q = DRAFT ? static_cast<const T *>(a.draft) + (uint64_t)row0 * a.draft_stride : nullptr;

    // The scalars of nodes [first, first + kNodes), by `threads` threads.
    const auto gather = [&](uint32_t first, uint32_t mine, uint32_t threads) {
        for (uint32_t i = first + mine; i < min(n, first + kNodes); i += threads) {
            Node x{0, __saturatef(__ldg(a.uniform + row0 + i)), 0.0f, 0.0f};
            int32_t up = -1;
            if (i) {
                up = parent_of(a, row0, i);
                x.token = __ldg(a.tokens + row0 + i);
                if (node_ok(a, up, x.token, i)) {
                    x.p = prob(__ldg(P + (uint64_t)up * a.probs_stride + x.token));
                    if (DRAFT) x.q = prob(__ldg(Q + (uint64_t)up * a.draft_stride + x.token));
                    if (DRAFT ? below(x.u, x.q, 1ull << 44, x.p, true, 1.0) : x.u < x.p) x.u = -x.u;
                    else x.u = fabsf(x.u);
                } else {
                    bad = true;
                }
            }
            parent[i - first] = up;
            node[i - first] = x;
        }
    };
    gather(0, tid, kVerifyThreads);
#pragma unroll 1
    for (uint32_t i = kNodes + tid; i < n; i += kVerifyThreads)
        bad |= !node_ok(a, parent_of(a, row0, i), __ldg(a.tokens + row0 + i), i);
    bad = __syncthreads_or(bad);                 // the same in every CTA of the cluster
    if (bad || n == 0) {
        if (rank == 0) {
            if (tid == 0) {
                a.accepted[request] = 0;
                a.next[request] = -1;
                if (a.ctx_out) a.ctx_out[request] = __ldg(a.ctx_len + request);
                if (bad && !a.checked) set_first(a.status, SKV_ERR_INVALID_ARG);
            }
            for (uint32_t i = tid; i < n; i += kVerifyThreads) {
                a.rows[row0 + i] = -1;
                if (a.kept) a.kept[row0 + i] = -1;
            }
        }
        return;
    }
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");      // waited for before the first sum
    bool started = false;
    // (not from node[0]: the walking warp may be at later nodes, which take its place, before every warp has read it)
    const float u0 = __saturatef(__ldg(a.uniform + row0));

    // A part of the vocabulary per CTA, of which shared memory holds a piece. With draft probabilities the rest is read
    // anew for each sum; without them the only sum passes through shared memory piece by piece. A run per warp
    // of each piece, and of the rest.
    const uint32_t first = min(rank * a.per_cta, a.vocab), last = min(first + a.per_cta, a.vocab);
    const uint32_t m = min(a.per_held, last - first), far0 = first + m;
    const uint32_t pieces = DRAFT ? 1u : (a.per_cta + a.per_held - 1u) / a.per_held;
    T *const sp = reinterpret_cast<T *>(row_memory), *const sq = sp + a.per_held + 32u / sizeof(T);
    uint32_t parity = 0, n_gone = 0;
    uint32_t held = ~0u;                         // whose rows, both, shared memory holds

    struct Run {
        const T *p, *q;
        uint32_t n, e0;                          // its length, and its first element
    };
    // This warp's run of the piece of `here` elements from e0 on that shared memory holds, and of the rest.
    const auto held_run = [&](uint32_t cur, uint32_t e0, uint32_t here) {
        const uint32_t r0 = min(warp * a.per_warp, here);
        Run r{sp + place_in_unit(P + (uint64_t)cur * a.probs_stride + e0) + r0, nullptr, min(a.per_warp, here - r0), e0 + r0};
        if (DRAFT) r.q = sq + place_in_unit(Q + (uint64_t)cur * a.draft_stride + e0) + r0;
        return r;
    };
    const auto far_run = [&](uint32_t cur) {
        const uint32_t r0 = min(warp * a.per_warp_far, last - far0);
        Run r{P + (uint64_t)cur * a.probs_stride + far0 + r0, nullptr, min(a.per_warp_far, last - far0 - r0), far0 + r0};
        if (DRAFT) r.q = Q + (uint64_t)cur * a.draft_stride + far0 + r0;
        return r;
    };
    // Every copy is in; without draft probabilities rejected tokens weigh nothing.
    const auto arrive = [&](uint32_t cur, uint32_t e0, uint32_t here) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        if (!DRAFT && n_gone) {
            T *p = sp + place_in_unit(P + (uint64_t)cur * a.probs_stride + e0);
            for (uint32_t g = tid; g < n_gone; g += kVerifyThreads)
                if ((uint32_t)gone[g] - e0 < here) p[(uint32_t)gone[g] - e0] = T(0);
            __syncthreads();
        }
    };
    // The warp's sum of R over its run of the rest, from global memory: up to 16 loads of a lane on their way.
    const auto sum_far = [&](const Run &r, float c) {
        Units u{0u, 0u};
        if (c != 0.0f) {
#pragma unroll 1
            for (uint32_t i0 = lane; i0 < r.n; i0 += 256u) {
                T x[8], y[8];
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) {
                    const bool in = i0 + 32u * j < r.n;
                    x[j] = in ? r.p[i0 + 32u * j] : T(0);
                    y[j] = in ? r.q[i0 + 32u * j] : T(0);
                }
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) add_units(u, rest_of(prob(x[j]), prob(y[j]), c));
            }
        } else {
#pragma unroll 1
            for (uint32_t i0 = lane; i0 < r.n; i0 += 512u) {
                T x[16];
#pragma unroll
                for (uint32_t j = 0; j < 16; ++j) x[j] = i0 + 32u * j < r.n ? r.p[i0 + 32u * j] : T(0);
#pragma unroll
                for (uint32_t j = 0; j < 16; ++j) add_units(u, prob(x[j]));
            }
        }
        return warp_total(u);
    };
    // Sum of R over the row of `cur`; every warp's own is in sums[parity ^ 1] then, of this CTA's runs in run_sum.
    const auto sum_row = [&](uint32_t cur, float c) -> unsigned long long {
        const bool both = DRAFT && c != 0.0f, reload = held != cur;
        unsigned long long sum = 0;
#pragma unroll 1
        for (uint32_t k = 0; k < pieces; ++k) {
            const uint32_t e0 = min(first + k * a.per_held, last), here = min(a.per_held, last - e0);
            if (reload) {
                __syncthreads();                 // what was here is read
                fetch_run(sp, P + (uint64_t)cur * a.probs_stride, a.vocab, e0, here);
                if (both) fetch_run(sq, Q + (uint64_t)cur * a.draft_stride, a.vocab, e0, here);
            }
            if (DRAFT) {
                unsigned long long far = 0;
                if (a.per_warp_far) far = sum_far(far_run(cur), c);
                if (lane == 0) run_sum[kVerifyWarps + warp] = far;
                sum += far;
            }
            if (reload) arrive(cur, e0, here);
            const Run r = held_run(cur, e0, here);
            Units u{0u, 0u};
            if (both) {
#pragma unroll 4
                for (uint32_t i = lane; i < r.n; i += 32u) add_units(u, rest_of(prob(r.p[i]), prob(r.q[i]), c));
            } else {
#pragma unroll 8
                for (uint32_t i = lane; i < r.n; i += 32u) add_units(u, prob(r.p[i]));
            }
            const unsigned long long near = warp_total(u);
            if (lane == 0) run_sum[k * kVerifyWarps + warp] = near;
            sum += near;
        }
        held = both ? cur : ~0u;
        if (!started) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        started = true;
        if (lane < C) *cluster.map_shared_rank(&sums[parity][rank * kVerifyWarps + warp], lane) = sum;
        cluster.sync();
        unsigned long long whole = 0;
#pragma unroll
        for (uint32_t j = 0; j < kVerifyCluster * kVerifyWarps / 32u; ++j)
            if (32u * j + lane < C * kVerifyWarps) whole += sums[parity][32u * j + lane];
        parity ^= 1u;
        return sum_of_warp(whole);
    };

    // The walk, the same in every warp of the cluster (without draft probabilities one warp's, for the others of its CTA).
    uint32_t batch = 0, at = 1, cur = 0, taken = 1;      // batch: first node in shared memory
    float c = 0.0f;
    unsigned long long total = 0;
    bool fresh = false;                          // total and the sums are those of (cur, c)
    double Z = 1.0, s = 1.0;                     // Z: without draft probabilities
    bool whole = true;                           // s is 1 (a warp's test of it in binary64 costs a hundred clocks)
    if (rank == 0 && tid == 0) a.rows[row0] = (int32_t)row0;
#pragma unroll 1
    while (DRAFT || warp == 0) {
        // the next child
        const uint32_t end = min(n, batch + kNodes);
        uint32_t found = end;
#pragma unroll 1
        for (uint32_t b = at; b < end; b += 32u) {
            const uint32_t i = b + lane;
            const uint32_t m = __ballot_sync(~0u, i < end && parent[i - batch] == (int32_t)cur);
            if (m) {
                found = b + __ffs(m) - 1u;
                break;
            }
        }
        at = found;
        if (found == end) {
            if (end == n) break;
            batch += kNodes;
            if (DRAFT) {
                __syncthreads();
                gather(batch, tid, kVerifyThreads);
                __syncthreads();
            } else {
                __syncwarp();
                gather(batch, lane, 32u);
                __syncwarp();
            }
            continue;
        }
        const Node x = node[found - batch];
        bool take;
        if (DRAFT) {
            if (c != 0.0f && !fresh) {
                total = sum_row(cur, c);
                fresh = true;
            }
            take = c == 0.0f ? signbit(x.u) : below(fabsf(x.u), x.q, total, rest_of(x.p, x.q, c), whole, s);
            if (!take) {
                // c + Z / s: c and Z are whole numbers of 2^-44 (c is 0, or from 1 on)
                float to = c;
                if (whole && c < 0x1p18f) to = __ull2float_rn((unsigned long long)(c * 0x1p44f) + (c == 0.0f ? 1ull << 44 : total)) * 0x1p-44f;
                else if (s > 0.0) to = (float)((double)c + (c == 0.0f ? 1.0 : (double)total * 0x1p-44) / s);
                fresh = fresh && to == c;
                c = to;
                if (a.distinct) {
                    s = fmax(s - (double)x.q, 0.0);
                    whole = false;
                }
            }
        } else {
            bool again = false;
            for (uint32_t j = lane; j < n_gone; j += 32u) again |= gone[j] == x.token;
            again = __any_sync(~0u, again);
            const float r = again ? 0.0f : x.p;
            take = n_gone ? below(fabsf(x.u), Z, r) : signbit(x.u);
            if (!take && !again) {
                Z = fmax(Z - (double)r, 0.0);
                if (lane == 0) gone[n_gone] = x.token;
                ++n_gone;
                __syncwarp();
            }
        }
        if (take) {
            if (rank == 0 && tid == 0) a.rows[row0 + taken] = (int32_t)(row0 + found);
            ++taken;
            cur = found;
            c = 0.0f, Z = 1.0, s = 1.0, whole = true, n_gone = 0, fresh = false;
        }
        at = found + 1u;
    }
    if (!DRAFT) {
        if (tid == 0) walk = {cur, taken, n_gone};
        __syncthreads();
        cur = walk.cur, taken = walk.taken, n_gone = walk.n_gone;
    }
    if (!fresh) total = sum_row(cur, c);
    if (total == 0ull && (c != 0.0f || n_gone)) {                 // nothing left of the target: its own row
        c = 0.0f, n_gone = 0;
        held = ~0u;
        total = sum_row(cur, c);
    }

    // The drawn number: floor(u total). The CTA in whose part it falls finds the warp's run, the warp the element.
    const float u = u0 > 0.0f ? fminf(u0, 0x1.fffffep-1f) : 0.0f;
    unsigned long long left = min((unsigned long long)__double2ull_rd((double)u * (double)total), total ? total - 1ull : 0ull);
    const unsigned long long *all = sums[parity ^ 1u];
    unsigned long long before = 0;
    for (uint32_t j = lane; j < rank * kVerifyWarps; j += 32u) before += all[j];
    before = sum_of_warp(before);
    const unsigned long long mine = sum_of_warp(lane < kVerifyWarps ? all[rank * kVerifyWarps + lane] : 0ull);
    if (total && left >= before && left - before < mine) {
        left -= before;
        // the run, of this CTA's in order
        const uint32_t runs = (DRAFT ? 2u : pieces) * kVerifyWarps;
        uint32_t e = 0;
        unsigned long long x, upto;
        while (true) {
            x = e + lane < runs ? run_sum[e + lane] : 0ull;
            upto = prefix_of_warp(x);
            const uint32_t in = __ballot_sync(~0u, left >= upto - x && left < upto);
            if (in) {
                const uint32_t l = __ffs(in) - 1u;
                left -= __shfl_sync(~0u, upto - x, l);
                e += l;
                break;
            }
            left -= __shfl_sync(~0u, upto, 31);
            e += 32u;
        }
        const uint32_t k = DRAFT ? 0u : e / kVerifyWarps, e0 = min(first + k * a.per_held, last), here = min(a.per_held, last - e0);
        if (k + 1u < pieces) {                   // (the last piece is there)
            __syncthreads();
            fetch_run(sp, P + (uint64_t)cur * a.probs_stride, a.vocab, e0, here);
            arrive(cur, e0, here);
        }
        if (warp == e % kVerifyWarps) {
            const Run r = DRAFT && e >= kVerifyWarps ? far_run(cur) : held_run(cur, e0, here);
            const auto rest = [&](uint32_t i) { return DRAFT ? rest_of(prob(r.p[i]), c != 0.0f ? prob(r.q[i]) : 0.0f, c) : prob(r.p[i]); };
            // stretches of it, one per lane, until a lane has one element
            uint32_t from = 0, n = r.n;
            while (n > 32u) {
                const uint32_t each = (n + 31u) / 32u;
                Units u{0u, 0u};
                for (uint32_t i = min(lane * each, n); i < min((lane + 1u) * each, n); ++i) add_units(u, rest(from + i));
                x = total_of(u.high, (int32_t)u.low);
                upto = prefix_of_warp(x);
                const uint32_t l = __ffs(__ballot_sync(~0u, left >= upto - x && left < upto)) - 1u;
                left -= __shfl_sync(~0u, upto - x, l);
                from += l * each;
                n = min(each, n - l * each);
            }
            x = lane < n ? units_of_prob(rest(from + lane)) : 0ull;
            upto = prefix_of_warp(x);
            if (left >= upto - x && left < upto) a.next[request] = (int32_t)(r.e0 + from + lane);
        }
    }
    if (rank == 0) {
        if (tid == 0) {
            a.accepted[request] = (int32_t)taken;
            if (!total) a.next[request] = -1;
            if (a.ctx_out) a.ctx_out[request] = __ldg(a.ctx_len + request) + (int32_t)taken;
        }
        for (uint32_t i = tid; i < n; i += kVerifyThreads) {
            if (i >= taken) a.rows[row0 + i] = -1;
            if (a.kept) a.kept[row0 + i] = i < taken ? __ldg(a.slots + row0 + i) : -1;
        }
    }
}

template <typename T, bool DRAFT>
static bool launch_verify(const VerifyArgs &a, uint32_t cluster, uint32_t bytes, cudaStream_t st) {
    static std::atomic<uint64_t> ready{0}, large{0};
    if (!allow_cluster(reinterpret_cast<const void *>(verify_kernel<T, DRAFT>), ready) ||
        !raise_smem(reinterpret_cast<const void *>(verify_kernel<T, DRAFT>), kRowBytes<DRAFT>, large))
        return false;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.n_requests + a.checked) * cluster);
    cfg.blockDim = dim3(kThreads<DRAFT>);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_kernel<T, DRAFT>, a) == cudaSuccess;
}

}  // namespace skv

using namespace skv;

extern "C" int32_t skv_tree_verify(uint32_t dtype, const void *probs, uint64_t probs_stride, const void *draft_probs,
                                   uint64_t draft_stride, uint32_t vocab, uint32_t distinct, uint32_t n_rows, uint32_t n_requests,
                                   const int32_t *cu_new, const int32_t *tokens, const int32_t *parents, const float *uniform,
                                   const int64_t *slots, const int32_t *ctx_len, int32_t *accepted, int32_t *rows, int64_t *kept,
                                   int32_t *ctx_out, int32_t *next, int32_t *status, void *stream) {
    const uint64_t most = uint64_t(1) << 40;
    const uint32_t size = dtype == SKV_PROB_F32 ? 4u : 2u;
    if ((dtype != SKV_PROB_F32 && dtype != SKV_PROB_BF16) || vocab == 0 || vocab > (1u << 19) || distinct > 1u ||
        n_rows > 0x7FFFFFFFu || n_requests > (1u << 26) || probs_stride > most || draft_stride > most ||
        (n_rows > 1 && (probs_stride < vocab || (draft_probs && draft_stride < vocab))))
        return SKV_ERR_INVALID_ARG;
    if (!status || !cu_new || (n_requests && (!accepted || !next)) || (n_rows && (!probs || !tokens || !uniform || !rows)) ||
        (slots == nullptr) != (kept == nullptr) || (ctx_len == nullptr) != (ctx_out == nullptr))
        return SKV_ERR_INVALID_ARG;
    const void *words[] = {cu_new, tokens, parents, uniform, ctx_len, accepted, rows, ctx_out, next, status};
    for (const void *p : words)
        if (!aligned(p, 4)) return SKV_ERR_INVALID_ARG;
    if (!aligned(slots, 8) || !aligned(kept, 8) || !aligned(probs, size) || !aligned(draft_probs, size)) return SKV_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (n_requests == 0) return cudaMemsetAsync(status, 0, sizeof(int32_t), st) == cudaSuccess ? SKV_OK : SKV_ERR_CUDA;
    // A cluster of its own looks through up to 4,096 rows of requests whose lengths it holds for errors; beyond, a launch clears the status first (without and with
    // that cluster, vocabulary of 1,000: 64 requests of 8 nodes 12.5 and 9.9 us, 256 of 16 17.6 and 14.2, 256 of 30 16.8 and 18.0, 1,000 of 32
    // 26 and 78).
    VerifyArgs a{probs, draft_probs, probs_stride, draft_stride, vocab, distinct, n_rows, n_requests, cu_new, tokens, parents, uniform,
                 slots, ctx_len, accepted, rows, kept, ctx_out, next, status, n_rows <= 4096u && n_requests < kNodes * 4u, 0u, 0u, 0u, 0u};
    if (!a.checked && cudaMemsetAsync(status, 0, sizeof(int32_t), st) != cudaSuccess) return SKV_ERR_CUDA;
    uint32_t sms = 0;
    if (!device_sms(&sms)) return SKV_ERR_CUDA;
    // CTAs to a request, up to 16 of 2,048 elements or more: as many as about find a place at once, 1,024 threads to an SM (up to seven
    // eighths of it, as a cluster's CTAs need places near one another). More of them hold more of the rows and have less to add up, but what waits for a place
    // waits for whole requests. With draft probabilities 64 requests of up to 60 nodes over 151,936 tokens take 55 us with 8 to
    // each, 54 with 16, 82 with 4; 64 of 30 nodes over 50,257 tokens 23 with 8, 30 with 16, 27 with 4. Without, 24 requests of 27 nodes over
    // 50,257 tokens take 9 with 8 and 15 with 16; 40 over 151,936 16 with 4 and 20 with 8.
    const uint32_t sides = draft_probs ? 2u : 1u, threads = draft_probs ? kThreads<true> : kThreads<false>,
                   fits = (draft_probs ? kRowBytes<true> : kRowBytes<false>) / (sides * size) - 32u / size - 16u;
    const uint32_t room = draft_probs || fits < 32u * threads ? fits : 32u * threads;      // (kPieces to a part at most)
    uint32_t cluster = 1;
    while (cluster < kVerifyCluster && cluster * 2048u < vocab &&
           ((uint64_t)cluster * n_requests * threads <= 448ull * sms || cluster * most_part(threads) < vocab))
        cluster *= 2u;
    a.per_cta = (vocab + cluster - 1u) / cluster;
    a.per_held = ((a.per_cta < room ? a.per_cta : room) + 15u) & ~15u;
    a.per_warp = (a.per_held + threads - 1u) / threads * 32u;
    a.per_warp_far = draft_probs && a.per_cta > a.per_held ? (a.per_cta - a.per_held + threads - 1u) / threads * 32u : 0u;
    const uint32_t bytes = sides * (a.per_held * size + 32u);
    bool ok;
    if (dtype == SKV_PROB_F32) ok = draft_probs ? launch_verify<float, true>(a, cluster, bytes, st) : launch_verify<float, false>(a, cluster, bytes, st);
    else ok = draft_probs ? launch_verify<uint16_t, true>(a, cluster, bytes, st) : launch_verify<uint16_t, false>(a, cluster, bytes, st);
    return ok ? SKV_OK : SKV_ERR_CUDA;
}
