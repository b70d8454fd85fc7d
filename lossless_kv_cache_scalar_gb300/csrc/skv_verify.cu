// skv_verify.cu -- verification of drafted trees.
//
// A cluster of CTAs takes a request. Every CTA walks the tree for itself, from the same few scalars (the
// probabilities of the drafted tokens, all gathered at once before the walk): nothing has to be
// passed on. Only a sum over the vocabulary is shared: each CTA sums its range of the row as whole numbers of
// 2^-44, so that no order of adding matters, and hands the sum to the others through distributed
// shared memory. The CTA and the warp in whose ranges the drawn number falls find the token.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "skv_rows.cuh"

namespace skv {

namespace cg = cooperative_groups;

constexpr uint32_t kVerifyThreads = 512, kVerifyWarps = kVerifyThreads / 32u;
constexpr uint32_t kNodes = 512;                 // nodes of a request that are gathered at once
constexpr uint32_t kGone = 4096;                 // nodes of a request without draft probabilities
constexpr uint32_t kVerifyCluster = 8;
constexpr float kUnit = 0x1p44f;

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
};

// A probability as it counts: the nearer end outside [0, 1], NaN as 0.
__device__ __forceinline__ float clamp01(float p) { return fminf(fmaxf(p, 0.0f), 1.0f); }
__device__ __forceinline__ float prob_of(const float *p) { return clamp01(__ldg(p)); }
__device__ __forceinline__ float prob_of(const uint16_t *p) { return clamp01(__uint_as_float((uint32_t)__ldg(p) << 16)); }

__device__ __forceinline__ uint64_t units_of_prob(float r) { return (uint64_t)__float2ull_rn(r * kUnit); }

// R(y) of a row: with c 0 (no rejection yet) p itself, whatever q holds.
__device__ __forceinline__ float rest_of(float p, float q, float c) { return fmaxf(fmaf(-c, q, p), 0.0f); }

struct Node {
    int32_t parent, token;
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

template <typename T, bool DRAFT>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyArgs a) {
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t C = cluster.num_blocks(), rank = cluster.block_rank();
    const uint32_t request = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    __shared__ Node node[kNodes];
    __shared__ unsigned long long warp_sum[kVerifyWarps + 1];
    __shared__ unsigned long long cta_sum[2][kVerifyCluster];
    __shared__ int32_t gone[DRAFT ? 1 : kGone];  // rejected tokens of the node (no draft probabilities)
    __shared__ struct {
        uint32_t todo, cur, at, taken, n_gone;
        float c;
        double Z, s;
    } walk;

    if (request == a.n_requests) {               // the errors of every request
        bool bad = false;
        if (rank == 0) {
            for (uint32_t r = warp; r < a.n_requests; r += kVerifyWarps) {
                uint32_t row0, n;
                bad |= !rows_of(a, r, &row0, &n);
                for (uint32_t i = 1 + lane; i < n; i += 32u)
                    bad |= !node_ok(a, parent_of(a, row0, i), __ldg(a.tokens + row0 + i), i);
            }
            bad = __syncthreads_or(bad);
            if (tid == 0) *a.status = bad ? SKV_ERR_INVALID_ARG : SKV_OK;
        }
        return;
    }
    uint32_t row0, n;
    const bool in_order = rows_of(a, request, &row0, &n);
    bool bad = !in_order;
    const T *P = static_cast<const T *>(a.probs) + (uint64_t)row0 * a.probs_stride;
    const T *Q = DRAFT ? static_cast<const T *>(a.draft) + (uint64_t)row0 * a.draft_stride : nullptr;

    // The scalars of nodes [first, first + kNodes).
    const auto gather = [&](uint32_t first) {
        const uint32_t i = first + tid;
        if (i < n) {
            Node x{-1, 0, __ldg(a.uniform + row0 + i), 0.0f, 0.0f};
            if (i) {
                x.parent = parent_of(a, row0, i);
                x.token = __ldg(a.tokens + row0 + i);
                if (node_ok(a, x.parent, x.token, i)) {
                    x.p = prob_of(P + (uint64_t)x.parent * a.probs_stride + x.token);
                    if (DRAFT) x.q = prob_of(Q + (uint64_t)x.parent * a.draft_stride + x.token);
                } else {
                    bad = true;
                }
            }
            node[tid] = x;
        }
    };
    static_assert(kNodes == kVerifyThreads, "a thread per node");
    gather(0);
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
    const float u0 = node[0].u;

    // Ranges of the vocabulary: a run per CTA, in it a run of whole 32s per warp.
    const uint32_t per_warp = (a.vocab + C * kVerifyThreads - 1u) / (C * kVerifyThreads) * 32u, per_cta = per_warp * kVerifyWarps;
    const uint32_t first = min(rank * per_cta, a.vocab), last = min(first + per_cta, a.vocab);
    const uint32_t w0 = min(first + warp * per_warp, last), w1 = min(w0 + per_warp, last);
    uint32_t parity = 0;

    // Sum of R over the row of `cur`: of each warp's range, of each CTA's; returns the whole.
    const auto sum_row = [&](uint32_t cur, float c) -> unsigned long long {
        const T *p = P + (uint64_t)cur * a.probs_stride;
        const T *q = DRAFT ? Q + (uint64_t)cur * a.draft_stride : nullptr;
        const bool with = DRAFT && c != 0.0f;
        unsigned long long sum = 0;
        constexpr uint32_t U = 8;
#pragma unroll 1
        for (uint32_t y = w0 + lane; y < w1; y += 32u * U) {
            float x[U], z[U];
#pragma unroll
            for (uint32_t j = 0; j < U; ++j) {
                const bool in = y + 32u * j < w1;
                x[j] = in ? prob_of(p + y + 32u * j) : 0.0f;
                z[j] = with && in ? prob_of(q + y + 32u * j) : 0.0f;
            }
#pragma unroll
            for (uint32_t j = 0; j < U; ++j) sum += units_of_prob(rest_of(x[j], z[j], c));
        }
#pragma unroll
        for (uint32_t d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
        __syncthreads();                         // the last sums are read
        if (lane == 0) warp_sum[warp] = sum;
        __syncthreads();
        // rejected tokens weigh nothing
        if (!DRAFT) {
            for (uint32_t j = tid; j < walk.n_gone; j += kVerifyThreads) {
                const uint32_t y = (uint32_t)gone[j];
                if (y >= first && y < last) atomicAdd(&warp_sum[(y - first) / per_warp], 0ull - units_of_prob(prob_of(p + y)));
            }
            __syncthreads();
        }
        if (!started) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        started = true;
        if (warp == 0) {
            unsigned long long t = lane < kVerifyWarps ? warp_sum[lane] : 0ull;
#pragma unroll
            for (uint32_t d = 16; d; d >>= 1) t += __shfl_xor_sync(~0u, t, d);
            if (lane < C) *cluster.map_shared_rank(&cta_sum[parity][rank], lane) = t;
        }
        cluster.sync();
        unsigned long long whole = 0;
        for (uint32_t j = 0; j < C; ++j) whole += cta_sum[parity][j];
        parity ^= 1u;
        return whole;
    };

    if (tid == 0) {
        walk.cur = 0, walk.at = 1, walk.taken = 1, walk.n_gone = 0;
        walk.c = 0.0f, walk.Z = 1.0, walk.s = 1.0;
        if (rank == 0) a.rows[row0] = (int32_t)row0;
    }
    constexpr uint32_t kDone = 0, kSum = 1, kMore = 2;
    uint32_t batch = 0;                          // first node in shared memory
    unsigned long long total = 0;
    bool fresh = false;                          // total and the sums are those of (cur, c)
    uint32_t cur = 0;
    float c = 0.0f;
#pragma unroll 1
    while (true) {
        __syncthreads();
        if (warp == 0) {
            uint32_t at = walk.at, taken = walk.taken, n_gone = walk.n_gone, todo = kDone;
            uint32_t here = walk.cur;
            float cc = walk.c;
            double Z = walk.Z, s = walk.s;
            bool have = !DRAFT || cc == 0.0f || fresh;      // Z is that of (here, cc)
            if (fresh) Z = (double)total * 0x1p-44;
            const uint32_t end = min(n, batch + kNodes);
#pragma unroll 1
            while (true) {
                // the next child of `here`
                uint32_t found = end;
#pragma unroll 1
                for (uint32_t b = at; b < end; b += 32u) {
                    const uint32_t i = b + lane;
                    const uint32_t m = __ballot_sync(~0u, i < end && node[i - batch].parent == (int32_t)here);
                    if (m) {
                        found = b + __ffs(m) - 1u;
                        break;
                    }
                }
                at = found;
                if (found == end) {
                    todo = end < n ? kMore : kDone;
                    break;
                }
                if (!have) {
                    todo = kSum;
                    break;
                }
                const Node x = node[found - batch];
                bool take;
                if (DRAFT) {
                    const double rest = (double)rest_of(x.p, x.q, cc);
                    take = (double)x.u * (double)x.q * Z < rest * s;
                    if (!take) {
                        if (s > 0.0) cc = (float)((double)cc + Z / s);
                        if (a.distinct) s = fmax(s - (double)x.q, 0.0);
                        have = false;
                    }
                } else {
                    bool again = false;
                    for (uint32_t j = lane; j < n_gone; j += 32u) again |= gone[j] == x.token;
                    again = __any_sync(~0u, again);
                    const double p = again ? 0.0 : (double)x.p;
                    take = (double)x.u * Z < p;
                    if (!take && !again) {
                        Z = fmax(Z - p, 0.0);
                        if (lane == 0) gone[n_gone] = x.token;
                        ++n_gone;
                        __syncwarp();
                    }
                }
                if (take) {
                    if (rank == 0 && lane == 0) a.rows[row0 + taken] = (int32_t)(row0 + found);
                    ++taken;
                    here = found;
                    cc = 0.0f, Z = 1.0, s = 1.0, n_gone = 0, have = true;
                }
                at = found + 1u;
            }
            if (lane == 0) {
                walk.todo = todo, walk.cur = here, walk.at = at, walk.taken = taken, walk.n_gone = n_gone;
                walk.c = cc, walk.Z = Z, walk.s = s;
            }
        }
        __syncthreads();
        const uint32_t todo = walk.todo;
        fresh = fresh && cur == walk.cur && c == walk.c;
        cur = walk.cur, c = walk.c;
        if (todo == kDone) break;
        if (todo == kMore) {
            batch += kNodes;
            gather(batch);
        } else {
            total = sum_row(cur, c);
            fresh = true;
        }
    }
    if (!fresh) total = sum_row(cur, c);
    if (total == 0ull && (c != 0.0f || walk.n_gone)) {            // nothing left of the target: its own row
        __syncthreads();
        if (tid == 0) walk.n_gone = 0;
        c = 0.0f;
        __syncthreads();
        total = sum_row(cur, c);
    }
    const uint32_t taken = walk.taken;

    // The drawn number: floor(u total), from u's bits.
    const float u = u0 > 0.0f ? fminf(u0, 0x1.fffffep-1f) : 0.0f;
    const unsigned long long t = min((unsigned long long)__double2ull_rd((double)u * (double)total), total ? total - 1ull : 0ull);
    unsigned long long before = 0;
    for (uint32_t j = 0; j < rank; ++j) before += cta_sum[parity ^ 1u][j];
    const bool mine = total && t >= before && t - before < cta_sum[parity ^ 1u][rank];
    if (mine) {
        // the warp's range, then the element: strips of 32, dealt to the warps
        uint32_t w = 0;
        unsigned long long left = t - before;
        while (left >= warp_sum[w]) left -= warp_sum[w++];
        const uint32_t v0 = first + w * per_warp, v1 = min(v0 + per_warp, last);
        const T *p = P + (uint64_t)cur * a.probs_stride;
        const T *q = DRAFT ? Q + (uint64_t)cur * a.draft_stride : nullptr;
        const auto weight = [&](uint32_t y) -> unsigned long long {
            if (y >= v1) return 0ull;
            const unsigned long long x = units_of_prob(rest_of(prob_of(p + y), DRAFT && c != 0.0f ? prob_of(q + y) : 0.0f, c));
            if (!DRAFT)
                for (uint32_t j = 0; j < walk.n_gone; ++j)
                    if ((uint32_t)gone[j] == y) return 0ull;
            return x;
        };
        __syncthreads();                         // (the same CTA-wide condition) warp_sum is read
        for (uint32_t y0 = v0; y0 < v1; y0 += kVerifyThreads) {
            const uint32_t y = y0 + tid;
            const unsigned long long x = weight(y);
            unsigned long long run = x;
#pragma unroll
            for (uint32_t d = 1; d < 32; d <<= 1) {
                const unsigned long long z = __shfl_up_sync(~0u, run, d);
                if (lane >= d) run += z;
            }
            if (lane == 31) warp_sum[warp] = run;
            __syncthreads();
            unsigned long long low = 0, all = 0;
            for (uint32_t j = 0; j < kVerifyWarps; ++j) {
                if (j < warp) low += warp_sum[j];
                all += warp_sum[j];
            }
            run += low;
            if (left >= run - x && left < run) a.next[request] = (int32_t)y;
            __syncthreads();
            if (left < all) break;
            left -= all;
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
static bool launch_verify(const VerifyArgs &a, uint32_t cluster, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.n_requests + a.checked) * cluster);
    cfg.blockDim = dim3(kVerifyThreads);
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
    VerifyArgs a{probs, draft_probs, probs_stride, draft_stride, vocab, distinct, n_rows, n_requests, cu_new, tokens, parents, uniform,
                 slots, ctx_len, accepted, rows, kept, ctx_out, next, status, n_rows <= 8192u && n_requests <= 1024u};
    if (!a.checked && cudaMemsetAsync(status, 0, sizeof(int32_t), st) != cudaSuccess) return SKV_ERR_CUDA;
    uint32_t cluster = 1;
    while (cluster < kVerifyCluster && cluster * 4096u < vocab) cluster *= 2u;
    bool ok;
    if (dtype == SKV_PROB_F32) ok = draft_probs ? launch_verify<float, true>(a, cluster, st) : launch_verify<float, false>(a, cluster, st);
    else ok = draft_probs ? launch_verify<uint16_t, true>(a, cluster, st) : launch_verify<uint16_t, false>(a, cluster, st);
    return ok ? SKV_OK : SKV_ERR_CUDA;
}
