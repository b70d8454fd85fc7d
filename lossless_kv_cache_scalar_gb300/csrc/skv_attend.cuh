// skv_attend.cuh -- what the tree-attention kernels share: the split of the work
// over CTAs, the workspace they leave their parts in, and small arithmetic.
//
// Work split. The work of a call is a list of units: for every request with
// rows, for every KV head, for every tile of query rows (R rows: node-major, a
// node's query heads of that KV head together), for every run of UT positions,
// one unit. A fixed grid takes equal, consecutive shares of the list (CTA c the
// units [c U / G, (c + 1) U / G)), so ragged lengths cost no balance and the host
// needs no length. The units of one (request, head, row tile) are an item; a
// CTA that holds a whole item writes its output, and one that holds a part
// leaves maximum, sum and unnormalised output in the workspace. The small-row
// kernel's CTA that comes last to an item joins its parts (counters in the
// workspace, 0 between calls); the large-row kernel's parts are joined by a second
// kernel, whose rows are spread over the GPU. A part that goes on from an earlier CTA goes to
// place 0 of its CTA, one that starts its item (and is cut off by the share's end) to place 1.
//
// In the large-row kernel a run of positions counts kWide units with more than 128 rows and
// kNarrow with up to 128: half of the products, the same bytes (256 against 128 rows took 1.28
// to 1.42 times as long, in bf16 and e4m3, with 64 and 128 channels). A run belongs to the CTA
// in whose share its first unit lies. A list of a few runs per CTA counts every run once: then what
// matters is that no CTA has one more than another.
#pragma once

#include <atomic>

#include "skv_paged.h"

namespace skv {

// Grids: persistent CTAs, three per SM of 152 for the small-row kernel, one for
// the tcgen05 one. Constants, so that the workspace's size depends on no device.
constexpr uint32_t kCtasSmall = 456, kCtasLarge = 152;
constexpr uint32_t kWide = 4, kNarrow = 3;

// An item that starts in a CTA and goes on in the next ones.
struct Desc {
    uint32_t valid, request, head, rt;
    uint64_t last;                       // unit at which its last run begins
};

struct Plan {
    uint64_t total;     // U
    uint64_t active;    // CTAs with work
};

struct AttendWs {
    uint32_t *arrived;  // [CTA]: parts done of the item that starts in the CTA and goes on
    uint32_t *finished; // CTAs done, and the errors seen
    Plan *plan;
    int32_t *errs;      // one per CTA
    Desc *desc;         // one per CTA
    float *parts;       // [CTA][2] of part_floats: m[R], l[R], o[R][DP]
};

__host__ __device__ inline uint64_t part_floats(uint32_t R, uint32_t DP) { return (uint64_t)R * (2u + DP); }

constexpr uint32_t kSawInvalid = 1u << 16, kSawCorrupt = 1u << 17;
__host__ __device__ inline int32_t status_of(uint32_t word) {
    return word & kSawInvalid ? SKV_ERR_INVALID_ARG : word & kSawCorrupt ? SKV_ERR_CORRUPT : SKV_OK;
}

// Counters (SKV_ATTENTION_ZERO_BYTES), then plan, errs, descs.
constexpr uint64_t kWsPlan = SKV_ATTENTION_ZERO_BYTES, kWsErrs = kWsPlan + 256u, kWsDesc = kWsErrs + 768u;
constexpr uint64_t kWsHead = kWsDesc + 160u * sizeof(Desc);
static_assert(kWsHead % 32u == 0 && sizeof(Desc) == 24 && kCtasLarge * 4u <= 768u && kCtasSmall * 4u + 4u <= SKV_ATTENTION_ZERO_BYTES &&
              kCtasLarge <= 160u && kWsHead % 256u == 0, "workspace head");

inline AttendWs attend_ws(void *base) {
    uint8_t *p = static_cast<uint8_t *>(base);
    uint32_t *n = reinterpret_cast<uint32_t *>(p);
    return AttendWs{n + 1, n, reinterpret_cast<Plan *>(p + kWsPlan),
                    reinterpret_cast<int32_t *>(p + kWsErrs), reinterpret_cast<Desc *>(p + kWsDesc),
                    reinterpret_cast<float *>(p + kWsHead)};
}

// Request r's rows and lengths; n = 0 for one without rows, or in error.
struct ReqOf {
    uint32_t row0, n, ctx, len;
    int32_t err;
};

__device__ __forceinline__ ReqOf request_of(const AttendArgs &a, uint32_t r) {
    ReqOf o{0u, 0u, 0u, 0u, SKV_OK};
    const int32_t c = a.ctx_len[r], lo = a.cu_new[r], hi = a.cu_new[r + 1];
    if (lo < 0 || hi < lo || (uint32_t)hi > a.n_rows) o.err = SKV_ERR_INVALID_ARG;
    else if (hi > lo) {
        const int64_t len = (int64_t)c + (hi - lo);
        if (c < 0 || len > (int64_t)a.c.max_pages * a.c.page.d || len > INT32_MAX ||
            (a.mask && (uint64_t)(hi - lo) > 64ull * a.mask_words))
            o.err = SKV_ERR_INVALID_ARG;
        else o = ReqOf{(uint32_t)lo, (uint32_t)(hi - lo), (uint32_t)c, (uint32_t)len, SKV_OK};
    }
    return o;
}

// Whether node sees position p of its request.
__device__ __forceinline__ bool sees(const AttendArgs &a, const ReqOf &q, uint32_t node, uint32_t p) {
    if (p < q.ctx) return true;
    const uint32_t j = p - q.ctx;
    if (!a.mask) return j <= node;
    return (__ldg(a.mask + (uint64_t)(q.row0 + node) * a.mask_words + (j >> 6)) >> (j & 63u)) & 1u;
}

// Which of the 32 positions p0 .. p0 + 31 the row sees.
__device__ __forceinline__ uint32_t sees32(const AttendArgs &a, const ReqOf &q, uint32_t node, uint32_t p0, uint32_t p_end) {
    uint32_t bits = 0u;
    if (p0 >= p_end) return 0u;
    const uint32_t live = p_end - p0 >= 32u ? ~0u : (1u << (p_end - p0)) - 1u;
    const int64_t j0 = (int64_t)p0 - q.ctx;                          // drafted index of bit 0
    if (j0 < 0) bits = j0 <= -32 ? ~0u : (1u << (uint32_t)(-j0)) - 1u;
    if (j0 > -32) {
        if (!a.mask) {
            const int64_t n = (int64_t)node - j0 + 1;                // j <= node
            bits |= n >= 32 ? ~0u : n <= 0 ? 0u : (1u << (uint32_t)n) - 1u;
        } else {
            const uint64_t *m = a.mask + (uint64_t)(q.row0 + node) * a.mask_words;
            const uint32_t first = j0 < 0 ? 0u : (uint32_t)j0, word = first >> 6, sh = first & 63u;
            uint64_t x = word < a.mask_words ? __ldg(m + word) >> sh : 0ull;
            if (sh > 32u && word + 1 < a.mask_words) x |= __ldg(m + word + 1) << (64u - sh);
            bits |= j0 < 0 ? (uint32_t)x << (uint32_t)(-j0) : (uint32_t)x;
        }
    }
    return bits & live;
}

// Byte offset of position p of request r, head h, in either pool; ~0 for a page
// number outside the pool.
__device__ __forceinline__ uint64_t place_of(const PagedView &c, uint32_t r, uint32_t h, uint32_t p) {
    const uint32_t j = div_by(p, c.page);
    const uint32_t page = (uint32_t)__ldg(c.table + (uint64_t)r * c.table_stride + j);
    if (page >= c.n_pages) return ~0ull;
    return (uint64_t)page * c.page_stride + (uint64_t)(p - j * c.page.d) * c.token_stride + h * c.head_stride;
}

__device__ __forceinline__ uint16_t bf16_bits(float x) {
    const uint32_t b = __float_as_uint(x);
    if ((b & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((b >> 16) | 0x40u);
    return (uint16_t)((b + 0x7FFFu + ((b >> 16) & 1u)) >> 16);
}

__device__ __forceinline__ float e4m3_float(uint32_t b) {
    const uint32_t e = (b >> 3) & 15u, m = b & 7u;
    float v = e ? __uint_as_float(((e + 120u) << 23) | (m << 20)) : (float)m * 0.001953125f;
    if ((b & 127u) == 127u) v = __uint_as_float(0x7FC00000u);
    return (b & 128u) ? -v : v;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A row's weights are 2^(score - m) against a reference m that lags behind the row's largest score by
// up to 2^8 in weight. In fp16 (e4m3 caches) a weight below 2^-14 loses bits and one below 2^-25 is
// nothing, while a sink's neighbours can hold much of the output at 2^-27 each: there the reference is
// put 2^7 lower, so that weights reach 2^15 (of fp16's 65,504) and are off by 2^-32 of the row's largest at
// most. The quotient does not depend on the reference.
constexpr float kLag = 8.0f;
template <bool FP16>
constexpr float kLower = FP16 ? 7.0f : 0.0f;

// The weight of a part with maximum m against the whole's M (0 for a part with nothing).
__device__ __forceinline__ float part_weight(float m, float M) { return m == -INFINITY ? 0.0f : ex2(m - M); }

// A V value that is not finite, at a position that some rows do not see, would
// reach them through the matrix product as 0 * NaN. The kernels put 0 in
// its place there, and each row that does see it gets it added at the end: its
// weight is positive, so the sum is that infinity or NaN whatever its size.
// This returns what to add to channel d of the row of `node`, from the positions [p0, p1).
__device__ __forceinline__ float not_finite_sum(const AttendArgs &a, const ReqOf &q, uint32_t r, uint32_t h,
                                                uint32_t node, uint32_t d, uint32_t p0, uint32_t p1) {
    float s = 0.0f;
#pragma unroll 1
    for (uint32_t p = max(p0, q.ctx); p < p1; ++p) {
        if (!sees(a, q, node, p)) continue;
        const uint64_t at = place_of(a.c, r, h, p);
        if (at == ~0ull) continue;
        const float v = a.c.e4m3 ? e4m3_float(a.c.v[at + d])
                                 : __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(a.c.v + at)[d] << 16);
        if (!(fabsf(v) < INFINITY)) s += v;
    }
    return s;
}

// n / d. Most lists are short; for the others bit by bit, in a loop: what a short call costs most is
// fetching instructions that it runs once, and a 64-bit division is a hundred of them.
__device__ __forceinline__ uint64_t quotient(uint64_t n, uint64_t d) {
    if (!((n | d) >> 32)) return (uint32_t)n / (uint32_t)d;
    uint64_t q = 0, r = 0;
#pragma unroll 1
    for (int i = 63; i >= 0; --i) {
        r = (r << 1) | ((n >> i) & 1u);
        q <<= 1;
        if (r >= d) {
            r -= d;
            q |= 1u;
        }
    }
    return q;
}

// Where CTA c's share of the list starts: the request, and the unit within it.
struct Share {
    uint64_t U, active;
    uint64_t u0, u1;      // units [u0, u1)
    uint32_t r;
    uint64_t off;
    uint32_t wide, narrow;    // units of a run
};

// Units of request r, split into row tiles of R rows and runs of UT positions.
__device__ __forceinline__ uint64_t units_of(const AttendArgs &a, const ReqOf &q, uint32_t R, uint32_t UT, uint32_t wide,
                                             uint32_t narrow) {
    if (q.n == 0) return 0;
    const uint32_t rows = q.n * a.group, rts = (rows + R - 1) / R;
    const uint32_t per_run = rts * wide - (rows - (rts - 1) * R > 128u ? 0u : wide - narrow);
    return (uint64_t)((q.len + UT - 1) / UT) * ((uint64_t)a.c.n_heads * per_run);
}

// Every thread of the block calls this; sm is scratch of 2 blockDim / 32 + 4 words of 8 bytes.
// LARGE: the kernel with weighted runs and a joining kernel behind it, for which it leaves plan, error and
// descriptor.
template <uint32_t THREADS, bool LARGE>
__device__ __forceinline__ Share share_of(const AttendArgs &a, const AttendWs &ws, uint32_t R, uint32_t UT,
                                          unsigned long long *sm) {
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    constexpr uint32_t W = THREADS / 32u;
    constexpr uint32_t wide = LARGE ? kWide : 1u, narrow = LARGE ? kNarrow : 1u;
    unsigned long long mine = 0, first = 0;
    uint32_t runs = 0, first_runs = 0;          // modulo 2^32: used where the whole is small
    int32_t err = SKV_OK;
#pragma unroll 1
    for (uint32_t r = tid; r < a.c.n_requests; r += THREADS) {
        const ReqOf q = request_of(a, r);
        if (q.err) err = q.err;
        const uint64_t u = units_of(a, q, R, UT, wide, narrow);
        if (r == tid) first = u;
        mine += u;
        if (LARGE) {
            const uint32_t n = (uint32_t)units_of(a, q, R, UT, 1u, 1u);
            if (r == tid) first_runs = n;
            runs += n;
        }
    }
    unsigned long long t = mine;
#pragma unroll
    for (uint32_t d = 16; d; d >>= 1) t += __shfl_xor_sync(~0u, t, d);
    if (LARGE) runs = __reduce_add_sync(~0u, runs);
    if (lane == 0) {
        sm[warp] = t;
        if (LARGE) sm[W + 4 + warp] = runs;
    }
    err = __syncthreads_or(err) ? SKV_ERR_INVALID_ARG : SKV_OK;
    unsigned long long U = 0;
#pragma unroll
    for (uint32_t w = 0; w < W; ++w) U += sm[w];
    const bool even = LARGE && U <= 4u * kWide * gridDim.x;
    if (even) {
        U = 0;
#pragma unroll
        for (uint32_t w = 0; w < W; ++w) U += sm[W + 4 + w];
        first = first_runs;
    }
    // every share is at least a run (U >= 4 kWide CTAs where runs are weighted)
    const uint64_t active = U < gridDim.x ? U : gridDim.x;
    Share s{U, active, 0, 0, 0, 0, even ? 1u : wide, even ? 1u : narrow};
    if (LARGE && tid == 0) {
        ws.errs[blockIdx.x] = err;
        ws.desc[blockIdx.x].valid = 0u;
        if (blockIdx.x == 0) *ws.plan = Plan{U, active};
    }
    if (!LARGE && tid == 0 && blockIdx.x == 0 && err) {
        atomicOr(ws.finished, kSawInvalid);
    }
    if (blockIdx.x >= active) return s;
    s.u0 = quotient((uint64_t)blockIdx.x * U, active);
    s.u1 = quotient((uint64_t)(blockIdx.x + 1) * U, active);
    unsigned long long carry = 0;
#pragma unroll 1
    for (uint32_t base = 0; base < a.c.n_requests; base += THREADS) {
        const uint32_t r = base + tid;
        unsigned long long u = base == 0 ? first : 0ull;
        if (base && r < a.c.n_requests) u = units_of(a, request_of(a, r), R, UT, s.wide, s.narrow);
        unsigned long long x = u;
#pragma unroll
        for (uint32_t d = 1; d < 32; d <<= 1) {
            const unsigned long long y = __shfl_up_sync(~0u, x, d);
            if (lane >= d) x += y;
        }
        __syncthreads();
        if (lane == 31) sm[warp] = x;
        __syncthreads();
        unsigned long long before = carry, whole = 0;
#pragma unroll
        for (uint32_t w = 0; w < W; ++w) {
            if (w < warp) before += sm[w];
            whole += sm[w];
        }
        x += before - u;
        if (x <= s.u0 && s.u0 < x + u) {
            sm[W] = r;
            sm[W + 1] = s.u0 - x;
        }
        carry += whole;
        if (carry > s.u0) break;            // the same for every thread
    }
    __syncthreads();
    s.r = (uint32_t)sm[W];
    s.off = sm[W + 1];
    return s;
}

// The last CTA whose share starts at or before unit u: where u lies.
__device__ __forceinline__ uint32_t cta_of(uint64_t u, uint64_t U, uint64_t active) {
    return (uint32_t)quotient((u + 1) * active - 1, U);
}

// One row of an item whose parts lie in CTAs c .. c + n - 1 (place 1 of the first, then 0), by one warp: each
// part weighs exp2(m - M) with M the largest m, in the order of the CTAs. Four parts' outputs
// are on their way while the four before them, or the weights, are worked on.
__device__ __forceinline__ void join_row(const AttendArgs &a, const AttendWs &ws, const ReqOf &q, uint32_t head, uint32_t rt,
                                         uint32_t row, uint32_t R, uint32_t DP, uint32_t c, uint32_t n) {
    const uint32_t lane = threadIdx.x & 31u, all = rt * R + row, node = all / a.group;
    if (node >= q.n) return;
    const uint32_t g = head * a.group + all - node * a.group;
    const uint32_t size = (uint32_t)part_floats(R, DP);
    const float *next = ws.parts + (uint64_t)c * 2u * size, *first = next + size;
    const auto part = [&](uint32_t j) { return j ? next + (uint64_t)(2u * j) * size : first; };
    uint16_t *out = a.out + ((uint64_t)(q.row0 + node) * a.n_q_heads + g) * a.c.head_dim;
    const uint32_t x = 4u * lane;                                    // (64 channels: half of the lanes)
    float4 y[4];
    const auto fetch = [&](uint32_t j0) {
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j)
            y[j] = j0 + j < n && x < DP ? __ldcg(reinterpret_cast<const float4 *>(part(j0 + j) + 2u * R + row * DP + x)) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    fetch(0);
    float M = -INFINITY;
#pragma unroll 1
    for (uint32_t j = lane; j < n; j += 32u) M = fmaxf(M, __ldcg(part(j) + row));
#pragma unroll
    for (uint32_t d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, d));
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.0f, f = 0.0f;
#pragma unroll 1
    for (uint32_t j0 = 0; j0 < n; j0 += 4u) {
        if ((j0 & 31u) == 0) {                                   // lane j: the weight of part j0 + j
            f = 0.0f;
            if (j0 + lane < n) {
                f = part_weight(__ldcg(part(j0 + lane) + row), M);
                L += f * __ldcg(part(j0 + lane) + R + row);
            }
        }
        const float4 z[4] = {y[0], y[1], y[2], y[3]};
        if (j0 + 4u < n) fetch(j0 + 4u);
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            const float w = __shfl_sync(~0u, f, (j0 + j) & 31u);
            o.x += w * z[j].x, o.y += w * z[j].y, o.z += w * z[j].z, o.w += w * z[j].w;
        }
    }
#pragma unroll
    for (uint32_t d = 16; d; d >>= 1) L += __shfl_xor_sync(~0u, L, d);
    const float inv = L == 0.0f ? 0.0f : (a.c.v_scale ? __ldg(a.c.v_scale + head) : 1.0f) / L;
    if (x < a.c.head_dim) {
        uint2 b;
        b.x = (uint32_t)bf16_bits(o.x * inv) | (uint32_t)bf16_bits(o.y * inv) << 16;
        b.y = (uint32_t)bf16_bits(o.z * inv) | (uint32_t)bf16_bits(o.w * inv) << 16;
        if (L == 0.0f) b = make_uint2(0u, 0u);
        *reinterpret_cast<uint2 *>(out + x) = b;
    }
    if (a.lse && x == 0)
        a.lse[(uint64_t)(q.row0 + node) * a.n_q_heads + g] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// skv_attend.cu
bool raise_smem(const void *kernel, uint32_t bytes, std::atomic<uint64_t> &ready);
bool launch_join(const AttendArgs &a, const AttendWs &ws, uint32_t R, uint32_t DP, uint32_t ctas, cudaStream_t st);
// skv_attend_tc.cu: head_dim up to 128
bool launch_large(const AttendArgs &a, const AttendWs &ws, cudaStream_t st);
constexpr uint32_t kLargeRows = 256;

}  // namespace skv
