// skv_paged.cu -- block tables, slot maps and row writes of a paged KV cache.
//
// page_map: the prefix sums over requests are short (a few thousand entries),
// the slot map long (one 8-byte slot per new token), so every CTA computes the
// sums for itself from the same lengths and then writes its own range of slots:
// one launch, no word passed between CTAs. What a request's last page count
// and the ring's old head leave open, every CTA works out alike; the page of
// token i of a request is either an old table entry or the ring's next entry,
// both only read in this call, and the CTA that holds the first token of a new
// page writes that page's table entry. The ring's pushes go behind its end, where
// nothing is read. On the device a step of 8 requests takes 3 to 4 us (launch, two barriers
// and code fetched once) and one of 2,000 requests with 1.75 M tokens in a map of 4.0 M slots 18.5 us:
// with a token each it takes 12.4 in a map of 0.6 M slots (152 CTAs, each with all lengths and sums) and
// 16.4 in the large one (32 MB of slots, 5 us of HBM); the rest are the tokens' searches.
//
// append: each K and V row moves once, 16 bytes per thread and step; bound by HBM: 65,536 bf16 rows of
// 8 x 128 channels take 90 us (5.95 TB/s, 0.89 of a copy), 8 rows 2 us. Into e4m3 the same rows take 120 us
// against 60 of HBM: bound by issue, some 24 instructions per code for the exact quotient.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <atomic>

#include "skv_paged.h"

namespace skv {

bool raise_smem(const void *kernel, uint32_t bytes, std::atomic<uint64_t> &ready);      // skv_attend.cu

struct MapArgs {
    FastDiv page;
    uint32_t pool_pages, n_requests, max_pages, free_capacity;
    const int32_t *ctx_len, *new_len, *n_in, *free_in;
    int32_t *table, *n_out, *free_pages, *free_out, *cu;
    uint64_t table_stride;
    int64_t *slots;
    uint64_t slot_capacity;
    int32_t *status;
};

constexpr uint32_t kMapThreads = 1024;

struct MapOf {
    int32_t ctx, have;
    uint32_t add, need, back;
    int32_t err;
};

// Request r's lengths and what they ask for.
__device__ __forceinline__ MapOf map_of(const MapArgs &a, uint32_t r) {
    MapOf m{-1, 0, 0u, 0u, 0u, SKV_OK};
    if (r >= a.n_requests) return m;
    const int32_t c = a.ctx_len[r], w = a.new_len[r], h = a.n_in[r];
    m.ctx = c;
    m.have = h;
    if (w < 0 || h < 0 || (uint32_t)h > a.max_pages || (c < 0 && w > 0) ||
        (c >= 0 && ((int64_t)c > (int64_t)h * a.page.d || (int64_t)c + w > INT32_MAX))) {
        m.err = SKV_ERR_INVALID_ARG;
        return m;
    }
    m.add = (uint32_t)w;
    if (c < 0) {
        m.back = (uint32_t)h;
        return m;
    }
    const uint32_t len = (uint32_t)c + (uint32_t)w;
    const uint32_t full = div_by(len, a.page);
    const uint32_t want = full + (full * a.page.d != len);
    if (want > a.max_pages) m.err = SKV_ERR_CAPACITY;
    if (want > (uint32_t)h) m.need = want - (uint32_t)h;
    return m;
}

// Exclusive prefix sums of three counts over the block, and their totals.
template <uint32_t THREADS>
__device__ __forceinline__ void scan3(uint32_t (&x)[3], uint32_t (&total)[3], uint32_t (*part)[32]) {
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const uint32_t in[3] = {x[0], x[1], x[2]};
#pragma unroll
    for (uint32_t d = 1; d < 32; d <<= 1) {
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            const uint32_t y = __shfl_up_sync(~0u, x[j], d);
            if (lane >= d) x[j] += y;
        }
    }
    if (lane == 31) {
#pragma unroll
        for (int j = 0; j < 3; ++j) part[j][warp] = x[j];
    }
    __syncthreads();
    // every warp sums the warps' totals for itself: one barrier less
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const uint32_t p = lane < THREADS / 32u ? part[j][lane] : 0u;
        total[j] = __reduce_add_sync(~0u, p);
        x[j] += __reduce_add_sync(~0u, lane < warp ? p : 0u) - in[j];
    }
}

// A thread keeps ITEMS requests in a row, so that THREADS * ITEMS requests need one scan, and
// maps TOK tokens in a row. A step of a few hundred requests and slots is bound by barriers and by
// fetching instructions that run once: it takes 256 threads, one request and one token each.
template <uint32_t THREADS, uint32_t ITEMS, uint32_t TOK>
__global__ void __launch_bounds__(THREADS) map_kernel(MapArgs a) {
    constexpr uint32_t CHUNK = THREADS * ITEMS;
    extern __shared__ uint32_t dyn[];
    uint32_t *s_cu = dyn, *s_need = dyn + CHUNK + 1;
    int32_t *s_ctx = reinterpret_cast<int32_t *>(s_need + CHUNK), *s_have = s_ctx + CHUNK;
    __shared__ unsigned long long sum[3][32];
    __shared__ uint32_t part[3][32];
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    const int32_t head = a.free_in[0], count = a.free_in[1];

    // Totals in 64 bits and every error that the lengths hold, before anything is written.
    MapOf mine[ITEMS];
    unsigned long long t[3] = {0ull, 0ull, 0ull};
    bool bad = false, full = false;
#pragma unroll
    for (uint32_t k = 0; k < ITEMS; ++k) mine[k] = map_of(a, tid * ITEMS + k);
    const auto add = [&](const MapOf &m) {
        bad |= m.err == SKV_ERR_INVALID_ARG;
        full |= m.err == SKV_ERR_CAPACITY;
        t[0] += m.add;
        t[1] += m.need;
        t[2] += m.back;
    };
#pragma unroll
    for (uint32_t k = 0; k < ITEMS; ++k) add(mine[k]);
#pragma unroll 1
    for (uint32_t r = CHUNK + tid; r < a.n_requests; r += THREADS) add(map_of(a, r));
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        for (uint32_t d = 16; d; d >>= 1) t[j] += __shfl_xor_sync(~0u, t[j], d);
        if (lane == 0) sum[j][warp] = t[j];
    }
    const int worst = __syncthreads_or((bad ? 1 : 0) | (full ? 2 : 0)) ? (__syncthreads_or(bad) ? 1 : 2) : 0;
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        t[j] = lane < THREADS / 32u ? sum[j][lane] : 0ull;
        for (uint32_t d = 16; d; d >>= 1) t[j] += __shfl_xor_sync(~0u, t[j], d);
    }
    const bool ring_bad = count < 0 || (uint32_t)count > a.free_capacity || head < 0 ||
                          ((uint32_t)head >= a.free_capacity && (head != 0 || a.free_capacity != 0));
    int32_t err = SKV_OK;
    if (worst == 1 || ring_bad)
        err = SKV_ERR_INVALID_ARG;
    else if (worst || t[1] > (unsigned long long)count || t[0] > a.slot_capacity || t[0] > INT32_MAX ||
             (unsigned long long)count + t[2] > a.free_capacity)
        err = SKV_ERR_CAPACITY;

    // This CTA's share of the tokens' slots, and of the -1 behind them.
    const uint64_t total = err ? 0u : t[0], tail = a.slot_capacity - total;
    const uint64_t per = ((total + gridDim.x - 1) / gridDim.x + 3) & ~uint64_t(3);
    const uint64_t i0 = min((uint64_t)blockIdx.x * per, total), i1 = min(i0 + per, total);
    {
        const uint64_t each = ((tail + gridDim.x - 1) / gridDim.x + 1) & ~uint64_t(1);
        const uint64_t b0 = min((uint64_t)blockIdx.x * each, tail) + total, b1 = min((uint64_t)(blockIdx.x + 1u) * each, tail) + total;
        // 16 bytes at a time between the first and the last even entry
        const uint64_t e0 = min((b0 + 1) & ~uint64_t(1), b1), e1 = max(b1 & ~uint64_t(1), e0);
        const bool wide = ((uintptr_t)a.slots & 15u) == 0;
        if (wide) {
#pragma unroll 1
            for (uint64_t i = e0 + 2 * tid; i < e1; i += 2 * THREADS)
                *reinterpret_cast<longlong2 *>(a.slots + i) = make_longlong2(-1ll, -1ll);
            if (tid == 0 && b0 < e0) a.slots[b0] = -1;
            if (tid == 1 && e1 < b1) a.slots[e1] = -1;
        } else {
#pragma unroll 1
            for (uint64_t i = b0 + tid; i < b1; i += THREADS) a.slots[i] = -1;
        }
    }
    if (blockIdx.x == 0 && tid == 0) {
        if (gridDim.x == 1) *a.status = err;
        else if (err) set_first(a.status, err);
        const uint32_t cap = max(a.free_capacity, 1u);
        uint64_t to = (uint64_t)head + t[1];
        if (to >= cap) to -= cap;                     // head < cap, at most cap taken
        a.free_out[0] = err ? head : (int32_t)to;
        a.free_out[1] = err ? count : (int32_t)(count - t[1] + t[2]);
        a.cu[a.n_requests] = (int32_t)total;
    }
    if (err) {
        if (blockIdx.x == 0) {
            for (uint32_t r = tid; r < a.n_requests; r += THREADS) {
                a.n_out[r] = a.n_in[r];
                a.cu[r] = 0;
            }
        }
        return;
    }
    bool corrupt = false;
    uint32_t carry[3] = {0u, 0u, 0u};
#pragma unroll 1
    for (uint32_t base = 0; base < a.n_requests; base += CHUNK) {
        if (base) {
#pragma unroll
            for (uint32_t k = 0; k < ITEMS; ++k) mine[k] = map_of(a, base + tid * ITEMS + k);
        }
        uint32_t x[3] = {0u, 0u, 0u}, tot[3];
#pragma unroll
        for (uint32_t k = 0; k < ITEMS; ++k) {
            x[0] += mine[k].add;
            x[1] += mine[k].need;
            x[2] += mine[k].back;
        }
        __syncthreads();                              // the last chunk's sums and slots are done
        scan3<THREADS>(x, tot, part);
#pragma unroll
        for (int j = 0; j < 3; ++j) x[j] += carry[j];
        if (tid == 0) s_cu[CHUNK] = carry[0] + tot[0];
#pragma unroll
        for (uint32_t k = 0; k < ITEMS; ++k) {
            const MapOf &m = mine[k];
            const uint32_t at = tid * ITEMS + k, r = base + at;
            s_cu[at] = x[0];
            s_need[at] = x[1];
            s_ctx[at] = m.ctx;
            s_have[at] = m.have;
            if (r < a.n_requests && r % gridDim.x == blockIdx.x) {
                a.cu[r] = (int32_t)x[0];
                a.n_out[r] = m.ctx < 0 ? 0 : m.have + (int32_t)m.need;
            }
            // Pages of ended requests, one warp per request, requests dealt over the CTAs.
            uint32_t ended = __ballot_sync(~0u, m.back != 0u && r % gridDim.x == blockIdx.x);
#pragma unroll 1
            while (ended) {
                const uint32_t l = __ffs(ended) - 1u;
                ended &= ended - 1u;
                const uint32_t back = __shfl_sync(~0u, m.back, l), before = __shfl_sync(~0u, x[2], l);
                const int32_t *row = a.table + (uint64_t)__shfl_sync(~0u, r, l) * a.table_stride;
#pragma unroll 4
                for (uint32_t j = lane; j < back; j += 32u) {
                    const int32_t p = __ldg(row + j);        // not written in this call
                    corrupt |= (uint32_t)p >= a.pool_pages;
                    uint64_t to = (uint64_t)head + (uint32_t)count + before + j;      // below 2 free_capacity
                    if (to >= a.free_capacity) to -= a.free_capacity;
                    a.free_pages[to] = p;
                }
            }
            x[0] += m.add;
            x[1] += m.need;
            x[2] += m.back;
        }
        __syncthreads();
        // The slots of this chunk of requests that lie in this CTA's run.
        const uint64_t lo = max(i0, (uint64_t)s_cu[0]), hi = min(i1, (uint64_t)s_cu[CHUNK]);
        const uint32_t live = min(CHUNK, a.n_requests - base);
        // TOK tokens to a thread. (Entries that are read, old ones of the table and the ring's front, are
        // not written in this call.)
        #pragma unroll 1
        for (uint64_t i = (lo & ~uint64_t(TOK - 1)) + TOK * tid; i < hi; i += TOK * THREADS) {
            const uint32_t from = (uint32_t)max(i, lo), to = (uint32_t)min(i + TOK, hi);
            uint32_t f = 0, n = live;                             // last request with cu <= from
#pragma unroll 1
            while (n > 1) {
                const uint32_t h = n >> 1;
                if (s_cu[f + h] <= from) f += h;
                n -= h;
            }
            if (TOK == 4 && a.page.d >= 4u && i >= lo && s_cu[f + 1] >= (uint32_t)i + 4u && i + 4 <= hi &&
                ((uintptr_t)a.slots & 31u) == 0) {
                // four tokens of one request lie on at most two pages
                const uint32_t pos = (uint32_t)s_ctx[f] + (from - s_cu[f]), have = (uint32_t)s_have[f];
                const uint32_t j = div_by(pos, a.page), off = pos - j * a.page.d;
                int32_t *row = a.table + (uint64_t)(base + f) * a.table_stride + j;
                const bool over = off + 3u >= a.page.d;
                int32_t p[2];
#pragma unroll
                for (uint32_t k = 0; k < 2; ++k) {
                    uint64_t e = (uint64_t)head + s_need[f] + (j + k - have);
                    if (e >= a.free_capacity) e -= a.free_capacity;
                    p[k] = k == 0 || over ? __ldg(j + k < have ? row + k : a.free_pages + e) : 0;
                }
                if (off == 0u && j >= have) row[0] = p[0];
                if (over && j + 1u >= have) row[1] = p[1];
                const bool ok0 = (uint32_t)p[0] < a.pool_pages, ok1 = (uint32_t)p[1] < a.pool_pages;
                corrupt |= !ok0 || (over && !ok1);
                const int64_t s0 = (int64_t)p[0] * a.page.d + off, s1 = (int64_t)p[1] * a.page.d + off - a.page.d;
                int64_t v[4];
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k) {
                    const bool next = off + k >= a.page.d;
                    v[k] = (next ? ok1 : ok0) ? (next ? s1 : s0) + k : -1ll;
                }
                // a whole 32-byte sector at a time
                asm volatile("st.global.v4.b64 [%0], {%1,%2,%3,%4};" ::"l"(a.slots + i), "l"(v[0]), "l"(v[1]), "l"(v[2]), "l"(v[3]) : "memory");
                continue;
            }
#pragma unroll 1
            for (uint32_t x = from; x < to; ++x) {
                while (s_cu[f + 1] <= x) ++f;                     // past requests without tokens
                const uint32_t pos = (uint32_t)s_ctx[f] + (x - s_cu[f]), have = (uint32_t)s_have[f];
                const uint32_t j = div_by(pos, a.page), off = pos - j * a.page.d;
                int32_t *row = a.table + (uint64_t)(base + f) * a.table_stride + j;
                uint64_t e = (uint64_t)head + s_need[f] + (j - have);
                if (e >= a.free_capacity) e -= a.free_capacity;
                const int32_t p = __ldg(j < have ? row : a.free_pages + e);
                if (j >= have && off == 0u) *row = p;
                const bool ok = (uint32_t)p < a.pool_pages;
                corrupt |= !ok;
                a.slots[x] = ok ? (int64_t)p * a.page.d + off : -1ll;
            }
        }
#pragma unroll
        for (int j = 0; j < 3; ++j) carry[j] += tot[j];
    }
    if (corrupt) set_first(a.status, SKV_ERR_CORRUPT);
}

template <uint32_t THREADS, uint32_t ITEMS, uint32_t TOK>
static bool launch_map(const MapArgs &a, unsigned grid, cudaStream_t st) {
    constexpr uint32_t bytes = (4u * THREADS * ITEMS + 1u) * 4u;
    if (bytes > 48u * 1024u) {
        static std::atomic<uint64_t> ready{0};
        if (!raise_smem(reinterpret_cast<const void *>(map_kernel<THREADS, ITEMS, TOK>), bytes, ready)) return false;
    }
    map_kernel<THREADS, ITEMS, TOK><<<grid, THREADS, bytes, st>>>(a);
    return cudaGetLastError() == cudaSuccess;
}

struct AppendArgs {
    uint8_t *k, *v;                                   // pools
    uint64_t page_stride, token_stride, head_stride;  // bytes
    const float *k_scale, *v_scale;
    FastDiv page;
    uint64_t pool_tokens;
    const uint16_t *k_new, *v_new;
    uint64_t row_stride, row_head_stride;             // elements
    uint32_t n_src, n;
    FastDiv units, per_row;                           // units of 16 source bytes or 16 channels, per head and per row
    uint32_t narrow;                                  // 1: units and slots of this call fit 31 bits
    const int32_t *rows;
    const int64_t *slots;
    int32_t *status;
    uint32_t checked;                                 // 1: block 0 reports the errors
};

// A head's scale s, brought between 2^-85 and 2^64 together with the values (`by`, a power of two):
// there 1 / s and the remainders below are exact enough at either end of binary32. A value that
// leaves binary32 on the way saturates, or is 0, like its quotient.
struct ScaleOf {
    float by, s, r;
};

__device__ __forceinline__ ScaleOf scale_of(float s) {
    ScaleOf o;
    o.by = s < 0x1p-64f ? 0x1p64f : s > 0x1p64f ? 0x1p-64f : 1.0f;
    o.s = s * o.by;
    o.r = __fdiv_rn(1.0f, o.s);
    return o;
}

// The e4m3 code nearest to x / s. The binary32 quotient alone can land on a tie
// that the real quotient only comes near, so it is rounded to odd first: the
// remainder x - q s is exact in an fma for any q within a step of the quotient, and
// where it is not 0 the quotient is cut towards 0 and its last bit set, which keeps it
// off every border of the much coarser code grid. q: one product with the
// reciprocal of s and one correction by the remainder.
__device__ __forceinline__ uint32_t e4m3_of(float value, const ScaleOf &c) {
    const float x = value * c.by;
    float q = x * c.r;
    if (fabsf(q) >= 1.0e-30f && fabsf(q) < 1.0e30f) {
        q = fmaf(fmaf(-q, c.s, x), c.r, q);
        const float rem = fmaf(-q, c.s, x);
        uint32_t b = __float_as_uint(q);
        // the remainder's sign against the quotient's (s > 0): q is too large in magnitude
        if ((__float_as_uint(rem) ^ b) >> 31) --b;
        if (rem != 0.0f) q = __uint_as_float(b | 1u);
    }
    return (uint32_t)__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float bf16_float(uint32_t bits) { return __uint_as_float(bits << 16); }

// 16 bytes of codes from 16 channels of a bf16 row.
__device__ __forceinline__ uint4 quantise16(const uint4 a, const uint4 b, const ScaleOf &s) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[i] = e4m3_of(bf16_float(w[2 * i] & 0xFFFFu), s) | (e4m3_of(bf16_float(w[2 * i] >> 16), s) << 8) |
               (e4m3_of(bf16_float(w[2 * i + 1] & 0xFFFFu), s) << 16) | (e4m3_of(bf16_float(w[2 * i + 1] >> 16), s) << 24);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <bool E4M3>
__global__ void __launch_bounds__(256) append_kernel(AppendArgs a) {
    bool bad = false;
    if (a.checked && blockIdx.x == 0) {
        // loads of eight rounds in flight at once (checked: n <= 2,048)
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
            const uint32_t i = k * 256u + threadIdx.x;
            const int64_t s = i < a.n ? __ldg(a.slots + i) : -1;
            const uint32_t row = i < a.n && a.rows ? (uint32_t)__ldg(a.rows + i) : i;
            bad |= s >= 0 && ((uint64_t)s >= a.pool_tokens || row >= a.n_src);
        }
        bad = __syncthreads_or(bad);
        if (threadIdx.x == 0) *a.status = bad ? SKV_ERR_INVALID_ARG : SKV_OK;
        bad = false;
    }
    const uint64_t work = (uint64_t)a.n * a.per_row.d, step = (uint64_t)gridDim.x * blockDim.x;
    for (uint64_t w = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; w < work; w += step) {
        const uint32_t i = a.narrow ? div_by((uint32_t)w, a.per_row) : (uint32_t)(w / a.per_row.d);
        const uint32_t c = (uint32_t)(w - (uint64_t)i * a.per_row.d);
        const int64_t s = __ldg(a.slots + i);
        const uint32_t row = a.rows ? (uint32_t)__ldg(a.rows + i) : i;
        if (s < 0) continue;
        if ((uint64_t)s >= a.pool_tokens || row >= a.n_src) {
            bad = true;
            continue;
        }
        const uint32_t h = div_by(c, a.units), u = c - h * a.units.d;
        // a slot can pass 2^31 in a long cache
        const uint64_t p = a.narrow ? div_by((uint32_t)s, a.page) : (uint64_t)s / a.page.d;
        const uint64_t t = (uint64_t)s - p * a.page.d;
        const uint64_t dst = p * a.page_stride + t * a.token_stride + h * a.head_stride + 16u * (uint64_t)u;
        const uint64_t src = (uint64_t)row * a.row_stride + h * a.row_head_stride + (E4M3 ? 16u : 8u) * (uint64_t)u;
        if (E4M3) {
            const float ks = a.k_scale ? __ldg(a.k_scale + h) : 1.0f, vs = a.v_scale ? __ldg(a.v_scale + h) : 1.0f;
            const uint4 k0 = __ldg(reinterpret_cast<const uint4 *>(a.k_new + src)), k1 = __ldg(reinterpret_cast<const uint4 *>(a.k_new + src) + 1);
            const uint4 v0 = __ldg(reinterpret_cast<const uint4 *>(a.v_new + src)), v1 = __ldg(reinterpret_cast<const uint4 *>(a.v_new + src) + 1);
            // one code for both pools: half the instructions to fetch
#pragma unroll 1
            for (uint32_t pool = 0; pool < 2; ++pool) {
                *reinterpret_cast<uint4 *>((pool ? a.v : a.k) + dst) = quantise16(pool ? v0 : k0, pool ? v1 : k1, scale_of(pool ? vs : ks));
            }
        } else {
            const uint4 kc = __ldg(reinterpret_cast<const uint4 *>(a.k_new + src)), vc = __ldg(reinterpret_cast<const uint4 *>(a.v_new + src));
            *reinterpret_cast<uint4 *>(a.k + dst) = kc;
            *reinterpret_cast<uint4 *>(a.v + dst) = vc;
        }
    }
    if (bad && !a.checked) set_first(a.status, SKV_ERR_INVALID_ARG);
}

static bool device_sms(uint32_t *sms) {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return false;
    *sms = (uint32_t)n;
    return true;
}

}  // namespace skv

using namespace skv;

static bool aligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

extern "C" int32_t skv_paged_check(const skv_paged *c) {
    if (!c || c->version != SKV_FORMAT_VERSION || (c->dtype != SKV_BF16 && c->dtype != SKV_E4M3))
        return SKV_ERR_INVALID_ARG;
    if (c->n_heads == 0 || c->n_heads > 65535u || c->head_dim == 0 || c->head_dim > 256u || c->head_dim % 16u ||
        c->page_tokens == 0 || c->page_tokens > (1u << 20) || c->n_pages == 0 || c->n_pages > 0x7FFFFFFFu)
        return SKV_ERR_INVALID_ARG;
    if (!c->k_pages || !c->v_pages || !aligned(c->k_pages, 16) || !aligned(c->v_pages, 16)) return SKV_ERR_INVALID_ARG;
    const uint64_t unit = c->dtype == SKV_BF16 ? 8u : 16u, most = uint64_t(1) << 40;
    const uint64_t strides[3] = {c->page_stride, c->token_stride, c->head_stride};
    for (uint64_t s : strides)
        if (s % unit || s > most) return SKV_ERR_INVALID_ARG;
    if ((c->n_pages > 1 && c->page_stride == 0) || (c->page_tokens > 1 && c->token_stride == 0) ||
        (c->n_heads > 1 && c->head_stride == 0))
        return SKV_ERR_INVALID_ARG;
    if ((c->k_scale == nullptr) != (c->v_scale == nullptr) || (c->k_scale && c->dtype != SKV_E4M3) ||
        !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return SKV_ERR_INVALID_ARG;
    return SKV_OK;
}

extern "C" int32_t skv_page_map(uint32_t page_tokens, uint32_t pool_pages, uint32_t n_requests,
                                const int32_t *ctx_len, const int32_t *new_len, int32_t *block_table,
                                uint64_t table_stride, uint32_t max_pages, const int32_t *n_pages_in,
                                int32_t *n_pages_out, int32_t *free_pages, uint32_t free_capacity,
                                const int32_t *free_in, int32_t *free_out, int32_t *cu_new, int64_t *slots,
                                uint64_t slot_capacity, int32_t *status, void *stream) {
    if (page_tokens == 0 || page_tokens > (1u << 20) || pool_pages == 0 || pool_pages > 0x7FFFFFFFu ||
        free_capacity > 0x7FFFFFFFu || max_pages > 0x7FFFFFFFu || n_requests > 0x7FFFFFFFu ||
        (n_requests > 1 && table_stride < max_pages) || slot_capacity > (uint64_t(1) << 40))
        return SKV_ERR_INVALID_ARG;
    if (!free_in || !free_out || !cu_new || !status || (slot_capacity && !slots) || (free_capacity && !free_pages) ||
        (n_requests && (!ctx_len || !new_len || !n_pages_in || !n_pages_out || !block_table)))
        return SKV_ERR_INVALID_ARG;
    const void *words[] = {ctx_len, new_len, block_table, n_pages_in, n_pages_out, free_pages, free_in, free_out,
                           cu_new, status};
    for (const void *p : words)
        if (!aligned(p, 4)) return SKV_ERR_INVALID_ARG;
    if (!aligned(slots, 8) || free_in == free_out || (n_requests && n_pages_in == n_pages_out))
        return SKV_ERR_INVALID_ARG;
    uint32_t sms = 0;
    if (!device_sms(&sms)) return SKV_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    MapArgs a{fast_div(page_tokens), pool_pages, n_requests, max_pages, free_capacity, ctx_len, new_len, n_pages_in,
              free_in, block_table, n_pages_out, free_pages, free_out, cu_new, table_stride, slots, slot_capacity,
              status};
    // One CTA of 256 threads up to 256 requests and 2,048 slots, else a CTA of 1,024 per
    // 4,096 slots up to one per SM; several CTAs need the status cleared before them.
    if (n_requests <= 256u && slot_capacity <= 2048u) return launch_map<256, 1, 1>(a, 1, st) ? SKV_OK : SKV_ERR_CUDA;
    uint64_t grid = (slot_capacity + 4u * kMapThreads - 1) / (4u * kMapThreads);
    grid = grid < 1 ? 1 : grid > sms ? sms : grid;
    if (grid > 1 && cudaMemsetAsync(status, 0, sizeof(int32_t), st) != cudaSuccess) return SKV_ERR_CUDA;
    return launch_map<kMapThreads, 4, 4>(a, (unsigned)grid, st) ? SKV_OK : SKV_ERR_CUDA;
}

extern "C" int32_t skv_cache_append(const skv_paged *cache, const void *k, const void *v, uint64_t row_stride,
                                    uint64_t row_head_stride, uint32_t n_src, const int32_t *rows,
                                    const int64_t *slots, uint32_t n, int32_t *status, void *stream) {
    const int32_t r = skv_paged_check(cache);
    if (r != SKV_OK) return r;
    if (!status || !aligned(status, 4) || row_stride % 8u || row_head_stride % 8u || row_stride > (uint64_t(1) << 40) ||
        row_head_stride > (uint64_t(1) << 40))
        return SKV_ERR_INVALID_ARG;
    if (n && (!slots || !aligned(slots, 8) || !aligned(rows, 4) || (n_src && (!k || !v)) || !aligned(k, 16) ||
              !aligned(v, 16)))
        return SKV_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (n == 0) return cudaMemsetAsync(status, 0, sizeof(int32_t), st) == cudaSuccess ? SKV_OK : SKV_ERR_CUDA;
    uint32_t sms = 0;
    if (!device_sms(&sms)) return SKV_ERR_CUDA;
    const PagedView c = paged_view(*cache);
    AppendArgs a{static_cast<uint8_t *>(cache->k_pages), static_cast<uint8_t *>(cache->v_pages), c.page_stride,
                 c.token_stride, c.head_stride, c.k_scale, c.v_scale, c.page,
                 (uint64_t)cache->n_pages * cache->page_tokens, static_cast<const uint16_t *>(k),
                 static_cast<const uint16_t *>(v), row_stride, row_head_stride, n_src, n,
                 fast_div(cache->head_dim / (c.e4m3 ? 16u : 8u)), fast_div(cache->n_heads * (cache->head_dim / (c.e4m3 ? 16u : 8u))),
                 0u, rows, slots, status, n <= 2048u};
    const uint64_t work = (uint64_t)n * a.per_row.d;
    a.narrow = work < (uint64_t(1) << 31) && a.pool_tokens < (uint64_t(1) << 31);
    if (!a.checked && cudaMemsetAsync(status, 0, sizeof(int32_t), st) != cudaSuccess) return SKV_ERR_CUDA;
    uint64_t grid = (work + 255u) / 256u;
    if (grid > (uint64_t)sms * 8u) grid = (uint64_t)sms * 8u;
    if (c.e4m3) append_kernel<true><<<(unsigned)grid, 256, 0, st>>>(a);
    else append_kernel<false><<<(unsigned)grid, 256, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? SKV_OK : SKV_ERR_CUDA;
}
