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
// nothing is read. Bound by the launch for small steps and by the slot writes
// for large ones.
//
// append: each K and V row moves once, 16 bytes per thread and step; bound by HBM.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "skv_paged.h"

namespace skv {

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
__device__ __forceinline__ void scan3(uint32_t (&x)[3], uint32_t (&total)[3], uint32_t (*part)[32]) {
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    uint32_t in[3] = {x[0], x[1], x[2]};
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
    if (warp < 3) {
        uint32_t p = lane < (blockDim.x >> 5) ? part[warp][lane] : 0u;
        for (uint32_t d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(~0u, p, d);
            if (lane >= d) p += y;
        }
        part[warp][lane] = p;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        x[j] += (warp ? part[j][warp - 1] : 0u) - in[j];
        total[j] = part[j][31];
    }
    __syncthreads();
}

__global__ void __launch_bounds__(kMapThreads) map_kernel(MapArgs a) {
    __shared__ unsigned long long sum[3];
    __shared__ int32_t worst;
    __shared__ uint32_t part[3][32];
    __shared__ uint32_t s_cu[kMapThreads + 1], s_need[kMapThreads];
    __shared__ int32_t s_ctx[kMapThreads], s_have[kMapThreads];
    const uint32_t tid = threadIdx.x, lane = tid & 31u;

    // Totals in 64 bits and every error that the lengths hold, before anything is written.
    if (tid == 0) {
        sum[0] = sum[1] = sum[2] = 0ull;
        worst = 0;
    }
    __syncthreads();
    unsigned long long t[3] = {0ull, 0ull, 0ull};
    bool bad = false, full = false;
    for (uint32_t r = tid; r < a.n_requests; r += blockDim.x) {
        const MapOf m = map_of(a, r);
        bad |= m.err == SKV_ERR_INVALID_ARG;
        full |= m.err == SKV_ERR_CAPACITY;
        t[0] += m.add;
        t[1] += m.need;
        t[2] += m.back;
    }
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        for (uint32_t d = 16; d; d >>= 1) t[j] += __shfl_xor_sync(~0u, t[j], d);
        if (lane == 0 && t[j]) atomicAdd(&sum[j], t[j]);       // integers: any order gives the same sum
    }
    if (bad) atomicOr(&worst, 1);
    if (full) atomicOr(&worst, 2);
    __syncthreads();
    const int32_t head = a.free_in[0], count = a.free_in[1];
    const bool ring_bad = count < 0 || (uint32_t)count > a.free_capacity || head < 0 ||
                          ((uint32_t)head >= a.free_capacity && (head != 0 || a.free_capacity != 0));
    int32_t err = SKV_OK;
    if ((worst & 1) || ring_bad)
        err = SKV_ERR_INVALID_ARG;
    else if ((worst & 2) || sum[1] > (unsigned long long)count || sum[0] > a.slot_capacity || sum[0] > INT32_MAX ||
             (unsigned long long)count + sum[2] > a.free_capacity)
        err = SKV_ERR_CAPACITY;

    // This CTA's slots: a run of pairs.
    const uint64_t per = ((a.slot_capacity + gridDim.x - 1) / gridDim.x + 1) & ~uint64_t(1);
    const uint64_t i0 = min((uint64_t)blockIdx.x * per, a.slot_capacity);
    const uint64_t i1 = min(i0 + per, a.slot_capacity);
    const uint32_t total = err ? 0u : (uint32_t)sum[0];
    for (uint64_t i = max(i0, (uint64_t)total) + tid; i < i1; i += blockDim.x) a.slots[i] = -1;
    if (blockIdx.x == 0 && tid == 0) {
        if (gridDim.x == 1) *a.status = err;
        else if (err) set_first(a.status, err);
        const uint32_t cap = max(a.free_capacity, 1u);
        a.free_out[0] = err ? head : (int32_t)(((uint64_t)head + sum[1]) % cap);
        a.free_out[1] = err ? count : (int32_t)(count - sum[1] + sum[2]);
        a.cu[a.n_requests] = (int32_t)total;
    }
    if (err) {
        if (blockIdx.x == 0) {
            for (uint32_t r = tid; r < a.n_requests; r += blockDim.x) {
                a.n_out[r] = a.n_in[r];
                a.cu[r] = 0;
            }
        }
        return;
    }
    if (gridDim.x == 1) __syncthreads();          // the OK above comes before any CORRUPT below
    bool corrupt = false;
    uint32_t carry[3] = {0u, 0u, 0u};
    for (uint32_t base = 0; base < a.n_requests; base += blockDim.x) {
        const uint32_t r = base + tid;
        const MapOf m = map_of(a, r);
        uint32_t x[3] = {m.add, m.need, m.back}, tot[3];
        scan3(x, tot, part);
#pragma unroll
        for (int j = 0; j < 3; ++j) x[j] += carry[j];
        s_cu[tid] = x[0];
        s_need[tid] = x[1];
        s_ctx[tid] = m.ctx;
        s_have[tid] = m.have;
        if (tid == 0) s_cu[blockDim.x] = carry[0] + tot[0];
        if (blockIdx.x == 0 && r < a.n_requests) {
            a.cu[r] = (int32_t)x[0];
            a.n_out[r] = m.ctx < 0 ? 0 : m.have + (int32_t)m.need;
        }
        // Pages of ended requests, one warp per request, requests dealt over the CTAs.
        uint32_t ended = __ballot_sync(~0u, m.back != 0u && r % gridDim.x == blockIdx.x);
        while (ended) {
            const uint32_t l = __ffs(ended) - 1u;
            ended &= ended - 1u;
            const uint32_t back = __shfl_sync(~0u, m.back, l), before = __shfl_sync(~0u, x[2], l);
            const int32_t *row = a.table + (uint64_t)__shfl_sync(~0u, r, l) * a.table_stride;
            for (uint32_t j = lane; j < back; j += 32u) {
                const int32_t p = row[j];
                corrupt |= (uint32_t)p >= a.pool_pages;
                a.free_pages[((uint64_t)head + (uint32_t)count + before + j) % a.free_capacity] = p;
            }
        }
        __syncthreads();
        // The slots of this chunk of requests that lie in this CTA's run.
        const uint64_t lo = max(i0, (uint64_t)s_cu[0]), hi = min(i1, (uint64_t)s_cu[blockDim.x]);
        for (uint64_t i = lo + tid; i < hi; i += blockDim.x) {
            uint32_t f = 0, n = blockDim.x;                       // last request with cu <= i
            while (n > 1) {
                const uint32_t h = n >> 1;
                if (s_cu[f + h] <= (uint32_t)i) f += h;
                n -= h;
            }
            const uint32_t at = (uint32_t)i - s_cu[f], pos = (uint32_t)s_ctx[f] + at;
            const uint32_t j = div_by(pos, a.page), off = pos - j * a.page.d;
            int32_t p;
            if (j < (uint32_t)s_have[f]) {
                p = a.table[(uint64_t)(base + f) * a.table_stride + j];
            } else {
                uint64_t e = (uint64_t)head + s_need[f] + (j - (uint32_t)s_have[f]);
                if (e >= a.free_capacity) e -= a.free_capacity;
                p = a.free_pages[e];
                if (off == 0u) a.table[(uint64_t)(base + f) * a.table_stride + j] = p;
            }
            const bool ok = (uint32_t)p < a.pool_pages;
            corrupt |= !ok;
            a.slots[i] = ok ? (int64_t)p * a.page.d + off : -1;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 3; ++j) carry[j] += tot[j];
    }
    if (corrupt) set_first(a.status, SKV_ERR_CORRUPT);
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
    uint32_t n_heads, units;                          // units of 16 source bytes or 16 channels per head
    const int32_t *rows;
    const int64_t *slots;
    int32_t *status;
    uint32_t checked;                                 // 1: block 0 reports the errors
};

// The e4m3 code nearest to x / s. The binary32 quotient alone can land on a tie
// that the real quotient only comes near, so it is rounded to odd first: the
// remainder x - q s is exact in an fma, and where it is not 0 the quotient is
// cut towards 0 and its last bit set, which keeps it off every border of the
// much coarser code grid.
__device__ __forceinline__ uint32_t e4m3_of(float x, float s) {
    float q = __fdiv_rn(x, s);
    const float rem = fmaf(-q, s, x);
    if (fabsf(q) >= 1.0e-30f && fabsf(q) < 1.0e30f && rem != 0.0f) {
        uint32_t b = __float_as_uint(q);
        // the remainder's sign against the quotient's (s > 0): q is too large in magnitude
        if ((__float_as_uint(rem) ^ b) >> 31) --b;
        q = __uint_as_float(b | 1u);
    }
    return (uint32_t)__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float bf16_float(uint32_t bits) { return __uint_as_float(bits << 16); }

// 16 bytes of codes from 16 channels of a bf16 row (two 16-byte loads).
__device__ __forceinline__ uint4 quantise16(const uint16_t *src, float s) {
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(src)), b = __ldg(reinterpret_cast<const uint4 *>(src) + 1);
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
        for (uint32_t i = threadIdx.x; i < a.n; i += blockDim.x) {
            const int64_t s = a.slots[i];
            bad |= s >= 0 && ((uint64_t)s >= a.pool_tokens || (a.rows && (uint32_t)a.rows[i] >= a.n_src) ||
                              (!a.rows && i >= a.n_src));
        }
        bad = __syncthreads_or(bad);
        if (threadIdx.x == 0) *a.status = bad ? SKV_ERR_INVALID_ARG : SKV_OK;
        bad = false;
    }
    const uint32_t per_row = a.n_heads * a.units;
    const uint64_t work = (uint64_t)a.n * per_row, step = (uint64_t)gridDim.x * blockDim.x;
    for (uint64_t w = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; w < work; w += step) {
        const uint32_t i = (uint32_t)(w / per_row), c = (uint32_t)(w - (uint64_t)i * per_row);
        const int64_t s = __ldg(a.slots + i);
        if (s < 0) continue;
        const uint32_t row = a.rows ? (uint32_t)__ldg(a.rows + i) : i;
        if ((uint64_t)s >= a.pool_tokens || row >= a.n_src) {
            bad = true;
            continue;
        }
        const uint32_t h = c / a.units, u = c - h * a.units;
        // a slot can pass 2^31 in a long cache: 64-bit division by the page length
        const uint64_t p = (uint64_t)s / a.page.d, t = (uint64_t)s - p * a.page.d;
        const uint64_t dst = p * a.page_stride + t * a.token_stride + h * a.head_stride + 16u * (uint64_t)u;
        const uint64_t src = (uint64_t)row * a.row_stride + h * a.row_head_stride + (E4M3 ? 16u : 8u) * (uint64_t)u;
        uint4 kc, vc;
        if (E4M3) {
            kc = quantise16(a.k_new + src, a.k_scale ? __ldg(a.k_scale + h) : 1.0f);
            vc = quantise16(a.v_new + src, a.v_scale ? __ldg(a.v_scale + h) : 1.0f);
        } else {
            kc = __ldg(reinterpret_cast<const uint4 *>(a.k_new + src));
            vc = __ldg(reinterpret_cast<const uint4 *>(a.v_new + src));
        }
        *reinterpret_cast<uint4 *>(a.k + dst) = kc;
        *reinterpret_cast<uint4 *>(a.v + dst) = vc;
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
    uint64_t grid = (slot_capacity + 4u * kMapThreads - 1) / (4u * kMapThreads);
    grid = grid < 1 ? 1 : grid > sms ? sms : grid;
    if (grid > 1 && cudaMemsetAsync(status, 0, sizeof(int32_t), st) != cudaSuccess) return SKV_ERR_CUDA;
    map_kernel<<<(unsigned)grid, kMapThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? SKV_OK : SKV_ERR_CUDA;
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
                 static_cast<const uint16_t *>(v), row_stride, row_head_stride, n_src, n, cache->n_heads,
                 cache->head_dim / (c.e4m3 ? 16u : 8u), rows, slots, status, n <= 2048u};
    if (!a.checked && cudaMemsetAsync(status, 0, sizeof(int32_t), st) != cudaSuccess) return SKV_ERR_CUDA;
    const uint64_t work = (uint64_t)n * a.n_heads * a.units;
    uint64_t grid = (work + 255u) / 256u;
    if (grid > (uint64_t)sms * 8u) grid = (uint64_t)sms * 8u;
    if (c.e4m3) append_kernel<true><<<(unsigned)grid, 256, 0, st>>>(a);
    else append_kernel<false><<<(unsigned)grid, 256, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? SKV_OK : SKV_ERR_CUDA;
}
