// skv_rotate.cu -- norms and rotation of query and key heads, keys and values into the pages.
//
// A head's channels are cut into units of 16: two vectors of 8 channels that are rotated with each
// other (channels 8 u .. and rot_dim / 2 + 8 u .., or 16 neighbours), so a lane that holds a unit
// has both sides of its 8 pairs, and the angles of its 8 frequencies serve every head of the token.
// head_dim / 16 lanes (rounded up to a power of two) hold a head, a warp 32 / that many heads at
// once; the norm's sum is a few shuffles among them.
//
// Angles: position x frequency grows far beyond the bits that binary32 keeps of it. In turns, as a fraction of
// 2^64, the product modulo one turn is the low word of an integer product, and the sine
// is taken of a reduced angle in [-1/2, 1/2) turns.
#include <cuda_bf16.h>

#include "skv_rows.cuh"

namespace skv {

struct RotateArgs {
    const uint16_t *q, *k, *v;
    uint64_t q_row_stride, q_head_stride, row_stride, head_stride;      // elements
    uint16_t *q_out;
    uint32_t n_q_heads, n_heads, head_dim;
    uint32_t n, parts;                                                  // rows, warps per row
    FastDiv by_parts;
    // rotation
    const uint64_t *turns;
    const uint8_t *axis;
    const float *q_norm, *k_norm;
    const int32_t *positions;
    uint32_t rot_units, n_axes, interleaved;                            // rot_dim / 16
    float eps, inv_dim, amplitude;
    // cache
    uint8_t *k_pages, *v_pages;
    uint64_t page_stride, token_stride, page_head_stride;               // bytes
    const float *k_scale, *v_scale;
    FastDiv page;
    uint64_t pool_tokens;
    const int64_t *slots;
    int32_t *status;
    uint32_t checked;                                                   // 1: block 0 reports the errors
};

constexpr uint32_t kRotateThreads = 256;

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

__device__ __forceinline__ void unpack8(const uint4 &w, float *x) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(a[i] << 16);
        x[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float *x) {
    return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

__device__ __forceinline__ uint2 quantise8(const float *x, const ScaleOf &s) {
    uint32_t o[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        o[i] = e4m3_of(x[4 * i], s) | (e4m3_of(x[4 * i + 1], s) << 8) | (e4m3_of(x[4 * i + 2], s) << 16) |
               (e4m3_of(x[4 * i + 3], s) << 24);
    return make_uint2(o[0], o[1]);
}

// LANES lanes to a head.
template <uint32_t LANES, bool E4M3>
__global__ void __launch_bounds__(kRotateThreads) rotate_kernel(const RotateArgs a) {
    constexpr uint32_t HPW = 32u / LANES;
    if (a.checked && blockIdx.x == 0) {
        // loads of eight rounds in flight at once (checked: n <= 2,048)
        bool bad = false;
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) {
            const uint32_t i = j * kRotateThreads + threadIdx.x;
            const int64_t s = i < a.n ? __ldg(a.slots + i) : -1;
            bad |= s >= 0 && (uint64_t)s >= a.pool_tokens;
        }
        bad = __syncthreads_or(bad);
        if (threadIdx.x == 0) *a.status = bad ? SKV_ERR_INVALID_ARG : SKV_OK;
    }
    const uint64_t item = (uint64_t)blockIdx.x * (kRotateThreads / 32u) + (threadIdx.x >> 5);
    if (item >= (uint64_t)a.n * a.parts) return;
    const uint32_t lane = threadIdx.x & 31u, u = lane % LANES, own = lane / LANES;
    const uint32_t i = item >> 31 ? (uint32_t)(item / a.parts) : div_by((uint32_t)item, a.by_parts);
    const uint32_t part = (uint32_t)(item - (uint64_t)i * a.parts);
    const bool live = u < a.head_dim / 16u;
    const bool turned = u < a.rot_units;
    // channels of the unit's two vectors
    const uint32_t lo = turned && !a.interleaved ? 8u * u : 16u * u;
    const uint32_t hi = lo + (turned && !a.interleaved ? 8u * a.rot_units : 8u);

    const int64_t slot = __ldg(a.slots + i);
    float c[8], s[8];
    if (turned) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t ax = a.axis ? __ldg(a.axis + 8u * u + j) : 0u;
            if (ax >= a.n_axes) ax = 0u;
            const int64_t pos = __ldg(a.positions + (uint64_t)ax * a.n + i);
            const uint64_t t = __ldg(a.turns + 8u * u + j) * (uint64_t)pos;
            sincospif((float)(int32_t)(t >> 32) * 0x1p-31f, &s[j], &c[j]);
            c[j] *= a.amplitude;
            s[j] *= a.amplitude;
        }
    }
    uint64_t dst = 0;
    bool to_pages = slot >= 0;
    if (to_pages && (uint64_t)slot >= a.pool_tokens) {
        to_pages = false;
        if (!a.checked) set_first(a.status, SKV_ERR_INVALID_ARG);
    }
    if (to_pages) {
        const uint64_t p = a.pool_tokens >> 31 ? (uint64_t)slot / a.page.d : div_by((uint32_t)slot, a.page);
        dst = p * a.page_stride + ((uint64_t)slot - p * a.page.d) * a.token_stride;
    }
    const uint32_t heads = a.n_q_heads + (to_pages ? 2u * a.n_heads : 0u);
    float w[16];
    uint32_t kind = 3u;                                     // whose weights w holds
#pragma unroll 1
    for (uint32_t h0 = part * HPW; h0 < heads; h0 += a.parts * HPW) {
        const uint32_t h = h0 + own;
        const bool on = live && h < heads;
        const uint32_t what = h < a.n_q_heads ? 0u : h < a.n_q_heads + a.n_heads ? 1u : 2u;
        const uint32_t g = what == 0 ? h : what == 1 ? h - a.n_q_heads : h - a.n_q_heads - a.n_heads;
        const uint16_t *src = what == 0 ? a.q + (uint64_t)i * a.q_row_stride + (uint64_t)g * a.q_head_stride
                                        : (what == 1 ? a.k : a.v) + (uint64_t)i * a.row_stride + (uint64_t)g * a.head_stride;
        uint4 x0 = make_uint4(0u, 0u, 0u, 0u), x1 = x0;
        if (on) {
            x0 = *reinterpret_cast<const uint4 *>(src + lo);
            x1 = *reinterpret_cast<const uint4 *>(src + hi);
        }
        float x[16];
        unpack8(x0, x);
        unpack8(x1, x + 8);
        const float *norm = what == 0 ? a.q_norm : a.k_norm;
        if (on && kind != what && what < 2u && norm) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 y = __ldg(reinterpret_cast<const float4 *>(norm + (j < 2 ? lo : hi)) + (j & 1));
                w[4 * j] = y.x, w[4 * j + 1] = y.y, w[4 * j + 2] = y.z, w[4 * j + 3] = y.w;
            }
        }
        kind = what;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
        for (uint32_t d = 1; d < LANES; d <<= 1) sum += __shfl_xor_sync(~0u, sum, d);
        if (!on) continue;
        if (what < 2u) {
            if (norm) {
                const float r = rsqrtf(fmaf(sum, a.inv_dim, a.eps));
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] *= r * w[j];
            }
            if (turned) {
                if (a.interleaved) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float p = x[2 * j], q = x[2 * j + 1];
                        x[2 * j] = p * c[j] - q * s[j];
                        x[2 * j + 1] = p * s[j] + q * c[j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float p = x[j], q = x[j + 8];
                        x[j] = p * c[j] - q * s[j];
                        x[j + 8] = p * s[j] + q * c[j];
                    }
                }
            }
        }
        if (what == 0) {
            uint16_t *out = a.q_out + ((uint64_t)i * a.n_q_heads + g) * a.head_dim;
            *reinterpret_cast<uint4 *>(out + lo) = pack8(x);
            *reinterpret_cast<uint4 *>(out + hi) = pack8(x + 8);
        } else {
            uint8_t *to = (what == 1 ? a.k_pages : a.v_pages) + dst + (uint64_t)g * a.page_head_stride;
            if (E4M3) {
                const float *scale = what == 1 ? a.k_scale : a.v_scale;
                const ScaleOf sc = scale_of(scale ? __ldg(scale + g) : 1.0f);
                *reinterpret_cast<uint2 *>(to + lo) = quantise8(x, sc);
                *reinterpret_cast<uint2 *>(to + hi) = quantise8(x + 8, sc);
            } else {
                *reinterpret_cast<uint4 *>(to + 2u * lo) = what == 1 ? pack8(x) : x0;
                *reinterpret_cast<uint4 *>(to + 2u * hi) = what == 1 ? pack8(x + 8) : x1;
            }
        }
    }
}

template <uint32_t LANES>
static bool launch_rotate(const RotateArgs &a, bool e4m3, unsigned grid, cudaStream_t st) {
    if (e4m3) rotate_kernel<LANES, true><<<grid, kRotateThreads, 0, st>>>(a);
    else rotate_kernel<LANES, false><<<grid, kRotateThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess;
}

}  // namespace skv

using namespace skv;

extern "C" int32_t skv_rotary_check(const skv_rotary *r) {
    if (!r || r->version != SKV_FORMAT_VERSION || r->head_dim == 0 || r->head_dim > 256u || r->head_dim % 16u ||
        r->rot_dim % 16u || r->rot_dim > r->head_dim || r->n_axes == 0 || r->n_axes > 16u || r->interleaved > 1u)
        return SKV_ERR_INVALID_ARG;
    if (!(r->eps >= 0.0f) || r->eps > 3.0e38f || !(r->amplitude >= -3.0e38f && r->amplitude <= 3.0e38f)) return SKV_ERR_INVALID_ARG;
    if ((r->rot_dim && !r->turns) || !aligned(r->turns, 8) || !aligned(r->q_norm, 16) || !aligned(r->k_norm, 16))
        return SKV_ERR_INVALID_ARG;
    return SKV_OK;
}

extern "C" int32_t skv_rotate_append(const skv_paged *cache, const skv_rotary *rotary, const void *q, uint64_t q_row_stride,
                                     uint64_t q_head_stride, uint32_t n_q_heads, const void *k, const void *v, uint64_t row_stride,
                                     uint64_t row_head_stride, const int32_t *positions, const int64_t *slots, uint32_t n,
                                     void *q_out, int32_t *status, void *stream) {
    int32_t rc = skv_paged_check(cache);
    if (rc == SKV_OK) rc = skv_rotary_check(rotary);
    if (rc != SKV_OK) return rc;
    const uint64_t most = uint64_t(1) << 40;
    if (rotary->head_dim != cache->head_dim || !status || !aligned(status, 4) || row_stride % 8u || row_head_stride % 8u ||
        q_row_stride % 8u || q_head_stride % 8u || row_stride > most || row_head_stride > most || q_row_stride > most ||
        q_head_stride > most || n_q_heads > 65535u || n > 0x7FFFFFFFu)
        return SKV_ERR_INVALID_ARG;
    if (n && (!slots || !aligned(slots, 8) || !k || !v || !aligned(k, 16) || !aligned(v, 16) || !aligned(positions, 4) ||
              (rotary->rot_dim && !positions) || (n_q_heads && (!q || !q_out)) || !aligned(q, 16) || !aligned(q_out, 16)))
        return SKV_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (n == 0) return cudaMemsetAsync(status, 0, sizeof(int32_t), st) == cudaSuccess ? SKV_OK : SKV_ERR_CUDA;
    uint32_t sms = 0;
    if (!device_sms(&sms)) return SKV_ERR_CUDA;
    const PagedView c = paged_view(*cache);
    const uint32_t units = cache->head_dim / 16u;
    const uint32_t lanes = units <= 1 ? 1 : units <= 2 ? 2 : units <= 4 ? 4 : units <= 8 ? 8 : 16;
    // A warp takes a row's heads one group after the other; with few rows a row's groups go to several
    // warps, up to 16 warps per SM, each of which works the angles out again.
    const uint32_t groups = (n_q_heads + 2u * cache->n_heads + 32u / lanes - 1u) / (32u / lanes);
    uint32_t parts = 16u * sms / n;
    parts = parts < 1 ? 1 : parts > groups ? groups : parts;
    RotateArgs a{};
    a.q = static_cast<const uint16_t *>(q), a.k = static_cast<const uint16_t *>(k), a.v = static_cast<const uint16_t *>(v);
    a.q_row_stride = q_row_stride, a.q_head_stride = q_head_stride, a.row_stride = row_stride, a.head_stride = row_head_stride;
    a.q_out = static_cast<uint16_t *>(q_out);
    a.n_q_heads = n_q_heads, a.n_heads = cache->n_heads, a.head_dim = cache->head_dim;
    a.n = n, a.parts = parts, a.by_parts = fast_div(parts);
    a.turns = rotary->turns, a.axis = rotary->axis, a.q_norm = rotary->q_norm, a.k_norm = rotary->k_norm, a.positions = positions;
    a.rot_units = rotary->rot_dim / 16u, a.n_axes = rotary->n_axes, a.interleaved = rotary->interleaved;
    a.eps = rotary->eps, a.inv_dim = 1.0f / (float)cache->head_dim, a.amplitude = rotary->amplitude;
    a.k_pages = static_cast<uint8_t *>(cache->k_pages), a.v_pages = static_cast<uint8_t *>(cache->v_pages);
    a.page_stride = c.page_stride, a.token_stride = c.token_stride, a.page_head_stride = c.head_stride;
    a.k_scale = c.k_scale, a.v_scale = c.v_scale, a.page = c.page;
    a.pool_tokens = (uint64_t)cache->n_pages * cache->page_tokens;
    a.slots = slots, a.status = status, a.checked = n <= 2048u;
    if (!a.checked && cudaMemsetAsync(status, 0, sizeof(int32_t), st) != cudaSuccess) return SKV_ERR_CUDA;
    const uint64_t blocks = ((uint64_t)n * parts + kRotateThreads / 32u - 1) / (kRotateThreads / 32u);
    const unsigned grid = (unsigned)blocks;               // below 2^29
    bool ok;
    switch (lanes) {
        case 1: ok = launch_rotate<1>(a, c.e4m3, grid, st); break;
        case 2: ok = launch_rotate<2>(a, c.e4m3, grid, st); break;
        case 4: ok = launch_rotate<4>(a, c.e4m3, grid, st); break;
        case 8: ok = launch_rotate<8>(a, c.e4m3, grid, st); break;
        default: ok = launch_rotate<16>(a, c.e4m3, grid, st); break;
    }
    return ok ? SKV_OK : SKV_ERR_CUDA;
}
