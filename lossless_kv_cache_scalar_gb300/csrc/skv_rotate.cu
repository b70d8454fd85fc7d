// skv_rotate.cu -- norms and rotation of query and key heads, keys and values into the pages.
//
// A head's channels are cut into units of 16: two vectors of 8 channels that are rotated with each
// other (channels 8 u .. and rot_dim / 2 + 8 u .., or 16 neighbours), so a lane that holds a unit
// has both sides of its 8 pairs, and the angles of its 8 frequencies serve every head of the token.
// head_dim / 16 lanes (rounded up to a power of two) hold a head, a warp 32 / that many heads at
// once; the norm's sum is a few shuffles among them. Norm's weights and angle of a pair come as
// four products, worked out once per row; the root is multiplied in at the end.
//
// Angles: position x frequency grows far beyond the bits that binary32 keeps of it. In turns, as a fraction of
// 2^64, the product modulo one turn is the low word of an integer product, and the sine
// is taken of a reduced angle in [-1/2, 1/2) turns.
//
// Bound by HBM, and close behind by issue (some 200 instructions for a warp's 4 heads of 128 channels): 65,536 rows of 32
// query and 8 KV heads, bf16, 244 us (6.6 TB/s, 0.97 of a copy); 30,000 rows of 40 and 8 into e4m3 131 us (0.90). Blocks
// of 4 warps, 7 to an SM (72 registers): with 6 257 us, with 8 (64 registers, some of them spilled) 253 and 210. The loads of the
// next step are on their way while a step is worked on; two steps ahead gave nothing.
#include <cuda_bf16.h>

#include "skv_rows.cuh"

namespace skv {

struct RotateArgs {
    const uint16_t *q, *k, *v;
    uint64_t q_row_stride, q_head_stride, row_stride, head_stride;      // elements
    uint16_t *q_out;
    uint32_t n_q_heads, n_heads, head_dim;
    uint32_t n, parts;                                                  // rows, warps per row
    uint32_t q_steps, kv_steps;                                         // a warp's steps over the heads of a kind
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
    uint32_t checked;                                                   // 1: block 0 reports the errors, 2: and does nothing else
};

constexpr uint32_t kRotateThreads = 128, kRotateWarps = kRotateThreads / 32u, kRotateBlocks = 7;      // blocks per SM
constexpr uint32_t kRotateChecked = 2048;        // rows that a block looks through for errors beside its own

__device__ __forceinline__ uint32_t pack2(float2 x) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x.y), "f"(x.x));
    return r;
}

__device__ __forceinline__ float2 unpack2(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }

__device__ __forceinline__ void unpack8(const uint4 &w, float2 *x) {
    x[0] = unpack2(w.x), x[1] = unpack2(w.y), x[2] = unpack2(w.z), x[3] = unpack2(w.w);
}

__device__ __forceinline__ uint4 pack8(const float2 *x) { return make_uint4(pack2(x[0]), pack2(x[1]), pack2(x[2]), pack2(x[3])); }

__device__ __forceinline__ uint2 quantise8(const float2 *x, const ScaleOf &s) {
    return make_uint2(e4m3x4_of(x[0], x[1], s), e4m3x4_of(x[2], x[3], s));
}

// LANES lanes to a head.
template <uint32_t LANES, bool E4M3>
__global__ void __launch_bounds__(kRotateThreads, kRotateBlocks) rotate_kernel(const RotateArgs a) {
    constexpr uint32_t HPW = 32u / LANES;
    // What a pair (x, y) of a row's frequency is multiplied with, the norm's weights w among it, for queries and for
    // keys: x' = x (w_x cos) + y (-w_y sin), y' = x (w_x sin) + y (w_y cos). Four frequencies of each unit
    // side by side, a unit's eight in two rows of each of the four.
    __shared__ float4 coef[kRotateWarps][2][8][LANES];
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, u = lane % LANES, own = lane / LANES;
    if (a.checked && blockIdx.x == 0) {
        // every slot, loads of 16 rounds in flight at once
        bool bad = false;
#pragma unroll 1
        for (uint32_t i0 = threadIdx.x; i0 < a.n; i0 += kRotateChecked) {
#pragma unroll
            for (uint32_t j = 0; j < kRotateChecked / kRotateThreads; ++j) {
                const uint32_t i = i0 + j * kRotateThreads;
                const int64_t s = i < a.n ? __ldg(a.slots + i) : -1;
                bad |= s >= 0 && (uint64_t)s >= a.pool_tokens;
            }
        }
        bad = __syncthreads_or(bad);
        if (threadIdx.x == 0) *a.status = bad ? SKV_ERR_INVALID_ARG : SKV_OK;
        if (a.checked == 2u) return;
    }
    const uint32_t first = a.checked == 2u ? blockIdx.x - 1u : blockIdx.x, blocks = a.checked == 2u ? gridDim.x - 1u : gridDim.x;
    const bool live = u < a.head_dim / 16u;
    const bool turned = u < a.rot_units;
    // channels of the unit's two vectors
    const uint32_t lo = turned && !a.interleaved ? 8u * u : 16u * u;
    const uint32_t apart = turned && !a.interleaved ? 8u * a.rot_units : 8u, hi = lo + apart;
    const uint64_t items = (uint64_t)a.n * a.parts, q_next = (uint64_t)a.parts * HPW * a.q_head_stride;
    const uint32_t out_next = a.parts * HPW * a.head_dim;
#pragma unroll 1
    for (uint64_t item = (uint64_t)first * kRotateWarps + warp; item < items; item += (uint64_t)blocks * kRotateWarps) {
        const uint32_t i = items >> 31 ? (uint32_t)(item / a.parts) : div_by((uint32_t)item, a.by_parts);
        const uint32_t part = (uint32_t)(item - (uint64_t)i * a.parts);
        // Steps of HPW heads of one kind: queries, then keys, then values.
        uint4 x0 = make_uint4(0u, 0u, 0u, 0u), x1 = x0;
        const auto fetch = [&](const uint16_t *src, bool on) {
            if (!on) return;
            x0 = *reinterpret_cast<const uint4 *>(src);
            x1 = *reinterpret_cast<const uint4 *>(src + apart);
        };
        const auto fetch_kv = [&](uint32_t t) {
            const uint32_t is_v = t >= a.kv_steps, h = (is_v ? t - a.kv_steps : t) * HPW + own;
            fetch((is_v ? a.v : a.k) + (uint64_t)i * a.row_stride + (uint64_t)h * a.head_stride + lo, live && t < 2u * a.kv_steps && h < a.n_heads);
        };
        const uint16_t *src = a.q + (uint64_t)i * a.q_row_stride + (uint64_t)(part * HPW + own) * a.q_head_stride + lo;
        if (part < a.q_steps) fetch(src, live && part * HPW + own < a.n_q_heads);
        const int64_t slot = __ldg(a.slots + i);
        bool to_pages = slot >= 0;
        if (to_pages && (uint64_t)slot >= a.pool_tokens) {
            to_pages = false;
            if (!a.checked) set_first(a.status, SKV_ERR_INVALID_ARG);
        }
        if (part >= a.q_steps && to_pages) fetch_kv(part - a.q_steps);
        __syncwarp();                                   // the last row's coefficients are read
#pragma unroll 1
        for (uint32_t j = lane; j < 8u * a.rot_units; j += 32u) {
            uint32_t ax = a.axis ? __ldg(a.axis + j) : 0u;
            if (ax >= a.n_axes) ax = 0u;
            const int64_t pos = __ldg(a.positions + (uint64_t)ax * a.n + i);
            const uint64_t t = __ldg(a.turns + j) * (uint64_t)pos;
            float c, s;
            sincospif((float)(int32_t)(t >> 32) * 0x1p-31f, &s, &c);
            c *= a.amplitude;
            s *= a.amplitude;
            const uint32_t x = a.interleaved ? 2u * j : j, y = a.interleaved ? x + 1u : j + 8u * a.rot_units;
#pragma unroll
            for (uint32_t k = 0; k < 2; ++k) {
                const float *w = k ? a.k_norm : a.q_norm;
                const float wx = w ? __ldg(w + x) : 1.0f, wy = w ? __ldg(w + y) : 1.0f;
                float *to = reinterpret_cast<float *>(&coef[warp][k][j >> 2 & 1u][j >> 3]) + (j & 3u);
                constexpr uint32_t next = 2u * LANES * 4u;
                to[0] = wx * c;
                to[next] = -wy * s;
                to[2u * next] = wx * s;
                to[3u * next] = wy * c;
            }
        }
        __syncwarp();
        // Norm and rotation of a unit of a head: `of` 0 a query's, 1 a key's.
        const auto turn = [&](float2 (&x)[8], uint32_t of) {
            const float *norm = of ? a.k_norm : a.q_norm;
            float2 r2 = make_float2(1.0f, 1.0f);
            if (norm) {
                float2 sum2 = mul2(x[0], x[0]);
#pragma unroll
                for (int j = 1; j < 8; ++j) sum2 = fma2(x[j], x[j], sum2);
                float sum = sum2.x + sum2.y;
#pragma unroll
                for (uint32_t d = 1; d < LANES; d <<= 1) sum += __shfl_xor_sync(~0u, sum, d);
                r2.x = r2.y = rsqrtf(fmaf(sum, a.inv_dim, a.eps));
            }
            if (turned) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float4 A = coef[warp][of][k][u], B = coef[warp][of][2 + k][u], C = coef[warp][of][4 + k][u], D = coef[warp][of][6 + k][u];
                    if (a.interleaved) {
                        const float ca[4] = {A.x, A.y, A.z, A.w}, cb[4] = {B.x, B.y, B.z, B.w}, cc[4] = {C.x, C.y, C.z, C.w}, cd[4] = {D.x, D.y, D.z, D.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 p = x[4 * k + j];
                            x[4 * k + j] = make_float2(fmaf(p.x, ca[j], p.y * cb[j]), fmaf(p.x, cc[j], p.y * cd[j]));
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float2 p = x[2 * k + j], q = x[2 * k + j + 4];
                            x[2 * k + j] = fma2(p, j ? make_float2(A.z, A.w) : make_float2(A.x, A.y), mul2(q, j ? make_float2(B.z, B.w) : make_float2(B.x, B.y)));
                            x[2 * k + j + 4] = fma2(p, j ? make_float2(C.z, C.w) : make_float2(C.x, C.y), mul2(q, j ? make_float2(D.z, D.w) : make_float2(D.x, D.y)));
                        }
                    }
                }
            } else if (norm && live) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 w = __ldg(reinterpret_cast<const float4 *>(norm + lo) + j);        // (lo and hi side by side)
                    x[2 * j] = mul2(x[2 * j], make_float2(w.x, w.y));
                    x[2 * j + 1] = mul2(x[2 * j + 1], make_float2(w.z, w.w));
                }
            }
            if (norm) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = mul2(x[j], r2);
            }
        };
        uint16_t *out = a.q_out + ((uint64_t)i * a.n_q_heads + part * HPW + own) * a.head_dim + lo;
        uint32_t t = part;
#pragma unroll 1
        for (; t < a.q_steps; t += a.parts, out += out_next) {
            const bool on = live && t * HPW + own < a.n_q_heads;
            float2 x[8];
            unpack8(x0, x);
            unpack8(x1, x + 4);
            if (t + a.parts < a.q_steps) {
                src += q_next;
                fetch(src, live && (t + a.parts) * HPW + own < a.n_q_heads);
            } else if (to_pages) {
                fetch_kv(t + a.parts - a.q_steps);
            }
            turn(x, 0u);
            if (on) {
                *reinterpret_cast<uint4 *>(out) = pack8(x);
                *reinterpret_cast<uint4 *>(out + apart) = pack8(x + 4);
            }
        }
        if (!to_pages) continue;
        const uint64_t p = a.pool_tokens >> 31 ? (uint64_t)slot / a.page.d : div_by((uint32_t)slot, a.page);
        const uint64_t dst = p * a.page_stride + ((uint64_t)slot - p * a.page.d) * a.token_stride;
#pragma unroll 1
        for (t -= a.q_steps; t < 2u * a.kv_steps; t += a.parts) {
            const uint32_t is_v = t >= a.kv_steps, g = (is_v ? t - a.kv_steps : t) * HPW + own;
            const bool on = live && g < a.n_heads;
            uint8_t *to = (is_v ? a.v_pages : a.k_pages) + dst + (uint64_t)g * a.page_head_stride;
            if (!E4M3 && is_v) {                        // bits as they are
                if (on) {
                    *reinterpret_cast<uint4 *>(to + 2u * lo) = x0;
                    *reinterpret_cast<uint4 *>(to + 2u * hi) = x1;
                }
                fetch_kv(t + a.parts);
                continue;
            }
            float2 x[8];
            unpack8(x0, x);
            unpack8(x1, x + 4);
            fetch_kv(t + a.parts);
            if (!is_v) turn(x, 1u);
            if (!on) continue;
            if (E4M3) {
                const float *scale = is_v ? a.v_scale : a.k_scale;
                const ScaleOf sc = scale_of(scale ? __ldg(scale + g) : 1.0f);
                *reinterpret_cast<uint2 *>(to + lo) = quantise8(x, sc);
                *reinterpret_cast<uint2 *>(to + hi) = quantise8(x + 4, sc);
            } else {
                *reinterpret_cast<uint4 *>(to + 2u * lo) = pack8(x);
                *reinterpret_cast<uint4 *>(to + 2u * hi) = pack8(x + 4);
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
    // Few rows' groups of heads go to several warps each, up to 24 warps per SM (1,000 rows of 32 query and 8 KV heads of 128 channels, bf16:
    // 6.5 us with three, 6.8 with two, 8.4 with one). Each works the angles out for itself, which takes as long as some four groups. So
    // where a warp to a row fills the GPU, two are better only by a shorter last round: the rounds of both are counted. One and two
    // warps, us: 3,600 rows 13.0, 14.6; 4,300 21.5, 19.0; 6,000 29.2, 27.3; 16,384 65.0, 65.3; 65,536 244.5, 246.2. Into e4m3 from 4,300 on 21.2,
    // 19.4; 29.1, 27.9; 64.6, 65.7; 235.6, 253.1; with 8 query heads 12.7, 13.4; 15.4, 18.3; 38.8, 44.6; 140.6, 170.0. Counted
    // wrongly just behind two whole rounds: 8,600 rows 41.6 (taken), 38.2.
    const uint32_t per_step = 32u / lanes, q_steps = (n_q_heads + per_step - 1u) / per_step;
    const uint32_t kv_steps = (cache->n_heads + per_step - 1u) / per_step, groups = q_steps + 2u * kv_steps;
    uint32_t parts = 24u * sms / n;
    if (parts < 2u) {
        const uint64_t warps = (kRotateBlocks * sms - 1u) * kRotateWarps;
        const uint64_t one = (n + warps - 1u) / warps * (groups + 4u), two = (2ull * n + warps - 1u) / warps * ((groups + 1u) / 2u + 4u);
        parts = two < one ? 2u : 1u;
    }
    parts = parts > groups ? groups : parts;
    RotateArgs a{};
    a.q = static_cast<const uint16_t *>(q), a.k = static_cast<const uint16_t *>(k), a.v = static_cast<const uint16_t *>(v);
    a.q_row_stride = q_row_stride, a.q_head_stride = q_head_stride, a.row_stride = row_stride, a.head_stride = row_head_stride;
    a.q_out = static_cast<uint16_t *>(q_out);
    a.n_q_heads = n_q_heads, a.n_heads = cache->n_heads, a.head_dim = cache->head_dim;
    a.n = n, a.parts = parts, a.by_parts = fast_div(parts), a.q_steps = q_steps, a.kv_steps = kv_steps;
    a.turns = rotary->turns, a.axis = rotary->axis, a.q_norm = rotary->q_norm, a.k_norm = rotary->k_norm, a.positions = positions;
    a.rot_units = rotary->rot_dim / 16u, a.n_axes = rotary->n_axes, a.interleaved = rotary->interleaved;
    a.eps = rotary->eps, a.inv_dim = 1.0f / (float)cache->head_dim, a.amplitude = rotary->amplitude;
    a.k_pages = static_cast<uint8_t *>(cache->k_pages), a.v_pages = static_cast<uint8_t *>(cache->v_pages);
    a.page_stride = c.page_stride, a.token_stride = c.token_stride, a.page_head_stride = c.head_stride;
    a.k_scale = c.k_scale, a.v_scale = c.v_scale, a.page = c.page;
    a.pool_tokens = (uint64_t)cache->n_pages * cache->page_tokens;
    // Errors are looked for by one block (it writes the status once, where clearing it first is a launch of its own): up to 2,048 rows on
    // its way, up to 65,536 as all it does, beyond by whoever meets them. With the launch and so: 2,049 rows of one head of 16 channels
    // 6.4 and 3.7 us, 65,536 of them 65.7 and 62.2; 65,536 of 8 + 8 + 8 heads of 64 81.8 and 79.2, but 262,144 312 and 329.
    a.slots = slots, a.status = status, a.checked = n <= kRotateChecked ? 1u : n <= 65536u ? 2u : 0u;
    if (!a.checked && cudaMemsetAsync(status, 0, sizeof(int32_t), st) != cudaSuccess) return SKV_ERR_CUDA;
    const uint64_t blocks = ((uint64_t)n * parts + kRotateWarps - 1) / kRotateWarps;
    const uint64_t all = blocks + (a.checked == 2u);
    const unsigned grid = (unsigned)(all < kRotateBlocks * sms ? all : kRotateBlocks * sms);
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
