// skv_attend.cu -- attention of a tree of drafted tokens over a paged KV cache.
//
// For query row i (node j of request r) and query head g, over the positions p
// that the row sees: s_p = scale q . K_p, out = sum w_p V_p / sum w_p with
// w_p = exp(s_p - m), m the running maximum; what was summed under an older
// maximum is scaled by exp(m_old - m) (the ratio is unchanged).
//
// One CTA per (row, query head), 128 positions at a time: a thread per score,
// then a thread per channel.
#include "skv_paged.h"

namespace skv {

constexpr uint32_t kNone = 0xFFFFFFFFu;

__device__ __forceinline__ float code_value(const PagedView &c, const uint8_t *p, uint32_t d) {
    if (!c.e4m3) return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(p)[d] << 16);
    const uint32_t b = p[d], e = (b >> 3) & 15u, m = b & 7u;
    float v = e ? __uint_as_float(((e + 120u) << 23) | (m << 20)) : (float)m * 0.001953125f;
    if ((b & 127u) == 127u) v = __uint_as_float(0x7FC00000u);
    return (b & 128u) ? -v : v;
}

__device__ __forceinline__ uint16_t bf16_bits(float x) {
    uint32_t b = __float_as_uint(x);
    if ((b & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((b >> 16) | 0x40u);
    return (uint16_t)((b + 0x7FFFu + ((b >> 16) & 1u)) >> 16);
}

// Request r's rows and lengths; SKV_OK with n = 0 for one without rows.
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

__device__ __forceinline__ bool sees(const AttendArgs &a, const ReqOf &q, uint32_t node, uint32_t p) {
    if (p < q.ctx) return true;
    const uint32_t j = p - q.ctx;
    if (!a.mask) return j <= node;
    return (a.mask[(uint64_t)(q.row0 + node) * a.mask_words + (j >> 6)] >> (j & 63u)) & 1u;
}

__global__ void __launch_bounds__(128) attend_simple(AttendArgs a) {
    __shared__ float s_q[256], s_w[128], s_red[4];
    __shared__ uint64_t s_at[128];
    const uint32_t tid = threadIdx.x, row = blockIdx.x, g = blockIdx.y, h = g / a.group;
    uint32_t r = 0;
    ReqOf q{0u, 0u, 0u, 0u, SKV_OK};
    for (; r < a.c.n_requests; ++r) {
        q = request_of(a, r);
        if (q.err && tid == 0) set_first(a.status, q.err);
        if (q.n && row >= q.row0 && row < q.row0 + q.n) break;
    }
    if (r == a.c.n_requests) return;
    const uint32_t node = row - q.row0, D = a.c.head_dim;
    for (uint32_t d = tid; d < D; d += 128u)
        s_q[d] = __uint_as_float((uint32_t)a.q[(uint64_t)row * a.q_row_stride + (uint64_t)g * a.q_head_stride + d] << 16);
    __syncthreads();
    const float mul = a.scale * (a.c.k_scale ? a.c.k_scale[h] : 1.0f);
    float m = -INFINITY, l = 0.0f, o[2] = {0.0f, 0.0f};
    for (uint32_t p0 = 0; p0 < q.len; p0 += 128u) {
        const uint32_t p = p0 + tid;
        uint64_t at = ~0ull;
        float s = -INFINITY;
        if (p < q.len && sees(a, q, node, p)) {
            const uint32_t j = div_by(p, a.c.page);
            const int32_t page = a.c.table[(uint64_t)r * a.c.table_stride + j];
            if ((uint32_t)page < a.c.n_pages) {
                at = (uint64_t)page * a.c.page_stride + (uint64_t)(p - j * a.c.page.d) * a.c.token_stride +
                     h * a.c.head_stride;
                s = 0.0f;
                for (uint32_t d = 0; d < D; ++d) s = fmaf(s_q[d], code_value(a.c, a.c.k + at, d), s);
                s *= mul;
            } else set_first(a.status, SKV_ERR_CORRUPT);
        }
        s_at[tid] = at;
        float t = s;
        for (uint32_t d = 16; d; d >>= 1) t = fmaxf(t, __shfl_xor_sync(~0u, t, d));
        if ((tid & 31u) == 0) s_red[tid >> 5] = t;
        __syncthreads();
        const float top = fmaxf(m, fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])));
        const float base = top == -INFINITY ? 0.0f : top;
        s_w[tid] = at == ~0ull ? 0.0f : expf(s - base);
        const float keep = m == -INFINITY ? 0.0f : expf(m - base);
        m = top;
        __syncthreads();
        l *= keep;
        o[0] *= keep;
        o[1] *= keep;
        for (uint32_t i = 0; i < 128u; ++i) {
            if (s_at[i] == ~0ull) continue;
            l += s_w[i];
            if (tid < D) o[0] = fmaf(s_w[i], code_value(a.c, a.c.v + s_at[i], tid), o[0]);
            if (tid + 128u < D) o[1] = fmaf(s_w[i], code_value(a.c, a.c.v + s_at[i], tid + 128u), o[1]);
        }
        __syncthreads();
    }
    const float inv = (l == 0.0f ? 0.0f : 1.0f / l) * (a.c.v_scale ? a.c.v_scale[h] : 1.0f);
    uint16_t *out = a.out + ((uint64_t)row * a.n_q_heads + g) * D;
    if (tid < D) out[tid] = bf16_bits(l == 0.0f ? 0.0f : o[0] * inv);
    if (tid + 128u < D) out[tid + 128u] = bf16_bits(l == 0.0f ? 0.0f : o[1] * inv);
    if (a.lse && tid == 0) a.lse[(uint64_t)row * a.n_q_heads + g] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace skv

using namespace skv;

extern "C" int32_t skv_tree_attention_workspace_bytes(const skv_paged *cache, uint32_t n_q_heads, uint64_t *bytes) {
    const int32_t r = skv_paged_check(cache);
    if (r != SKV_OK) return r;
    if (!bytes || n_q_heads == 0 || n_q_heads % cache->n_heads) return SKV_ERR_INVALID_ARG;
    *bytes = 256;
    return SKV_OK;
}

extern "C" int32_t skv_tree_attention(const skv_paged *cache, const void *q, uint64_t q_row_stride,
                                      uint64_t q_head_stride, uint32_t n_q_heads, uint32_t n_rows,
                                      const int32_t *ctx_len, const int32_t *cu_new, const uint64_t *mask,
                                      uint32_t mask_words, uint32_t max_nodes, float scale, void *out, float *lse,
                                      int32_t *status, void *workspace, uint64_t ws_bytes, void *stream) {
    uint64_t need = 0;
    const int32_t r = skv_tree_attention_workspace_bytes(cache, n_q_heads, &need);
    if (r != SKV_OK) return r;
    const auto off = [](const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) != 0; };
    if (!status || off(status, 4) || !workspace || off(workspace, 256) || ws_bytes < need) return SKV_ERR_INVALID_ARG;
    if (cache->n_requests > 0x7FFFFFFEu || n_rows > 0x7FFFFFFFu || n_q_heads > 65535u || cache->max_pages > 0x7FFFFFFFu ||
        (cache->n_requests > 1 && cache->table_stride < cache->max_pages) || !(scale == scale) ||
        (mask != nullptr) != (mask_words != 0) || mask_words > (1u << 20))
        return SKV_ERR_INVALID_ARG;
    const uint64_t most = uint64_t(1) << 40;
    if (q_row_stride % 8u || q_head_stride % 8u || q_row_stride > most || q_head_stride > most) return SKV_ERR_INVALID_ARG;
    if (cache->n_requests && n_rows &&
        (!q || !out || !ctx_len || !cu_new || !cache->block_table || off(q, 16) || off(out, 16) || off(ctx_len, 4) ||
         off(cu_new, 4) || off(cache->block_table, 4) || off(mask, 8) || off(lse, 4)))
        return SKV_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(status, 0, sizeof(int32_t), st) != cudaSuccess) return SKV_ERR_CUDA;
    if (cache->n_requests == 0 || n_rows == 0) return SKV_OK;
    (void)max_nodes;
    AttendArgs a{paged_view(*cache), static_cast<const uint16_t *>(q), q_row_stride, q_head_stride, n_q_heads,
                 n_q_heads / cache->n_heads, n_rows, ctx_len, cu_new, mask, mask_words, scale,
                 static_cast<uint16_t *>(out), lse, status};
    attend_simple<<<dim3(n_rows, n_q_heads), 128, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? SKV_OK : SKV_ERR_CUDA;
}
