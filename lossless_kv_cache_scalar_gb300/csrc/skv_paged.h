// skv_paged.h -- argument blocks of the paged-cache operators (skv_paged.cu,
// skv_attend.cu): the device's view of a skv_paged and of each call.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "skv.h"

namespace skv {

// n / d and n % d for 0 <= n < 2^31 by a multiplication: with s = ceil(log2 d)
// and m = ceil(2^(31 + s) / d), floor(n m / 2^(31 + s)) = floor(n / d), since
// m d - 2^(31 + s) < d <= 2^s keeps the error n (m d - 2^(31+s)) / (d 2^(31+s))
// below 1 / d. m < 2^32 fits a word.
struct FastDiv {
    uint32_t d, m, s;
};

inline FastDiv fast_div(uint32_t d) {
    FastDiv f{d, 0, 0};
    while ((uint64_t(1) << f.s) < d) ++f.s;
    f.m = (uint32_t)(((uint64_t(1) << (31 + f.s)) + d - 1) / d);
    return f;
}

__device__ __forceinline__ uint32_t div_by(uint32_t n, FastDiv f) {
    return (uint32_t)(((uint64_t)n * f.m) >> (31 + f.s));
}

struct PagedView {
    const uint8_t *k;         // bytes
    const uint8_t *v;
    uint64_t page_stride;     // bytes
    uint64_t token_stride;
    uint64_t head_stride;
    const float *k_scale;     // or NULL
    const float *v_scale;
    const int32_t *table;
    uint64_t table_stride;
    FastDiv page;             // page_tokens
    uint32_t n_pages;
    uint32_t n_heads;
    uint32_t head_dim;
    uint32_t n_requests;
    uint32_t max_pages;
    uint32_t e4m3;
};

struct AttendArgs {
    PagedView c;
    const uint16_t *q;        // bf16 bits
    uint64_t q_row_stride;    // elements
    uint64_t q_head_stride;
    uint32_t n_q_heads;
    uint32_t group;           // n_q_heads / n_heads
    uint32_t n_rows;
    const int32_t *ctx_len;
    const int32_t *cu_new;
    const uint64_t *mask;     // or NULL
    uint32_t mask_words;
    float scale;
    uint16_t *out;
    float *lse;               // or NULL
    int32_t *status;
    uint32_t box;             // positions of a tensor copy, 0: none fits the page length
    uint32_t span;            // positions of a tile: 128 / box boxes, or 128
    uint32_t folded;          // 1: a copy brings both 64-channel blocks of a head of 128 channels
};

// Positions of a tensor copy for a page length: the largest divisor of it that is a
// multiple of 8 (the swizzle's period) and of which whole boxes fill at least 112 of a
// tile's 128 rows; 0 if the length is no multiple of 8. A copy costs some 45 clocks
// beside its rows: with boxes of 8 a page of 24 took 410 us where whole pages (five of 24, 120 of
// 128 rows used) take 245, 209 with both blocks of a head in one box, and a page of 256 190 (19 requests x 16,384 positions x 8 heads x 128 channels, bf16, 64 rows).
inline uint32_t paged_box(uint32_t page) {
    for (uint32_t b = page < 128u ? page : 128u; b >= 8u; --b)
        if (b % 8u == 0 && page % b == 0 && 128u / b * b >= 112u) return b;
    return 0u;
}

inline PagedView paged_view(const skv_paged &c) {
    const uint64_t b = c.dtype == SKV_BF16 ? 2u : 1u;
    PagedView v;
    v.k = static_cast<const uint8_t *>(c.k_pages);
    v.v = static_cast<const uint8_t *>(c.v_pages);
    v.page_stride = c.page_stride * b;
    v.token_stride = c.token_stride * b;
    v.head_stride = c.head_stride * b;
    v.k_scale = c.k_scale;
    v.v_scale = c.v_scale;
    v.table = c.block_table;
    v.table_stride = c.table_stride;
    v.page = fast_div(c.page_tokens);
    v.n_pages = c.n_pages;
    v.n_heads = c.n_heads;
    v.head_dim = c.head_dim;
    v.n_requests = c.n_requests;
    v.max_pages = c.max_pages;
    v.e4m3 = c.dtype == SKV_E4M3;
    return v;
}

__device__ __forceinline__ void set_first(int32_t *status, int32_t code) {
    atomicCAS(status, SKV_OK, code);
}

}  // namespace skv
