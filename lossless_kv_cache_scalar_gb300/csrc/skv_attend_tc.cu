// skv_attend_tc.cu -- tree attention for more than 16 query rows per KV head, on
// the fifth-generation tensor cores (the mathematics: skv_attend.cu; the split of
// the work: skv_attend.cuh).
//
// A part has up to 256 query rows (node-major, the query heads of one KV head)
// and runs over its positions in tiles of 128. Two streams share the tensor
// cores so that one computes weights while the other multiplies:
//   more than 128 rows   stream s holds rows 128 s .. 128 s + 127 and every tile
//                        enters both: a K or V tile is read once for 256 rows
//   up to 128 rows       both streams hold the same rows and take the tiles in
//                        turn; their two results are joined at the end
// A job is one stream with one tile; jobs alternate between the streams.
//   warps 0-3, 4-7  the weights of stream 0 and 1, one thread per row
//   warps 8-11      queries; 8-bit tiles raised to fp16; pages of other lengths, row by row
//   warp 12         one lane issues the matrix products
//   warp 13         tensor copies of K and V into the ring, page by page
//   warps 14, 15    only give up their registers
// Per job: S = Q K^T (128 x 128, accumulated in tensor memory), the row's thread
// turns S into weights and writes them over S as 16-bit values, O += W V with the
// weights read from tensor memory. K lies in shared memory as [position][channel],
// channels contiguous (K-major operand); V lies the same way and is the
// MN-major operand of the second product, so neither is transposed. Both in
// rows of 128 bytes with the 128-byte swizzle.
//
// The reference of a row's weights lags behind the row's largest score (kLag), so the output in
// tensor memory is rarely scaled anew; sums stay binary32.
//
// Bound: from 129 rows on by the products (2 x 128 x 128 x DP per job, 2^12 multiply-adds per clock) and the
// first product's shared-memory reads (8 KB for 64 clocks of work); below that by the pages' bytes.
// Measured, us, 19 requests x 16,384 positions x 8 heads x 128 channels, pages of 256, 8 query heads per KV
// head: bf16 64 rows 190 (6.7 TB/s: a copy's rate), 256 rows 244 (1,340 TFLOP/s); e4m3 64 rows 182, 256 rows
// 250. Why not larger jobs or deeper buffers: two streams of 128 x 128 scores and their outputs fill
// tensor memory; jobs of 64 positions with two score buffers each took 13% longer.
#include <cuda.h>

#include "skv_attend.cuh"

namespace skv {

constexpr uint32_t kTcThreads = 512, kTcRows = kLargeRows, kTile = 128;

template <int DP, bool E>
struct TcShape {
    static constexpr uint32_t block = kTile * 128;              // 128 rows of 128 bytes: 64 channels
    static constexpr uint32_t tile = block * (DP / 64);         // one K, V or 128-row Q tile in 16-bit values
    static constexpr uint32_t ring = 4 * (128 / DP);            // tiles
    static constexpr uint32_t raw = E ? 2 * (128 / DP) : 0;     // tiles of 8-bit codes on their way to the ring
    static constexpr uint32_t raw_tile = kTile * DP;
    static constexpr uint32_t raw_at = (2 + ring) * tile;       // from the queries' start
    // where rows are copied one by one, their offsets: four tiles' (then no codes are on their way)
    static constexpr uint32_t offsets = 4 * kTile * 8;
    static constexpr uint32_t smem = raw_at + (E ? raw * raw_tile : offsets);
};

// The parts of a CTA's share, in order; every role walks them for itself.
struct Walk {
    uint64_t at, u1;                                // units: the item's start, the share's end
    uint32_t r, tiles, rts, h, rt;
    ReqOf q;
    uint32_t n;                                     // parts so far
    // the part: tiles [tile, tile_end) of the item
    uint32_t tile, tile_end, rows, weight;          // rows of this row tile, units of a tile
    uint32_t wide, narrow;

    __device__ __forceinline__ void request(const AttendArgs &a) {
        tiles = (q.len + a.span - 1) / a.span;
        rts = (q.n * a.group + kTcRows - 1) / kTcRows;
        h = rt = 0;
    }
    __device__ __forceinline__ void item(const AttendArgs &a) {
        rows = min(kTcRows, q.n * a.group - rt * kTcRows);
        weight = both() ? wide : narrow;
    }
    // The tiles that start before the share's end.
    __device__ __forceinline__ void part() {
        const uint64_t left = u1 > at ? u1 - at : 0u;
        tile_end = left >= (uint64_t)tiles * weight ? tiles : ((uint32_t)left + weight - 1) / weight;
    }
    __device__ __forceinline__ void advance(const AttendArgs &a) {
        at += (uint64_t)tiles * weight;
        tile = tile_end = 0;
        if (at >= u1) return;
        if (++rt == rts) {
            rt = 0;
            if (++h == a.c.n_heads) {
                do q = request_of(a, ++r);
                while (q.n == 0);
                request(a);
            }
        }
        item(a);
        part();
    }
    __device__ __forceinline__ void start(const AttendArgs &a, const Share &s) {
        u1 = s.u1;
        r = s.r;
        n = 0;
        wide = s.wide;
        narrow = s.narrow;
        q = request_of(a, r);
        request(a);
        const uint32_t last = q.n * a.group - (rts - 1) * kTcRows > kTile ? wide : narrow;
        const uint64_t full = (uint64_t)tiles * wide, head = (rts - 1) * full + (uint64_t)tiles * last;
        h = (uint32_t)quotient(s.off, head);
        uint64_t off = s.off - h * head;
        rt = min((uint32_t)quotient(off, full), rts - 1);
        off -= rt * full;
        at = s.u0 - off;
        item(a);
        tile = (uint32_t)quotient(off + weight - 1, weight);
        part();
        if (tile >= tiles) advance(a);
    }
    __device__ __forceinline__ bool more() const { return tile < tile_end; }
    __device__ __forceinline__ bool both() const { return rows > kTile; }          // 129 rows on: every tile in both streams
    __device__ __forceinline__ uint32_t count() const { return tile_end - tile; }
    __device__ __forceinline__ void next(const AttendArgs &a) {
        ++n;
        if (tile_end < tiles) tile = tile_end;      // the share ends in this item
        else advance(a);
    }
};

struct TcShared {
    unsigned long long plan[2 * kTcThreads / 32 + 4];
    unsigned long long full[8], empty[8];        // ring
    unsigned long long landed[8], taken[8];      // tensor copies that the filling warps finish
    int32_t pages[4][16];                        // page numbers of a tile's boxes
    unsigned long long s_full[2], p_ready[2], o_done[2], q_full, q_empty, drain;
    uint8_t scaled[2][kTcRows];                  // e4m3: exponent of each row's scale, 127 + e
    float m1[kTile], l1[kTile];                  // stream 1's maxima and sums, for the join
    uint32_t hurt[4];                            // part by part: a V value that is not finite was put to 0
    uint32_t tmem;
    uint32_t gave_up, stopped;                   // a wait ran out; no tensor copy is started any more
    Walk walk[2];                                // the weights' threads keep their registers for scores
};

__device__ __forceinline__ uint32_t s32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void bar_init(const void *b, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(s32(b)), "r"(n) : "memory");
}

__device__ __forceinline__ void bar_arrive(const void *b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(s32(b)) : "memory");
}

// One arrival for a warp: what its lanes did before is ordered before it.
__device__ __forceinline__ void warp_arrive(const void *b) {
    __syncwarp();
    if ((threadIdx.x & 31u) == 0u) bar_arrive(b);
}

// How a wait looks at its barrier (try_wait sleeps on it for a while, test_wait does not) and when it
// runs out. A test builds the kernel with a limit of its own.
#ifndef SKV_WAIT_CLOCKS
#define SKV_WAIT_CLOCKS 4000000000ll
#define SKV_BAR_TRY "mbarrier.try_wait"
#else
#define SKV_BAR_TRY "mbarrier.test_wait"
#endif

__device__ __forceinline__ bool bar_try(uint32_t at, uint32_t parity) {
    uint32_t ok;
    asm volatile("{.reg .pred p; " SKV_BAR_TRY ".parity.shared::cta.b64 p, [%1], %2; selp.b32 %0, 1, 0, p;}"
                 : "=r"(ok) : "r"(at), "r"(parity) : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool bar_try(const void *b, uint32_t parity) { return bar_try(s32(b), parity); }

// Waits for the phase of that parity, at most about two seconds; false where it gave up. From
// the first wait that runs out on, every wait of the CTA that is not over gives up at once, and
// the CTA runs to its end on whatever it holds (all addresses stay in bounds), to report TIMEOUT.
__device__ __forceinline__ bool bar_wait(TcShared &sm, const void *b, uint32_t parity) {
    if (bar_try(b, parity)) return true;
    const long long t0 = clock64();
    while (!bar_try(b, parity)) {
        if (*reinterpret_cast<volatile uint32_t *>(&sm.gave_up)) return false;
        if (clock64() - t0 > SKV_WAIT_CLOCKS) {
            *reinterpret_cast<volatile uint32_t *>(&sm.gave_up) = 1u;
            return false;
        }
    }
    return true;
}

// For whoever gave up on a tile and is about to go on as if it had come: the place that it frees then may
// still be on its way, and a barrier armed twice for copies in one phase is undefined. So
// first, with a limit, no more copies are started.
__device__ __forceinline__ void copies_stopped(const TcShared &sm) {
    const long long t0 = clock64();
    while (!*reinterpret_cast<const volatile uint32_t *>(&sm.stopped) && clock64() - t0 < 4000000000ll) {}
}

// For what is on its way itself, whether the CTA gave up or not.
__device__ __forceinline__ void bar_last(uint32_t at, uint32_t parity) {
    const long long t0 = clock64();
    while (!bar_try(at, parity) && clock64() - t0 < 4000000000ll) {}
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tc_commit(const void *b) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(s32(b)) : "memory");
}

// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elected() {
    uint32_t ok;
    asm volatile("{.reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.b32 %0, 1, 0, p;}" : "=r"(ok));
    return ok != 0;
}

// Shared-memory operand: 128-byte swizzle, 8-row groups `group` bytes apart (bits 32-45);
// lead: distance of 64-channel blocks where the contiguous dimension is not the
// product's (bits 16-29).
__device__ __forceinline__ uint64_t tc_operand(uint32_t at, uint32_t lead, uint32_t group) {
    return (uint64_t)((at >> 4) & 0x3FFFu) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(group >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, bool add) {
    asm volatile("{.reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;}" ::"r"(d),
                 "l"(a), "l"(b), "r"(kind), "r"((uint32_t)add) : "memory");
}

__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t kind, bool add) {
    asm volatile("{.reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;}" ::"r"(d),
                 "r"(a), "l"(b), "r"(kind), "r"((uint32_t)add) : "memory");
}

#define SKV_R4(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])
#define SKV_I4(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])

// One box of a pool: `rows` positions of one page and head, from channel x on.
__device__ __forceinline__ void tc_box(uint32_t dst, const CUtensorMap *map, uint32_t x, uint32_t h, uint32_t token, int32_t page,
                                       const void *bar) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
                 ::"r"(dst), "l"(map), "r"(s32(bar)), "r"(x), "r"(h), "r"(token), "r"(page) : "memory");
}

// The same with both 64-channel blocks of a head in one box, eight positions of one, then of the other.
__device__ __forceinline__ void tc_box_folded(uint32_t dst, const CUtensorMap *map, uint32_t block, uint32_t eight, int32_t page,
                                              const void *bar) {
    asm volatile("cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %3, %4, %5, %6}], [%2];"
                 ::"r"(dst), "l"(map), "r"(s32(bar)), "r"(0), "r"(block), "r"(eight), "r"(page) : "memory");
}

// 32 columns of this warp's 32 rows of tensor memory.
__device__ __forceinline__ void tc_ld32(uint32_t (&r)[32], uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : SKV_R4(r, 0), SKV_R4(r, 4), SKV_R4(r, 8), SKV_R4(r, 12), SKV_R4(r, 16), SKV_R4(r, 20), SKV_R4(r, 24), SKV_R4(r, 28)
        : "r"(at) : "memory");
}

__device__ __forceinline__ void tc_ld16(uint32_t (&r)[16], uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : SKV_R4(r, 0), SKV_R4(r, 4), SKV_R4(r, 8), SKV_R4(r, 12) : "r"(at) : "memory");
}

__device__ __forceinline__ void tc_st16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::SKV_I4(r, 0),
        SKV_I4(r, 4), SKV_I4(r, 8), SKV_I4(r, 12), "r"(at) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Two binary32 values in one 64-bit register: one instruction for both.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
    return (uint64_t)__float_as_uint(lo) | ((uint64_t)__float_as_uint(hi) << 32);
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 32 bytes to a 32-byte boundary.
__device__ __forceinline__ void store32(void *at, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f, uint32_t g,
                                        uint32_t h) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(f),
                 "r"(g), "r"(h) : "memory");
}

// The 128 threads of one stream's weights.
__device__ __forceinline__ void group_sync(uint32_t s) { asm volatile("bar.sync %0, 128;" ::"r"(3u + s) : "memory"); }

template <bool E>
__device__ __forceinline__ uint32_t tc_pack(float lo, float hi) {
    uint32_t r;
    if (E) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight e4m3 codes as fp16.
__device__ __forceinline__ uint4 tc_raise8(uint32_t a, uint32_t b) {
    uint4 r;
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h;}" : "=r"(r.x), "=r"(r.y) : "r"(a));
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h;}" : "=r"(r.z), "=r"(r.w) : "r"(b));
    return r;
}

__device__ __forceinline__ uint2 ld_shared8(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ void st_shared16(uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Which tile fills the e-th place of a part of T tiles, in the order in which the
// products need them: K0 V0 K1 V1 ... where both streams take every tile, else
// K0 K1 V0 K2 V1 K3 ... V(T-2) V(T-1).
__device__ __forceinline__ uint32_t fill_of(bool both, uint32_t T, uint32_t e, bool &is_v) {
    if (both || T == 1) {
        is_v = e & 1u;
        return e >> 1;
    }
    if (e < 2) {
        is_v = false;
        return e;
    }
    is_v = !(e & 1u) || e == 2 * T - 1;
    return e == 2 * T - 1 ? T - 1 : is_v ? (e - 2) / 2 : (e - 2) / 2 + 2;
}

// A tile's layout in the ring: 64-channel blocks one after the other, or, where a box brings both
// (a.folded), eight positions of one and of the other in turn.
template <int DP, bool E>
__device__ __forceinline__ uint32_t block_of(const AttendArgs &a) { return !E && DP == 128 && a.folded ? 1024u : TcShape<DP, E>::block; }
__device__ __forceinline__ uint32_t group_of(const AttendArgs &a) { return a.folded ? 2048u : 1024u; }

// The part's query rows as the first product's operand, by the 128 filling threads.
template <int DP, bool E>
__device__ __forceinline__ void fill_queries(const AttendArgs &a, const Walk &w, TcShared &sm, uint32_t q_at) {
    using S = TcShape<DP, E>;
    const uint32_t t = threadIdx.x - 256u;
    const bool both = w.both();
    if (w.n) bar_wait(sm, &sm.q_empty, (w.n - 1) & 1u);
    if (t == 0) sm.hurt[w.n & 3u] = 0u;
    asm volatile("bar.sync 2, 128;" ::: "memory");                   // the last part's offsets are read, the flag is down
    const uint32_t q_rows = both ? 256u : 128u;
    // a negative scale turns the queries, so that the weights' threads look for the largest score in any case
    const bool turned = a.scale * (a.c.k_scale ? __ldg(a.c.k_scale + w.h) : 1.0f) < 0.0f;
    if (!E) {
        constexpr uint32_t CH = DP / 8;                          // 16-byte chunks of a row
        for (uint32_t x = t; x < q_rows * CH; x += 128u) {
            const uint32_t row = x / CH, ch = x % CH, all = w.rt * kTcRows + row, node = all / a.group, g = all - node * a.group;
            const bool live = node < w.q.n && ch * 8u < a.c.head_dim;
            const uint16_t *src = live ? a.q + (uint64_t)(w.q.row0 + node) * a.q_row_stride +
                                             (uint64_t)(w.h * a.group + g) * a.q_head_stride + ch * 8u : a.q;
            const uint32_t dst = q_at + (row >> 7) * S::tile + (ch >> 3) * S::block + (row & 127u) * 128u + (((ch ^ row) & 7u) << 4);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16u : 0u) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (turned) {
            for (uint32_t x = t; x < q_rows * CH; x += 128u) {       // this thread's own copies
                const uint32_t row = x / CH, ch = x % CH;
                const uint32_t at = q_at + (row >> 7) * S::tile + (ch >> 3) * S::block + (row & 127u) * 128u + (((ch ^ row) & 7u) << 4);
                const uint2 lo = ld_shared8(at), hi = ld_shared8(at + 8u);
                st_shared16(at, make_uint4(lo.x ^ 0x80008000u, lo.y ^ 0x80008000u, hi.x ^ 0x80008000u, hi.y ^ 0x80008000u));
            }
        }
    } else {
        // fp16 after a power-of-two scale per row (skv_attend.cu): one thread per row
        for (uint32_t row = t; row < q_rows; row += 128u) {
            const uint32_t all = w.rt * kTcRows + row, node = all / a.group, g = all - node * a.group;
            const bool live = node < w.q.n;
            const uint4 *src = reinterpret_cast<const uint4 *>(
                live ? a.q + (uint64_t)(w.q.row0 + node) * a.q_row_stride + (uint64_t)(w.h * a.group + g) * a.q_head_stride : a.q);
            float top = 0.0f;
            const uint32_t chunks = live ? a.c.head_dim / 8u : 0u;
            for (uint32_t ch = 0; ch < chunks; ++ch) {
                const uint4 v = __ldg(src + ch);
                const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[i] << 16)), fabsf(__uint_as_float(x[i] & 0xFFFF0000u))));
            }
            const uint32_t e = __float_as_uint(top) >> 23;
            const bool usual = e > 2u && e < 252u;
            const float down = (usual ? __uint_as_float((254u - e) << 23) : 1.0f) * (turned ? -1.0f : 1.0f);
            sm.scaled[w.n & 1u][row] = (uint8_t)(usual ? e : 127u);
            for (uint32_t ch = 0; ch < DP / 8u; ++ch) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (ch < chunks) {
                    v = __ldg(src + ch);
                    uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[i] = tc_pack<true>(__uint_as_float(x[i] << 16) * down, __uint_as_float(x[i] & 0xFFFF0000u) * down);
                    v = make_uint4(x[0], x[1], x[2], x[3]);
                }
                st_shared16(q_at + (row >> 7) * S::tile + (ch >> 3) * S::block + (row & 127u) * 128u + (((ch ^ row) & 7u) << 4), v);
            }
        }
    }
    proxy_fence();
    warp_arrive(&sm.q_full);
}

// Pages whose length is no multiple of 8: every row is looked up and copied by itself.
template <int DP, bool E>
__device__ __forceinline__ void fill_role(const AttendArgs &a, const Share &sh, TcShared &sm, uint32_t q_at, uint32_t ring_at,
                                          uint64_t (*at_of)[kTile], bool &corrupt) {
    using S = TcShape<DP, E>;
    const uint32_t t = threadIdx.x - 256u;
    const uint32_t row_bytes = a.c.head_dim * (E ? 1u : 2u);
    uint32_t pos = 0;                                                // tiles begun, over all parts
    Walk w;
    for (w.start(a, sh); w.more(); w.next(a)) {
        const bool both = w.both();
        const uint32_t T = w.count(), p_end = min(w.q.len, w.tile_end * kTile);
        fill_queries<DP, E>(a, w, sm, q_at);
        // ---- K and V tiles
        // Offsets of a tile's positions: a thread each, into one of four places, a tile ahead.
        uint64_t next_at = ~0ull;
        const auto look_up = [&](uint32_t k) {
            next_at = ~0ull;
            const uint32_t p = (w.tile + k) * kTile + t;
            if (k < T && p < p_end) {
                next_at = place_of(a.c, w.r, w.h, p);
                corrupt |= next_at == ~0ull;
            }
        };
        look_up(0);
        const auto offsets = [&](uint32_t k) {
            at_of[k & 3u][t] = next_at;
            asm volatile("bar.sync 2, 128;" ::: "memory");
            look_up(k + 1);
        };
        if (!E) {
            constexpr uint32_t CH = DP / 8, PER = kTile * CH / 128;   // chunks per row, copies per thread
            constexpr uint32_t LAG = 2;                               // tiles in flight behind the newest
            // Tile e of the part has landed: clear what is not finite among drafted V, tell the products.
            const auto landed = [&](uint32_t e) {
                bool is_v;
                const uint32_t k = fill_of(both, T, e, is_v), slot = (pos + e) % S::ring;
                const uint32_t p0 = (w.tile + k) * kTile;
                if (is_v && p0 + kTile > w.q.ctx) {
                    bool found = false;
                    for (uint32_t i = 0; i < PER; ++i) {
                        const uint32_t x = i * 128u + t, row = x / CH, ch = x % CH;
                        if (p0 + row < w.q.ctx) continue;
                        const uint32_t at = ring_at + slot * S::tile + (ch >> 3) * S::block + row * 128u + (((ch ^ row) & 7u) << 4);
                        uint32_t v[4];
                        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at) : "memory");
                        bool hit = false;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if ((v[j] & 0x7F80u) == 0x7F80u) v[j] &= 0xFFFF0000u, hit = true;
                            if ((v[j] & 0x7F800000u) == 0x7F800000u) v[j] &= 0xFFFFu, hit = true;
                        }
                        if (hit) st_shared16(at, make_uint4(v[0], v[1], v[2], v[3]));
                        found |= hit;
                    }
                    if (found) *reinterpret_cast<volatile uint32_t *>(&sm.hurt[w.n & 3u]) = 1u;
                }
                proxy_fence();
                warp_arrive(&sm.full[slot]);
            };
            for (uint32_t e = 0; e < 2 * T; ++e) {
                bool is_v;
                const uint32_t k = fill_of(both, T, e, is_v), slot = (pos + e) % S::ring;
                if (!is_v) offsets(k);
                bar_wait(sm, &sm.empty[slot], (((pos + e) / S::ring) & 1u) ^ 1u);
                const uint8_t *base = is_v ? a.c.v : a.c.k;
#pragma unroll
                for (uint32_t i = 0; i < PER; ++i) {
                    const uint32_t x = i * 128u + t, row = x / CH, ch = x % CH;
                    const uint64_t at = at_of[k & 3u][row];
                    const bool live = at != ~0ull && ch * 16u < row_bytes;
                    const uint32_t dst = ring_at + slot * S::tile + (ch >> 3) * S::block + row * 128u + (((ch ^ row) & 7u) << 4);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(base + (live ? at + ch * 16u : 0ull)),
                                 "r"(live ? 16u : 0u) : "memory");
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (e >= LAG) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(LAG) : "memory");
                    landed(e - LAG);
                }
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            for (uint32_t e = 2 * T > LAG ? 2 * T - LAG : 0u; e < 2 * T; ++e) landed(e);
        } else {
            constexpr uint32_t CH = DP / 16, PER = kTile * CH / 128;  // 16 codes each
            uint4 now[PER], next[PER];
            const auto load = [&](uint32_t e, uint4(&v)[PER]) {
                bool is_v;
                const uint32_t k = fill_of(both, T, e, is_v);
                if (!is_v) offsets(k);
                const uint8_t *base = is_v ? a.c.v : a.c.k;
#pragma unroll
                for (uint32_t i = 0; i < PER; ++i) {
                    const uint32_t x = i * 128u + t, row = x / CH, ch = x % CH;
                    const uint64_t at = at_of[k & 3u][row];
                    v[i] = at != ~0ull && ch * 16u < row_bytes ? __ldg(reinterpret_cast<const uint4 *>(base + at + ch * 16u))
                                                               : make_uint4(0u, 0u, 0u, 0u);
                }
            };
            load(0, now);
            for (uint32_t e = 0; e < 2 * T; ++e) {
                if (e + 1 < 2 * T) load(e + 1, next);
                bool is_v;
                const uint32_t k = fill_of(both, T, e, is_v), slot = (pos + e) % S::ring;
                const uint32_t p0 = (w.tile + k) * kTile;
                bar_wait(sm, &sm.empty[slot], (((pos + e) / S::ring) & 1u) ^ 1u);
                bool found = false;
#pragma unroll
                for (uint32_t i = 0; i < PER; ++i) {
                    const uint32_t x = i * 128u + t, row = x / CH, ch = x % CH;
                    uint32_t c[4] = {now[i].x, now[i].y, now[i].z, now[i].w};
                    if (is_v && p0 + row >= w.q.ctx) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int b = 0; b < 32; b += 8)
                                if (((c[j] >> b) & 0x7Fu) == 0x7Fu) c[j] &= ~(0xFFu << b), found = true;
                    }
                    const uint32_t at = ring_at + slot * S::tile + (ch >> 2) * S::block + row * 128u;
                    const uint32_t c0 = 2u * ch;
                    st_shared16(at + (((c0 ^ row) & 7u) << 4),
                                tc_raise8(c[0], c[1]));
                    st_shared16(at + ((((c0 + 1u) ^ row) & 7u) << 4),
                                tc_raise8(c[2], c[3]));
                }
                if (found) *reinterpret_cast<volatile uint32_t *>(&sm.hurt[w.n & 3u]) = 1u;
                proxy_fence();
                warp_arrive(&sm.full[slot]);
#pragma unroll
                for (uint32_t i = 0; i < PER; ++i) now[i] = next[i];
            }
        }
        pos += 2 * T;
    }
}

// Pages of a multiple of 8 positions: a tile holds `span` positions in boxes of `box`, a
// divisor of the page length, so that no box crosses a page (paged_box). A lane
// per box looks the page up one tile ahead and starts the box's copies; a page number
// outside the pool is outside the tensor and reads 0. Boxes past the part's end are
// not copied: their scores are not used and finish_role clears their V.
template <int DP, bool E>
__device__ __forceinline__ void box_role(const AttendArgs &a, const Share &sh, TcShared &sm, uint32_t ring_at, uint32_t raw_at,
                                         const CUtensorMap *kmap, const CUtensorMap *vmap, bool &corrupt) {
    using S = TcShape<DP, E>;
    const uint32_t lane = threadIdx.x & 31u, boxes = a.span / a.box;
    constexpr uint32_t kRaw = E ? S::raw : 1;
    uint32_t pos = 0, filled = 0;                                    // tiles begun over all parts; tiles copied
    bool ok = true;
    Walk w;
    for (w.start(a, sh); ok && w.more(); w.next(a)) {
        const bool both = w.both();
        const uint32_t T = w.count(), p_end = min(w.q.len, w.tile_end * a.span);
        int32_t next_page = 0;
        const auto look_up = [&](uint32_t k) {
            const uint32_t p = (w.tile + k) * a.span + lane * a.box;
            if (k < T && lane < boxes && p < p_end) {
                next_page = __ldg(a.c.table + (uint64_t)w.r * a.c.table_stride + div_by(p, a.c.page));
                if ((uint32_t)next_page >= a.c.n_pages) {
                    corrupt = true;
                    next_page = (int32_t)a.c.n_pages;
                }
            }
        };
        look_up(0);
        for (uint32_t e = 0; e < 2 * T; ++e) {
            bool is_v;
            const uint32_t k = fill_of(both, T, e, is_v), n = pos + e, p0 = (w.tile + k) * a.span;
            if (!is_v) {
                if (lane < 16u) sm.pages[k & 3u][lane] = next_page;
                __syncwarp();
                look_up(k + 1);
            }
            const uint32_t slot = n % S::ring;
            const void *bar;
            uint32_t dst;
            if (E) {
                const uint32_t raw = n % kRaw;
                ok = bar_wait(sm, &sm.taken[raw], ((n / kRaw) & 1u) ^ 1u);
                bar = &sm.landed[raw];
                dst = raw_at + raw * S::raw_tile;
            } else {
                ok = bar_wait(sm, &sm.empty[slot], ((n / S::ring) & 1u) ^ 1u);
                bar = is_v && p0 + a.span > w.q.ctx ? &sm.landed[slot] : &sm.full[slot];
                dst = ring_at + slot * S::tile;
            }
            const uint32_t live = min(boxes, (p_end - p0 + a.box - 1) / a.box);
            if (lane == 0 && ok)                                     // (at worst armed and then left alone)
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(s32(bar)), "r"(live * a.box * DP * (E ? 1u : 2u)) : "memory");
            ok = __all_sync(~0u, ok);
            if (!ok) {
                filled = n;
                break;
            }
            if (lane < live) {
                const int32_t page = sm.pages[k & 3u][lane];
                const uint32_t p = p0 + lane * a.box, token = p - div_by(p, a.c.page) * a.c.page.d;
                const CUtensorMap *map = is_v ? vmap : kmap;
                if (E) {
                    tc_box(dst + lane * a.box * DP, map, 0u, w.h, token, page, bar);
                } else if (DP == 128 && a.folded) {
                    tc_box_folded(dst + lane * a.box * 256u, map, 2u * w.h, token >> 3, page, bar);
                } else {
#pragma unroll
                    for (uint32_t b = 0; b < DP / 64; ++b)
                        tc_box(dst + b * S::block + lane * a.box * 128u, map, 64u * b, w.h, token, page, bar);
                }
            }
            __syncwarp();
        }
        pos += 2 * T;
    }
    if (ok) filled = pos;
    __syncwarp();
    if (lane == 0) *reinterpret_cast<volatile uint32_t *>(&sm.stopped) = 1u;
    // No copy is on its way into this CTA's shared memory when the roles meet at the end: lane i waits for the
    // last of the tiles that went to place i (in bf16 a V tile with drafted positions is full only once it has landed).
    constexpr uint32_t places = E ? kRaw : S::ring;
    if (lane < places && lane < filled) bar_last(s32(E ? &sm.landed[lane] : &sm.full[lane]), ((filled - 1u - lane) / places) & 1u);
    __syncwarp();
}

// Beside box_role: queries; every tile of an 8-bit cache raised to fp16; and in V tiles with
// drafted positions, what is not finite there, and what lies past the end, put to 0.
template <int DP, bool E>
__device__ __forceinline__ void finish_role(const AttendArgs &a, const Share &sh, TcShared &sm, uint32_t q_at, uint32_t ring_at,
                                            uint32_t raw_at) {
    using S = TcShape<DP, E>;
    const uint32_t t = threadIdx.x - 256u;
    const uint32_t block = block_of<DP, E>(a), group = group_of(a);
    uint32_t pos = 0, turns = 0;                                     // turns: parity of landed[] by slot (bf16)
    bool good = true;                                                // (bf16) no tile was given up
    Walk w;
    for (w.start(a, sh); w.more(); w.next(a)) {
        const bool both = w.both();
        const uint32_t T = w.count(), p_end = min(w.q.len, w.tile_end * a.span);
        fill_queries<DP, E>(a, w, sm, q_at);
        for (uint32_t e = 0; e < 2 * T; ++e) {
            bool is_v;
            const uint32_t k = fill_of(both, T, e, is_v), n = pos + e, p0 = (w.tile + k) * a.span, slot = n % S::ring;
            const bool edge = is_v && p0 + a.span > w.q.ctx;
            if (!E && !edge) continue;
            const uint32_t first = w.q.ctx > p0 ? w.q.ctx - p0 : 0u, last = min(a.span, p_end - p0);     // drafted rows [first, last)
            bool found = false;
            if (!E) {
                if (!bar_wait(sm, &sm.landed[slot], (turns >> slot) & 1u)) good = false;
                turns ^= 1u << slot;
                constexpr uint32_t CH = DP / 8;
                for (uint32_t x = first * CH + t; x < kTile * CH; x += 128u) {
                    const uint32_t row = x / CH, ch = x % CH;
                    const uint32_t at = ring_at + slot * S::tile + (ch >> 3) * block + (row >> 3) * group + (row & 7u) * 128u + (((ch ^ row) & 7u) << 4);
                    uint32_t v[4];
                    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at) : "memory");
                    bool hit = false;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if ((v[j] & 0x7F80u) == 0x7F80u) v[j] &= 0xFFFF0000u, hit = true;
                        if ((v[j] & 0x7F800000u) == 0x7F800000u) v[j] &= 0xFFFFu, hit = true;
                    }
                    if (row >= last) st_shared16(at, make_uint4(0u, 0u, 0u, 0u));
                    else if (hit) st_shared16(at, make_uint4(v[0], v[1], v[2], v[3])), found = true;
                }
            } else {
                constexpr uint32_t kRaw = E ? S::raw : 1;
                const uint32_t raw = n % kRaw;
                if (!bar_wait(sm, &sm.landed[raw], (n / kRaw) & 1u)) copies_stopped(sm);
                __syncwarp();
                // Thread: 16 codes of channels 16 ch .. of every (128 / CH)th row. The eight bytes that go first
                // differ between the two 64-channel blocks, so that eight lanes' stores lie on different banks.
                constexpr uint32_t CH = DP / 16, PER = kTile * CH / 128, STEP = 128 / CH;
                const uint32_t ch = t % CH, row0 = t / CH, turn = (ch >> 2) & 1u;
                const uint32_t from = raw_at + raw * S::raw_tile + t * 16u + turn * 8u, to = ring_at + slot * S::tile + (ch >> 2) * S::block + row0 * 128u;
                const uint32_t to0 = to + (((2u * ch + turn) ^ row0) & 7u) * 16u, to1 = to + (((2u * ch + 1u - turn) ^ row0) & 7u) * 16u;
                uint2 c[PER][2];
#pragma unroll
                for (uint32_t i = 0; i < PER; ++i) {
                    c[i][0] = ld_shared8(from + i * 2048u);
                    c[i][1] = ld_shared8((from ^ 8u) + i * 2048u);
                }
                warp_arrive(&sm.taken[raw]);
                bar_wait(sm, &sm.empty[slot], ((n / S::ring) & 1u) ^ 1u);
                if (edge) {
#pragma unroll
                    for (uint32_t i = 0; i < PER; ++i) {
                        const uint32_t row = row0 + i * STEP;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t &x = j & 1 ? c[i][j >> 1].y : c[i][j >> 1].x;
#pragma unroll
                            for (int b = 0; b < 32; b += 8)
                                if (row >= first && row < last && ((x >> b) & 0x7Fu) == 0x7Fu) x &= ~(0xFFu << b), found = true;
                            if (row >= last) x = 0u;
                        }
                    }
                }
#pragma unroll
                for (uint32_t i = 0; i < PER; ++i) {
                    st_shared16(to0 + i * STEP * 128u, tc_raise8(c[i][0].x, c[i][0].y));
                    st_shared16(to1 + i * STEP * 128u, tc_raise8(c[i][1].x, c[i][1].y));
                }
            }
            if (found) *reinterpret_cast<volatile uint32_t *>(&sm.hurt[w.n & 3u]) = 1u;
            proxy_fence();
            if (E) {
                warp_arrive(&sm.full[slot]);
            } else {
                asm volatile("bar.sync 2, 128;" ::: "memory");
                if (t == 0 && good) bar_arrive(&sm.full[slot]);
            }
        }
        pos += 2 * T;
    }
}

template <int DP, bool E>
__device__ __forceinline__ void product_role(const AttendArgs &a, const Share &sh, TcShared &sm, uint32_t q_at, uint32_t ring_at,
                                             uint32_t tmem) {
    using S = TcShape<DP, E>;
    // binary32 accumulators; both inputs fp16 (0) or bf16 (1); 128 rows
    constexpr uint32_t kind0 = (1u << 4) | ((E ? 0u : 1u) << 7) | ((E ? 0u : 1u) << 10) | (8u << 24);
    constexpr uint32_t kind_s = kind0 | ((kTile >> 3) << 17), kind_o = kind0 | (1u << 16) | (((uint32_t)DP >> 3) << 17);
    // The whole warp walks the jobs and one lane issues: what the operands' descriptors are
    // made of is the same in every lane, so it stays in uniform registers (a branch
    // for one thread moves every descriptor there anew).
    tmem = __shfl_sync(~0u, tmem, 0);
    const uint32_t block = block_of<DP, E>(a), group = group_of(a);
    const uint64_t q_op = tc_operand(q_at, 16u, 1024u), k_op = tc_operand(ring_at, 16u, group), v_op = tc_operand(ring_at, block, group);
    uint32_t pos = 0, jobs[2] = {0u, 0u};
    Walk w;
    for (w.start(a, sh); __shfl_sync(~0u, (int)w.more(), 0); w.next(a)) {
        const bool both = __shfl_sync(~0u, (int)w.both(), 0);
        const uint32_t T = __shfl_sync(~0u, w.count(), 0), J = both ? 2 * T : T;
        bar_wait(sm, &sm.q_full, w.n & 1u);
        uint32_t k_slot = 0, v_slot = 0;
        const auto take = [&](uint32_t &slot) {
            slot = pos % S::ring;
            if (!bar_wait(sm, &sm.full[slot], (pos / S::ring) & 1u)) copies_stopped(sm);
            ++pos;
        };
        const auto scores = [&](uint32_t j) {
            const uint32_t s = j & 1u;
            if (!both || s == 0) take(k_slot);
            __syncwarp();
            tc_fence_after();
            if (elected()) {
                const uint64_t qa = q_op + (both && s ? S::tile >> 4 : 0u), ka = k_op + ((k_slot * S::tile) >> 4);
#pragma unroll
                for (uint32_t k = 0; k < DP / 16; ++k) {
                    const uint32_t in = ((k & 3u) * 32u) >> 4;
                    tc_mma_ss(tmem + s * kTile, qa + (((k >> 2) * S::block) >> 4) + in, ka + (((k >> 2) * block) >> 4) + in, kind_s, k != 0);
                }
                tc_commit(&sm.s_full[s]);
                if (!both || s) tc_commit(&sm.empty[k_slot]);
                if (j + 1 == J) tc_commit(&sm.q_empty);
            }
            __syncwarp();
        };
        scores(0);
        if (J > 1) scores(1);
        for (uint32_t j = 0; j < J; ++j) {
            const uint32_t s = j & 1u;
            if (!both || s == 0) take(v_slot);
            bar_wait(sm, &sm.p_ready[s], jobs[s] & 1u);
            ++jobs[s];
            __syncwarp();
            tc_fence_after();
            if (elected()) {
                const uint64_t va = v_op + ((v_slot * S::tile) >> 4);
#pragma unroll
                for (uint32_t k = 0; k < kTile / 16; ++k)
                    tc_mma_ts(tmem + 256u + s * DP, tmem + s * kTile + k * 8u, va + ((k * 2u * group) >> 4), kind_o, j > 1 || k != 0);
                tc_commit(&sm.o_done[s]);
                if (!both || s) tc_commit(&sm.empty[v_slot]);
            }
            __syncwarp();
            if (j + 2 < J) scores(j + 2);
        }
    }
    // Nothing of this CTA is left in the tensor cores when the roles meet at the end.
    if (elected()) tc_commit(&sm.drain);
    __syncwarp();
    bar_last(s32(&sm.drain), 0u);
}

template <int DP, bool E>
__device__ __forceinline__ void weight_role(const AttendArgs &a, const AttendWs &ws, const Share &sh, TcShared &sm, uint32_t tmem) {
    const uint32_t s = threadIdx.x >> 7, t = threadIdx.x & 127u, lanes = (t & ~31u) << 16;
    const uint32_t at_s = tmem + lanes + s * kTile, at_o = tmem + lanes + 256u + s * DP;
    uint32_t jobs = 0, others = 0;                                   // of this stream and of stream 1, over all parts
    Walk &w = sm.walk[s];
    if (t == 0) w.start(a, sh);
    group_sync(s);
    while (w.more()) {
        const bool both = w.both();
        const uint32_t T = w.count(), p_end = min(w.q.len, w.tile_end * a.span);
        const uint32_t row = both ? s * kTile + t : t;               // of the row tile
        const uint32_t all = w.rt * kTcRows + row, node = all / a.group, g = w.h * a.group + all - node * a.group;
        const bool live = row < w.rows, warp_live = (row & ~31u) < w.rows;
        // (no wait for the queries here: a part of few jobs can be two phases behind the filling warps)
        float mul = a.scale * (a.c.k_scale ? __ldg(a.c.k_scale + w.h) : 1.0f) * 1.4426950408889634f;
        // (a negative scale has turned the queries;) at least 2^-149, so that -infinity times it stays that
        if (!E) mul = fmaxf(fabsf(mul), 0x1p-149f);
        float m = -INFINITY, l = 0.0f;
        uint32_t done = 0;                                           // jobs of this part
        for (uint32_t k = both ? 0u : s; k < T; k += both ? 1u : 2u, ++done, ++jobs) {
            bar_wait(sm, &sm.s_full[s], jobs & 1u);
            __syncwarp();
            tc_fence_after();
            if (E && done == 0) mul = fmaxf(fabsf(mul) * __uint_as_float((uint32_t)sm.scaled[w.n & 1u][row] << 23), 0x1p-149f);
            const uint32_t p0 = (w.tile + k) * a.span;
            const bool edge = p0 + a.span > w.q.ctx || p0 + a.span > p_end, cut = a.span < kTile;
            if (warp_live) {
                // a span below 128 positions (at least 112) ends inside the last 32 columns
                uint32_t bits[4] = {~0u, ~0u, ~0u, cut ? (1u << (a.span - 96u)) - 1u : ~0u};
                if (edge && live) {
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t seen = sees32(a, w.q, node, p0 + 32u * c, p_end);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k == c) bits[k] &= seen;
                    }
                }
                __syncwarp();
                // the row's 128 scores, all in registers; -infinity where it does not see
                uint32_t x[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tc_ld32(x[c], at_s + 32u * c);
                tc_wait_ld();
                if (edge) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!((bits[c] >> i) & 1u)) x[c][i] = 0xFF800000u;
                } else if (cut) {
#pragma unroll
                    for (int i = 16; i < 32; ++i)
                        if (!((bits[3] >> i) & 1u)) x[3][i] = 0xFF800000u;
                }
                float far[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; i += 2) far[c] = max3(far[c], __uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]));
                far[0] = fmaxf(fmaxf(far[0], far[1]), fmaxf(far[2], far[3]));
                const float top = far[0] * mul;                      // in base 2
                const bool move = top > m + (kLag + kLower<E>) || (m == -INFINITY && top > m);
                const float keep = move ? part_weight(m, top - kLower<E>) : 1.0f;
                if (move) m = top - kLower<E>;
                l *= keep;
                if (__any_sync(~0u, move) && done) {
                    bar_wait(sm, &sm.o_done[s], (jobs - 1u) & 1u);
                    __syncwarp();
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < DP / 16; ++c) {              // 16 at a time: the scores stay in registers
                        uint32_t y[16];
                        tc_ld16(y, at_o + 16u * c);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * keep);
                        tc_st16(at_o + 16u * c, y);
                    }
                    tc_wait_st();
                }
                const float base = m == -INFINITY ? 0.0f : m;
                const uint64_t mul2 = pair_of(mul, mul), base2 = pair_of(-base, -base);
                uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t y[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        uint64_t z = fma2((uint64_t)x[c][i] | ((uint64_t)x[c][i + 1] << 32), mul2, base2);
                        const float w0 = ex2(__uint_as_float((uint32_t)z)), w1 = ex2(__uint_as_float((uint32_t)(z >> 32)));
                        sum2[(i >> 1) & 1] = add2(sum2[(i >> 1) & 1], pair_of(w0, w1));
                        y[i / 2] = tc_pack<E>(w0, w1);
                    }
                    tc_st16(at_s + 16u * c, y);
                }
                sum2[0] = add2(sum2[0], sum2[1]);
                l += __uint_as_float((uint32_t)sum2[0]) + __uint_as_float((uint32_t)(sum2[0] >> 32));
                tc_wait_st();
            }
            tc_fence_before();
            warp_arrive(&sm.p_ready[s]);
        }
        // ---- the part's result
        if (!both) {
            if (s == 1) {
                sm.m1[t] = done ? m : -INFINITY;
                sm.l1[t] = l;
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
        }
        others += both ? T : T / 2;
        if (done && (both || s == 0)) {
            bar_wait(sm, &sm.o_done[s], (jobs - 1u) & 1u);
            if (!both && T > 1) bar_wait(sm, &sm.o_done[1], (others - 1u) & 1u);
            __syncwarp();
            tc_fence_after();
            if (warp_live) {
                const bool whole = w.tile == 0 && w.tile_end == w.tiles, two = !both && T > 1;
                const bool hurt = *reinterpret_cast<volatile uint32_t *>(&sm.hurt[w.n & 3u]) != 0u;
                float f0 = 1.0f, f1 = 0.0f;
                if (two) {
                    const float m1 = sm.m1[t], M = fmaxf(m, m1);
                    f0 = part_weight(m, M);
                    f1 = part_weight(m1, M);
                    l = f0 * l + f1 * sm.l1[t];
                    m = M;
                }
                const float norm = !whole ? 1.0f : l == 0.0f ? 0.0f : (a.c.v_scale ? __ldg(a.c.v_scale + w.h) : 1.0f) / l;
                f0 *= norm;
                f1 *= norm;
                const uint32_t place = w.tile ? 0u : 1u;
                float *part = ws.parts + ((uint64_t)blockIdx.x * 2u + place) * part_floats(kTcRows, DP);
                uint16_t *out = a.out + ((uint64_t)(w.q.row0 + node) * a.n_q_heads + g) * a.c.head_dim;
#pragma unroll 1
                for (int c = 0; c < DP / 32; ++c) {
                    uint32_t x[32];
                    __syncwarp();
                    tc_ld32(x, at_o + 32u * c);
                    tc_wait_ld();
                    if (two) {
                        uint32_t y[32];
                        tc_ld32(y, at_o + DP + 32u * c);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            x[i] = __float_as_uint(__uint_as_float(x[i]) * f0 + __uint_as_float(y[i]) * f1);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f0);
                    }
                    if (hurt && live) {
#pragma unroll 1
                        for (int i = 0; i < 32; ++i) {
                            if (32u * c + i >= a.c.head_dim) break;
                            const float add = not_finite_sum(a, w.q, w.r, w.h, node, 32u * c + i, w.tile * a.span, p_end);
#pragma unroll
                            for (int j = 0; j < 32; ++j)             // registers have no index of their own
                                if (j == i) x[j] = __float_as_uint(__uint_as_float(x[j]) + add);
                        }
                    }
                    if (live && whole) {
                        uint32_t y[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            y[i] = l == 0.0f ? 0u : tc_pack<false>(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
#pragma unroll
                        for (int i = 0; i < 16; i += 8) {
                            if (32u * c + 2 * i >= a.c.head_dim) break;
                            if (((uintptr_t)out & 31u) == 0) {
                                store32(out + 32u * c + 2 * i, y[i], y[i + 1], y[i + 2], y[i + 3], y[i + 4], y[i + 5], y[i + 6], y[i + 7]);
                            } else {
                                *reinterpret_cast<uint4 *>(out + 32u * c + 2 * i) = make_uint4(y[i], y[i + 1], y[i + 2], y[i + 3]);
                                *reinterpret_cast<uint4 *>(out + 32u * c + 2 * i + 8) = make_uint4(y[i + 4], y[i + 5], y[i + 6], y[i + 7]);
                            }
                        }
                    } else if (live) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8)              // a whole 32-byte sector per lane and store
                            store32(part + 2u * kTcRows + row * DP + 32u * c + i, x[i], x[i + 1], x[i + 2], x[i + 3], x[i + 4],
                                    x[i + 5], x[i + 6], x[i + 7]);
                    }
                }
                if (live && whole && a.lse)
                    a.lse[(uint64_t)(w.q.row0 + node) * a.n_q_heads + g] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
                if (live && !whole) {
                    part[row] = m;
                    part[kTcRows + row] = l;
                }
                if (threadIdx.x == 0 && w.tile == 0 && !whole)
                    ws.desc[blockIdx.x] = Desc{1u, w.r, w.h, w.rt, w.at + (uint64_t)(w.tiles - 1) * w.weight};
            }
            tc_fence_before();
        }
        // stream 1 goes on once its output has been read
        if (!both) asm volatile("bar.sync 1, 256;" ::: "memory");
        else group_sync(s);
        if (t == 0) w.next(a);
        group_sync(s);
    }
}

template <int DP, bool E>
__global__ void __launch_bounds__(kTcThreads, 1) attend_large(const AttendArgs a, const AttendWs ws,
                                                              const __grid_constant__ CUtensorMap kmap,
                                                              const __grid_constant__ CUtensorMap vmap) {
    using S = TcShape<DP, E>;
    extern __shared__ __align__(1024) uint8_t dyn[];
    __shared__ TcShared sm;
    const uint32_t tid = threadIdx.x, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Share sh = share_of<kTcThreads, true>(a, ws, kTcRows, a.span, sm.plan);
    if (sh.u0 == sh.u1) return;
    const uint32_t q_at = s32(dyn), ring_at = q_at + 2u * S::tile, raw_at = q_at + S::raw_at;
    if (tid == 0) {
        for (uint32_t i = 0; i < 8; ++i) {
            bar_init(&sm.full[i], a.box && !E ? 1u : 4u);     // the copies' own arrival, or four warps'
            bar_init(&sm.empty[i], 1u);
            bar_init(&sm.landed[i], 1u);
            bar_init(&sm.taken[i], 4u);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            bar_init(&sm.s_full[i], 1u);
            bar_init(&sm.p_ready[i], 4u);
            bar_init(&sm.o_done[i], 1u);
        }
        bar_init(&sm.q_full, 4u);
        bar_init(&sm.q_empty, 1u);
        bar_init(&sm.drain, 1u);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sm.gave_up = 0u;
        sm.stopped = a.box ? 0u : 1u;
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(s32(&sm.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    if (a.span < kTile) {
        // rows of the ring (and of the codes behind it) that no copy reaches: read as 0, not as what was there
        const uint32_t rows = kTile - a.span;
        for (uint32_t x = tid; x < S::ring * (DP / 64u) * rows * 8u; x += kTcThreads) {
            const uint32_t row = a.span + x / 8u % rows, of = x / (rows * 8u);
            st_shared16(ring_at + of / (DP / 64u) * S::tile + of % (DP / 64u) * block_of<DP, E>(a) + (row >> 3) * group_of(a) + (row & 7u) * 128u +
                            x % 8u * 16u, make_uint4(0u, 0u, 0u, 0u));
        }
        for (uint32_t x = tid; x < S::raw * rows * (DP / 16u); x += kTcThreads)
            st_shared16(raw_at + x / (rows * (DP / 16u)) * S::raw_tile + a.span * DP + x % (rows * (DP / 16u)) * 16u, make_uint4(0u, 0u, 0u, 0u));
        proxy_fence();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    bool corrupt = false;
    // 512 threads of 128 registers, dealt out anew: per lane of the four groups 2 x 184 + 88 + 56 (bf16) and
    // 2 x 184 + 96 + 48 (e4m3, whose second group converts) = 4 x 128.
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        weight_role<DP, E>(a, ws, sh, sm, tmem);
    } else if (warp < 12) {
        if (E) asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (a.box) finish_role<DP, E>(a, sh, sm, q_at, ring_at, raw_at);
        else fill_role<DP, E>(a, sh, sm, q_at, ring_at, reinterpret_cast<uint64_t(*)[kTile]>(dyn + S::raw_at), corrupt);
    } else {
        if (E) asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 13 && a.box) box_role<DP, E>(a, sh, sm, ring_at, raw_at, &kmap, &vmap, corrupt);
        if (warp == 12) product_role<DP, E>(a, sh, sm, q_at, ring_at, tmem);
    }
    __syncwarp();
    tc_fence_before();
    corrupt = __syncthreads_or(corrupt);
    if (warp == 12) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
    if (tid == 0) {
        if (sm.gave_up) ws.errs[blockIdx.x] = SKV_ERR_TIMEOUT;
        else if (corrupt && ws.errs[blockIdx.x] == SKV_OK) ws.errs[blockIdx.x] = SKV_ERR_CORRUPT;
    }
}

// The driver's tensor-map encoder, through the runtime (the library does not link libcuda).
typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiled encoder() {
    static std::atomic<EncodeTiled> known{nullptr};
    EncodeTiled f = known.load(std::memory_order_acquire);
    if (!f) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        f = reinterpret_cast<EncodeTiled>(p);
        known.store(f, std::memory_order_release);
    }
    return f;
}

// A pool as a tensor [page][token][head][channel] read in boxes of `box` tokens of one head; folded: as
// [page][token / 8][64-channel block][token % 8][channel], both blocks of a head in a box.
static bool pool_map(CUtensorMap *map, const PagedView &c, const uint8_t *pool, uint32_t DP, bool folded) {
    const EncodeTiled f = encoder();
    if (!f) return false;
    const bool e = c.e4m3;
    const uint64_t page_stride = c.n_pages > 1 ? c.page_stride : 16u;
    if (folded) {
        const cuuint64_t dims[5] = {64u, 8u, 2u * c.n_heads, c.page.d / 8u, c.n_pages};
        const cuuint64_t strides[4] = {c.token_stride, 128u, 8u * c.token_stride, page_stride};
        const cuuint32_t box[5] = {64u, 8u, 2u, paged_box(c.page.d) / 8u, 1u}, one[5] = {1u, 1u, 1u, 1u, 1u};
        return f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<uint8_t *>(pool), dims, strides, box, one,
                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    }
    const cuuint64_t dims[4] = {c.head_dim, c.n_heads, c.page.d, c.n_pages};
    // the stride of a dimension of one entry is never used, but has to be a valid one
    const cuuint64_t strides[3] = {c.n_heads > 1 ? c.head_stride : 16u, c.page.d > 1 ? c.token_stride : 16u,
                                   page_stride};
    const cuuint32_t box[4] = {e ? DP : 64u, 1u, paged_box(c.page.d), 1u}, one[4] = {1u, 1u, 1u, 1u};
    // L2 fetches no more than a row: what lies behind it is another head's, wanted much later
    const uint32_t row = c.head_dim * (e ? 1u : 2u);
    const CUtensorMapL2promotion fetch = row >= 256u ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                       : row >= 128u ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_NONE;
    return f(map, e ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint8_t *>(pool), dims, strides,
             box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, e ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
             fetch, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP, bool E>
static bool launch(AttendArgs a, const AttendWs &ws, cudaStream_t st) {
    static std::atomic<uint64_t> ready{0};
    constexpr uint32_t bytes = TcShape<DP, E>::smem;
    static_assert(bytes + (sizeof(TcShared) + 1023) / 1024 * 1024 <= 232448 && TcShape<DP, E>::ring <= 8 && TcShape<DP, E>::raw <= 8, "shared memory of a CTA");
    if (!raise_smem(reinterpret_cast<const void *>(attend_large<DP, E>), bytes, ready)) return false;
    CUtensorMap kmap = {}, vmap = {};
    // strides reach 2^41 bytes, a tensor map's less than 2^40
    a.box = a.c.page_stride < (uint64_t(1) << 40) && a.c.token_stride < (uint64_t(1) << 40) && a.c.head_stride < (uint64_t(1) << 40)
                ? paged_box(a.c.page.d) : 0u;
    // heads side by side, as the coder lays pages out: half as many boxes, which counts where they are small
    a.folded = !E && a.c.head_dim == 128u && a.box && a.box < 128u && (a.c.n_heads == 1u || a.c.head_stride == 256u);
    if (a.box && !(pool_map(&kmap, a.c, a.c.k, DP, a.folded) && pool_map(&vmap, a.c, a.c.v, DP, a.folded))) a.box = a.folded = 0u;    // row by row
    a.span = a.box ? kTile / a.box * a.box : kTile;
    attend_large<DP, E><<<kCtasLarge, kTcThreads, bytes, st>>>(a, ws, kmap, vmap);
    return cudaGetLastError() == cudaSuccess && launch_join(a, ws, kTcRows, DP, kCtasLarge, st);
}

bool launch_large(const AttendArgs &a, const AttendWs &ws, cudaStream_t st) {
    if (a.c.e4m3) return a.c.head_dim <= 64 ? launch<64, true>(a, ws, st) : launch<128, true>(a, ws, st);
    return a.c.head_dim <= 64 ? launch<64, false>(a, ws, st) : launch<128, false>(a, ws, st);
}

}  // namespace skv
