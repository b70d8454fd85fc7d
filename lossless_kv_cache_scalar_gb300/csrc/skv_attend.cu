// skv_attend.cu -- attention of a tree of drafted tokens over a paged KV cache.
//
// For query row i (node j of request r) and query head g, over the positions p
// that the row sees: s_p = scale q . K_p, out = sum w_p V_p / sum w_p with
// w_p = exp(s_p - m), m the running maximum; what was summed under an older
// maximum is scaled by exp(m_old - m) (the ratio is unchanged). All in base 2:
// the scores are scaled by log2 e once.
//
// attend_small serves up to 16 query rows per KV head (single tokens, small
// trees). It is bound by reading the pages: every K and V value enters one
// 16-row product, 2 x 16 multiply-adds per code, far below what even the
// warp-level matrix instructions need to keep up with HBM. So each warp is a
// stream of its own: it takes every fourth run of 16 positions (32 of an
// e4m3 cache) of its CTA's share through a private ring in shared memory, filled 16 bytes at a time by
// asynchronous copies that look the page up per position (a page may end
// anywhere, a row may lie at any 16-byte multiple), and keeps its own maximum,
// sum and output; no barrier inside the loop. The four are joined at the end of
// a part. Three CTAs of 4 warps per SM, 64 KB of ring each, half of it in flight: 64
// requests of 2,048 to 8,192 positions (332,000 in all) x 8 heads x 128 channels, one token, 8 query heads
// each, take 212 us in bf16 (1.36 GB at 6.40 TB/s, 0.95 of a copy) and 128 us in e4m3 (5.3 TB/s, bound by
// issue: the conversions); two CTAs of 96 KB took 3% and 6% longer.
//
// An e4m3 cache is raised to fp16 in registers (every e4m3 value is an fp16
// value). The order of the channels inside a product is free as long as both
// operands agree, and so is the order of the output's columns: both are chosen so
// that a thread's 16 bytes of K, and of V per position, are what its fragments
// need. The queries become fp16 after a power-of-two scale per row that brings the
// largest magnitude to [1, 2): bf16's 8 bits fit, and what is below 2^-14 of the
// largest is off by at most 2^-25 of it. Weights are rounded to the type of the
// product (fp16: half a step 2^-11, or 2^-32 of the row's largest; bf16: 2^-8); their sum stays binary32.
#include "skv_attend.cuh"

namespace skv {

constexpr uint32_t kWarps = 4;

template <int DP, bool E>
struct SmallShape {
    static constexpr uint32_t bytes = E ? 1 : 2;
    static constexpr uint32_t run = E ? 32 : 16;           // positions of a warp at a time
    static constexpr uint32_t unit = kWarps * run;
    static constexpr uint32_t groups = run / 16;
    static constexpr uint32_t row = DP * bytes;            // bytes of a position's row in the ring
    static constexpr uint32_t chunks = row / 16;
    static constexpr uint32_t half = run * row;           // K, then V
    static constexpr uint32_t stage = 2 * half;
    static constexpr uint32_t want = 16384 / stage;        // 16 KB per warp
    static constexpr uint32_t stages = want < 2 ? 2 : want > 8 ? 8 : want;
    static constexpr uint32_t ring = stages * stage;
    static constexpr uint32_t per_sm = DP == 256 ? 1 : 3;  // CTAs
    static constexpr uint32_t joined = kWarps * (16 * (DP + 4) + 32) * 4;
    static constexpr uint32_t smem = kWarps * ring > joined ? kWarps * ring : joined;
};

__device__ __forceinline__ uint32_t smem_of(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}

__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}

template <bool E>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (E)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool E>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if (E) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four e4m3 codes as two pairs of fp16.
__device__ __forceinline__ void raise4(uint32_t codes, uint32_t &lo, uint32_t &hi) {
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h;}"
        : "=r"(lo), "=r"(hi) : "r"(codes));
}

__device__ __forceinline__ uint32_t lds32(uint32_t at) {
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
    return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 r;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at) : "memory");
    return r;
}

// Chunk order inside a row of the ring, so that what the eight lanes of one
// shared-memory phase read lies in eight different 16-byte columns: bf16 matrices
// take the same chunk of 8 rows; e4m3 K takes chunks 0-3 of two rows, e4m3 V two
// chunks of every other row.
template <int DP, bool E>
__device__ __forceinline__ uint32_t swz_k(uint32_t row, uint32_t chunk) {
    if (!E) return chunk ^ (row & 7u);
    return DP >= 128 ? chunk ^ ((row & 1u) << 2) : chunk;
}
template <int DP, bool E>
__device__ __forceinline__ uint32_t swz_v(uint32_t row, uint32_t chunk) {
    if (!E) return chunk ^ (row & 7u);
    return DP >= 128 ? chunk ^ (row & 6u) : chunk ^ ((row >> 1) & 3u);
}

// The rows (two per thread: lane / 4 and 8 more) of a part's query tile as matrix fragments.
template <int DP, bool E>
struct QueryFrags {
    uint32_t f[DP / 16][4];
    float mul[2];          // product -> score in base 2; at least 2^-149, so that -infinity times it stays that
};

template <int DP, bool E>
__device__ __forceinline__ void load_queries(const AttendArgs &a, const ReqOf &q, uint32_t h, uint32_t rt,
                                             QueryFrags<DP, E> &x) {
    const uint32_t lane = threadIdx.x & 31u, c = lane & 3u;
    // a negative scale turns the queries, so that the largest product is the largest score
    const float scale = a.scale * (a.c.k_scale ? __ldg(a.c.k_scale + h) : 1.0f) * 1.4426950408889634f, mul = fabsf(scale);
    const bool turned = scale < 0.0f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const uint32_t r = rt * 16u + (lane >> 2) + 8u * half, node = r / a.group, g = r - node * a.group;
        const bool live = node < q.n;
        const uint16_t *src = a.q + (uint64_t)(q.row0 + node) * a.q_row_stride + (uint64_t)(h * a.group + g) * a.q_head_stride;
        float top = 0.0f;
        if (!E) {
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const uint32_t d = 16u * k + 8u * s + 2u * c;
                    x.f[k][half + 2 * s] = (live && d < a.c.head_dim ? __ldg(reinterpret_cast<const uint32_t *>(src + d)) : 0u) ^ (turned ? 0x80008000u : 0u);
                }
            }
            x.mul[half] = fmaxf(mul, 0x1p-149f);
        } else {
#pragma unroll
            for (int b = 0; b < DP / 64; ++b) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // channels 64 b + 16 c + 4 j + {0, 1} and + {2, 3}
                    const uint32_t d = 64u * b + 16u * c + 4u * j;
                    const uint2 w = live && d < a.c.head_dim ? __ldg(reinterpret_cast<const uint2 *>(src + d)) : make_uint2(0u, 0u);
                    x.f[4 * b + j][half] = w.x;
                    x.f[4 * b + j][half + 2] = w.y;
                    top = fmaxf(top, fmaxf(fmaxf(fabsf(__uint_as_float(w.x << 16)), fabsf(__uint_as_float(w.x & 0xFFFF0000u))),
                                           fmaxf(fabsf(__uint_as_float(w.y << 16)), fabsf(__uint_as_float(w.y & 0xFFFF0000u)))));
                }
            }
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
            // 2^-e with e the exponent of the largest magnitude; 1 for 0, tiny and infinite rows
            const uint32_t e = __float_as_uint(top) >> 23;
            const bool usual = e > 2u && e < 252u;
            const float down = (usual ? __uint_as_float((254u - e) << 23) : 1.0f) * (turned ? -1.0f : 1.0f);
            x.mul[half] = fmaxf(usual ? mul * __uint_as_float(e << 23) : mul, 0x1p-149f);
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const uint32_t w = x.f[k][half + 2 * s];
                    x.f[k][half + 2 * s] = pack2<true>(__uint_as_float(w << 16) * down, __uint_as_float(w & 0xFFFF0000u) * down);
                }
            }
        }
    }
}

// o[k] += weight * output of the warp's k-th row (warp + 4 k), over `here` parts, in their order.
template <int DP, uint32_t ROWS, class At>
__device__ __forceinline__ void add_parts(float4 (&o)[4], const float *s_f, uint32_t rows, uint32_t here, At at) {
    const uint32_t warp = threadIdx.x >> 5;
    constexpr uint32_t PARTS = 8u / ROWS;
#pragma unroll 1
    for (uint32_t j0 = 0; j0 < here; j0 += PARTS) {
        float4 y[PARTS][ROWS];
#pragma unroll
        for (uint32_t j = 0; j < PARTS; ++j)
#pragma unroll
            for (uint32_t k = 0; k < ROWS; ++k) {
                y[j][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (j0 + j < here && warp + 4u * k < rows)
                    y[j][k] = __ldcg(reinterpret_cast<const float4 *>(at(j0 + j) + (warp + 4u * k) * DP));
            }
#pragma unroll
        for (uint32_t j = 0; j < PARTS; ++j)
#pragma unroll
            for (uint32_t k = 0; k < ROWS; ++k) {
                const float f = j0 + j < here ? s_f[(warp + 4u * k) * 33u + j0 + j] : 0.0f;
                o[k].x += f * y[j][k].x, o[k].y += f * y[j][k].y, o[k].z += f * y[j][k].z, o[k].w += f * y[j][k].w;
            }
    }
}

// The 16 rows of an item whose n parts lie in CTAs c .. c + n - 1 (place 1 of the first, then 0), by a CTA:
// each part weighs exp2(m - M) with M the largest m, in the order of the CTAs. Eight threads per row
// find the weights of 32 parts at a time; then a thread adds up four channels of four rows, so
// that the rows wait for L2 together (one after the other a warp's four rows took 5 us of 19).
template <int DP>
__device__ __forceinline__ void join_item(const AttendArgs &a, const AttendWs &ws, const ReqOf &q, uint32_t h, uint32_t rt,
                                          uint32_t c, uint32_t n, float *scratch) {
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5, row8 = tid >> 3, sub = tid & 7u;
    const uint32_t rows = min(16u, q.n * a.group - rt * 16u);
    constexpr uint32_t size = 16u * (2u + DP);
    const float *next = ws.parts + (uint64_t)c * 2u * size;
    const auto part = [&](uint32_t j) { return j ? next + (uint64_t)(2u * j) * size : next + size; };
    float *s_f = scratch, *s_ml = scratch + 16 * 33;
    const float vs = a.c.v_scale ? __ldg(a.c.v_scale + h) : 1.0f;
    float M = -INFINITY, L = 0.0f;
    if (row8 < rows) {
#pragma unroll 4
        for (uint32_t j = sub; j < n; j += 8u) M = fmaxf(M, __ldcg(part(j) + row8));
    }
#pragma unroll
    for (uint32_t d = 4; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, d));
#pragma unroll 1
    for (uint32_t x0 = 0; x0 < DP; x0 += 128u) {                     // 256 channels: two rounds; 64: half of the lanes
        const uint32_t x = x0 + 4u * lane;
        float4 o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (uint32_t j0 = 0; j0 < n; j0 += 32u) {
            __syncthreads();
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
                const uint32_t j = 8u * i + sub;
                float f = 0.0f;
                if (j0 + j < n && row8 < rows) {
                    f = part_weight(__ldcg(part(j0 + j) + row8), M);
                    if (x0 == 0) L += f * __ldcg(part(j0 + j) + 16u + row8);
                }
                s_f[row8 * 33u + j] = f;
            }
            __syncthreads();
            const uint32_t here = min(32u, n - j0);
            if (x < DP) {
                // eight loads on their way: four rows of two parts, two of four, or one of eight
                if (rows > 8u) add_parts<DP, 4>(o, s_f, rows, here, [&](uint32_t j) { return part(j0 + j) + 32u + x; });
                else if (rows > 4u) add_parts<DP, 2>(o, s_f, rows, here, [&](uint32_t j) { return part(j0 + j) + 32u + x; });
                else add_parts<DP, 1>(o, s_f, rows, here, [&](uint32_t j) { return part(j0 + j) + 32u + x; });
            }
        }
        if (x0 == 0) {
#pragma unroll
            for (uint32_t d = 4; d; d >>= 1) L += __shfl_xor_sync(~0u, L, d);
            if (sub == 0) {
                s_ml[row8] = M;
                s_ml[16u + row8] = L;
            }
            __syncthreads();
        }
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
            const uint32_t row = warp + 4u * k;
            if (row >= rows) continue;
            const uint32_t all = rt * 16u + row, node = all / a.group, g = h * a.group + all - node * a.group;
            const float l = s_ml[16u + row], inv = l == 0.0f ? 0.0f : vs / l;
            if (x < a.c.head_dim) {
                uint2 y;
                y.x = l == 0.0f ? 0u : pack2<false>(o[k].x * inv, o[k].y * inv);
                y.y = l == 0.0f ? 0u : pack2<false>(o[k].z * inv, o[k].w * inv);
                *reinterpret_cast<uint2 *>(a.out + ((uint64_t)(q.row0 + node) * a.n_q_heads + g) * a.c.head_dim + x) = y;
            }
            if (a.lse && x == 0)
                a.lse[(uint64_t)(q.row0 + node) * a.n_q_heads + g] = l == 0.0f ? -INFINITY : (s_ml[row] + log2f(l)) * 0.6931471805599453f;
        }
    }
}

// The end of a CTA with work: one word counts the CTAs in its low half and holds the kinds of
// error above; the last CTA writes the status and clears it.
__device__ __forceinline__ void finish(const AttendArgs &a, const AttendWs &ws, int32_t err, uint32_t active) {
    if (err) atomicOr(ws.finished, err == SKV_ERR_CORRUPT ? kSawCorrupt : kSawInvalid);
    const uint32_t was = atomicAdd(ws.finished, 1u);
    if ((was & 0xFFFFu) == active - 1u) {
        *a.status = status_of(was);
        *ws.finished = 0u;
    }
}

template <int DP, bool E>
__global__ void __launch_bounds__(kWarps * 32, SmallShape<DP, E>::per_sm) attend_small(AttendArgs a, AttendWs ws) {
    using S = SmallShape<DP, E>;
    extern __shared__ __align__(1024) uint8_t ring_all[];
    __shared__ unsigned long long sm_plan[2 * kWarps + 4];
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5, c4 = lane & 3u, g8 = lane >> 2;
    __shared__ uint32_t sm_last;
    const Share sh = share_of<kWarps * 32, false>(a, ws, 16u, S::unit, sm_plan);
    if (sh.u0 == sh.u1) {
        if (sh.active == 0 && blockIdx.x == 0 && tid == 0) *a.status = status_of(atomicExch(ws.finished, 0u));
        return;
    }
    const uint32_t ring = smem_of(ring_all) + warp * S::ring;
    const uint32_t row_bytes = a.c.head_dim * S::bytes;
    bool corrupt = false;

    uint32_t r = sh.r;
    ReqOf q = request_of(a, r);
    constexpr uint32_t G = S::groups;
    uint32_t tiles = (q.len + S::unit - 1) / S::unit, rts = (q.n * a.group + 15u) / 16u;
    uint64_t item = quotient(sh.off, tiles);
    uint32_t tile = (uint32_t)(sh.off - item * tiles);
    for (uint64_t u = sh.u0; u < sh.u1;) {
        // one part: head h, row tile rt, tiles [tile, tile_end) of the request
        const uint32_t h = (uint32_t)quotient(item, rts), rt = (uint32_t)(item - (uint64_t)h * rts);
        const uint32_t tile_end = (uint32_t)min((uint64_t)tiles, tile + (sh.u1 - u));
        const uint32_t p_begin = tile * S::unit, p_end = min(q.len, tile_end * S::unit);
        const uint32_t runs = (p_end - p_begin + S::run - 1) / S::run;
        const uint32_t mine = runs > warp ? (runs - warp + kWarps - 1) / kWarps : 0u;
        bool hurt = false;                       // this warp put 0 for a value that is not finite

        // The page of this lane's position in run i of this warp, one run ahead of its copies.
        uint64_t next_at = ~0ull;
        auto look_up = [&](uint32_t i) {
            next_at = ~0ull;
            const uint32_t p = p_begin + (warp + i * kWarps) * S::run + (lane & (S::run - 1u));
            if (i < mine && p < p_end) {
                next_at = place_of(a.c, r, h, p);
                corrupt |= next_at == ~0ull;
            }
        };
        auto issue = [&](uint32_t i) {
            if (i < mine) {
                const uint32_t st = ring + (i % S::stages) * S::stage;
#pragma unroll
                for (uint32_t n = 0; n < (S::run * S::chunks + 31) / 32; ++n) {
                    const uint32_t x = n * 32u + lane, row = x / S::chunks, ch = x % S::chunks;
                    const uint64_t at = __shfl_sync(~0u, next_at, row & (S::run - 1u));
                    if (row < S::run) {
                        const bool live = at != ~0ull && ch * 16u < row_bytes;
                        const uint64_t off = live ? at + ch * 16u : 0ull;
                        copy16(st + row * S::row + swz_k<DP, E>(row, ch) * 16u, a.c.k + off, live ? 16u : 0u);
                        copy16(st + S::half + row * S::row + swz_v<DP, E>(row, ch) * 16u, a.c.v + off, live ? 16u : 0u);
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            look_up(i + 1);
        };
        look_up(0);
        QueryFrags<DP, E> qf;
        float o[DP / 8][4];
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

        // the first turns only fill the ring
#pragma unroll 1
        for (int32_t turn = 1 - (int32_t)S::stages; turn < (int32_t)mine; ++turn) {
            if (turn >= 0) {
                asm volatile("cp.async.wait_group %0;" ::"n"(S::stages - 2) : "memory");
                __syncwarp();
            }
            const uint32_t i = (uint32_t)turn;
            issue(i + S::stages - 1);
            if (turn < 0) {
                if (turn == -1) load_queries<DP, E>(a, q, h, rt, qf);
                continue;
            }
            const uint32_t st = ring + (i % S::stages) * S::stage, sv = st + S::half;
            const uint32_t p0 = p_begin + (warp + i * kWarps) * S::run;
            const bool edge = p0 + S::run > q.ctx || p0 + S::run > p_end;
            if (edge && p0 + S::run > q.ctx) {
                // drafted positions: values that are not finite leave the product
                bool found = false;
#pragma unroll 1
                for (uint32_t x = lane; x < S::run * S::chunks; x += 32u) {
                    const uint32_t row = x / S::chunks;
                    if (p0 + row < q.ctx) continue;
                    const uint32_t at = sv + x * 16u;
                    const uint4 w4 = lds128(at);
                    uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
                    bool hit = false;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
#pragma unroll
                        for (int b = 0; b < (E ? 4 : 2); ++b) {
                            const uint32_t bits = E ? 0x7Fu << (8 * b) : 0x7F80u << (16 * b), all = E ? 0xFFu << (8 * b) : 0xFFFFu << (16 * b);
                            if ((w[j] & bits) == bits) {
                                w[j] &= ~all;
                                hit = true;
                            }
                        }
                    }
                    if (hit)
                        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
                    found |= hit;
                }
                hurt |= found;
                __syncwarp();
            }
            float s[2 * G][4];
#pragma unroll
            for (int n = 0; n < 2 * (int)G; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
            if (!E) {
#pragma unroll
                for (int y = 0; y < (int)G; ++y) {
                    const uint32_t row = 16u * y + (lane & 7u) + ((lane >> 4) << 3), hi = (lane >> 3) & 1u;
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k) {
                        uint32_t b[4];
                        ldm4(b, st + row * S::row + swz_k<DP, E>(row, 2u * k + hi) * 16u);
                        mma16<E>(s[2 * y], qf.f[k], b[0], b[1]);
                        mma16<E>(s[2 * y + 1], qf.f[k], b[2], b[3]);
                    }
                }
            } else {
#pragma unroll
                for (int b = 0; b < DP / 64; ++b) {
#pragma unroll
                    for (int n = 0; n < 2 * (int)G; ++n) {
                        const uint32_t row = 8u * n + g8;
                        const uint4 w4 = lds128(st + row * S::row + swz_k<DP, E>(row, 4u * b + c4) * 16u);
                        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t lo, hi;
                            raise4(w[j], lo, hi);
                            mma16<E>(s[n], qf.f[4 * b + j], lo, hi);
                        }
                    }
                }
            }
            // positions a row does not see: -infinity
            if (edge) {
                uint32_t seen[2] = {0u, 0u};
#pragma unroll 1
                for (uint32_t half = 0; half < 2; ++half) {
                    const uint32_t bits = sees32(a, q, min((rt * 16u + g8 + 8u * half) / a.group, q.n - 1u), p0, p_end);
                    if (half) seen[1] = bits;
                    else seen[0] = bits;
                }
#pragma unroll
                for (int n = 0; n < 2 * (int)G; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!((seen[e >> 1] >> (8u * n + 2u * c4 + (e & 1))) & 1u)) s[n][e] = -INFINITY;
            }
            float top[2] = {-INFINITY, -INFINITY}, base[2];
#pragma unroll
            for (int n = 0; n < 2 * (int)G; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], s[n][e]);
            // the reference of a row's weights lags (kLag; sums are binary32), so the output is rarely scaled anew
            bool move[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                top[half] = fmaxf(top[half], __shfl_xor_sync(~0u, top[half], 1));
                top[half] = fmaxf(top[half], __shfl_xor_sync(~0u, top[half], 2)) * qf.mul[half];
                move[half] = top[half] > m[half] + (kLag + kLower<E>) || (m[half] == -INFINITY && top[half] > m[half]);
                top[half] -= kLower<E>;
            }
            if (__any_sync(~0u, move[0] || move[1])) {
                float keep[2];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    keep[half] = move[half] ? part_weight(m[half], top[half]) : 1.0f;
                    if (move[half]) m[half] = top[half];
                    l[half] *= keep[half];
                }
#pragma unroll
                for (int j = 0; j < DP / 8; ++j) {
                    o[j][0] *= keep[0];
                    o[j][1] *= keep[0];
                    o[j][2] *= keep[1];
                    o[j][3] *= keep[1];
                }
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) base[half] = m[half] == -INFINITY ? 0.0f : -m[half];
            uint32_t pa[G][4];
#pragma unroll
            for (int n = 0; n < 2 * (int)G; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[n][e] = ex2(fmaf(s[n][e], qf.mul[e >> 1], base[e >> 1]));
                    l[e >> 1] += s[n][e];
                }
                pa[n >> 1][2 * (n & 1)] = pack2<E>(s[n][0], s[n][1]);
                pa[n >> 1][2 * (n & 1) + 1] = pack2<E>(s[n][2], s[n][3]);
            }
#pragma unroll
            for (int y = 0; y < (int)G; ++y) {
                if (!E) {
                    const uint32_t row = 16u * y + (lane & 15u), hi = lane >> 4;
#pragma unroll
                    for (int j = 0; j < DP / 16; ++j) {
                        uint32_t b[4];
                        ldm4t(b, sv + row * S::row + swz_v<DP, E>(row, 2u * j + hi) * 16u);
                        mma16<E>(o[2 * j], pa[y], b[0], b[1]);
                        mma16<E>(o[2 * j + 1], pa[y], b[2], b[3]);
                    }
                } else {
                    // column n of the output tile i is channel (DP / 8) n + i: a thread's bytes of four positions
                    constexpr int CW = DP / 32;              // words of one position
                    constexpr int PW = CW < 4 ? CW : 4;      // at a time
#pragma unroll
                    for (int part = 0; part < CW; part += PW) {
                        uint32_t w[4][4];
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const uint32_t row = 16u * y + 2u * c4 + (t & 1) + 8u * (t >> 1);
                            const uint32_t byte = g8 * (DP / 8) + part * 4u;
                            const uint32_t at = sv + row * S::row + swz_v<DP, E>(row, byte >> 4) * 16u + (byte & 15u);
                            if (PW == 4) {
                                const uint4 x = lds128(at);
                                w[t][0] = x.x, w[t][1] = x.y, w[t][2] = x.z, w[t][3] = x.w;
                            } else {
#pragma unroll
                                for (int j = 0; j < PW; ++j) w[t][j] = lds32(at + 4u * j);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < PW; ++j) {
                            const uint32_t lo0 = __byte_perm(w[0][j], w[1][j], 0x5140), lo1 = __byte_perm(w[0][j], w[1][j], 0x7362);
                            const uint32_t hi0 = __byte_perm(w[2][j], w[3][j], 0x5140), hi1 = __byte_perm(w[2][j], w[3][j], 0x7362);
                            const int i = (part + j) * 4;
                            uint32_t b[4][2];
                            raise4(lo0, b[0][0], b[1][0]);
                            raise4(hi0, b[0][1], b[1][1]);
                            raise4(lo1, b[2][0], b[3][0]);
                            raise4(hi1, b[2][1], b[3][1]);
#pragma unroll
                            for (int x = 0; x < 4; ++x) mma16<E>(o[i + x], pa[y], b[x][0], b[x][1]);
                        }
                    }
                }
            }
            __syncwarp();
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            l[half] += __shfl_xor_sync(~0u, l[half], 1);
            l[half] += __shfl_xor_sync(~0u, l[half], 2);
        }
        // the rings become the place where the four warps meet
        const bool any_hurt = __syncthreads_or(hurt);
        float *so = reinterpret_cast<float *>(ring_all) + warp * 16u * (DP + 4);
        float *sml = reinterpret_cast<float *>(ring_all) + kWarps * 16u * (DP + 4);     // [warp][2][16]
        if (c4 == 0) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                sml[warp * 32u + g8 + 8u * half] = m[half];
                sml[warp * 32u + 16u + g8 + 8u * half] = l[half];
            }
        }
#pragma unroll
        for (int j = 0; j < DP / 8; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t row = g8 + 8u * (e >> 1), n = 2u * c4 + (e & 1);
                so[row * (DP + 4) + (E ? n * (DP / 8) + j : 8u * j + n)] = o[j][e];
            }
        }
        __syncthreads();
        const bool whole = tile == 0 && tile_end == tiles;
        const uint32_t place = tile ? 0u : 1u;
        float *part = ws.parts + ((uint64_t)blockIdx.x * 2u + place) * part_floats(16u, DP);
        const float vs = a.c.v_scale ? __ldg(a.c.v_scale + h) : 1.0f;
        // thread: 4 channels of every (512 / DP)th row
#pragma unroll 1
        for (uint32_t x = tid; x < 16u * (DP / 4); x += kWarps * 32) {
            const uint32_t row = x / (DP / 4), d = (x % (DP / 4)) * 4u;
            const uint32_t all = rt * 16u + row, node = all / a.group, g = h * a.group + all - node * a.group;
            if (node >= q.n) continue;
            float M = -INFINITY, L = 0.0f, f[kWarps];
#pragma unroll
            for (uint32_t w = 0; w < kWarps; ++w) M = fmaxf(M, sml[w * 32u + row]);
#pragma unroll
            for (uint32_t w = 0; w < kWarps; ++w) {
                f[w] = part_weight(sml[w * 32u + row], M);
                L += f[w] * sml[w * 32u + 16u + row];
            }
            float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (uint32_t w = 0; w < kWarps; ++w) {
                const float4 y = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(ring_all) +
                                                                   (w * 16u + row) * (DP + 4) + d);
                v[0] += f[w] * y.x, v[1] += f[w] * y.y, v[2] += f[w] * y.z, v[3] += f[w] * y.w;
            }
            if (any_hurt && d < a.c.head_dim) {
#pragma unroll 1
                for (uint32_t j = 0; j < 4; ++j) {
                    const float add = not_finite_sum(a, q, r, h, node, d + j, p_begin, p_end);
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i)
                        if (i == j) v[i] += add;
                }
            }
            if (whole) {
                const float inv = L == 0.0f ? 0.0f : vs / L;
                if (d < a.c.head_dim) {
                    uint2 y;
                    y.x = L == 0.0f ? 0u : pack2<false>(v[0] * inv, v[1] * inv);
                    y.y = L == 0.0f ? 0u : pack2<false>(v[2] * inv, v[3] * inv);
                    *reinterpret_cast<uint2 *>(a.out + ((uint64_t)(q.row0 + node) * a.n_q_heads + g) * a.c.head_dim + d) = y;
                }
                if (a.lse && d == 0)
                    a.lse[(uint64_t)(q.row0 + node) * a.n_q_heads + g] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
            } else {
                if (d == 0) {
                    part[row] = M;
                    part[16u + row] = L;
                }
                *reinterpret_cast<float4 *>(part + 32u + row * DP + d) = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
        if (!whole) {
            // the CTA that brings the item's last part joins them all
            const uint64_t unit0 = u - tile;
            const uint32_t c0 = cta_of(unit0, sh.U, sh.active), n = cta_of(unit0 + tiles - 1, sh.U, sh.active) - c0 + 1u;
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                sm_last = atomicAdd(ws.arrived + c0, 1u) == n - 1u;
                if (sm_last) ws.arrived[c0] = 0u;
            }
            __syncthreads();
            if (sm_last) {
                __threadfence();
                join_item<DP>(a, ws, q, h, rt, c0, n, reinterpret_cast<float *>(ring_all));
            }
        }
        u += tile_end - tile;
        tile = 0;
        ++item;
        if (u < sh.u1 && item == (uint64_t)a.c.n_heads * rts) {
            do q = request_of(a, ++r);
            while (q.n == 0);
            tiles = (q.len + S::unit - 1) / S::unit;
            rts = (q.n * a.group + 15u) / 16u;
            item = 0;
        }
        __syncthreads();                         // the rings are free again
    }
    corrupt = __syncthreads_or(corrupt);
    if (tid == 0) finish(a, ws, corrupt ? SKV_ERR_CORRUPT : SKV_OK, (uint32_t)sh.active);
}

// Joins the parts that attend_large leaves: block (c, y) every eighth eight rows of the
// item that starts in CTA c and goes on, a warp per row. All blocks are resident at
// once, so that descriptor and request are waited for once, not once per eight rows
// (152 x 32 blocks of eight rows each took 31 us behind a 515 us call, 152 x 4 took 21). Block (0, 0)
// turns the CTAs' error words into the status: the first that has one.
constexpr uint32_t kJoinBlocks = 8;

__global__ void __launch_bounds__(256, 4) attend_join(AttendArgs a, AttendWs ws, uint32_t R, uint32_t DP, uint32_t ctas) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, c = blockIdx.x;
    if (blockIdx.x == 0 && blockIdx.y == 0 && warp == 0) {
        int32_t e[(kCtasLarge + 31u) / 32u], err = SKV_OK;
#pragma unroll
        for (uint32_t i = 0; i < (kCtasLarge + 31u) / 32u; ++i)      // all in flight at once
            e[i] = i * 32u + lane < ctas ? __ldcg(ws.errs + i * 32u + lane) : SKV_OK;
#pragma unroll
        for (uint32_t i = 0; i < (kCtasLarge + 31u) / 32u; ++i) {
            const uint32_t any = __ballot_sync(~0u, e[i] != SKV_OK);
            if (any && err == SKV_OK) err = __shfl_sync(~0u, e[i], __ffs(any) - 1);
        }
        if (lane == 0) *a.status = err;
    }
    const Desc d = ws.desc[c];
    const Plan plan = *ws.plan;
    if (!d.valid) return;
    const ReqOf q = request_of(a, d.request);
    const uint32_t last = cta_of(d.last, plan.total, plan.active);
    const uint32_t rows = min(R, q.n * a.group - d.rt * R);
    for (uint32_t row = blockIdx.y * 8u + warp; row < rows; row += kJoinBlocks * 8u)
        join_row(a, ws, q, d.head, d.rt, row, R, DP, c, last - c + 1u);
}

// Dynamic shared memory above 48 KB is asked for once per kernel and device.
bool raise_smem(const void *kernel, uint32_t bytes, std::atomic<uint64_t> &ready) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (bit && (ready.load(std::memory_order_relaxed) & bit)) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) return false;
    ready.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

bool launch_join(const AttendArgs &a, const AttendWs &ws, uint32_t R, uint32_t DP, uint32_t ctas, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, kJoinBlocks);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attend_join, a, ws, R, DP, ctas) == cudaSuccess;
}

template <int DP, bool E>
static bool launch_small(const AttendArgs &a, const AttendWs &ws, cudaStream_t st) {
    using S = SmallShape<DP, E>;
    static_assert(S::smem <= 232448, "shared memory of a CTA");
    static std::atomic<uint64_t> ready{0};                 // devices where the limit is set
    if (!raise_smem(reinterpret_cast<const void *>(attend_small<DP, E>), S::smem, ready)) return false;
    attend_small<DP, E><<<kCtasSmall / 3 * S::per_sm, kWarps * 32, S::smem, st>>>(a, ws);
    return cudaGetLastError() == cudaSuccess;
}

}  // namespace skv

using namespace skv;

extern "C" int32_t skv_tree_attention_workspace_bytes(const skv_paged *cache, uint32_t n_q_heads, uint64_t *bytes) {
    const int32_t r = skv_paged_check(cache);
    if (r != SKV_OK) return r;
    if (!bytes || n_q_heads == 0 || n_q_heads % cache->n_heads) return SKV_ERR_INVALID_ARG;
    const uint32_t DP = cache->head_dim <= 64 ? 64 : cache->head_dim <= 128 ? 128 : 256;
    const uint64_t small = 2u * kCtasSmall * part_floats(16u, DP), large = DP <= 128 ? 2u * kCtasLarge * part_floats(kLargeRows, DP) : 0;
    *bytes = kWsHead + sizeof(float) * (small > large ? small : large);
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
    if (cache->n_requests > 0x7FFFFFFEu || n_q_heads > 65535u ||
        (uint64_t)n_rows * (n_q_heads / cache->n_heads) > 0x7FFFFFFFu || cache->max_pages > 0x7FFFFFFFu ||
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
    if (cache->n_requests == 0 || n_rows == 0)
        return cudaMemsetAsync(status, 0, sizeof(int32_t), st) == cudaSuccess ? SKV_OK : SKV_ERR_CUDA;
    const AttendArgs a{paged_view(*cache), static_cast<const uint16_t *>(q), q_row_stride, q_head_stride, n_q_heads,
                       n_q_heads / cache->n_heads, n_rows, ctx_len, cu_new, mask, mask_words, scale,
                       static_cast<uint16_t *>(out), lse, status};
    const AttendWs ws = attend_ws(workspace);
    const uint32_t d = cache->head_dim;
    bool ok;
    // The tcgen05 kernel pays 128 rows whatever their number, the small-row kernel reads the pages once per
    // 16 rows. us for small / tcgen05, 8 KV heads of 128 channels, 8 query heads each, bf16: 16 requests x
    // 16,000 positions: 16 rows 172 / 177, 32 rows 329 / 174; 4 x 3,000: 16 rows 24 / 25, 32 rows 29 / 25; e4m3, 16 x
    // 16,000: 16 rows 106 / 167, 32 rows 202 / 165. Head sizes above 128 do not fit tensor memory twice.
    if ((uint64_t)max_nodes * a.group > 16u && d <= 128)
        ok = launch_large(a, ws, st);
    else if (cache->dtype == SKV_E4M3)
        ok = d <= 64 ? launch_small<64, true>(a, ws, st) : d <= 128 ? launch_small<128, true>(a, ws, st) : launch_small<256, true>(a, ws, st);
    else
        ok = d <= 64 ? launch_small<64, false>(a, ws, st) : d <= 128 ? launch_small<128, false>(a, ws, st) : launch_small<256, false>(a, ws, st);
    return ok ? SKV_OK : SKV_ERR_CUDA;
}
