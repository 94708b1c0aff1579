// delta_mma.cuh -- pieces of the gated delta rule's tensor-core kernels: warp
// matrix products on bf16 fragments, swizzled tiles, values split in two bf16
// terms, and the strictly lower triangular inverse of a block of 64 steps.
//
// A warp keeps 16 rows of the state, transposed products and all, in the
// accumulator layout of m16n8k16, which is also the layout of the next
// product's left operand: the chain state -> errors -> state never leaves the
// warp's registers, and the warps of the chain never wait for one another.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "delta_rule.cuh"
#include "tc_ptx.cuh"

namespace ssm {
namespace delta {
namespace mma {

using bf = __nv_bfloat16;

__device__ __forceinline__ void product(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void load4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void load4t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void store4(uint32_t at, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ void store4t(uint32_t at, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

// A kernel launched behind another one may begin while that one runs: it lets
// the next one do the same, and waits before it reads what the one before wrote.
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Two values as bf16, the first in the low half.
__device__ __forceinline__ uint32_t pack(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// Two values as the sum of two bf16 each: 16 bits of each value are kept.
__device__ __forceinline__ void split(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack(a, b);
    lo = pack(a - low(hi), b - high(hi));
}

// Tiles of bf16 in shared memory, as tensor copies leave them: ROWS rows of 64
// columns, and for WIDTH = 128 as many again behind them; the 16-byte pieces of
// a row exchanged by its number, so that eight rows' pieces of one column lie
// in eight different groups of banks.
template <int WIDTH, int ROWS = kBlock>
__device__ __forceinline__ uint32_t place(uint32_t tile, int row, int col) {      // col: a multiple of 8
    const int half = WIDTH > 64 ? (col >> 6) * (ROWS * 128) : 0;
    return tile + half + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4);
}
// The address that this lane gives for four 8 x 8 pieces: rows r, r + 8 by
// columns c, c + 8 in the order (r, c), (r + 8, c), (r, c + 8), (r + 8, c + 8).
template <int WIDTH, int ROWS = kBlock>
__device__ __forceinline__ uint32_t four(uint32_t tile, int r, int c) {
    const int lane = threadIdx.x % 32;
    return place<WIDTH, ROWS>(tile, r + (lane & 15), c + (lane >> 4) * 8);
}
// The same in the order (r, c), (r, c + 8), (r + 8, c), (r + 8, c + 8).
template <int WIDTH, int ROWS = kBlock>
__device__ __forceinline__ uint32_t four_across(uint32_t tile, int r, int c) {
    const int lane = threadIdx.x % 32;
    return place<WIDTH, ROWS>(tile, r + (lane & 7) + (lane >> 4) * 8, c + ((lane >> 3) & 1) * 8);
}

__device__ __forceinline__ uint4 load16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void put_values(uint32_t at, const float (&v)[4]) {
    asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(at), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
}
__device__ __forceinline__ float4 get_values(uint32_t at) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}

// Rows from `rows` on of a 64 x WIDTH tile become 0: a tensor copy brings the
// next sequence's.
template <int WIDTH>
__device__ __forceinline__ void clear_rows(uint32_t tile, int rows, int tid, int threads) {
    for (int i = tid; i < (kBlock - rows) * WIDTH / 8; i += threads)
        asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(place<WIDTH>(tile, rows + i / (WIDTH / 8), i % (WIDTH / 8) * 8)), "r"(0) : "memory");
}

// Copies that report to a barrier in shared memory; one thread asks for them.
__device__ __forceinline__ void box(uint32_t to, const CUtensorMap *map, uint64_t *bar, int col, int head, int row) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(to),
        "l"(map), "r"(col), "r"(head), "r"(row), "r"(tc::smem_addr(bar))
        : "memory");
}
template <int WIDTH>
__device__ __forceinline__ void boxes(uint32_t to, const CUtensorMap *map, uint64_t *bar, int head, int row) {
#pragma unroll
    for (int c = 0; c < WIDTH; c += 64) box(to + c * kBlock * 2, map, bar, c, head, row);
}
__device__ __forceinline__ void bulk(uint32_t to, const void *from, int bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(from),
                 "r"(bytes), "r"(tc::smem_addr(bar))
                 : "memory");
}
constexpr uint64_t kWaitLimitNs = 2000000000ull;
__device__ __forceinline__ void linger() {
    const uint64_t t0 = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t0 < kWaitLimitNs) __nanosleep(1000);
}
// Waits for a barrier's phase; gives up after the limit, and says so in *abort and *error.
__device__ __forceinline__ void wait_for(uint64_t *bar, int phase, int *abort, unsigned int *error,
                                         uint64_t limit_ns = kWaitLimitNs) {
    if (tc::mbar_wait_bounded(bar, phase, abort, limit_ns)) return;
    *reinterpret_cast<volatile int *>(abort) = 1;
    atomicOr(error, 1u);
}

// by v, and 0 for by = 0 whatever v holds.
__device__ __forceinline__ float kept(float by, float v) { return by == 0.0f ? 0.0f : by * v; }

// Whether this lane's rows g and g + 8 of the state hold what is not finite (bits 0 and 1).
template <int N>
__device__ __forceinline__ unsigned not_finite(const float (&st)[N][4]) {
    unsigned bad = 0;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) bad |= (__float_as_uint(st[n][e]) & 0x7f800000u) == 0x7f800000u ? 1u << e / 2 : 0u;
    bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
    return bad | __shfl_xor_sync(0xffffffffu, bad, 2);
}
// Those rows become 0 in the packed columns of 16 steps that the state still
// reaches (`start` above 0): a cut keeps the state out of the steps behind it,
// but 0 times what it holds may not be 0.
__device__ __forceinline__ void drop(uint32_t (&w)[4], unsigned bad, const float *start) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float2 by = *reinterpret_cast<const float2 *>(start + 8 * h + threadIdx.x % 4 * 2);
        const uint32_t keep = (by.x > 0.0f ? 0u : 0xffffu) | (by.y > 0.0f ? 0u : 0xffff0000u);
        if (bad & 1) w[2 * h] &= keep;
        if (bad & 2) w[2 * h + 1] &= keep;
    }
}

// d += a b for 64 columns (from column 16 `from`) of b.
__device__ __forceinline__ void across(float (&d)[8][4], const uint32_t (&a)[4], const uint32_t (&b)[4][4], int from = 0) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        if (t < from) continue;
        product(d[2 * t], a, b[t][0], b[t][1]);
        product(d[2 * t + 1], a, b[t][2], b[t][3]);
    }
}

// The same up to column 16 `to`.
__device__ __forceinline__ void across_to(float (&d)[8][4], const uint32_t (&a)[4], const uint32_t (&b)[4][4], int to) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        if (t > to) continue;
        product(d[2 * t], a, b[t][0], b[t][1]);
        product(d[2 * t + 1], a, b[t][2], b[t][3]);
    }
}

// 16 columns of the state as a left operand of two terms.
template <int KP>
__device__ __forceinline__ void operand(uint32_t (&hi)[4], uint32_t (&lo)[4], const float (&s)[KP / 8][4], int k) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        split(s[2 * k + h][0], s[2 * k + h][1], hi[2 * h], lo[2 * h]);
        split(s[2 * k + h][2], s[2 * k + h][3], hi[2 * h + 1], lo[2 * h + 1]);
    }
}

// w = st tile^T, 16 x 64: 16 columns of the state at a time, as an operand of
// two terms whose first term `use` gets as well.  The pieces of the tile and the
// terms of the next 16 columns are made between the products of these.
template <int KP, typename Use>
__device__ __forceinline__ void through_tile(float (&w)[8][4], const float (&st)[KP / 8][4], uint32_t tile, Use use) {
    uint32_t b[2][4][4], hi[2][4], lo[2][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) load4(b[0][t], four_across<KP>(tile, 16 * t, 0));
    operand<KP>(hi[0], lo[0], st, 0);
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) w[n][e] = 0.0f;
#pragma unroll
    for (int k = 0; k < KP / 16; ++k) {
        const int now = k % 2, next = 1 - now;
        const bool more = k + 1 < KP / 16;
        if (more)
#pragma unroll
            for (int t = 0; t < 4; ++t) load4(b[next][t], four_across<KP>(tile, 16 * t, 16 * (k + 1)));
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            product(w[2 * t], hi[now], b[now][t][0], b[now][t][1]);
            product(w[2 * t + 1], hi[now], b[now][t][2], b[now][t][3]);
            if (more) {
                const float(&s)[4] = st[2 * (k + 1) + t / 2];
                split(s[t % 2 * 2], s[t % 2 * 2 + 1], hi[next][t], lo[next][t]);
            }
        }
        use(k, hi[now]);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            product(w[2 * t], lo[now], b[now][t][0], b[now][t][1]);
            product(w[2 * t + 1], lo[now], b[now][t][2], b[now][t][3]);
        }
    }
}

// The state's 16 rows += (hi + lo) times the 64 x KP tile; a tile's pieces are
// loaded ahead of the products before them.
template <int KP>
__device__ __forceinline__ void add_outer(float (&st)[KP / 8][4], const uint32_t (&hi)[4][4], const uint32_t (&lo)[4][4],
                                          uint32_t tile) {
    constexpr int parts = KP / 64;          // 64 columns at a time
    uint32_t b[2][4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) load4t(b[0][k], four<KP>(tile, 0, 16 * k));
#pragma unroll
    for (int i = 0; i < 4 * parts; ++i) {
        const int t = i / parts, k0 = i % parts * 4, next_t = (i + 1) / parts, next_k = (i + 1) % parts * 4;
        if (i + 1 < 4 * parts)
#pragma unroll
            for (int k = 0; k < 4; ++k) load4t(b[(i + 1) % 2][k], four<KP>(tile, 16 * next_t, 16 * (next_k + k)));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            product(st[2 * (k0 + k)], hi[t], b[i % 2][k][0], b[i % 2][k][1]);
            product(st[2 * (k0 + k) + 1], hi[t], b[i % 2][k][2], b[i % 2][k][3]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            product(st[2 * (k0 + k)], lo[t], b[i % 2][k][0], b[i % 2][k][1]);
            product(st[2 * (k0 + k) + 1], lo[t], b[i % 2][k][2], b[i % 2][k][3]);
        }
    }
}

// A warp's 16 columns of a 64-row result, from transposed accumulators: into
// rows of 32 bytes in shared memory, and from there to rows `step` apart.
__device__ __forceinline__ void store_turned(uint32_t room, int t, const float (&w)[8][4]) {
    const int lane = threadIdx.x % 32;
    uint32_t r[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        r[2 * h] = pack(w[2 * t + h][0], w[2 * t + h][1]);
        r[2 * h + 1] = pack(w[2 * t + h][2], w[2 * t + h][3]);
    }
    store4t(room + (16 * t + (lane >> 4) * 8 + (lane & 7)) * 32 + ((lane >> 3) & 1) * 16, r);
}
__device__ __forceinline__ void write_turned(bf *out, int64_t step, int rows, int width, uint32_t room) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = (i * 32 + lane) / 2, v = lane % 2 * 8;
        const uint4 w = load16(room + t * 32 + v * 2);
        if (t < rows && v < width) *reinterpret_cast<uint4 *>(out + t * step + v) = w;
    }
}

// What a step's decays come to, beside the sums of Decays.
struct alignas(16) Factors {
    float start[kBlock], start_scaled[kBlock], end[kBlock], beta[kBlock];
    float last;     // Gam_C
};

// ---- pairs of steps ------------------------------------------------------------
constexpr int kPairThreads = 128;
constexpr int kPairStride = kBlock + 4;     // floats

// D_ts (a_t . b_s) for rows 16 j.. of `a` and the 16-column blocks 0..j of
// `b`: `put(n, h, t, s, x, y)` takes two neighbours of block n with their decays
// (h: which of the four of a lane).
template <int KP, typename Put>
__device__ __forceinline__ void pair_products(uint32_t a, uint32_t b, int j, const Decays &d, Put put) {
    uint32_t fa[KP / 16][4];
#pragma unroll
    for (int k = 0; k < KP / 16; ++k) load4(fa[k], four<KP>(a, 16 * j, 16 * k));
    const int lane = threadIdx.x % 32, c = lane % 4 * 2, t = 16 * j + lane / 4;
    const float hi0 = d.hi[t], lo0 = d.lo[t], hi1 = d.hi[t + 8], lo1 = d.lo[t + 8];
    const int cut0 = d.cut[t], cut1 = d.cut[t + 8];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        if (n > j) break;
        float m[2][4] = {};
#pragma unroll
        for (int k = 0; k < KP / 16; ++k) {
            uint32_t fb[4];
            load4(fb, four_across<KP>(b, 16 * n, 16 * k));
            product(m[0], fa[k], fb[0], fb[1]);
            product(m[1], fa[k], fb[2], fb[3]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = 16 * n + 8 * h + c;
            const float2 hi = *reinterpret_cast<const float2 *>(d.hi + r), lo = *reinterpret_cast<const float2 *>(d.lo + r);
            const int2 cut = *reinterpret_cast<const int2 *>(d.cut + r);
            // above the diagonal the exponent may be large; put() drops those
            put(n, 2 * h, t, r, cut0 == cut.x ? m[h][0] * ex2((hi0 - hi.x) + (lo0 - lo.x)) : 0.0f,
                cut0 == cut.y ? m[h][1] * ex2((hi0 - hi.y) + (lo0 - lo.y)) : 0.0f);
            put(n, 2 * h + 1, t + 8, r, cut1 == cut.x ? m[h][2] * ex2((hi1 - hi.x) + (lo1 - lo.x)) : 0.0f,
                cut1 == cut.y ? m[h][3] * ex2((hi1 - hi.y) + (lo1 - lo.y)) : 0.0f);
        }
    }
}

// Two values as the sum of three bf16 each: all 24 bits.
__device__ __forceinline__ void split3(float a, float b, uint32_t (&t)[3]) {
    t[0] = pack(a, b);
    a -= low(t[0]), b -= high(t[0]);
    t[1] = pack(a, b);
    t[2] = pack(a - low(t[1]), b - high(t[1]));
}

// c += a b for 16 x 16 floats of rows `stride` apart each, b's two blocks of
// eight columns, in bf16 matrix products of three terms that leave out what is
// below 2^-24 of a product; from b's column `from` on.  a's column s is scaled by
// -by_s; LOWER: only what lies below a's (A) or b's (B) diagonal counts.
template <bool LOWER_A, bool LOWER_B, int N>
__device__ __forceinline__ void join(float (&c)[N][4], const float *a, const float *by, const float *b, int from = 0) {
    const int lane = threadIdx.x % 32, g = lane / 4, c2 = lane % 4 * 2;
    uint32_t at[3][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float2 f = *reinterpret_cast<const float2 *>(by + 8 * h + c2);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = g + 8 * e, s = 8 * h + c2;
            float2 v = *reinterpret_cast<const float2 *>(a + t * kPairStride + s);
            if (LOWER_A) v.x = s < t ? v.x : 0.0f, v.y = s + 1 < t ? v.y : 0.0f;
            uint32_t w[3];
            split3(-f.x * v.x, -f.y * v.y, w);
#pragma unroll
            for (int i = 0; i < 3; ++i) at[i][2 * h + e] = w[i];
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        uint32_t bt[2][3];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int s = 8 * h + c2, r = from + 8 * n + g;
            float x = b[s * kPairStride + r], y = b[(s + 1) * kPairStride + r];
            if (LOWER_B) x = r < s ? x : 0.0f, y = r < s + 1 ? y : 0.0f;
            split3(x, y, bt[h]);
        }
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
            for (int j = 0; i + j < 3; ++j) product(c[n], at[i], bt[0][j], bt[1][j]);
    }
}
template <int N>
__device__ __forceinline__ void get_block(float (&c)[N][4], const float *from) {
    const int lane = threadIdx.x % 32, g = lane / 4, c2 = lane % 4 * 2;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float2 v = *reinterpret_cast<const float2 *>(from + (g + 8 * e) * kPairStride + 8 * n + c2);
            c[n][2 * e] = v.x, c[n][2 * e + 1] = v.y;
        }
}
template <int N>
__device__ __forceinline__ void put_block(const float (&c)[N][4], float *to) {
    const int lane = threadIdx.x % 32, g = lane / 4, c2 = lane % 4 * 2;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float2 *>(to + (g + 8 * e) * kPairStride + 8 * n + c2) = make_float2(c[n][2 * e], c[n][2 * e + 1]);
}

// N with (I + A beta) N = A for A strictly lower triangular (64 x 64 floats in
// `m`, zeros on and above the diagonal of its 16 x 16 blocks on the diagonal),
// so that (I + A beta)^-1 = I - N beta.  N takes A's place; what lies above
// the diagonal blocks is overwritten.  Blocks of 16 by substitution in fp32,
// then pairs of blocks joined,
//   N21 = (I - N22 beta2) A21 (I - beta1 N11),
// in matrix products on all 24 bits of either side: the chains take 16 bits of N,
// but with beta near 2 and keys alike what is joined cancels (on 16 bits N was off
// by 2e-4, the state by 1.2e-3; 8192 blocks took 131 us in place of 139).
// Multiply-adds there were bound by their shared-memory operands.  128 threads.
__device__ __forceinline__ void lower_solve(float *m, const float *beta, int tid) {
    const int warp = tid / 32;
    {
        const int b = warp * 16, j = tid % 16;
        float x[16], by[16];        // the column, and beta times it
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = m[(b + i) * kPairStride + b + j];
#pragma unroll
            for (int s = 0; s < 16; s += 4) {
                if (s >= i) break;
                const float4 a = *reinterpret_cast<const float4 *>(m + (b + i) * kPairStride + b + s);
                x[i] -= a.x * by[s];
                if (s + 1 < i) x[i] -= a.y * by[s + 1];
                if (s + 2 < i) x[i] -= a.z * by[s + 2];
                if (s + 3 < i) x[i] -= a.w * by[s + 3];
            }
            by[i] = beta[b + i] * x[i];
        }
        __syncwarp();
        if (tid % 32 < 16)
#pragma unroll
            for (int i = 0; i < 16; ++i) m[(b + i) * kPairStride + b + j] = x[i];
    }
    __syncthreads();
    {
        // two pairs of 16: a warp has eight columns of one
        const int first = warp / 2 * 32, second = first + 16, c = warp % 2 * 8;
        float *lower = m + second * kPairStride + first, *upper = m + first * kPairStride + second;
        float o[1][4];
        get_block(o, lower + c);
        join<false, true, 1>(o, lower, beta + first, m + first * kPairStride + first, c);
        put_block(o, upper + c);
        __syncthreads();
        join<true, false, 1>(o, m + second * kPairStride + second, beta + second, upper + c);
        put_block(o, lower + c);
    }
    __syncthreads();
    {
        // one pair of 32: a warp has 16 x 16 of it
        const int t = warp / 2 * 16, c = warp % 2 * 16;
        float *lower = m + 32 * kPairStride, *upper = m + 32;
        float o[2][4];
        get_block(o, lower + t * kPairStride + c);
        if (c == 0) join<false, true, 2>(o, lower + t * kPairStride, beta, m);
        else join<false, true, 2>(o, lower + t * kPairStride + 16, beta + 16, m + 16 * kPairStride + 16);
        if (c == 0) join<false, false, 2>(o, lower + t * kPairStride + 16, beta + 16, m + 16 * kPairStride);
        put_block(o, upper + t * kPairStride + c);
        __syncthreads();
        const float *n22 = m + (32 + t) * kPairStride + 32;
        if (t == 0) join<true, false, 2>(o, n22, beta + 32, upper + c);
        else {
            join<false, false, 2>(o, n22, beta + 32, upper + c);
            join<true, false, 2>(o, n22 + 16, beta + 48, upper + 16 * kPairStride + c);
        }
        put_block(o, lower + t * kPairStride + c);
    }
    __syncthreads();
}

// What the chains need of a block besides its tokens, made once by
// pairs_kernel: -N in two bf16 terms, P (with the scale), the factors, and for
// the gradients P's second term; tiles of 64 x 64 with their pieces exchanged
// as place<64> does.  Blocks of 16 x 16 above P's diagonal are unspecified.
constexpr int kTile = kBlock * kBlock * 2;
constexpr int kRecord = (3 * kTile + int(sizeof(Factors)) + 127) / 128 * 128, kBothRecord = kRecord + kTile;
cudaError_t take_device_error(unsigned int *out);
// `states`: of the kept ones, those of places that no block has become 0 (null: none are kept).
cudaError_t make_pairs(const Shape &s, const CUtensorMap &q, const CUtensorMap &k, const bf *g, const bf *beta,
                       unsigned char *records, bool both, bf *states, cudaStream_t st);

// Dynamic shared memory for a kernel, allowed once a device.
template <auto KERNEL>
cudaError_t allow(int bytes) {
    static std::atomic<uint64_t> known{0};
    int device = 0;
    if (cudaError_t e = cudaGetDevice(&device)) return e;
    if (device < 64 && known.load(std::memory_order_acquire) >> device & 1) return cudaSuccess;
    if (cudaError_t e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) return e;
    if (device < 64) known.fetch_or(uint64_t(1) << device, std::memory_order_release);
    return cudaSuccess;
}
// Read and clear a unit's error word (host side, synchronous).
inline cudaError_t take_error(const unsigned int &symbol, unsigned int *out) {
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, symbol, sizeof(v));
    if (e == cudaSuccess && v) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(symbol, &zero, sizeof(zero));
    }
    *out = v;
    return e;
}

// A map of a tensor (rows, heads, cols) for boxes of 64 rows x 64 columns of a
// head, or (`across`) of 64 heads x 64 columns of a row; what lies outside
// reads as 0.
inline bool map_of(CUtensorMap *map, const bf *base, int64_t rows, int heads, int cols, bool across = false) {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> cached{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 fn = cached.load(std::memory_order_acquire);
    if (fn == nullptr) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return false;
        fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        cached.store(fn, std::memory_order_release);
    }
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(heads), cuuint64_t(rows)};
    const cuuint64_t strides[2] = {cuuint64_t(cols) * 2, cuuint64_t(cols) * heads * 2};
    const cuuint32_t box[3] = {64, across ? kBlock : 1u, across ? 1u : kBlock}, each[3] = {1, 1, 1};
    const auto encode = [&] {
        return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<bf *>(base), dims, strides, box, each,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    // A host thread that has made no call of the runtime yet has no context for the driver's.  Setting the
    // device that it has gives it one, and unlike an allocation's call may be made while a graph is captured.
    int device = 0;
    return encode() || (cudaGetDevice(&device) == cudaSuccess && cudaSetDevice(device) == cudaSuccess && encode());
}
// A launch that may begin while the kernel before it in the stream runs.
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), unsigned grid, unsigned threads, int bytes, cudaStream_t st, A... args) {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(grid), c.blockDim = dim3(threads);
    c.dynamicSmemBytes = size_t(bytes), c.stream = st;
    c.attrs = &at, c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

// Sizes whose rows 16-byte copies can take, and whose states fit a warp's registers.
inline bool fits(const Shape &s) {
    return s.K <= 128 && s.K % 8 == 0 && s.V % 8 == 0 && s.rows() <= 0x7fffffff - kBlock;
}
inline int64_t record_bytes(const Shape &s) { return s.slots() * s.H * kRecord; }
// ... and whose block fits shared memory.
inline bool fits_bwd(const Shape &s) { return fits(s) && s.V <= 128; }
// Blocks a part, or 0 for whole sequences: a chain is one head's slice of 64
// values, at most one a SM at a time.  In parts, every block is walked about
// twice more (its own 64 rows and the K rows that its turning of the state
// takes, then the outputs), so that parts pay where the chains fill a small
// share of the SMs, 152 as on every GB300 (the size functions follow the same
// rule and need no device; results are right whatever a GPU has).  The bound lies
// between the sizes measured on either side, calls of one sequence, whole against
// in parts:
//   16384 steps, K = V = 128: 8 heads 743 / 287 us, 24 heads 815 / 667, 32 heads 850 / 888
//   4096 steps,  K = V = 128: 8 heads 194 / 128, 16 heads 203 / 167, 32 heads 220 / 259
//   16384 steps, K = 128, V = 64: 16 heads 777 / 364, 32 heads 841 / 694
//   16384 steps, K = V = 64: 32 heads 644 / 445, 64 heads 758 / 764
// and, of the lengths, 8 heads: 1024 steps 58 / 65, 1536 steps 81 / 71, 2048 steps 103 / 88.
inline int part_blocks(const Shape &s) {
    const int64_t slices = (s.V + 63) / 64, keys = (s.K + 63) / 64, chains = s.n * int64_t(s.H) * slices;
    const int64_t longest = (s.L + kBlock - 1) / kBlock;
    if (longest < 24 || chains * (3 * slices + keys) > 228 * slices) return 0;
    const int64_t total = s.slots() * s.H * slices, part = (total + 151) / 152;
    return int(part < 8 ? 8 : part);
}
inline int64_t part_places(const Shape &s, int part) {
    const int64_t longest = (s.L + kBlock - 1) / kBlock;
    return s.offsets ? s.L / (int64_t(kBlock) * part) + s.n : (longest + part - 1) / part * s.n;
}
struct FwdScratch {
    int64_t added, turned, entering, bytes;
    int part;
};
inline FwdScratch fwd_scratch(const Shape &s) {
    const auto up = [](int64_t b) { return (b + 255) / 256 * 256; };
    FwdScratch r{};
    r.part = part_blocks(s);
    r.bytes = r.added = r.turned = r.entering = up(record_bytes(s));
    if (r.part) {
        const int64_t heads = part_places(s, r.part) * s.H * 4;
        r.turned = r.added + up(heads * s.V * s.K);
        r.entering = r.turned + up(heads * s.K * s.K);
        r.bytes = r.entering + up(heads * s.V * s.K);
    }
    return r;
}

inline int dbeta_parts(const Shape &s) { return (s.V + 63) / 64 * 4; }

}  // namespace mma
}  // namespace delta
}  // namespace ssm
