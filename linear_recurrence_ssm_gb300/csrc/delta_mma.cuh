// delta_mma.cuh -- pieces of the gated delta rule's tensor-core kernels: warp
// matrix products on bf16 fragments, swizzled tiles, values split in two bf16
// terms, and the strictly lower triangular inverse of a block of 64 steps.
//
// A warp keeps 16 rows of the state, transposed products and all, in the
// accumulator layout of m16n8k16, which is also the layout of the next
// product's left operand: the chain state -> errors -> state never leaves the
// warp's registers, and the warps of the chain never wait for one another.
#pragma once

#include "delta_rule.cuh"

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

// Tiles of bf16 in shared memory: rows of WIDTH elements (64 or 128), the
// 16-byte pieces of a row exchanged by its number, so that eight rows' pieces
// of one column lie in eight different groups of banks.
template <int WIDTH>
__device__ __forceinline__ uint32_t place(uint32_t tile, int row, int col) {      // col: a multiple of 8
    return tile + row * (WIDTH * 2) + (((col >> 3) ^ (row & 7)) << 4);
}
// The address that this lane gives for four 8 x 8 pieces: rows r, r + 8 by
// columns c, c + 8 in the order (r, c), (r + 8, c), (r, c + 8), (r + 8, c + 8).
template <int WIDTH>
__device__ __forceinline__ uint32_t four(uint32_t tile, int r, int c) {
    const int lane = threadIdx.x % 32;
    return place<WIDTH>(tile, r + (lane & 15), c + (lane >> 4) * 8);
}
// The same in the order (r, c), (r, c + 8), (r + 8, c), (r + 8, c + 8).
template <int WIDTH>
__device__ __forceinline__ uint32_t four_across(uint32_t tile, int r, int c) {
    const int lane = threadIdx.x % 32;
    return place<WIDTH>(tile, r + (lane & 7) + (lane >> 4) * 8, c + ((lane >> 3) & 1) * 8);
}

// `rows` rows of `width` elements (a multiple of 8) into a tile of 64 x WIDTH, zeros around them.
template <int WIDTH, int THREADS>
__device__ __forceinline__ void copy_tile(uint32_t tile, const bf *src, int64_t step, int rows, int width, int tid) {
#pragma unroll
    for (int i = 0; i < kBlock * WIDTH / 8 / THREADS; ++i) {
        const int at = i * THREADS + tid, row = at / (WIDTH / 8), col = at % (WIDTH / 8) * 8;
        const bool in = row < rows && col < width;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(place<WIDTH>(tile, row, col)),
                     "l"(in ? src + row * step + col : src), "r"(in ? 16 : 0)
                     : "memory");
    }
}

__device__ __forceinline__ uint4 load16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to), "l"(from) : "memory");
}

// by v, and 0 for by = 0 whatever v holds.
__device__ __forceinline__ float kept(float by, float v) { return by == 0.0f ? 0.0f : by * v; }

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

// N with (I + A beta) N = A for A strictly lower triangular (64 x 64 floats in
// `m`, zeros on and above the diagonal of its 16 x 16 blocks on the diagonal),
// so that (I + A beta)^-1 = I - N beta.  N takes A's place; what lies above
// the diagonal blocks is overwritten.  Blocks of 16 by substitution, then
// pairs of blocks joined:
//   N21 = (I - N22 beta2) A21 (I - beta1 N11).
// All in fp32: the errors of a solve feed every later step.  128 threads.
__device__ __forceinline__ void lower_solve(float *m, const float *beta, int tid) {
    {
        const int b = tid / 32 * 16, j = tid % 16;
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
#pragma unroll
    for (int size = 16; size <= 32; size *= 2) {
        // four columns of a row of the lower left block; the upper right one holds A21 (I - beta1 N11)
        const int per = size / 4, items = size / 16;
#pragma unroll
        for (int i = 0; i < items; ++i) {
            const int at = i * 128 + tid, p = at / (size * per), t = at / per % size, c = at % per * 4;
            const int first = p * 2 * size, second = first + size;
            float4 o = *reinterpret_cast<const float4 *>(m + (second + t) * kPairStride + first + c);
#pragma unroll
            for (int s = 0; s < size; s += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(m + (second + t) * kPairStride + first + s);
                const float4 w = *reinterpret_cast<const float4 *>(beta + first + s);
                const float av[4] = {a.x * w.x, a.y * w.y, a.z * w.z, a.w * w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 n = *reinterpret_cast<const float4 *>(m + (first + s + e) * kPairStride + first + c);
                    // N11 is strictly lower, but its upper part may hold a smaller pair's left-overs
                    o.x -= s + e > c ? av[e] * n.x : 0.0f;
                    o.y -= s + e > c + 1 ? av[e] * n.y : 0.0f;
                    o.z -= s + e > c + 2 ? av[e] * n.z : 0.0f;
                    o.w -= s + e > c + 3 ? av[e] * n.w : 0.0f;
                }
            }
            *reinterpret_cast<float4 *>(m + (first + t) * kPairStride + second + c) = o;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < items; ++i) {
            const int at = i * 128 + tid, p = at / (size * per), t = at / per % size, c = at % per * 4;
            const int first = p * 2 * size, second = first + size;
            float4 o = *reinterpret_cast<const float4 *>(m + (first + t) * kPairStride + second + c);
#pragma unroll
            for (int s = 0; s < size; s += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(m + (second + t) * kPairStride + second + s);
                const float4 w = *reinterpret_cast<const float4 *>(beta + second + s);
                const float av[4] = {s < t ? a.x * w.x : 0.0f, s + 1 < t ? a.y * w.y : 0.0f,
                                     s + 2 < t ? a.z * w.z : 0.0f, s + 3 < t ? a.w * w.w : 0.0f};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 n = *reinterpret_cast<const float4 *>(m + (first + s + e) * kPairStride + second + c);
                    o.x -= av[e] * n.x, o.y -= av[e] * n.y, o.z -= av[e] * n.z, o.w -= av[e] * n.w;
                }
            }
            *reinterpret_cast<float4 *>(m + (second + t) * kPairStride + first + c) = o;
        }
        __syncthreads();
    }
}

// What the chains need of a block besides its tokens, made once by
// pairs_kernel: -N in two bf16 terms, P (with the scale), the factors, and for
// the gradients P's second term; tiles of 64 x 64 with their pieces exchanged
// as place<64> does.  Blocks of 16 x 16 above P's diagonal are unspecified.
constexpr int kTile = kBlock * kBlock * 2;
constexpr int kRecord = (3 * kTile + int(sizeof(Factors)) + 127) / 128 * 128, kBothRecord = kRecord + kTile;
cudaError_t make_pairs(const Shape &s, const bf *q, const bf *k, const bf *g, const bf *beta, unsigned char *records,
                       bool both, cudaStream_t st);

// Sizes whose rows 16-byte copies can take, and whose states fit a warp's registers.
inline bool fits(const Shape &s) { return s.K <= 128 && s.K % 8 == 0 && s.V % 8 == 0; }
inline int64_t record_bytes(const Shape &s) { return s.slots() * s.H * kRecord; }
// ... and whose block fits shared memory.
inline bool fits_bwd(const Shape &s) { return fits(s) && s.V <= 128; }
inline int dbeta_parts(const Shape &s) { return (s.V + 63) / 64 * 4; }

}  // namespace mma
}  // namespace delta
}  // namespace ssm
