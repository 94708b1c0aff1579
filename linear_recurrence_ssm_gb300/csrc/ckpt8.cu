// ckpt8.cu -- 8-bit activation checkpoints: a row's groups of 64 columns, each
// with a scale of its own (gated_scan.cuh has the rounding rule).
//
// Both directions stream: 3 bytes an element of bf16.  Eight lanes share a
// group (8 elements each, one 16-byte access of bf16), a warp takes 16 rows of
// one group with four rows in flight a lane, and the eight warps of a block
// take neighbouring groups, so that a block reads 1 KB of every row and writes
// 64 bytes of neighbouring scales.  Where rows do not start on vectors, lanes
// take single elements, a warp a whole group of 64.  16384 x 2048 bf16: save
// 20.5 us (5.0 TB/s), load 18.5 us (5.5 TB/s), 15 us of bytes each and 3 us of
// start.  8 rows a warp measured the same, 4 rows 28.7 us, 32 rows 30.7 us;
// one division a row instead of one a lane took save from 24.6 to 20.5 us.
#include "gated_scan.cuh"

namespace ssm {
namespace ckpt8 {
using namespace gated;

constexpr int kRows = 16, kWarps = 8;

struct Block {
    int64_t row0, group;
};
// Blocks count through the groups, eight at a time, then the rows.
__device__ __forceinline__ Block block_of(int64_t groups) {
    const uint32_t across = uint32_t((groups + kWarps - 1) / kWarps), row = blockIdx.x / across;
    return {int64_t(row) * kRows, int64_t(blockIdx.x - row * across) * kWarps + threadIdx.x / 32};
}

// |v| as bits: their order is that of the values, NaN on top
__device__ __forceinline__ uint32_t size_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Eight elements as they are read; the largest's size_bits; one as fp32.
struct Eight16 {
    uint32_t w[4];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { *reinterpret_cast<uint4 *>(w) = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
        return max(m << 16, m & 0xffff0000u);
    }
    __device__ __forceinline__ float at(int k) const {
        return __uint_as_float(k % 2 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
    }
};
struct Eight32 {
    float v[8];
    __device__ __forceinline__ void load(const float *p) {
        reinterpret_cast<float4 *>(v)[0] = reinterpret_cast<const float4 *>(p)[0];
        reinterpret_cast<float4 *>(v)[1] = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) m = max(m, size_bits(v[k]));
        return m;
    }
    __device__ __forceinline__ float at(int k) const { return v[k]; }
};
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
    uint4 w;
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4 *>(p) = w;
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
// cols is a multiple of 8, x starts on 16 bytes and q on 8.
template <typename T>
__global__ void __launch_bounds__(32 * kWarps)
save_vectors_kernel(const T *__restrict__ x, int8_t *__restrict__ q, float *__restrict__ scale, int64_t rows,
                    int64_t cols) {
    const Block b = block_of((cols + kGroup - 1) / kGroup);
    const int lane = threadIdx.x % 32;
    const int64_t e = b.group * kGroup + lane % 8 * 8;
    if (b.group * kGroup >= cols) return;
    const int64_t first = b.row0 + lane / 8, at = first * cols + e, step = 4 * cols;
    const int left = int(min(rows - first, int64_t(kRows)));      // rows of this lane: 0, 4, ... below it
    std::conditional_t<sizeof(T) == 4, Eight32, Eight16> v[kRows / 4];
#pragma unroll
    for (int i = 0; i < kRows / 4; ++i) {
        v[i] = {};
        if (4 * i < left && e < cols) v[i].load(x + at + i * step);
    }
    // lane 8 r + i divides for row 4 i + r
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < kRows / 4; ++i) {
        uint32_t top = v[i].top();
#pragma unroll
        for (int d = 1; d < 8; d *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        if (lane % 8 == i) mine = top;
    }
    const float t = __uint_as_float(mine), inv = inverse_of(t);
    if (lane % 8 < kRows / 4 && 4 * (lane % 8) < left)
        scale[b.group * rows + first + 4 * (lane % 8)] = scale_of(t);
#pragma unroll
    for (int i = 0; i < kRows / 4; ++i) {
        const float by = __shfl_sync(0xffffffffu, inv, (lane & 24) + i);
        uint32_t n[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) n[k] = quantised(v[i].at(k), by);
        uint2 w;
        w.x = __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
        w.y = __byte_perm(__byte_perm(n[4], n[5], 0x0040), __byte_perm(n[6], n[7], 0x0040), 0x5410);
        if (4 * i < left && e < cols) *reinterpret_cast<uint2 *>(q + at + i * step) = w;
    }
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps)
load_vectors_kernel(const int8_t *__restrict__ q, const float *__restrict__ scale, T *__restrict__ x, int64_t rows,
                    int64_t cols) {
    const Block b = block_of((cols + kGroup - 1) / kGroup);
    const int lane = threadIdx.x % 32;
    const int64_t e = b.group * kGroup + lane % 8 * 8;
    if (e >= cols) return;
    const int64_t first = b.row0 + lane / 8, at = first * cols + e, step = 4 * cols;
    const int left = int(min(rows - first, int64_t(kRows)));
    uint2 w[kRows / 4];
    float s[kRows / 4];
#pragma unroll
    for (int i = 0; i < kRows / 4; ++i) {
        if (4 * i >= left) break;
        w[i] = *reinterpret_cast<const uint2 *>(q + at + i * step);
        s[i] = scale[b.group * rows + first + 4 * i];
    }
#pragma unroll
    for (int i = 0; i < kRows / 4; ++i) {
        if (4 * i >= left) break;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = float(int8_t((k < 4 ? w[i].x : w[i].y) >> (k % 4 * 8))) * s[i];
        store8(x + at + i * step, v);
    }
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps)
save_elements_kernel(const T *__restrict__ x, int8_t *__restrict__ q, float *__restrict__ scale, int64_t rows,
                     int64_t cols) {
    const Block b = block_of((cols + kGroup - 1) / kGroup);
    const int lane = threadIdx.x % 32;
    const int64_t e = b.group * kGroup + lane;
    if (b.group * kGroup >= cols) return;
    const bool in0 = e < cols, in1 = e + 32 < cols;
    float v[kRows][2];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t at = (b.row0 + i) * cols + e;
        const bool in = b.row0 + i < rows;
        v[i][0] = in && in0 ? to_f32(x[at]) : 0.0f;
        v[i][1] = in && in1 ? to_f32(x[at + 32]) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const float t = __uint_as_float(__reduce_max_sync(0xffffffffu, max(size_bits(v[i][0]), size_bits(v[i][1]))));
        const float inv = inverse_of(t);
        const int64_t at = (b.row0 + i) * cols + e;
        if (b.row0 + i < rows) {
            if (in0) q[at] = int8_t(quantised(v[i][0], inv));
            if (in1) q[at + 32] = int8_t(quantised(v[i][1], inv));
            if (lane == i) scale[b.group * rows + b.row0 + i] = scale_of(t);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps)
load_elements_kernel(const int8_t *__restrict__ q, const float *__restrict__ scale, T *__restrict__ x, int64_t rows,
                     int64_t cols) {
    const Block b = block_of((cols + kGroup - 1) / kGroup);
    const int64_t e = b.group * kGroup + threadIdx.x % 32;
    if (b.group * kGroup >= cols) return;
    const bool in0 = e < cols, in1 = e + 32 < cols;
    int8_t n[kRows][2];
    float s[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t at = (b.row0 + i) * cols + e;
        const bool in = b.row0 + i < rows;
        n[i][0] = in && in0 ? q[at] : 0;
        n[i][1] = in && in1 ? q[at + 32] : 0;
        s[i] = in ? scale[b.group * rows + b.row0 + i] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t at = (b.row0 + i) * cols + e;
        if (b.row0 + i >= rows) break;
        if (in0) put(x + at, float(n[i][0]) * s[i]);
        if (in1) put(x + at + 32, float(n[i][1]) * s[i]);
    }
}

// The grid's blocks; 0 where there are too many.
static unsigned blocks_for(int64_t rows, int64_t cols) {
    const int64_t groups = (cols + kGroup - 1) / kGroup;
    const int64_t n = (rows + kRows - 1) / kRows * ((groups + kWarps - 1) / kWarps);
    return n <= 0x7fffffff ? unsigned(n) : 0;
}
static bool vectors(const void *x, const void *q, int64_t cols) {
    return cols % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 && reinterpret_cast<uintptr_t>(q) % 8 == 0;
}

template <typename T>
cudaError_t save(const T *x, int8_t *q, float *scale, int64_t rows, int64_t cols, cudaStream_t st) {
    const unsigned grid = blocks_for(rows, cols);
    if (grid == 0) return cudaErrorInvalidConfiguration;
    if (vectors(x, q, cols))
        save_vectors_kernel<T><<<grid, 32 * kWarps, 0, st>>>(x, q, scale, rows, cols);
    else
        save_elements_kernel<T><<<grid, 32 * kWarps, 0, st>>>(x, q, scale, rows, cols);
    return cudaGetLastError();
}

template <typename T>
cudaError_t load(const int8_t *q, const float *scale, T *x, int64_t rows, int64_t cols, cudaStream_t st) {
    const unsigned grid = blocks_for(rows, cols);
    if (grid == 0) return cudaErrorInvalidConfiguration;
    if (vectors(x, q, cols))
        load_vectors_kernel<T><<<grid, 32 * kWarps, 0, st>>>(q, scale, x, rows, cols);
    else
        load_elements_kernel<T><<<grid, 32 * kWarps, 0, st>>>(q, scale, x, rows, cols);
    return cudaGetLastError();
}

template cudaError_t save<float>(const float *, int8_t *, float *, int64_t, int64_t, cudaStream_t);
template cudaError_t save<__nv_bfloat16>(const __nv_bfloat16 *, int8_t *, float *, int64_t, int64_t,
                                         cudaStream_t);
template cudaError_t load<float>(const int8_t *, const float *, float *, int64_t, int64_t, cudaStream_t);
template cudaError_t load<__nv_bfloat16>(const int8_t *, const float *, __nv_bfloat16 *, int64_t, int64_t,
                                         cudaStream_t);

}  // namespace ckpt8
}  // namespace ssm
