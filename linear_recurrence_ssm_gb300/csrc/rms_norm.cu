// rms_norm.cu -- root-mean-square norm over rows, with the residual's addition
// and an output in 8 bits, and its gradients.
//
//   s = x + residual,  r = (mean s^2 + eps)^-1/2,  y = s r w
//   dx = ds + r (w dy - s r^2 mean(w dy s)),  dw = sum over rows of dy s r
//
// Memory bound: every element is read once and kept in registers between the
// row's sum and its outputs.  A row takes the lanes that its vectors of eight
// need at two to four vectors a lane; short rows share a block.
#include <type_traits>

#include "gated_scan.cuh"

namespace ssm {
namespace norm {
using gated::inverse_of;
using gated::kGroup;
using gated::quantised;
using gated::scale_of;

constexpr int kVec = 8;                 // elements of an access
constexpr int kParts = 608;             // most partial sums of dw

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16(v); }

__device__ __forceinline__ void load8(float (&v)[kVec], const float *p) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(float (&v)[kVec], const __nv_bfloat16 *p) {
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float *p, const float (&v)[kVec]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[kVec]) {
    uint4 w;
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4 *>(p) = w;
}

// The sum over the LANES threads that share a row (a block holds 1 or more
// such groups); every thread of the group gets it.  `mem`: a float a warp.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float *mem) {
#pragma unroll
    for (int o = (LANES < 32 ? LANES : 32) / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (LANES > 32) {
        constexpr int warps = LANES > 32 ? LANES / 32 : 1;
        const int warp = threadIdx.x / 32, first = warp / warps * warps;
        __syncthreads();
        if (threadIdx.x % 32 == 0) mem[warp] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < warps; ++i) v += mem[first + i];
    }
    return v;
}

template <typename T>
struct FwdArgs {
    const T *x, *residual;
    const float *weight;
    T *sum, *y;
    int8_t *q;
    float *scale, *rstd;
    int64_t rows, cols;
    float eps;
};

constexpr int threads_for(int lanes) { return lanes > 256 ? lanes : 256; }

template <typename T, int LANES, int VECS>
__global__ void __launch_bounds__(threads_for(LANES)) fwd_kernel(const FwdArgs<T> p) {
    __shared__ float mem[32];
    constexpr int per_block = threads_for(LANES) / LANES;
    const int lane = threadIdx.x % LANES;
    const int64_t row = int64_t(blockIdx.x) * per_block + threadIdx.x / LANES;
    const bool there = row < p.rows;
    const int64_t at = row * p.cols;
    float v[VECS][kVec], squares = 0.0f;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int c = (i * LANES + lane) * kVec;
        if (there && c < p.cols) {
            load8(v[i], p.x + at + c);
            if (p.residual) {
                float r[kVec];
                load8(r, p.residual + at + c);
#pragma unroll
                for (int e = 0; e < kVec; ++e) v[i][e] += r[e];
                store8(p.sum + at + c, v[i]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[i][e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) squares += v[i][e] * v[i][e];
    }
    const float rstd = 1.0f / sqrtf(row_sum<LANES>(squares, mem) / float(p.cols) + p.eps);
    if (there && lane == 0 && p.rstd) p.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int c = (i * LANES + lane) * kVec;
        const bool in = there && c < p.cols;
        float w[kVec];
        if (in && p.weight) {
            load8(w, p.weight + c);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) w[e] = 1.0f;
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[i][e] = v[i][e] * rstd * w[e];
        if (p.q) {
            // eight lanes share a group of 64 columns
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < kVec; ++e) top = max(top, __float_as_uint(v[i][e]) & 0x7fffffffu);
#pragma unroll
            for (int o = 1; o < 8; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float t = __uint_as_float(top), inv = inverse_of(t);
            uint32_t n[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) n[e] = quantised(v[i][e], inv);
            uint2 o;
            o.x = __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
            o.y = __byte_perm(__byte_perm(n[4], n[5], 0x0040), __byte_perm(n[6], n[7], 0x0040), 0x5410);
            if (in) {
                *reinterpret_cast<uint2 *>(p.q + at + c) = o;
                if (lane % 8 == 0) p.scale[int64_t(c / kGroup) * p.rows + row] = scale_of(t);
            }
        } else if (in) {
            store8(p.y + at + c, v[i]);
        }
    }
}

// Any width and alignment: a block a row, the sum recomputed for the second pass.
template <typename T>
__global__ void __launch_bounds__(256) fwd_elements_kernel(const FwdArgs<T> p) {
    __shared__ float mem[32];
    const int64_t row = blockIdx.x, at = row * p.cols;
    const auto value = [&](int64_t c) {
        return to_f32(p.x[at + c]) + (p.residual ? to_f32(p.residual[at + c]) : 0.0f);
    };
    float squares = 0.0f;
    for (int64_t c = threadIdx.x; c < p.cols; c += 256) {
        const float v = value(c);
        squares += v * v;
    }
    const float rstd = 1.0f / sqrtf(row_sum<256>(squares, mem) / float(p.cols) + p.eps);
    if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;
    // a warp takes a group of 64 columns at a time; the sum may lie where x or the residual lay
    const int lane = threadIdx.x % 32;
    for (int64_t g = threadIdx.x / 32; g * kGroup < p.cols; g += 8) {
        float v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t c = g * kGroup + 32 * h + lane;
            v[h] = 0.0f;
            if (c < p.cols) {
                const float s = value(c);
                if (p.residual) put(p.sum + at + c, s);
                v[h] = s * rstd * (p.weight ? p.weight[c] : 1.0f);
            }
        }
        if (p.q) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, max(__float_as_uint(v[0]) & 0x7fffffffu,
                                                                     __float_as_uint(v[1]) & 0x7fffffffu));
            const float t = __uint_as_float(top), inv = inverse_of(t);
            if (lane == 0) p.scale[g * p.rows + row] = scale_of(t);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t c = g * kGroup + 32 * h + lane;
                if (c < p.cols) p.q[at + c] = int8_t(quantised(v[h], inv));
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t c = g * kGroup + 32 * h + lane;
                if (c < p.cols) put(p.y + at + c, v[h]);
            }
        }
    }
}

template <typename T>
struct BwdArgs {
    const T *dy, *s, *residual, *ds;     // s, or x and the residual that make it up
    const float *weight, *rstd;
    T *dx;
    float *dweight, *parts;
    int64_t rows, cols;
};

// A thread keeps its columns over all rows of its block: dw's partial sums
// stay in registers.  Each group of LANES threads writes one part.
template <typename T, int LANES, int VECS>
__global__ void __launch_bounds__(threads_for(LANES)) bwd_kernel(const BwdArgs<T> p) {
    __shared__ float mem[32];
    constexpr int per_block = threads_for(LANES) / LANES;
    const int lane = threadIdx.x % LANES;
    const int64_t part = int64_t(blockIdx.x) * per_block + threadIdx.x / LANES, step = int64_t(gridDim.x) * per_block;
    const float inv_cols = 1.0f / float(p.cols);
    float dw[VECS][kVec] = {};
    // groups of a block take the same turns, for the barriers of row_sum
    for (int64_t row0 = int64_t(blockIdx.x) * per_block; row0 < p.rows; row0 += step) {
        const int64_t row = row0 + threadIdx.x / LANES, at = row * p.cols;
        const bool there = row < p.rows;
        const float rstd = there ? p.rstd[row] : 0.0f;
        float s[VECS][kVec], d[VECS][kVec], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const int c = (i * LANES + lane) * kVec;
            if (there && c < p.cols) {
                load8(s[i], p.s + at + c);
                load8(d[i], p.dy + at + c);
                if (p.residual) {
                    float r[kVec];
                    load8(r, p.residual + at + c);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) s[i][e] += r[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e) s[i][e] = d[i][e] = 0.0f;
            }
            float w[kVec];
            if (p.weight && c < p.cols) {
                load8(w, p.weight + c);
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e) w[e] = 1.0f;
            }
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                s[i][e] *= rstd;
                dw[i][e] += d[i][e] * s[i][e];
                d[i][e] *= w[e];
                sum += d[i][e] * s[i][e];
            }
        }
        const float mean = row_sum<LANES>(sum, mem) * inv_cols;
        if (!there) continue;
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const int c = (i * LANES + lane) * kVec;
            if (c >= p.cols) continue;
            float o[kVec];
            if (p.ds) {
                load8(o, p.ds + at + c);
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e) o[e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < kVec; ++e) o[e] += rstd * (d[i][e] - s[i][e] * mean);
            store8(p.dx + at + c, o);
        }
    }
    if (p.dweight)
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const int c = (i * LANES + lane) * kVec;
            if (c < p.cols) store8(p.parts + part * p.cols + c, dw[i]);
        }
}

template <typename T>
__global__ void __launch_bounds__(256) bwd_elements_kernel(const BwdArgs<T> p) {
    __shared__ float mem[32];
    const int64_t row = blockIdx.x, at = row * p.cols;
    const float rstd = p.rstd[row];
    const auto value = [&](int64_t c) { return to_f32(p.s[at + c]) + (p.residual ? to_f32(p.residual[at + c]) : 0.0f); };
    const auto wd = [&](int64_t c) { return to_f32(p.dy[at + c]) * (p.weight ? p.weight[c] : 1.0f); };
    float sum = 0.0f;
    for (int64_t c = threadIdx.x; c < p.cols; c += 256) sum += wd(c) * (value(c) * rstd);
    const float mean = row_sum<256>(sum, mem) / float(p.cols);
    for (int64_t c = threadIdx.x; c < p.cols; c += 256)
        put(p.dx + at + c, (p.ds ? to_f32(p.ds[at + c]) : 0.0f) +
                               rstd * (wd(c) - value(c) * rstd * mean));
}

// dw's partial sums, a thread a column, a block row a part of the rows.
template <typename T>
__global__ void __launch_bounds__(256) weight_elements_kernel(const BwdArgs<T> p) {
    const int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (c >= p.cols) return;
    float sum = 0.0f;
    for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
        const int64_t i = row * p.cols + c;
        const float s = to_f32(p.s[i]) + (p.residual ? to_f32(p.residual[i]) : 0.0f);
        sum += to_f32(p.dy[i]) * (s * p.rstd[row]);
    }
    p.parts[blockIdx.y * p.cols + c] = sum;
}

// dw from its parts: 32 columns a block, the parts over the warps, joined in
// their order.
__global__ void __launch_bounds__(256) weight_kernel(const float *parts, float *dweight, int n, int64_t cols) {
    __shared__ float mem[8][32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t c = int64_t(blockIdx.x) * 32 + lane;
    float sum[4] = {};
    if (c < cols)
        for (int i = warp; i < n; i += 32)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + 8 * j < n) sum[j] += parts[int64_t(i + 8 * j) * cols + c];
    mem[warp][lane] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    __syncthreads();
    if (warp == 0 && c < cols) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += mem[i][lane];
        dweight[c] = v;
    }
}

static bool on16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename T, int LANES, int VECS>
static cudaError_t go(const FwdArgs<T> &a, cudaStream_t st) {
    constexpr int per_block = threads_for(LANES) / LANES;
    const int64_t grid = (a.rows + per_block - 1) / per_block;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    fwd_kernel<T, LANES, VECS><<<unsigned(grid), threads_for(LANES), 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t fwd(const FwdArgs<T> &a, cudaStream_t st) {
    const int64_t vecs = a.cols / kVec;
    if (a.cols % kVec == 0 && vecs <= 4096 && on16(a.x) && on16(a.residual) && on16(a.weight) && on16(a.sum) &&
        on16(a.y) && reinterpret_cast<uintptr_t>(a.q) % 8 == 0) {
        if (vecs <= 8) return go<T, 8, 1>(a, st);
        if (vecs <= 16) return go<T, 16, 1>(a, st);
        if (vecs <= 32) return go<T, 32, 1>(a, st);
        if (vecs <= 64) return go<T, 64, 1>(a, st);
        if (vecs <= 128) return go<T, 64, 2>(a, st);
        if (vecs <= 256) return go<T, 128, 2>(a, st);
        if (vecs <= 512) return go<T, 256, 2>(a, st);
        if (vecs <= 1024) return go<T, 256, 4>(a, st);
        return go<T, 1024, 4>(a, st);
    }
    if (a.rows > 0x7fffffff) return cudaErrorInvalidConfiguration;
    fwd_elements_kernel<T><<<unsigned(a.rows), 256, 0, st>>>(a);
    return cudaGetLastError();
}

static cudaError_t fold(const float *parts, float *dweight, int64_t n, int64_t cols, cudaStream_t st) {
    weight_kernel<<<unsigned((cols + 31) / 32), 256, 0, st>>>(parts, dweight, int(n), cols);
    return cudaGetLastError();
}

template <typename T, int LANES, int VECS>
static cudaError_t go(const BwdArgs<T> &a, cudaStream_t st) {
    constexpr int per_block = threads_for(LANES) / LANES;
    static_assert(kParts % per_block == 0, "whole blocks of parts");
    const int64_t blocks = (a.rows + per_block - 1) / per_block;
    const int64_t grid = blocks < kParts / per_block ? blocks : kParts / per_block;
    bwd_kernel<T, LANES, VECS><<<unsigned(grid), threads_for(LANES), 0, st>>>(a);
    if (cudaError_t e = cudaGetLastError()) return e;
    return a.dweight ? fold(a.parts, a.dweight, grid * per_block, a.cols, st) : cudaSuccess;
}

template <typename T>
cudaError_t bwd(const BwdArgs<T> &a, cudaStream_t st) {
    const int64_t vecs = a.cols / kVec;
    if (a.cols % kVec == 0 && vecs <= 2048 && on16(a.dy) && on16(a.s) && on16(a.residual) && on16(a.ds) && on16(a.weight) && on16(a.dx) &&
        on16(a.parts)) {
        if (vecs <= 8) return go<T, 8, 1>(a, st);
        if (vecs <= 16) return go<T, 16, 1>(a, st);
        if (vecs <= 32) return go<T, 32, 1>(a, st);
        if (vecs <= 64) return go<T, 64, 1>(a, st);
        if (vecs <= 128) return go<T, 128, 1>(a, st);
        if (vecs <= 256) return go<T, 128, 2>(a, st);
        if (vecs <= 512) return go<T, 256, 2>(a, st);
        if (vecs <= 1024) return go<T, 512, 2>(a, st);
        return go<T, 1024, 2>(a, st);
    }
    if (a.rows > 0x7fffffff) return cudaErrorInvalidConfiguration;
    bwd_elements_kernel<T><<<unsigned(a.rows), 256, 0, st>>>(a);
    if (cudaError_t e = cudaGetLastError()) return e;
    if (!a.dweight) return cudaSuccess;
    const unsigned n = unsigned(a.rows < kParts ? a.rows : kParts);
    weight_elements_kernel<T><<<dim3(unsigned((a.cols + 255) / 256), n), 256, 0, st>>>(a);
    if (cudaError_t e = cudaGetLastError()) return e;
    return fold(a.parts, a.dweight, n, a.cols, st);
}

template <typename T>
cudaError_t launch_fwd(const T *x, const T *residual, const float *weight, float eps, T *sum, T *y, int8_t *q,
                       float *scale, float *rstd, int64_t rows, int64_t cols, cudaStream_t st) {
    return fwd(FwdArgs<T>{x, residual, weight, sum, y, q, scale, rstd, rows, cols, eps}, st);
}
template <typename T>
cudaError_t launch_bwd(const T *dy, const T *s, const T *residual, const float *weight, const float *rstd, const T *ds, T *dx,
                       float *dweight, float *scratch, int64_t rows, int64_t cols, cudaStream_t st) {
    return bwd(BwdArgs<T>{dy, s, residual, ds, weight, rstd, dx, dweight, scratch, rows, cols}, st);
}

using bf = __nv_bfloat16;
template cudaError_t launch_fwd<float>(const float *, const float *, const float *, float, float *, float *, int8_t *,
                                       float *, float *, int64_t, int64_t, cudaStream_t);
template cudaError_t launch_fwd<bf>(const bf *, const bf *, const float *, float, bf *, bf *, int8_t *, float *,
                                    float *, int64_t, int64_t, cudaStream_t);
template cudaError_t launch_bwd<float>(const float *, const float *, const float *, const float *, const float *,
                                       const float *, float *, float *, float *, int64_t, int64_t, cudaStream_t);
template cudaError_t launch_bwd<bf>(const bf *, const bf *, const bf *, const float *, const float *, const bf *, bf *, float *,
                                    float *, int64_t, int64_t, cudaStream_t);

}  // namespace norm
}  // namespace ssm
