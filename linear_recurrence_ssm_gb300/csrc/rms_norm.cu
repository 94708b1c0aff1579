// rms_norm.cu -- root-mean-square norm over rows, with the residual's addition
// and an output in 8 bits, and its gradients.
//
//   s = x + residual,  r = (mean s^2 + eps)^-1/2,  y = s r w
//   dx = ds + r (w dy - s r^2 mean(w dy s)),  dw = sum over rows of dy s r
//
// Memory bound: every element is read once and kept in registers between the
// row's sum and its outputs.  A row of up to 256 columns takes 8, 16 or 32
// lanes, a longer one a thread block of as many warps as its vectors of eight
// need at one to four a thread.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "gated_scan.cuh"
#include "kept_by_device.cuh"

namespace ssm {
namespace norm {
using gated::inverse_of;
using gated::kGroup;
using gated::quantised;
using gated::scale_of;

constexpr int kVec = 8;                 // elements of an access
constexpr int kParts = 1216;            // most partial sums of dw

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

// The sums over the threads that share a row: LANES of a warp, or the whole
// block (LANES = 0).  `mem`: a float a warp and row; the next call of the same
// block needs other ones.
template <int LANES, int ROWS>
__device__ __forceinline__ void row_sums(float (&v)[ROWS], float (*mem)[ROWS]) {
#pragma unroll
    for (int o = (LANES == 0 ? 32 : LANES) / 2; o > 0; o /= 2)
#pragma unroll
        for (int r = 0; r < ROWS; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], o);
    if (LANES == 0) {
        const int warp = threadIdx.x / 32;
        if (threadIdx.x % 32 == 0)
#pragma unroll
            for (int r = 0; r < ROWS; ++r) mem[warp][r] = v[r];
        __syncthreads();
        const int lane = threadIdx.x % 32;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            v[r] = lane < int(blockDim.x / 32) ? mem[lane][r] : 0.0f;
#pragma unroll
            for (int o = 16; o > 0; o /= 2) v[r] += __shfl_xor_sync(0xffffffffu, v[r], o);
        }
    }
}

// Eight elements as they lie in memory.
template <typename T>
struct Raw {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (auto &x : w) x = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < int(sizeof(T) / 2); ++i) w[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void add_to(float (&v)[kVec]) const {
        float x[kVec];
        load8(x, reinterpret_cast<const T *>(w));
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] += x[e];
    }
};

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

template <typename T, int LANES, int VECS>
__global__ void __launch_bounds__(LANES ? 256 : 1024) fwd_kernel(const FwdArgs<T> p) {
    __shared__ float mem[32][1];
    const int lanes = LANES ? LANES : int(blockDim.x), lane = threadIdx.x % lanes;
    const int64_t row = int64_t(blockIdx.x) * (blockDim.x / lanes) + threadIdx.x / lanes;
    const bool there = row < p.rows;
    const int64_t at = row * p.cols;
    float v[VECS][kVec], squares[1] = {0.0f};
    {
        // all loads ahead of the first store, which the compiler may not pass
        Raw<T> x[VECS], r[VECS];
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const int c = (i * lanes + lane) * kVec;
            x[i].clear(), r[i].clear();
            if (there && c < p.cols) {
                x[i].load(p.x + at + c);
                if (p.residual) r[i].load(p.residual + at + c);
            }
        }
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const int c = (i * lanes + lane) * kVec;
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[i][e] = 0.0f;
            x[i].add_to(v[i]);
            if (p.residual) {
                r[i].add_to(v[i]);
                if (there && c < p.cols) store8(p.sum + at + c, v[i]);
            }
#pragma unroll
            for (int e = 0; e < kVec; ++e) squares[0] += v[i][e] * v[i][e];
        }
    }
    row_sums<LANES, 1>(squares, mem);
    const float rstd = 1.0f / sqrtf(squares[0] / float(p.cols) + p.eps);
    if (there && lane == 0 && p.rstd) p.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int c = (i * lanes + lane) * kVec;
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
    __shared__ float mem[32][1];
    const int64_t row = blockIdx.x, at = row * p.cols;
    const auto value = [&](int64_t c) {
        return to_f32(p.x[at + c]) + (p.residual ? to_f32(p.residual[at + c]) : 0.0f);
    };
    float squares[1] = {0.0f};
    for (int64_t c = threadIdx.x; c < p.cols; c += 256) {
        const float v = value(c);
        squares[0] += v * v;
    }
    row_sums<0, 1>(squares, mem);
    const float rstd = 1.0f / sqrtf(squares[0] / float(p.cols) + p.eps);
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

// A thread keeps its columns over all rows of its block, so that dw's partial
// sums stay in registers; a block writes one part.  ROWS rows at a time, all
// their loads ahead of the sums; what was read is kept as it was read and
// unpacked twice, which takes half the registers of its values.  A block a row
// is held to 64 registers, for more rows in flight on a SM (fp32, 16384 x 2560
// without the residual, dw included: 102 us, with 79 registers 115).
template <typename T, int LANES, int VECS, int ROWS>
__global__ void __launch_bounds__(LANES ? 256 : 512, LANES || VECS == 1 ? 2 : 1) bwd_kernel(const BwdArgs<T> p) {
    __shared__ float mem[2][32][ROWS];
    __shared__ float fold[LANES ? 8 : 1][LANES ? LANES * kVec : 1];
    const int lanes = LANES ? LANES : int(blockDim.x), lane = threadIdx.x % lanes;
    const int groups = blockDim.x / lanes;              // rows side by side
    const float inv_cols = 1.0f / float(p.cols);
    float dw[VECS][kVec] = {};
    // groups of a block take the same turns, for the barriers of row_sums
    int turn = 0;
    for (int64_t row0 = int64_t(blockIdx.x) * groups * ROWS; row0 < p.rows; row0 += int64_t(gridDim.x) * groups * ROWS) {
        const int64_t row = row0 + threadIdx.x / lanes;         // and row + groups
        Raw<T> s[ROWS][VECS], d[ROWS][VECS], more[ROWS][VECS], other[ROWS][VECS];
        float rstd[ROWS], sum[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const bool there = row + r * groups < p.rows;
            const int64_t at = (row + r * groups) * p.cols;
            rstd[r] = there ? p.rstd[row + r * groups] : 0.0f;
#pragma unroll
            for (int i = 0; i < VECS; ++i) {
                const int c = (i * lanes + lane) * kVec;
                const bool in = there && c < p.cols;
                s[r][i].clear(), d[r][i].clear(), more[r][i].clear(), other[r][i].clear();
                if (in) s[r][i].load(p.s + at + c), d[r][i].load(p.dy + at + c);
                if (in && p.residual) other[r][i].load(p.residual + at + c);
                if (in && p.ds) more[r][i].load(p.ds + at + c);
            }
        }
        // s r and w dy of one vector
        const auto unpack = [&](int r, int i, float (&x)[kVec], float (&y)[kVec], bool first) {
            const int c = (i * lanes + lane) * kVec;
            float w[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) x[e] = y[e] = 0.0f, w[e] = 1.0f;
            s[r][i].add_to(x);
            if (p.residual) other[r][i].add_to(x);
            d[r][i].add_to(y);
            if (p.weight && c < p.cols) load8(w, p.weight + c);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                x[e] *= rstd[r];
                if (first) dw[i][e] += y[e] * x[e];
                y[e] *= w[e];
            }
        };
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            sum[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < VECS; ++i) {
                float x[kVec], y[kVec];
                unpack(r, i, x, y, true);
#pragma unroll
                for (int e = 0; e < kVec; ++e) sum[r] += y[e] * x[e];
            }
        }
        row_sums<LANES, ROWS>(sum, mem[turn]);
        turn ^= 1;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (row + r * groups >= p.rows) break;
            const int64_t at = (row + r * groups) * p.cols;
            const float mean = sum[r] * inv_cols;
#pragma unroll
            for (int i = 0; i < VECS; ++i) {
                const int c = (i * lanes + lane) * kVec;
                if (c >= p.cols) continue;
                float x[kVec], y[kVec], o[kVec];
                unpack(r, i, x, y, false);
#pragma unroll
                for (int e = 0; e < kVec; ++e) o[e] = rstd[r] * (y[e] - x[e] * mean);
                more[r][i].add_to(o);
                store8(p.dx + at + c, o);
            }
        }
    }
    if (!p.dweight) return;
    if constexpr (LANES > 0) {
        // the groups of a warp, then the warps
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
#pragma unroll
            for (int o = LANES; o < 32; o *= 2) dw[0][e] += __shfl_xor_sync(0xffffffffu, dw[0][e], o);
            if (threadIdx.x % 32 < LANES) fold[threadIdx.x / 32][(threadIdx.x % 32) * kVec + e] = dw[0][e];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < p.cols; c += 256) {
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) v += fold[i][c];
            p.parts[blockIdx.x * p.cols + c] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const int c = (i * lanes + lane) * kVec;
            if (c < p.cols) store8(p.parts + blockIdx.x * p.cols + c, dw[i]);
        }
    }
}

// The same for bf16 rows of a whole block: what the next row holds is on its
// way to shared memory, a thread's own pieces to its own places, so that no
// barrier but the row's sum is needed, and values are unpacked once.  16384 x
// 2560 with the residual and ds: 75 us, from registers 89 (3 and 4 rows on their
// way: 76, 82); without them 56 and 78.  fp32 rows have twice the bytes in
// flight for the same instructions and gain nothing: 102 from registers, 136 so.
using bf = __nv_bfloat16;
constexpr int kStages = 2;

template <int VECS>
__global__ void __launch_bounds__(512, VECS == 1 ? 2 : 1) bwd_ring_kernel(const BwdArgs<bf> p) {
    extern __shared__ uint4 ring[];
    __shared__ float mem[2][32][1];
    const int tid = threadIdx.x, threads = blockDim.x;
    const int of_tensor = VECS * threads, tensors = 2 + (p.residual != nullptr) + (p.ds != nullptr);
    const float inv_cols = 1.0f / float(p.cols);
    float w[VECS][kVec], dw[VECS][kVec] = {};
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int c = (i * threads + tid) * kVec;
        if (p.weight && c < p.cols) {
            load8(w[i], p.weight + c);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) w[i][e] = 1.0f;
        }
    }
    const auto ask = [&](int stage, int64_t row) {
        uint32_t to = smem_u32(ring + stage * tensors * of_tensor + tid);
        const auto tensor = [&](const bf *from) {
#pragma unroll
            for (int i = 0; i < VECS; ++i) {
                const int c = (i * threads + tid) * kVec;
                if (row < p.rows && c < p.cols)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to + i * threads * 16),
                                 "l"(from + row * p.cols + c)
                                 : "memory");
            }
            to += of_tensor * 16;
        };
        tensor(p.s), tensor(p.dy);
        if (p.residual) tensor(p.residual);
        if (p.ds) tensor(p.ds);
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
    const int64_t step = gridDim.x;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) ask(i, blockIdx.x + i * step);
    int stage = 0, turn = 0;
    float rstd = p.rstd[blockIdx.x];
    for (int64_t row = blockIdx.x; row < p.rows; row += step) {
        ask(stage == 0 ? kStages - 1 : stage - 1, row + (kStages - 1) * step);
        asm volatile("cp.async.wait_group %0;\n" ::"n"(kStages - 1) : "memory");
        const uint4 *at = ring + stage * tensors * of_tensor + tid;
        const auto take = [&](int tensor, int i) {
            Raw<bf> v;
            v.w[0] = at[tensor * of_tensor + i * threads];
            return v;
        };
        float x[VECS][kVec], y[VECS][kVec], sum[1] = {0.0f};       // s r, and w dy
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) x[i][e] = y[i][e] = 0.0f;
            if ((i * threads + tid) * kVec < p.cols) {
                take(0, i).add_to(x[i]);
                if (p.residual) take(2, i).add_to(x[i]);
                take(1, i).add_to(y[i]);
            }
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                x[i][e] *= rstd;
                dw[i][e] += y[i][e] * x[i][e];
                y[i][e] *= w[i][e];
                sum[0] += y[i][e] * x[i][e];
            }
        }
        const float next = row + step < p.rows ? p.rstd[row + step] : 0.0f;
        row_sums<0, 1>(sum, mem[turn]);
        turn ^= 1;
        const float mean = sum[0] * inv_cols;
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const int c = (i * threads + tid) * kVec;
            if (c >= p.cols) continue;
            float o[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) o[e] = rstd * (y[i][e] - x[i][e] * mean);
            if (p.ds) take(tensors - 1, i).add_to(o);
            store8(p.dx + row * p.cols + c, o);
        }
        rstd = next;
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    if (!p.dweight) return;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int c = (i * threads + tid) * kVec;
        if (c < p.cols) store8(p.parts + blockIdx.x * p.cols + c, dw[i]);
    }
}

template <typename T>
__global__ void __launch_bounds__(256) bwd_elements_kernel(const BwdArgs<T> p) {
    __shared__ float mem[32][1];
    const int64_t row = blockIdx.x, at = row * p.cols;
    const float rstd = p.rstd[row];
    const auto value = [&](int64_t c) { return to_f32(p.s[at + c]) + (p.residual ? to_f32(p.residual[at + c]) : 0.0f); };
    const auto wd = [&](int64_t c) { return to_f32(p.dy[at + c]) * (p.weight ? p.weight[c] : 1.0f); };
    float sum[1] = {0.0f};
    for (int64_t c = threadIdx.x; c < p.cols; c += 256) sum[0] += wd(c) * (value(c) * rstd);
    row_sums<0, 1>(sum, mem);
    const float mean = sum[0] / float(p.cols);
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

// dw from its parts: 32 columns a block, the parts over its 32 warps, joined
// in their order.
__global__ void __launch_bounds__(1024) weight_kernel(const float *parts, float *dweight, int n, int64_t cols) {
    __shared__ float mem[32][33];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t c = int64_t(blockIdx.x) * 32 + lane;
    float sum[4] = {};
    if (c < cols)
        for (int i = warp; i < n; i += 128)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + 32 * j < n) sum[j] += parts[int64_t(i + 32 * j) * cols + c];
    mem[warp][lane] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    __syncthreads();
    // warp w has column w
    float v = mem[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int64_t mine = int64_t(blockIdx.x) * 32 + warp;
    if (lane == 0 && mine < cols) dweight[mine] = v;
}

static bool on16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
// Threads for a row of `vecs` vectors at `each` a thread.
static unsigned threads_for(int64_t vecs, int each) { return unsigned(((vecs + each - 1) / each + 31) / 32 * 32); }

template <typename T, int LANES, int VECS>
static cudaError_t go(const FwdArgs<T> &a, cudaStream_t st) {
    const unsigned threads = LANES ? 256 : threads_for(a.cols / kVec, VECS), per = LANES ? 256 / LANES : 1;
    const int64_t grid = (a.rows + per - 1) / per;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    fwd_kernel<T, LANES, VECS><<<unsigned(grid), threads, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t fwd(const FwdArgs<T> &a, cudaStream_t st) {
    const int64_t vecs = a.cols / kVec;
    if (a.cols % kVec == 0 && vecs <= 4096 && on16(a.x) && on16(a.residual) && on16(a.weight) && on16(a.sum) &&
        on16(a.y) && reinterpret_cast<uintptr_t>(a.q) % 8 == 0) {
        // lanes of a warp up to 256 columns (bf16, 100000 x 256 with a residual: 38 us, as a block a row
        // 58; 400000 x 64: 37 and 210); then two vectors a thread (16384 x 2048 to 8 bits: 37.5, one
        // 43.6; 32768 x 1024: 37.5 and 42.6), four where 1024 threads would not do otherwise
        if (vecs <= 8) return go<T, 8, 1>(a, st);
        if (vecs <= 16) return go<T, 16, 1>(a, st);
        if (vecs <= 32) return go<T, 32, 1>(a, st);
        if (vecs <= 1024) return go<T, 0, 2>(a, st);
        return go<T, 0, 4>(a, st);
    }
    if (a.rows > 0x7fffffff) return cudaErrorInvalidConfiguration;
    fwd_elements_kernel<T><<<unsigned(a.rows), 256, 0, st>>>(a);
    return cudaGetLastError();
}

static cudaError_t fold(const float *parts, float *dweight, int64_t n, int64_t cols, cudaStream_t st) {
    weight_kernel<<<unsigned((cols + 31) / 32), 1024, 0, st>>>(parts, dweight, int(n), cols);
    return cudaGetLastError();
}

// The blocks of `threads` that run at a time, at most kParts: a kernel of as many
// has no last round that leaves SMs idle, and the fewest partial sums (fp32, two
// vectors a thread, 4096 x 8192: 1216 blocks 118 us, as many as run 101).
template <auto KERNEL>
static cudaError_t at_a_time(unsigned threads, int bytes, int tensors, int *blocks) {
    static KeptByDevice<5 * 17> kept;       // by tensors and warps
    return kept.get(tensors * 17 + int(threads) / 32, blocks, [&](int device, int *most) {
        int sms = 0, each = 0;
        if (cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device)) return e;
        if (cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&each, KERNEL, int(threads), size_t(bytes))) return e;
        *most = std::min(std::max(sms * each, 1), kParts);
        return cudaSuccess;
    });
}

template <typename T, int LANES, int VECS, int ROWS>
static cudaError_t go(const BwdArgs<T> &a, cudaStream_t st) {
    const unsigned threads = LANES ? 256 : threads_for(a.cols / kVec, VECS), per = ROWS * (LANES ? 256 / LANES : 1);
    const int64_t blocks = (a.rows + per - 1) / per;
    int most = 0;
    if (cudaError_t e = at_a_time<bwd_kernel<T, LANES, VECS, ROWS>>(threads, 0, 0, &most)) return e;
    const int64_t grid = blocks < most ? blocks : most;
    bwd_kernel<T, LANES, VECS, ROWS><<<unsigned(grid), threads, 0, st>>>(a);
    if (cudaError_t e = cudaGetLastError()) return e;
    return a.dweight ? fold(a.parts, a.dweight, grid, a.cols, st) : cudaSuccess;
}

template <int VECS>
static cudaError_t go_ring(const BwdArgs<bf> &a, cudaStream_t st) {
    const unsigned threads = threads_for(a.cols / kVec, VECS);
    const int tensors = 2 + (a.residual != nullptr) + (a.ds != nullptr);
    constexpr int each = VECS * 16 * kStages;       // bytes of a thread and tensor
    static_assert(512 * 4 * each <= 232448 - 1024, "shared memory");
    static std::atomic<uint64_t> allowed{0};        // by device: the limit of the widest rows
    int device = 0;
    if (cudaError_t e = cudaGetDevice(&device)) return e;
    if (device >= 64 || !(allowed.load(std::memory_order_acquire) >> device & 1)) {
        if (cudaError_t e = cudaFuncSetAttribute(bwd_ring_kernel<VECS>, cudaFuncAttributeMaxDynamicSharedMemorySize, 512 * 4 * each))
            return e;
        if (device < 64) allowed.fetch_or(uint64_t(1) << device, std::memory_order_release);
    }
    const int bytes = int(threads) * tensors * each;
    int most = 0;
    if (cudaError_t e = at_a_time<bwd_ring_kernel<VECS>>(threads, bytes, tensors, &most)) return e;
    const int64_t grid = a.rows < most ? a.rows : most;
    bwd_ring_kernel<VECS><<<unsigned(grid), threads, bytes, st>>>(a);
    if (cudaError_t e = cudaGetLastError()) return e;
    return a.dweight ? fold(a.parts, a.dweight, grid, a.cols, st) : cudaSuccess;
}

template <typename T>
cudaError_t bwd(const BwdArgs<T> &a, cudaStream_t st) {
    const int64_t vecs = a.cols / kVec;
    if (a.cols % kVec == 0 && vecs <= 1024 && on16(a.dy) && on16(a.s) && on16(a.residual) && on16(a.ds) && on16(a.weight) &&
        on16(a.dx) && on16(a.parts)) {
        // lanes of a warp up to 256 columns (bf16, 100000 x 256: 53 us, as a block a row 98); then one
        // vector a thread (fp32, 16384 x 2560: 102, two 100; 65536 x 512: 99 and 101), two where 512
        // threads would not do otherwise
        if (vecs <= 8) return go<T, 8, 1, 2>(a, st);
        if (vecs <= 16) return go<T, 16, 1, 2>(a, st);
        if (vecs <= 32) return go<T, 32, 1, 2>(a, st);
        if constexpr (sizeof(T) == 2) return vecs <= 512 ? go_ring<1>(a, st) : go_ring<2>(a, st);
        else return vecs <= 512 ? go<T, 0, 1, 1>(a, st) : go<T, 0, 2, 1>(a, st);
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
