// ckpt8.cu -- 8-bit activation checkpoints: a row's groups of 64 columns, each
// with a scale of its own (gated_scan.cuh has the rounding rule).
#include "gated_scan.cuh"

namespace ssm {
namespace ckpt8 {
using namespace gated;

template <typename T>
__global__ void __launch_bounds__(32)
save_kernel(const T *__restrict__ x, int8_t *__restrict__ q, float *__restrict__ scale, int64_t rows,
            int64_t cols) {
    const int64_t row = blockIdx.x, e = int64_t(blockIdx.y) * kGroup + threadIdx.x;
    float v[2];
    unsigned top = 0;
    for (int j = 0; j < 2; ++j) {
        v[j] = e + 32 * j < cols ? to_f32(x[row * cols + e + 32 * j]) : 0.0f;
        top = max(top, __float_as_uint(fabsf(v[j])));
    }
    const float t = __uint_as_float(__reduce_max_sync(0xffffffffu, top)), inv = inverse_of(t);
    for (int j = 0; j < 2; ++j)
        if (e + 32 * j < cols) q[row * cols + e + 32 * j] = int8_t(quantised(v[j], inv));
    if (threadIdx.x == 0) scale[blockIdx.y * rows + row] = scale_of(t);
}

template <typename T>
__global__ void __launch_bounds__(256)
load_kernel(const int8_t *__restrict__ q, const float *__restrict__ scale, T *__restrict__ x, int64_t rows,
            int64_t cols) {
    const int64_t e = int64_t(blockIdx.y) * 256 + threadIdx.x, row = blockIdx.x;
    if (e < cols) put(x + row * cols + e, float(q[row * cols + e]) * scale[e / kGroup * rows + row]);
}

template <typename T>
cudaError_t save(const T *x, int8_t *q, float *scale, int64_t rows, int64_t cols, cudaStream_t st) {
    save_kernel<T><<<dim3(unsigned(rows), unsigned((cols + kGroup - 1) / kGroup)), 32, 0, st>>>(
        x, q, scale, rows, cols);
    return cudaGetLastError();
}

template <typename T>
cudaError_t load(const int8_t *q, const float *scale, T *x, int64_t rows, int64_t cols, cudaStream_t st) {
    load_kernel<T><<<dim3(unsigned(rows), unsigned((cols + 255) / 256)), 256, 0, st>>>(q, scale, x, rows, cols);
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
