// gated_scan.cu -- the gated linear recurrence, forward and one token.
#include "gated_scan.cuh"

namespace ssm {
namespace gated {

// One thread for each channel of each sequence, step after step.
template <typename T>
__global__ void __launch_bounds__(64)
gated_fwd_kernel(const T *__restrict__ x, const T *__restrict__ gr, const T *__restrict__ gi,
                 const float *__restrict__ lam, float c, const uint8_t *__restrict__ reset,
                 const float *__restrict__ h0, T *__restrict__ y, float *__restrict__ h_final,
                 Kept kept, int64_t L, int64_t ED, int64_t rows) {
    constexpr bool ACC = sizeof(T) == 4;
    __shared__ float tops[3][2];
    const int64_t e = int64_t(blockIdx.x) * kGroup + threadIdx.x;
    const int64_t b = blockIdx.y;
    const bool in = e < ED;
    const float k = in ? log_decay(lam[e], c) : 0.0f;
    float h = h0 && in ? h0[b * ED + e] : 0.0f;
    const int64_t blocks = (L + kBlock - 1) / kBlock;
    for (int64_t t = 0; t < L; ++t) {
        const int64_t row = b * L + t, at = row * ED + e;
        const float v[3] = {in ? to_f32(x[at]) : 0.0f, in ? to_f32(gr[at]) : 0.0f,
                            in ? to_f32(gi[at]) : 0.0f};
        if (kept.states && in && t % kBlock == 0) kept.states[(b * blocks + t / kBlock) * ED + e] = h;
        if (kept.x_q) {
            int8_t *q[3] = {kept.x_q, kept.r_q, kept.i_q};
            float *s[3] = {kept.x_s, kept.r_s, kept.i_s};
            __syncthreads();
            for (int j = 0; j < 3; ++j) {
                // order of the bit patterns of |v| = order of the values, NaN on top
                const unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(v[j])));
                if (threadIdx.x % 32 == 0) tops[j][threadIdx.x / 32] = __uint_as_float(top);
            }
            __syncthreads();
            for (int j = 0; j < 3; ++j) {
                const float top = __uint_as_float(max(__float_as_uint(tops[j][0]), __float_as_uint(tops[j][1])));
                if (in) q[j][at] = int8_t(quantised(v[j], inverse_of(top)));
                if (threadIdx.x == 0) s[j][blockIdx.x * rows + row] = scale_of(top);
            }
        }
        if (in) {
            const float la = k * sigmoid<ACC>(v[1]), a = decay<ACC>(la);
            if (reset && reset[row]) {
                h = sigmoid<ACC>(v[2]) * v[0];
            } else {
                const float m = root<ACC>(one_minus_exp(2.0f * la, a));
                h = fmaf(a, h, m * sigmoid<ACC>(v[2]) * v[0]);
            }
            put(y + at, h);
        }
    }
    if (h_final && in) h_final[b * ED + e] = h;
}

template <typename T>
__global__ void __launch_bounds__(256)
gated_step_kernel(const T *__restrict__ x, const T *__restrict__ gr, const T *__restrict__ gi,
                  const float *__restrict__ lam, float c, float *__restrict__ states,
                  const int32_t *__restrict__ pages, T *__restrict__ y, int64_t ED, int64_t num_pages) {
    constexpr bool ACC = sizeof(T) == 4;
    const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x, b = blockIdx.y;
    if (e >= ED) return;
    const int64_t page = pages ? pages[b] : b, at = b * ED + e;
    if (page < 0 || page >= num_pages) {
        put(y + at, 0.0f);
        return;
    }
    const float la = log_decay(lam[e], c) * sigmoid<ACC>(to_f32(gr[at])), a = decay<ACC>(la);
    const float m = root<ACC>(one_minus_exp(2.0f * la, a));
    const float h = fmaf(a, states[page * ED + e], m * sigmoid<ACC>(to_f32(gi[at])) * to_f32(x[at]));
    states[page * ED + e] = h;
    put(y + at, h);
}

template <typename T>
cudaError_t launch_fwd(const T *x, const T *gr, const T *gi, const float *lam, float c,
                       const uint8_t *reset, const float *h0, T *y, float *h_final,
                       const Kept &kept, int64_t Bs, int64_t L, int64_t ED, int num_sms,
                       cudaStream_t st) {
    const dim3 grid(unsigned((ED + kGroup - 1) / kGroup), unsigned(Bs));
    gated_fwd_kernel<T><<<grid, kGroup, 0, st>>>(x, gr, gi, lam, c, reset, h0, y, h_final, kept, L, ED,
                                                 Bs * L);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_step(const T *x, const T *gr, const T *gi, const float *lam, float c,
                        float *states, const int32_t *pages, T *y, int64_t Bs, int64_t ED,
                        int64_t num_pages, cudaStream_t st) {
    const dim3 grid(unsigned((ED + 255) / 256), unsigned(Bs));
    gated_step_kernel<T><<<grid, 256, 0, st>>>(x, gr, gi, lam, c, states, pages, y, ED, num_pages);
    return cudaGetLastError();
}

#define SSM_GATED_INSTANTIATE(T)                                                                  \
    template cudaError_t launch_fwd<T>(const T *, const T *, const T *, const float *, float,     \
                                       const uint8_t *, const float *, T *, float *, const Kept &, \
                                       int64_t, int64_t, int64_t, int, cudaStream_t);             \
    template cudaError_t launch_step<T>(const T *, const T *, const T *, const float *, float,    \
                                        float *, const int32_t *, T *, int64_t, int64_t, int64_t, \
                                        cudaStream_t);
SSM_GATED_INSTANTIATE(float)
SSM_GATED_INSTANTIATE(__nv_bfloat16)

}  // namespace gated
}  // namespace ssm
