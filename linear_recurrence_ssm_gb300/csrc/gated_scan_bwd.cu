// gated_scan_bwd.cu -- gradients of the gated linear recurrence.
//
// With g_t = dL/dh_t:  g_t = dy_t + u_{t+1},  u_t = a_t g_t,  u_L = dh_final
//   dx = g m s_i            dgate_i = g m x s_i (1 - s_i)
//   G  = la g (a h_{t-1} - (a^2 / m) s_i x)     (0 at a reset)
//   dgate_r = G (1 - s_r)   dlam = sum of G, times sigmoid(lam) / softplus(lam)
// h inside a block of 64 steps is recomputed from the state kept at its start.
#include "gated_scan.cuh"

namespace ssm {
namespace gated_bwd {
using namespace gated;

template <typename T>
__global__ void __launch_bounds__(64)
gated_bwd_kernel(const T *__restrict__ x, const T *__restrict__ gr, const T *__restrict__ gi,
                 const float *__restrict__ lam, float c, const uint8_t *__restrict__ reset,
                 const T *__restrict__ dy, const float *__restrict__ dh_final, Kept kept,
                 T *__restrict__ dx, T *__restrict__ dr, T *__restrict__ di,
                 float *__restrict__ part, float *__restrict__ dh0, int64_t L, int64_t ED,
                 int64_t rows) {
    constexpr bool ACC = sizeof(T) == 4;
    const int64_t e = int64_t(blockIdx.x) * kGroup + threadIdx.x, b = blockIdx.y;
    if (e >= ED) return;
    const float k = decay_rate(lam[e], c);
    const int64_t blocks = (L + kBlock - 1) / kBlock;
    float u = dh_final ? dh_final[b * ED + e] : 0.0f, sum = 0.0f;
    float before[kBlock];
    for (int64_t blk = blocks - 1; blk >= 0; --blk) {
        float h = kept.states[(b * blocks + blk) * ED + e];
        const int64_t t0 = blk * kBlock;
        const int n = int(min(int64_t(kBlock), L - t0));
        auto get = [&](const T *p, const int8_t *q, const float *s, int64_t row) {
            return q ? float(q[row * ED + e]) * s[blockIdx.x * rows + row] : to_f32(p[row * ED + e]);
        };
        for (int j = 0; j < n; ++j) {
            const int64_t row = b * L + t0 + j;
            before[j] = h;
            const float xv = get(x, kept.x_q, kept.x_s, row), si = sigmoid2<ACC>(both(get(gi, kept.i_q, kept.i_s, row))).x;
            float2 a2, w2;
            decay2<ACC, true>(both(k * sigmoid2<ACC>(both(get(gr, kept.r_q, kept.r_s, row))).x), a2, w2);
            const float a = a2.x, m = root2<ACC>(one_minus_square(w2)).x;
            h = reset && reset[row] ? si * xv : fmaf(a, h, m * si * xv);
        }
        for (int j = n - 1; j >= 0; --j) {
            const int64_t row = b * L + t0 + j, at = row * ED + e;
            const float xv = get(x, kept.x_q, kept.x_s, row), si = sigmoid2<ACC>(both(get(gi, kept.i_q, kept.i_s, row))).x;
            const float sr = sigmoid2<ACC>(both(get(gr, kept.r_q, kept.r_s, row))).x, la = -k * sr;
            float2 a2, w2;
            decay2<ACC, true>(both(k * sr), a2, w2);
            const float a = a2.x;
            const bool cut = reset && reset[row];
            const float m = cut ? 1.0f : root2<ACC>(one_minus_square(w2)).x;
            const float g = to_f32(dy[at]) + u;
            // m -> 0 only together with la, and la / m -> 0
            const float G = cut ? 0.0f : la * g * (a * before[j] - a * a / fmaxf(m, 1e-30f) * si * xv);
            const float gm = g * m * si;
            put(dx + at, gm);
            put(di + at, gm * xv * (1.0f - si));
            put(dr + at, G * (1.0f - sr));
            sum += G;
            u = cut ? 0.0f : a * g;
        }
    }
    if (dh0) dh0[b * ED + e] = u;
    part[b * ED + e] = sum;
}

// dlam from the sequences' sums, in their order.
__global__ void __launch_bounds__(256)
dlam_kernel(const float *__restrict__ part, const float *__restrict__ lam, float *__restrict__ dlam,
            int64_t n, int64_t ED) {
    const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (e >= ED) return;
    float s = 0.0f;
    for (int64_t b = 0; b < n; ++b) s += part[b * ED + e];
    dlam[e] = s * dlog_decay_over(lam[e]);
}

template <typename T>
cudaError_t launch(const T *x, const T *gr, const T *gi, const float *lam, float c,
                   const uint8_t *reset, const T *dy, const float *dh_final, const Kept &kept, T *dx,
                   T *dr, T *di, float *dlam, float *dh0, int64_t Bs, int64_t L, int64_t ED,
                   int num_sms, cudaStream_t st) {
    float *part = nullptr;
    cudaError_t err = cudaMallocAsync(&part, size_t(Bs * ED) * sizeof(float), st);
    if (err != cudaSuccess) return err;
    const dim3 grid(unsigned((ED + kGroup - 1) / kGroup), unsigned(Bs));
    gated_bwd_kernel<T><<<grid, kGroup, 0, st>>>(x, gr, gi, lam, c, reset, dy, dh_final, kept, dx, dr, di,
                                                 part, dh0, L, ED, Bs * L);
    err = cudaGetLastError();
    if (err == cudaSuccess) {
        dlam_kernel<<<unsigned((ED + 255) / 256), 256, 0, st>>>(part, lam, dlam, Bs, ED);
        err = cudaGetLastError();
    }
    const cudaError_t e2 = cudaFreeAsync(part, st);
    return err != cudaSuccess ? err : e2;
}

#define SSM_GATED_BWD_INSTANTIATE(T)                                                              \
    template cudaError_t launch<T>(const T *, const T *, const T *, const float *, float,         \
                                   const uint8_t *, const T *, const float *, const Kept &, T *,  \
                                   T *, T *, float *, float *, int64_t, int64_t, int64_t, int,    \
                                   cudaStream_t);
SSM_GATED_BWD_INSTANTIATE(float)
SSM_GATED_BWD_INSTANTIATE(__nv_bfloat16)

}  // namespace gated_bwd
}  // namespace ssm
