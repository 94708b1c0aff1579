// gated_scan.cuh -- the gated linear recurrence's arithmetic, shared by its
// forward, backward and single-token kernels.
//
//   s_r = 1 / (1 + e^-gate_r),  s_i = 1 / (1 + e^-gate_i)
//   la  = -c softplus(lam) s_r,  a = e^la,  m = sqrt(1 - e^(2 la))
//   h   = a h + m s_i x
// A reset step has a = 0 and m = 1.
#pragma once

#include "ssm_common.cuh"

namespace ssm {
namespace gated {

constexpr int kBlock = 64;   // steps between two kept states

// Inputs of one pass: the tensors themselves, or their 8-bit checkpoint.
struct Kept {
    float *states;                  // (Bs, ceil(L / 64), ED)
    int8_t *x_q, *r_q, *i_q;        // (Bs, L, ED)
    float *x_s, *r_s, *i_s;         // (ceil(ED / 64), Bs * L)
};

// -c softplus(lam); e^lam overflows above 88, where softplus(lam) = lam.
__device__ __forceinline__ float log_decay(float lam, float c) {
    return -c * (lam > 20.0f ? lam : log1pf(expf(lam)));
}

// sigmoid(lam) / softplus(lam): la's derivative with respect to lam, over la.
// Both tend to e^lam for lam -> -inf, the quotient to 1.
__device__ __forceinline__ float dlog_decay_over(float lam) {
    if (lam < -20.0f) return 1.0f;
    return 1.0f / ((1.0f + expf(-lam)) * (lam > 20.0f ? lam : log1pf(expf(lam))));
}

// 1 / (1 + e^-v).  ACC (fp32 tensors) uses the accurate functions; bf16
// tensors the special-function unit, whose ~2^-22 is far below the 2^-9 of
// their rounding.
template <bool ACC>
__device__ __forceinline__ float sigmoid(float v) {
    if (ACC) return 1.0f / (1.0f + expf(-v));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + ex2(-SSM_LOG2E * v)));
    return r;
}

template <bool ACC>
__device__ __forceinline__ float decay(float la) {
    return ACC ? expf(la) : ex2(SSM_LOG2E * la);
}

// 1 - e^u, u = 2 la <= 0, without the cancellation of 1 - a^2 for slow decays
// (a -> 1): for u > -0.7, -u times a fifth-degree fit of (e^u - 1) / u on
// [-0.7, 0] (Chebyshev nodes, relative error 1.2e-8 in exact arithmetic);
// below that 1 - a^2 loses less than two bits.
__device__ __forceinline__ float one_minus_exp(float u, float a) {
    float p = 0x1.0f0144p-10f;
    p = fmaf(p, u, 0x1.08671cp-7f);
    p = fmaf(p, u, 0x1.5491aap-5f);
    p = fmaf(p, u, 0x1.554d72p-3f);
    p = fmaf(p, u, 0x1.ffffc4p-2f);
    p = fmaf(p, u, 1.0f);
    return u > -0.7f ? -u * p : fmaf(-a, a, 1.0f);
}

template <bool ACC>
__device__ __forceinline__ float root(float v) {
    if (ACC) return sqrtf(v);
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// ---- 8-bit checkpoints ------------------------------------------------------
// A group of 64 columns of one row shares a scale: top = max |x|,
// scale = top * fl(1 / 127), q = rint(x * fl(127 / top)).  The products are
// rounded on their own (no fused multiply-add), so q does not depend on the
// code around it.  A group below 2^-100 is stored as zeros: 127 / top would
// overflow soon after.
constexpr int kGroup = 64;
constexpr float kTiny = 0x1p-100f;

__device__ __forceinline__ float scale_of(float top) {
    return top < kTiny ? 0.0f : __fmul_rn(top, 1.0f / 127.0f);
}
__device__ __forceinline__ float inverse_of(float top) {
    return top < kTiny ? 0.0f : __fdiv_rn(127.0f, top);
}
__device__ __forceinline__ int quantised(float x, float inv) {
    return min(127, max(-127, __float2int_rn(__fmul_rn(x, inv))));
}

}  // namespace gated
}  // namespace ssm
