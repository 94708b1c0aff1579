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

constexpr int kBlock = SSM_GATED_BLOCK;   // steps between two kept states

// A thread-block cluster's barrier and the address of a variable in another
// of its blocks' shared memory.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void put_remote(const float4 *at, uint32_t rank, float4 v) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z),
                 "f"(v.w)
                 : "memory");
}

// Inputs of one pass: the tensors themselves, or their 8-bit checkpoint.
struct Kept {
    float *states;                  // (Bs, ceil(L / 64), ED)
    int8_t *x_q, *r_q, *i_q;        // (Bs, L, ED)
    float *x_s, *r_s, *i_s;         // (ceil(ED / 64), Bs * L)
};
__device__ __forceinline__ void put_remote_u32(const uint32_t *at, uint32_t rank, uint32_t v) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// c softplus(lam); e^lam overflows above 88, where softplus(lam) = lam.
__device__ __forceinline__ float decay_rate(float lam, float c) {
    return c * (lam > 20.0f ? lam : log1pf(expf(lam)));
}

// sigmoid(lam) / softplus(lam): la's derivative with respect to lam, over la.
// Both tend to e^lam for lam -> -inf, the quotient to 1.
__device__ __forceinline__ float dlog_decay_over(float lam) {
    if (lam < -20.0f) return 1.0f;
    return 1.0f / ((1.0f + expf(-lam)) * (lam > 20.0f ? lam : log1pf(expf(lam))));
}

// ---- packed pairs (two neighbouring channels, one instruction) --------------
__device__ __forceinline__ unsigned long long bits2(float2 v) {
    return *reinterpret_cast<unsigned long long *>(&v);
}
__device__ __forceinline__ float2 from2(unsigned long long v) { return *reinterpret_cast<float2 *>(&v); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return from2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return from2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return from2(r);
}

__device__ __forceinline__ float rcp_fast(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float sqrt_fast(float v) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// 1 / (1 + e^-v).  ACC (fp32 tensors) uses the accurate functions; bf16
// tensors the special-function unit, whose ~2^-22 is far below the 2^-9 of
// their rounding.
template <bool ACC>
__device__ __forceinline__ float2 sigmoid2(float2 v) {
    if (ACC) return make_float2(1.0f / (1.0f + expf(-v.x)), 1.0f / (1.0f + expf(-v.y)));
    const float2 s = mul2(v, both(-SSM_LOG2E));
    const float2 d = add2(make_float2(ex2(s.x), ex2(s.y)), both(1.0f));
    return make_float2(rcp_fast(d.x), rcp_fast(d.y));
}

// Decays from t = -la >= 0: a = e^-t and w = 1 - a, w to full relative
// accuracy, so that 1 - a^2 = w (2 - w) does not cancel for slow decays (a -> 1)
// and a = 1 - w is rounded once.  For t < 0.7, w = t Q(t) with Q a
// fifth-degree fit of (1 - e^-t) / t on [0, 0.7] (Chebyshev nodes; relative
// error 1.2e-8 in exact arithmetic); from 0.7 on 1 - a loses at most one bit.
// WIDE says that t may exceed 0.7: t <= c softplus(lam), so a warp knows from
// its channels alone.
constexpr float kSlow = 0.7f;
template <bool ACC, bool WIDE>
__device__ __forceinline__ void decay2(float2 t, float2 &a, float2 &w) {
    float2 q = fma2(t, both(-0x1.0f0144p-10f), both(0x1.08671cp-7f));
    q = fma2(q, t, both(-0x1.5491aap-5f));
    q = fma2(q, t, both(0x1.554d72p-3f));
    q = fma2(q, t, both(-0x1.ffffc4p-2f));
    q = fma2(q, t, both(1.0f));
    w = mul2(q, t);
    a = fma2(w, both(-1.0f), both(1.0f));
    if (WIDE) {
        float2 e;
        if (ACC) {
            e = make_float2(expf(-t.x), expf(-t.y));
        } else {
            const float2 s = mul2(t, both(-SSM_LOG2E));
            e = make_float2(ex2(s.x), ex2(s.y));
        }
        const float2 we = fma2(e, both(-1.0f), both(1.0f));
        if (t.x >= kSlow) a.x = e.x, w.x = we.x;
        if (t.y >= kSlow) a.y = e.y, w.y = we.y;
    }
}

// 1 - a^2
__device__ __forceinline__ float2 one_minus_square(float2 w) { return mul2(w, fma2(w, both(-1.0f), both(2.0f))); }

template <bool ACC>
__device__ __forceinline__ float2 root2(float2 v) {
    return ACC ? make_float2(sqrtf(v.x), sqrtf(v.y)) : make_float2(sqrt_fast(v.x), sqrt_fast(v.y));
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
    // an infinite top gives NaN: no value of the group can be told
    return top < kTiny ? 0.0f : __fmul_rn(top, 1.0f / 127.0f) + (top - top);
}
__device__ __forceinline__ float inverse_of(float top) {
    return top < kTiny ? 0.0f : __fdiv_rn(127.0f, top);
}
// q in the low byte.  Adding 1.5 2^23 rounds to an integer, ties to even; the
// two operations are the intrinsics that the compiler may not join (packed
// mul and add are joined into a multiply-add, which rounds once too few).
__device__ __forceinline__ uint32_t quantised(float x, float inv) {
    return __float_as_uint(__fadd_rn(__fmul_rn(x, inv), 12582912.0f));
}

// 4-byte copy; `src_bytes` < 4 zero-fills the rest (0 = pure zero fill).
__device__ __forceinline__ void cp_async4(void *smem_dst, const void *gsrc, int src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(smem_u32(smem_dst)), "l"(gsrc),
                 "r"(src_bytes)
                 : "memory");
}

}  // namespace gated
}  // namespace ssm
