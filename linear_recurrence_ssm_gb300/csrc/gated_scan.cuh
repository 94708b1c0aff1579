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
// w is kept above kLeast, far below what it adds to, so that t = 0 needs no
// case of its own where (1 - a^2)^(-1/2) is taken.
constexpr float kSlow = 0.7f, kLeast = 1e-30f;
__device__ __forceinline__ float2 slow_loss(float2 t) {
    float2 q = fma2(t, both(-0x1.0f0144p-10f), both(0x1.08671cp-7f));
    q = fma2(q, t, both(-0x1.5491aap-5f));
    q = fma2(q, t, both(0x1.554d72p-3f));
    q = fma2(q, t, both(-0x1.ffffc4p-2f));
    q = fma2(q, t, both(1.0f));
    return fma2(q, t, both(kLeast));
}
template <bool ACC, bool WIDE>
__device__ __forceinline__ void decay2(float2 t, float2 &a, float2 &w) {
    w = slow_loss(t);
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

// v^(-1/2), for v > 0
template <bool ACC>
__device__ __forceinline__ float2 rsqrt2(float2 v) {
    float2 r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(v.x));
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(v.y));
    if (ACC) {   // one Newton step: r + r (1 - v r^2) / 2
        const float2 d = fma2(mul2(v, r), mul2(r, both(-1.0f)), both(1.0f));
        r = fma2(mul2(r, both(0.5f)), d, r);
    }
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

// ---- a warp's rows of a tile ----------------------------------------------------
// A tile is 64 steps x 64 channels; each of a block's 8 warps owns 8 steps, a
// lane two channels.  A warp copies its own rows ahead of their use, so no
// block barrier stands between a copy and its use.
constexpr int kWarps = 8, kSteps = kBlock / kWarps, kThreads = 32 * kWarps;
constexpr int kMaxCluster = 8;

// W is the widest copy that every row's start allows: 16 bytes, 4 (rows of
// narrow elements then start anywhere in their first word, and need one word
// more), or 1 for plain loads of elements, which wait for their data.
template <typename T, int W>
constexpr bool kShifted = W == 4 && sizeof(T) < 4;
template <typename T, int W>
constexpr int kPitch = 64 * int(sizeof(T)) + (kShifted<T, W> ? 16 : 0);

template <typename T, int W>
__device__ __forceinline__ void copy_rows(uint8_t *to, const T *from, int64_t row0, int n_rows, int e0, int ED) {
    constexpr int kSize = int(sizeof(T));
    const int lane = threadIdx.x % 32;
    if constexpr (W == 16 || (W == 4 && kSize == 4)) {
        constexpr int kChunks = 64 * kSize / W, kPer = W / kSize;
#pragma unroll
        for (int i = 0; i < kSteps * kChunks / 32; ++i) {
            const int row = (i * 32 + lane) / kChunks, e = (i * 32 + lane) % kChunks * kPer;
            const bool in = row < n_rows && e0 + e < ED;
            const T *src = in ? from + (row0 + row) * ED + e0 + e : from;
            uint8_t *dst = to + row * kPitch<T, W> + e * kSize;
            if constexpr (W == 16)
                cp_async16(dst, src, in ? 16 : 0);
            else
                cp_async4(dst, src, in ? 4 : 0);
        }
    } else if constexpr (W == 4) {
        constexpr int kPer = 4 / kSize, kWords = 64 / kPer + 1;
#pragma unroll
        for (int row = 0; row < kSteps; ++row) {
            const int64_t begin = (row0 + row) * ED, end = begin + ED;
            // the word that holds the row's first element; the tensor starts on a word
            const int64_t first = (begin + e0) & ~int64_t(kPer - 1);
#pragma unroll
            for (int k = 0; k < (kWords + 31) / 32; ++k) {
                const int word = lane + 32 * k;
                if (word >= kWords) continue;
                const int64_t e = first + kPer * word;
                const bool in = row < n_rows && e < end;
                // nothing behind the row's end, which may be the tensor's
                const int bytes = in ? int(min(int64_t(kPer), end - e)) * kSize : 0;
                cp_async4(to + row * kPitch<T, W> + 4 * word, in ? from + e : from, bytes);
            }
        }
    } else {
#pragma unroll
        for (int row = 0; row < kSteps; ++row)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int e = lane + 32 * k;
                T v = T(0.0f);
                if (row < n_rows && e0 + e < ED) v = from[(row0 + row) * ED + e0 + e];
                *reinterpret_cast<T *>(to + row * kPitch<T, W> + e * kSize) = v;
            }
    }
}

// Elements between a row's first word and its first element.
template <typename T, int W>
__device__ __forceinline__ uint32_t shift_of(int64_t row, int ED) {
    return kShifted<T, W> ? uint32_t(row) * uint32_t(ED) & (4 / uint32_t(sizeof(T)) - 1) : 0;
}

// The lane's two channels of a copied row (int8: the integers).
template <typename T, int W>
__device__ __forceinline__ float2 pair_at(const uint8_t *row, uint32_t shift) {
    const int lane = threadIdx.x % 32;
    if constexpr (sizeof(T) == 4) {
        return *reinterpret_cast<const float2 *>(row + 8 * lane);
    } else if constexpr (sizeof(T) == 2) {
        uint32_t w = *reinterpret_cast<const uint32_t *>(row + 4 * lane);
        if (W == 4 && shift) w = __funnelshift_r(w, *reinterpret_cast<const uint32_t *>(row + 4 * lane + 4), 16);
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
        uint32_t w;
        if (kShifted<T, W>)
            w = row[2 * lane + shift] | row[2 * lane + shift + 1] << 8;
        else
            w = *reinterpret_cast<const uint16_t *>(row + 2 * lane);
        // 2^23 + (q + 128) as a bit pattern, less 2^23 + 128: exact
        w ^= 0x8080u;
        return add2(make_float2(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440)),
                                __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441))),
                    both(-8388736.0f));
    }
}

__device__ __forceinline__ void put2(float *p, float2 v) { *reinterpret_cast<float2 *>(p) = v; }
__device__ __forceinline__ void put2(__nv_bfloat16 *p, float2 v) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __float22bfloat162_rn(v);
}
// A lane's two channels of one row, as one store where `pairs`.
template <typename T>
__device__ __forceinline__ void put_pair(T *p, float2 v, bool pairs, bool in0, bool in1) {
    if (pairs) {
        if (in0) put2(p, v);
    } else {
        if (in0) put(p, v.x);
        if (in1) put(p + 1, v.y);
    }
}

template <typename T>
inline int widest_copy(uintptr_t at, int64_t ED) {
    return ED * int64_t(sizeof(T)) % 16 == 0 && at % 16 == 0 ? 16 : at % 4 == 0 ? 4 : 1;
}

// Blocks of a cluster take neighbouring tiles of a sequence at once: as many
// as bring the GPU two blocks an SM, none with less than two tiles.
inline int cluster_for(int64_t Bs, int64_t L, int64_t ED, int num_sms) {
    const int64_t chains = (ED + 63) / 64 * Bs, tiles = (L + kBlock - 1) / kBlock;
    int c = 1;
    while (c < kMaxCluster && chains * c * 2 <= 3 * num_sms && c * 2 <= tiles) c *= 2;
    return c;
}

}  // namespace gated
}  // namespace ssm
