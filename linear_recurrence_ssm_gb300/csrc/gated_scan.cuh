// gated_scan.cuh -- the gated linear recurrence's arithmetic, shared by its
// forward, backward and single-token kernels.
//
//   s_r = 1 / (1 + e^-gate_r),  s_i = 1 / (1 + e^-gate_i)
//   la  = -c softplus(lam) s_r,  a = e^la,  m = sqrt(1 - e^(2 la))
//   h   = a h + m s_i x
// A reset step has a = 0 and m = 1.
#pragma once

#include "ssm_common.cuh"
#include "tc_ptx.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <limits.h>
#include <type_traits>

namespace ssm {
namespace gated {

constexpr int kBlock = SSM_GATED_BLOCK;   // steps between two kept states

// Inputs of one pass: the tensors themselves, or their 8-bit checkpoint.
struct Kept {
    float *states;                  // (Bs, ceil(L / 64), ED)
    int8_t *x_q, *r_q, *i_q;        // (Bs, L, ED)
    float *x_s, *r_s, *i_s;         // (ceil(ED / 64), Bs * L)
};

// ---- exchange between the blocks of a cluster --------------------------------
// Each block sends its tile's piece to every other block of the cluster, as
// asynchronous stores that count towards the receiver's mbarrier: no block
// waits for its own stores to arrive anywhere, as a cluster barrier would have
// it do (its release took 1.2 of 7 cycles an instruction).  Two buffers are
// enough: a block sends for turn s + 2 only after it has received every piece
// of turn s + 1, and each of those was sent after its sender had read turn s.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

constexpr int kMaxCluster = 16, kRest = 4;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr int exchange_bytes(int cluster) { return 2 * (cluster - 1) * 32 * 16; }

__device__ __forceinline__ bool aborted(const int *abort) { return *reinterpret_cast<const volatile int *>(abort); }
// What a block does before it leaves after a wait that ran out: copies and
// pieces on their way into its shared memory get the same time again.
__device__ __forceinline__ void linger(uint64_t limit_ns = kWaitLimitNs) {
    const uint64_t t0 = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t0 < limit_ns) __nanosleep(1000);
}
struct alignas(16) Exchange {
    uint64_t full[2];
    int abort;      // a wait ran out: this block waits no more, its results are unspecified

    // What block `from` of the others sent to block `at`; C - 1 slots a buffer follow this structure.
    __device__ __forceinline__ float4 *piece(int buf, int C, int at, int from) {
        return reinterpret_cast<float4 *>(this + 1) + (buf * (C - 1) + from - (from > at)) * 32;
    }
    // One thread; a cluster barrier follows.
    __device__ __forceinline__ void init() {
        tc::mbar_init(&full[0], 1);
        tc::mbar_init(&full[1], 1);
        tc::mbar_fence_init();
    }
    // One warp: block `rank`'s piece to block k.
    __device__ __forceinline__ void send(int buf, int C, int rank, int k, float4 v) {
        if (aborted(&abort)) return;
        uint32_t to, bar;
        asm("mapa.shared::cluster.u32 %0, %1, %2;"
            : "=r"(to)
            : "r"(smem_u32(piece(buf, C, k, rank) + threadIdx.x % 32)), "r"(k));
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(smem_u32(&full[buf])), "r"(k));
        asm volatile(
            "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
            "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
            : "memory");
    }
    // One thread, once a turn: C - 1 pieces will come.
    __device__ __forceinline__ void expect(int buf, int C) {
        if (aborted(&abort)) return;      // the phase before may never complete
        tc::mbar_arrive_expect_tx(&full[buf], uint32_t(C - 1) * 32 * 16);
    }
    __device__ __forceinline__ bool arrived(int buf, uint32_t parity) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n"
            " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(smem_u32(&full[buf])), "r"(parity)
            : "memory");
        return ok != 0;
    }
    // Every thread; gives up after limit_ns and then reports in *error.
    __device__ __forceinline__ void wait(int buf, uint32_t parity, unsigned int *error,
                                         uint64_t limit_ns = kWaitLimitNs) {
        if (arrived(buf, parity)) return;
        const uint64_t t0 = tc::globaltimer_ns();
        while (!arrived(buf, parity)) {
            if (*reinterpret_cast<volatile int *>(&abort)) return;
            if (tc::globaltimer_ns() - t0 > limit_ns) {
                *reinterpret_cast<volatile int *>(&abort) = 1;
                atomicOr(error, 1u);
                return;
            }
        }
    }
};

// Waits for a warp's own copies; the same limit.
__device__ __forceinline__ void wait_or_abort(uint64_t *bar, uint32_t parity, int *abort, unsigned int *error,
                                              uint64_t limit_ns = kWaitLimitNs) {
    if (tc::mbar_wait_bounded(bar, parity, abort, limit_ns)) return;
    *reinterpret_cast<volatile int *>(abort) = 1;
    atomicOr(error, 1u);
}

// Self-test of the above, one warp in each of two blocks of a cluster: the
// first block waits for a piece that the other one never sends (for_copy: for
// a copy that was never asked for), gives up, and then does what a kernel does
// in its remaining turns -- which has to wait no more and send nothing.
__device__ __forceinline__ void run_out(bool for_copy, unsigned int *error) {
    constexpr uint64_t kLimitNs = 20000000ull;
    constexpr int kTurns = 100;
    __shared__ struct {
        Exchange ex;
        float4 pieces[exchange_bytes(2) / int(sizeof(float4))];
        uint64_t copied;
    } sh;
    const int rank = int(cluster_rank());
    if (threadIdx.x == 0) {
        sh.ex.init();
        sh.ex.abort = 0;
        tc::mbar_init(&sh.copied, 1);
        tc::mbar_fence_init();
    }
    __syncwarp();
    cluster_sync();
    if (rank == 0) {
        if (for_copy) wait_or_abort(&sh.copied, 0, &sh.ex.abort, error, kLimitNs);
        __syncwarp();
        for (int turn = 0; turn < kTurns; ++turn) {
            const int buf = turn & 1;
            if (threadIdx.x == 0) sh.ex.expect(buf, 2);
            if (turn > 0) sh.ex.send(buf, 2, 0, 1, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
            __syncwarp();
            sh.ex.wait(buf, turn >> 1 & 1, error, kLimitNs);
            wait_or_abort(&sh.copied, 0, &sh.ex.abort, error, kLimitNs);
        }
        if (aborted(&sh.ex.abort)) linger(kLimitNs);
    }
    __syncwarp();
    cluster_sync();
}

// A piece's A carries in its first channel's sign whether a step of it dropped
// the state before, of both channels: the carried state may be an infinity or
// NaN, which 0 times it would keep.  A is then -0, or a NaN with the sign where
// a gate behind the drop was NaN; arithmetic makes no NaN with a sign.
__device__ __forceinline__ bool drops(float A) { return __float_as_int(A) < 0; }

// c softplus(lam); e^lam overflows above 88, where softplus(lam) = lam.  Rates
// above 2^127 are taken as that: an infinite one would make NaN of a gate that
// is shut (times 0) and of a decay of 0 (its logarithm times it).  NaN stays.
__device__ __forceinline__ float decay_rate(float lam, float c) {
    const float rate = c * (lam > 20.0f ? lam : log1pf(expf(lam)));
    return rate > 0x1p127f ? 0x1p127f : rate;
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
// e^v for v <= 88.  bf16 tensors take the special-function unit's exponential
// of v log2(e) as it is: ~2^-22, far below the 2^-9 of their rounding.  ACC
// (fp32 tensors) adds what that product's rounding and log2(e)'s own lose,
// carried to first order.
template <bool ACC>
__device__ __forceinline__ float2 exp_pair(float2 v) {
    const float2 s = mul2(v, both(SSM_LOG2E));
    const float2 e = make_float2(ex2(s.x), ex2(s.y));
    if (!ACC) return e;
    // log2(e) = 0x1.715476p+0 + 0x1.4ae0cp-26 (the next bits)
    const float2 lost = fma2(v, both(0x1.4ae0cp-26f), fma2(v, both(SSM_LOG2E), mul2(s, both(-1.0f))));
    return fma2(mul2(e, lost), both(0x1.62e43p-1f), e);      // ln 2
}
// -1 / (1 + e^-v): the sign costs nothing here and saves one where 1 - s or
// -la is wanted.
template <bool ACC>
__device__ __forceinline__ float2 nsigmoid2(float2 v) {
    if (!ACC) {
        const float2 s = mul2(v, both(-SSM_LOG2E));
        const float2 d = fma2(make_float2(ex2(s.x), ex2(s.y)), both(-1.0f), both(-1.0f));
        return make_float2(rcp_fast(d.x), rcp_fast(d.y));
    }
    // e^88 keeps d finite, and its reciprocal is below the smallest normal
    // number; e^-88 is nothing beside 1
    float x, y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(v.x), "f"(-88.0f));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(v.y), "f"(-88.0f));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(x), "f"(88.0f));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(y), "f"(88.0f));
    const float2 d = fma2(exp_pair<true>(make_float2(-x, -y)), both(-1.0f), both(-1.0f));
    const float2 r = make_float2(rcp_fast(d.x), rcp_fast(d.y));
    return fma2(fma2(mul2(d, both(-1.0f)), r, both(1.0f)), r, r);      // one Newton step
}

// Decays from la <= 0: a = e^la and em = a - 1, em to full relative accuracy,
// so that a^2 - 1 = em (1 + a) does not cancel for slow decays (a -> 1) and
// a = 1 + em is rounded once.  For la > -0.4, em = la Q(la) with Q a
// fourth-degree fit of (e^la - 1) / la on [-0.4, 0] (Chebyshev nodes; relative
// error 5.2e-8 in exact arithmetic); from there on a - 1 loses at most two
// bits.  WIDE says that la may be below -0.4: |la| <= c softplus(lam), so a
// warp knows from its channels alone.
// em is kept below -kLeast, so that la = 0 needs no case of its own where
// (1 - a^2)^(-1/2) is taken (flushed if 1 - a^2 were subnormal): far below what
// it adds to for every -la above 2^-100, whose m is 2^-50.
constexpr float kSlow = 0.4f, kLeast = 0x1p-125f;
__device__ __forceinline__ float2 slow_em1(float2 la) {
    float2 q = fma2(la, both(0x1.cf2208p-8f), both(0x1.51d0aap-5f));
    q = fma2(q, la, both(0x1.5535acp-3f));
    q = fma2(q, la, both(0x1.ffff38p-2f));
    q = fma2(q, la, both(1.0f));
    return fma2(q, la, both(-kLeast));
}
template <bool ACC, bool WIDE>
__device__ __forceinline__ void decay2(float2 la, float2 &a, float2 &em) {
    em = slow_em1(la);
    a = add2(em, both(1.0f));
    if (WIDE) {
        float2 v = la;
        if (ACC) {      // e^-1000 = 0 in fp32; what log2(e) v loses has to stay finite
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(v.x) : "f"(la.x), "f"(-1000.0f));
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(v.y) : "f"(la.y), "f"(-1000.0f));
        }
        const float2 e = exp_pair<ACC>(v);
        const float2 em_e = add2(e, both(-1.0f));
        if (la.x <= -kSlow) a.x = e.x, em.x = em_e.x;
        if (la.y <= -kSlow) a.y = e.y, em.y = em_e.y;
    }
}

// a^2 - 1 = em (1 + a)
__device__ __forceinline__ float2 square_less_one(float2 a, float2 em) { return fma2(em, a, em); }

// (1 - e^(2 la))^(1/2) / (-la)^(1/2) on [-0.4, 0]: a fourth-degree fit as
// above, relative error 6.9e-8.
__device__ __forceinline__ float2 slow_root(float2 la) {
    float2 q = fma2(la, both(0x1.0ca10cp-6f), both(0x1.65e174p-4f));
    q = fma2(q, la, both(0x1.2d8d8ap-2f));
    q = fma2(q, la, both(0x1.6a08fap-1f));
    return fma2(q, la, both(0x1.6a09e6p+0f));
}

__device__ __forceinline__ float rsqrt_fast(float v) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
template <bool ACC>
__device__ __forceinline__ float2 reciprocal_of_minus(float2 v) {
    float2 r = make_float2(rcp_fast(-v.x), rcp_fast(-v.y));
    if (ACC) r = fma2(fma2(v, r, both(1.0f)), r, r);     // one Newton step
    return r;
}
// (-v)^(-1/2), for v < 0
template <bool ACC>
__device__ __forceinline__ float2 rsqrt_of_minus(float2 v) {
    float2 r = make_float2(rsqrt_fast(-v.x), rsqrt_fast(-v.y));
    if (ACC) {   // one Newton step: r + r (1 + v r^2) / 2
        const float2 d = fma2(mul2(v, r), r, both(1.0f));
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

// ---- pieces of the time axis: h -> A h + H (A of two channels, H of two) -----
template <bool RESET>
__device__ __forceinline__ float2 after(float4 piece, float2 h) {
    const float2 on = fma2(make_float2(piece.x, piece.y), h, make_float2(piece.z, piece.w));
    return RESET && drops(piece.x) ? make_float2(piece.z, piece.w) : on;
}
// One piece, then another.
template <bool RESET>
__device__ __forceinline__ float4 joined(float4 first, float4 second) {
    float2 A = mul2(make_float2(first.x, first.y), make_float2(second.x, second.y));
    const float2 H = after<RESET>(second, make_float2(first.z, first.w));
    // -0 times -0 or NaN would lose the sign
    if (RESET) A.x = __int_as_float(__float_as_int(A.x) | (__float_as_int(first.x) & INT_MIN));
    return RESET && drops(second.x) ? second : make_float4(A.x, A.y, H.x, H.y);
}

// ---- a warp's rows of a tile ----------------------------------------------------
// A tile is 64 steps x 64 channels; each of a block's warps owns STEPS of the
// steps, a lane two channels.  A warp copies its own rows ahead of their use,
// so no block barrier stands between a copy and its use.

// W says how: 16, tensor copies (rows are multiples of 16 bytes); 8, copies of
// 16 bytes from the granule that holds a row's first element, one more than
// the 64 channels fill; 1, plain loads of elements, which wait for their data
// (tensors that do not start on 16 bytes).
template <typename T, int W>
constexpr int kPitch = 64 * int(sizeof(T)) + (W == 8 ? 16 : 0);

template <typename T, int W, int STEPS>
__device__ __forceinline__ void copy_rows(uint8_t *to, const T *from, int64_t row0, int n_rows, int e0, int ED) {
    constexpr int kSize = int(sizeof(T));
    const int lane = threadIdx.x % 32;
    if constexpr (W == 8) {
        constexpr int kChunks = 64 * kSize / 16, kRows = 32 / kChunks;      // of one instruction
        // offsets from the granule of the first row's first element fit 32 bits (ED < 2^26)
        const int64_t begin = (row0 * ED + e0) * kSize;
        const uint8_t *base = reinterpret_cast<const uint8_t *>(from) + (begin & ~int64_t(15));
        const uint32_t lead = uint32_t(begin) & 15, pitch = uint32_t(ED) * kSize;
        const int width = min(64, ED - e0) * kSize;
        // The lane's granule `chunk` of a row; nothing behind the row's end, which may be the tensor's.
        auto copy = [&](int row, int chunk) {
            const uint32_t at = lead + uint32_t(row) * pitch, first = at & ~15u;
            const int bytes = min(16, int(at - first) + width - 16 * chunk);
            if (row < n_rows && bytes > 0) cp_async16(to + row * kPitch<T, W> + 16 * chunk, base + (first + 16 * chunk), bytes);
        };
#pragma unroll
        for (int i = 0; i < STEPS; i += kRows) copy(i + lane / kChunks, lane % kChunks);
        if (lane < STEPS) copy(lane, kChunks);
    } else {
#pragma unroll
        for (int row = 0; row < STEPS; ++row)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int e = lane + 32 * k;
                if (row < n_rows && e0 + e < ED)
                    *reinterpret_cast<T *>(to + row * kPitch<T, W> + e * kSize) = from[(row0 + row) * ED + e0 + e];
            }
    }
}

// Zeros in a warp's whole ring, before its first copy: columns behind the
// row's end are never copied to.
__device__ __forceinline__ void clear_ring(uint8_t *ring, int bytes) {
    for (int i = threadIdx.x % 32 * 16; i < bytes; i += 32 * 16)
        *reinterpret_cast<uint4 *>(ring + i) = make_uint4(0, 0, 0, 0);
    __syncwarp();
}

// Bytes between a copied row's first granule and its first element.
template <typename T, int W>
__device__ __forceinline__ uint32_t shift_of(int64_t row, int ED) {
    return W == 8 ? uint32_t(row) * uint32_t(ED) * uint32_t(sizeof(T)) & 15 : 0;
}

// A lane's two channels: neighbours where rows are stored as boxes (and read
// in pairs), else lane and lane + 32, so that every load and store of single
// elements is of neighbours.
template <int W>
constexpr int kNext = W == 16 ? 1 : 32;
template <int W>
__device__ __forceinline__ int first_channel() {
    const int lane = threadIdx.x % 32;
    return W == 16 ? 2 * lane : lane;
}

// The lane's two channels of a copied row (int8: the integers).
template <typename T, int W>
__device__ __forceinline__ float2 pair_at(const uint8_t *row, uint32_t shift) {
    // in bytes and in 32 bits: as T * plus an unsigned index the bf16 gradients took 2 % more
    const T *p = reinterpret_cast<const T *>(row + shift + int(sizeof(T)) * first_channel<W>());
    if constexpr (sizeof(T) == 4) {
        return W == 16 ? *reinterpret_cast<const float2 *>(p) : make_float2(p[0], p[32]);
    } else if constexpr (sizeof(T) == 2) {
        if (W != 16) return make_float2(to_f32(p[0]), to_f32(p[32]));
        const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
        // 2^23 + (q + 128) as a bit pattern, less 2^23 + 128: exact
        const uint8_t *b = reinterpret_cast<const uint8_t *>(p);
        const uint32_t w = (W == 16 ? *reinterpret_cast<const uint16_t *>(b) : uint32_t(b[0]) | uint32_t(b[32]) << 8) ^ 0x8080u;
        return add2(make_float2(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440)),
                                __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441))),
                    both(-8388736.0f));
    }
}

__device__ __forceinline__ void put2(float *p, float2 v) { *reinterpret_cast<float2 *>(p) = v; }
__device__ __forceinline__ void put2(__nv_bfloat16 *p, float2 v) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __float22bfloat162_rn(v);
}
// A lane's two channels of one row, element by element.
template <int W, typename T>
__device__ __forceinline__ void put_pair(T *p, float2 v, bool in0, bool in1) {
    if (in0) put(p, v.x);
    if (in1) put(p + kNext<W>, v.y);
}
// The two channels of a vector over the channels.
template <int W>
__device__ __forceinline__ float2 get_pair(const float *p, bool in0, bool in1) {
    return make_float2(in0 ? p[0] : 0.0f, in1 ? p[kNext<W>] : 0.0f);
}

// ---- tensor copies of boxes of STEPS rows x 64 channels --------------------------
// The driver's tensor-map encoder.  Only a successful lookup is kept.
inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> cached{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 fn = cached.load(std::memory_order_acquire);
    if (fn != nullptr) return fn;
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
        fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        cached.store(fn, std::memory_order_release);
    }
    return fn;
}
template <typename T>
inline bool rows_map(CUtensorMap *m, const T *base, int64_t Bs, int64_t L, int64_t ED, int steps) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {cuuint64_t(ED), cuuint64_t(L), cuuint64_t(Bs)};
    const cuuint64_t strides[2] = {cuuint64_t(ED) * sizeof(T), cuuint64_t(L) * cuuint64_t(ED) * sizeof(T)};
    const cuuint32_t box[3] = {64, cuuint32_t(steps), 1}, each[3] = {1, 1, 1};
    return fn(m, sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                 : sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                  : CU_TENSOR_MAP_DATA_TYPE_UINT8,
              3, const_cast<T *>(base), dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
__device__ __forceinline__ void tma_store_3d(const void *tmap, const void *src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(tmap),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

// How a kernel's blocks share the work: blocks of `warps` warps, each with 64
// channels of a sequence (a chain) and one of its C shares of the time axis, C
// blocks a cluster.  Sequences behind the first `first` have clusters of
// `rest_cluster` blocks, in a launch of their own (0: there are none).
struct Split {
    int warps = 0, cluster = 1, rest_cluster = 0;
    int64_t first = 0;
    double us = 0.0;
    cudaError_t err = cudaSuccess;      // of the questions to the driver; nothing else counts then
};

// Which sequences a launch has, in its arguments.
struct Share {
    int cluster = 1;      // blocks a cluster
    int first = 0;        // its first sequence
    int sums = 0;         // blocks' sums before its first one's
    int order = 0;        // 1: a launch for the rest follows; 2: it is that one
};
// At a block's start: the next launch of this pass may begin once every block
// of this one has.  The rest needs no result of the first launch.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_launch() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// At a block's end: what comes after the rest comes after the first launch, too.
__device__ __forceinline__ void wait_for_first(const Share &s) {
    if (s.order == 2) wait_for_launch();
}

// Starts `seqs` sequences in clusters of args.share.cluster blocks.  With
// `resident`: asks for the blocks that run at a time instead.  The kernel's
// limit of shared memory is that of the largest cluster whatever this launch
// takes: the limit belongs to the kernel, and another host thread may set it
// between this call's setting and its launch.  (A limit alone costs no places.)
template <typename Args, typename Maps>
inline cudaError_t start_clusters(void (*kern)(Args, Maps), int smem, int warps, int64_t seqs, int64_t ED, const Args &args,
                                  const Maps &maps, cudaStream_t st, int *resident = nullptr) {
    const int C = args.share.cluster;
    cudaError_t err =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem + exchange_bytes(kMaxCluster));
    smem += exchange_bytes(C);
    if (err == cudaSuccess && C > 8)
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned((ED + 63) / 64 * C), unsigned(seqs));
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {unsigned(C), 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = args.share.order == 2 ? 2 : 1;
    if (resident) {
        int clusters = 0;
        err = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
        *resident = clusters * C;
        return err;
    }
    return cudaLaunchKernelEx(&cfg, kern, args, maps);
}

// One pass over all sequences.
template <typename Args, typename Maps>
inline cudaError_t start_split(void (*kern)(Args, Maps), int smem, const Split &how, int64_t Bs, int64_t ED, Args args,
                               const Maps &maps, cudaStream_t st) {
    const bool rest = how.rest_cluster != 0;
    args.share = {how.cluster, 0, 0, rest ? 1 : 0};
    const cudaError_t err = start_clusters(kern, smem, how.warps, how.first, ED, args, maps, st);
    if (err != cudaSuccess || !rest) return err;
    args.share = {how.rest_cluster, int(how.first), int(how.first) * how.cluster, 2};
    return start_clusters(kern, smem, how.warps, Bs - how.first, ED, args, maps, st);
}

// What a turn (one tile of a block) takes, in microseconds: alone on its SM,
// for each other block there, for an exchange with a cluster of two and for
// each further block of the cluster; and what a block's start takes.  Measured.
struct Turn {
    double alone, shared, exchange, hop, start;
};

constexpr double kLaunchUs = 1.0;

// Blocks of one kernel that run at a time, by device and C; asked for once.
// An answer is kept, a failure is not.
struct Places {
    static constexpr int kDevices = 64;
    std::atomic<int> of[kDevices][kMaxCluster + 1];
};

// Chooses C for one kernel (blocks of `warps` warps, `tile` steps) by the time
// that its rounds of blocks would take.  A last round that a few sequences
// would have for themselves goes to larger clusters, so that it is as short as
// the GPU is empty; of kRest blocks at most, since a cluster waits until all
// its places are free (gradients of Bs=32 L=2048 ED=1536 274 us, with the last
// round by 4 blocks 267, by 6 286, by 8 283).  It has to save kLaunchUs: where
// the sums were even, two launches took longer (forward of Bs=5 L=4096 ED=2048
// 72.5 us, in two launches 74.9).
template <typename Args, typename Maps>
inline Split best_split(void (*kern)(Args, Maps), int smem, int warps, int tile, const Turn &t,
                        int64_t Bs, int64_t L, int64_t ED, int num_sms, Places &places) {
    Split best;
    int device = 0;
    best.err = cudaGetDevice(&device);
    if (best.err == cudaSuccess && device >= Places::kDevices) best.err = cudaErrorInvalidDevice;
    if (best.err != cudaSuccess) return best;
    std::atomic<int> *cache = places.of[device];
    const int64_t groups = (ED + 63) / 64, tiles = (L + tile - 1) / tile;
    const int widest = int(std::min<int64_t>(kMaxCluster, tiles));
    int slots[kMaxCluster + 1];
    for (int C = 1; C <= widest; ++C) {
        slots[C] = cache[C].load(std::memory_order_relaxed);
        if (slots[C] == 0) {
            Args one{};
            one.share.cluster = C;
            best.err = start_clusters(kern, smem, warps, 1, ED, one, Maps{}, nullptr, &slots[C]);
            if (best.err != cudaSuccess) return best;
            // one cluster less than the driver counts: when all it counts
            // were asked for (40 of 7), some waited for a second round
            slots[C] = slots[C] > C ? slots[C] - C : slots[C] > 0 ? slots[C] : -1;
            cache[C].store(slots[C], std::memory_order_relaxed);
        }
    }
    // one round of `blocks` blocks
    auto round = [&](int C, int64_t blocks) {
        if (blocks == 0) return 0.0;
        const double others = double((blocks + num_sms - 1) / num_sms - 1);
        const double turn = t.alone + others * t.shared + (C > 1 ? t.exchange + (C - 1) * t.hop : 0.0);
        return double((tiles + C - 1) / C) * turn + t.start;
    };
    auto launch = [&](int64_t seqs, int most) {
        Split best;
        for (int C = 1; C <= most; ++C) {
            if (slots[C] < C) continue;
            const int64_t blocks = seqs * groups * C;
            const double us = double(blocks / slots[C]) * round(C, slots[C]) + round(C, blocks % slots[C]);
            if (best.warps == 0 || us < best.us) best.warps = warps, best.cluster = C, best.us = us;
        }
        best.first = seqs;
        return best;
    };
    best = launch(Bs, widest);
    for (int C = 1; C <= widest && best.warps != 0; ++C) {
        if (slots[C] < C) continue;
        const int64_t rounds = Bs * groups * C / slots[C], first = rounds * slots[C] / (C * groups);
        if (first == 0 || first == Bs) continue;
        const double whole = double(rounds) * round(C, slots[C]);
        if (whole >= best.us) continue;
        const Split rest = launch(Bs - first, std::min(widest, kRest));
        const double us = whole + rest.us + kLaunchUs;
        if (rest.warps != 0 && us < best.us) best.cluster = C, best.first = first, best.rest_cluster = rest.cluster, best.us = us;
    }
    return best;
}

template <typename T>
inline int widest_copy(uintptr_t at, int64_t ED) {
    return at % 16 != 0 || ED >= (1 << 26) ? 1 : ED * int64_t(sizeof(T)) % 16 == 0 ? 16 : 8;
}


}  // namespace gated
}  // namespace ssm
