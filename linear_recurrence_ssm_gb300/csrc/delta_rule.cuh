// delta_rule.cuh -- what the kernels of the gated delta rule share: the
// problem, the tokens of a sequence, and the decays inside a block of 64 steps.
//
// Per head, with a state S (V x K) in fp32 and a_t = e^(g_t):
//   x_t = v_t - a_t S_{t-1} k_t,  u_t = beta_t x_t
//   S_t = a_t S_{t-1} + u_t k_t^T,  y_t = scale S_t q_t
// Over a block of C = 64 steps from S0, with gamma the running sum of g,
// D_ts = e^(gamma_t - gamma_s), Gam_t = e^(gamma_t), E_t = e^(gamma_C - gamma_t),
// Ab_ts = D_ts k_t.k_s (s < t) and P_ts = D_ts q_t.k_s (s <= t):
//   W = V - Gam K S0^T,  (I + Ab beta) X = W,  U = beta X
//   Y = scale (Gam Q S0^T + P U),  S1 = Gam_C S0 + U^T E K
// and back, with dS the adjoint of S1:
//   dU = scale P^T dY + E K dS^T,  (I + Ab^T beta) Z = dU
//   dV = beta Z,  dbeta_t = Z_t.x_t
//   dS0 = Gam_C dS + scale (Gam dY)^T Q - (Gam beta Z)^T K
//   dP = scale dY U^T (s <= t),  dAb = -(beta Z) U^T (s < t)
//   dQ = scale Gam dY S0 + (dP D) K
//   dK = (dP D)^T Q + E U dS - Gam beta Z S0 + (dAb D) K + (dAb D)^T K
//   dg_t = sum_{r >= t} (row_r) + sum_{s < t <= r} (dP P + dAb Ab)_rs
//        + sum_{s < t} E_s u_s.(dS k_s) + Gam_C <S0, dS>,
//   row_r = Gam_r (scale dY_r.(S0 q_r) - beta_r Z_r.(S0 k_r)):
// each term of dg_t crosses step t, so nothing large cancels.
#pragma once

#include "ssm_common.cuh"

namespace ssm {
namespace delta {

constexpr int kBlock = 64;      // steps taken at once, and between two kept states

struct Shape {
    const int32_t *offsets;     // (n + 1) starts of the packed sequences, or null: n sequences of L tokens
    int64_t L;                  // tokens of a sequence, or of all packed ones
    int n, G, H, K, V;
    float scale;
    int64_t rows() const { return offsets ? L : L * n; }
    // Blocks that any offsets can need, each with a place of its own.
    int64_t slots() const { return offsets ? L / kBlock + n : (L + kBlock - 1) / kBlock * n; }
    int64_t states() const { return int64_t(H) * V * K; }
};

// A sequence: its tokens, its blocks, and the place of its first block.  Bad
// offsets are brought into 0..L and a sequence that would end before it starts
// is empty: every access stays inside the arrays.
struct Span {
    int64_t first, slot;
    int len, blocks;
};
__device__ __forceinline__ Span span_of(const Shape &s, int i) {
    if (!s.offsets) {
        const int blocks = int((s.L + kBlock - 1) / kBlock);
        return {int64_t(i) * s.L, int64_t(i) * blocks, int(s.L), blocks};
    }
    const int L = int(s.L);
    const int b = min(max(s.offsets[i], 0), L), e = min(max(s.offsets[i + 1], b), L);
    return {b, int64_t(b / kBlock) + i, e - b, (e - b + kBlock - 1) / kBlock};
}

// A long sequence of few heads is taken in parts of `blocks` blocks of 64
// steps: parts have places as blocks have, and an empty sequence has one part.
__device__ __forceinline__ int64_t first_part(const Shape &s, const Span &span, int i, int blocks) {
    if (s.offsets) return span.first / (int64_t(kBlock) * blocks) + i;
    return int64_t(i) * ((span.blocks + blocks - 1) / blocks);
}
__device__ __forceinline__ int parts_of(const Span &span, int blocks) {
    return max(1, (span.blocks + blocks - 1) / blocks);
}

// The sequence whose block has place `slot`, or -1.  All threads of the thread
// block; `found` is in shared memory.
__device__ __forceinline__ int sequence_of(const Shape &s, int64_t slot, int *found) {
    if (!s.offsets) return int(slot / ((s.L + kBlock - 1) / kBlock));
    if (threadIdx.x == 0) *found = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < s.n; i += blockDim.x) {
        const Span span = span_of(s, i);
        if (slot >= span.slot && slot < span.slot + span.blocks) atomicMax(found, i);
    }
    __syncthreads();
    return *found;
}

// The same for a part's place.
__device__ __forceinline__ int part_sequence_of(const Shape &s, int64_t place, int blocks, int *found) {
    if (!s.offsets) {
        const int whole = int((s.L + kBlock - 1) / kBlock);
        return int(place / ((whole + blocks - 1) / blocks));
    }
    if (threadIdx.x == 0) *found = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < s.n; i += blockDim.x) {
        const Span span = span_of(s, i);
        const int64_t first = first_part(s, span, i, blocks);
        if (place >= first && place < first + parts_of(span, blocks)) atomicMax(found, i);
    }
    __syncthreads();
    return *found;
}

// The sums of log2 decays inside a block, as two floats: differences of far
// steps keep their relative accuracy after the exponential.  A decay below
// e^-100 is 0 in fp32: such a step counts as a cut, adds nothing to the sum,
// and no pair reaches across it (-infinity is a cut).
struct alignas(16) Decays {
    float hi[kBlock], lo[kBlock], beta[kBlock];
    int cut[kBlock];
    __device__ __forceinline__ float between(int t, int s) const {
        return cut[t] == cut[s] ? ex2((hi[t] - hi[s]) + (lo[t] - lo[s])) : 0.0f;
    }
    __device__ __forceinline__ float start(int t) const { return cut[t] == 0 ? ex2(hi[t] + lo[t]) : 0.0f; }
    __device__ __forceinline__ float end(int t) const { return between(kBlock - 1, t); }
};
constexpr float kCut = -100.0f;

// One warp: the running sums of `rows` steps; steps behind them do not decay
// and write nothing (beta = 0).  `g` and `beta` start at the first step,
// `stride` is the heads of a token.  A lane has steps `lane` and `lane + 32`.
struct Gates {
    float g[2], beta[2];
    template <typename T>
    __device__ __forceinline__ void load(const T *from_g, const T *from_beta, int64_t stride, int rows) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int t = 32 * half + int(threadIdx.x % 32);
            g[half] = t < rows ? to_f32(from_g[t * stride]) : 0.0f;
            beta[half] = t < rows ? to_f32(from_beta[t * stride]) : 0.0f;
        }
    }
};
// A sum of two floats' exact sum and what it leaves over.
__device__ __forceinline__ void add_to(float &hi, float &lo, float more_hi, float more_lo) {
    const float s = __fadd_rn(hi, more_hi), b = __fsub_rn(s, hi);
    lo = __fadd_rn(__fadd_rn(lo, more_lo), __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(more_hi, b)));
    hi = s;
}
__device__ __forceinline__ void sum_decays(Decays &d, const Gates &w) {
    const int lane = threadIdx.x % 32;
    float sum_hi = 0.0f, sum_lo = 0.0f;
    int cuts = 0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int t = 32 * half + lane;
        const bool cut = w.g[half] < kCut;
        const float v = cut ? 0.0f : w.g[half];
        // g log2(e): the constant in two floats, the product's remainder from a fused multiply-add
        float hi = __fmul_rn(v, 1.44269502162933349609375f);
        float lo = __fmaf_rn(v, 1.925963033500011e-8f, __fmaf_rn(v, 1.44269502162933349609375f, -hi));
        int c = cut;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const float x = __shfl_up_sync(0xffffffffu, hi, o), y = __shfl_up_sync(0xffffffffu, lo, o);
            const int n = __shfl_up_sync(0xffffffffu, c, o);
            if (lane >= o) {
                add_to(hi, lo, x, y);
                c += n;
            }
        }
        add_to(hi, lo, sum_hi, sum_lo);
        c += cuts;
        d.hi[t] = hi;
        d.lo[t] = lo;
        d.cut[t] = c;
        d.beta[t] = w.beta[half];
        sum_hi = __shfl_sync(0xffffffffu, hi, 31), sum_lo = __shfl_sync(0xffffffffu, lo, 31);
        cuts = __shfl_sync(0xffffffffu, c, 31);
    }
}
template <typename T>
__device__ __forceinline__ void load_decays(Decays &d, const T *g, const T *beta, int64_t stride, int rows) {
    Gates w;
    w.load(g, beta, stride, rows);
    sum_decays(d, w);
}

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16(v); }

// `width` elements of the rows of `out`, `step` elements apart, that no sequence covers become 0: those
// before the first sequence (its blocks write them) and behind the last.
template <typename T>
__device__ __forceinline__ void clear_uncovered(const Shape &s, int seq, T *out, int64_t step, int width) {
    if (!s.offsets) return;
    int64_t a = 0, b = 0;
    for (int part = 0; part < 2; ++part) {
        if (part == 0) {
            if (seq != 0) continue;
            a = 0, b = span_of(s, 0).first;
        } else {
            if (seq != s.n - 1) continue;
            const Span last = span_of(s, s.n - 1);
            a = last.first + last.len, b = s.L;
        }
        for (int64_t i = threadIdx.x; i < (b - a) * width; i += blockDim.x)
            put(out + (a + i / width) * step + i % width, 0.0f);
    }
}

// The kept state of a place that no block has becomes 0.
template <typename T>
__device__ __forceinline__ void clear_state(const Shape &s, int64_t slot, int head, T *states) {
    T *out = states + (slot * s.H + head) * int64_t(s.V) * s.K;
    for (int i = threadIdx.x; i < s.V * s.K; i += blockDim.x) put(out + i, 0.0f);
}

// What the backward pass keeps between its kernels, one after another in the
// caller's scratch.
struct Scratch {
    int64_t ds, dbeta, dq, dk, records, bytes;
};
// `shares`: floats of dbeta's parts; `records`: bytes.
inline Scratch scratch_of(const Shape &s, int elem, int64_t shares, int64_t records) {
    const auto up = [](int64_t b) { return (b + 255) / 256 * 256; };
    Scratch r;
    r.ds = 0;
    r.dbeta = up(s.slots() * s.states() * elem);
    r.dq = r.dbeta + up(shares * 4);
    const int64_t per_head = s.H > s.G ? up(s.rows() * s.H * s.K * 4) : 0;
    r.dk = r.dq + per_head;
    r.records = r.dk + per_head;
    r.bytes = r.records + up(records);
    return r;
}

template <typename T>
struct FwdArgs {
    Shape s;
    const T *q, *k, *v, *g, *beta;
    const float *h0;
    T *y;
    float *h_final;
    T *states, *errors;     // kept for the gradients, or null
    unsigned char *scratch; // the records of all blocks
    // sequences in parts of `part` blocks (0: whole): what each part adds to a
    // state, (places, H, V, K), what it makes of one, (places, H, K, K), and
    // the states that enter the parts, (places, H, V, K)
    int part;
    float *added, *turned, *entering;
};
template <typename T>
struct BwdArgs {
    Shape s;
    const T *q, *k, *g, *beta, *dy;
    const float *dh_final;
    const T *states, *errors;
    T *dq, *dk, *dv, *dg, *dbeta;
    float *dh0;
    T *ds;                  // scratch: the adjoint of every block's last state
    float *dbeta_part, *dq_head, *dk_head;
    unsigned char *records;
};
namespace general {
int64_t shares(const Shape &s);
int64_t made_bytes(const Shape &s);
template <typename T>
cudaError_t fold(const BwdArgs<T> &a, cudaStream_t st);
}

}  // namespace delta
}  // namespace ssm
