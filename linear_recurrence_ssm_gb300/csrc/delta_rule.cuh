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

// The sums of log2 decays inside a block, as two floats: differences of far
// steps keep their relative accuracy after the exponential.  A decay below
// e^-100 is 0 in fp32: such a step counts as a cut, adds nothing to the sum,
// and no pair reaches across it (-infinity is a cut).
struct Decays {
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
// and write nothing (beta = 0).  `at` is the first step's gate, `stride` the
// heads of a token.
template <typename T>
__device__ __forceinline__ void load_decays(Decays &d, const T *g, const T *beta, int64_t stride, int rows) {
    const int lane = threadIdx.x % 32;
    double sum = 0.0;
    int cuts = 0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int t = 32 * half + lane;
        const float v = t < rows ? to_f32(g[t * stride]) : 0.0f;
        const bool cut = v < kCut;
        double w = cut ? 0.0 : double(v) * 1.4426950408889634;
        int c = cut;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const double x = __shfl_up_sync(0xffffffffu, w, o);
            const int y = __shfl_up_sync(0xffffffffu, c, o);
            if (lane >= o) w += x, c += y;
        }
        w += sum, c += cuts;
        const float hi = float(w);
        d.hi[t] = hi;
        d.lo[t] = float(w - double(hi));
        d.cut[t] = c;
        d.beta[t] = t < rows ? to_f32(beta[t * stride]) : 0.0f;
        sum = __shfl_sync(0xffffffffu, w, 31);
        cuts = __shfl_sync(0xffffffffu, c, 31);
    }
}

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16(v); }

// What the backward pass keeps between its kernels, one after another in the
// caller's scratch.
struct Scratch {
    int64_t ds, dbeta, dq, dk, bytes;
};
inline Scratch scratch_of(const Shape &s, int elem, int slices) {
    const auto up = [](int64_t b) { return (b + 255) / 256 * 256; };
    Scratch r;
    r.ds = 0;
    r.dbeta = up(s.slots() * s.states() * elem);
    r.dq = r.dbeta + up(int64_t(slices) * s.rows() * s.H * 4);
    const int64_t per_head = s.H > s.G ? up(s.rows() * s.H * s.K * 4) : 0;
    r.dk = r.dq + per_head;
    r.bytes = r.dk + per_head;
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
};

}  // namespace delta
}  // namespace ssm
