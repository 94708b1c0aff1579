// gated_scan_bwd.cu -- gradients of the gated linear recurrence.
//
// With g_t = dL/dh_t:  g_t = dy_t + u_{t+1},  u_t = a_t g_t,  u_L = dh_final
//   dx = g m s_i            dgate_i = g m x s_i (1 - s_i)
//   G  = la g (a h_{t-1} - (a^2 / m) s_i x)     (0 at a reset)
//   dgate_r = G (1 - s_r)   dlam = sum of G, times sigmoid(lam) / softplus(lam)
//
// The tiles are the forward pass's (gated_scan.cu), walked from the end.  A
// warp's piece of the time axis has two results, that of its states and that
// of its adjoints u; one exchange a tile carries both.  The states of a tile
// start from the kept one, so only the adjoint passes between tiles, and
// between the blocks of a cluster.  a, s_r, s_i and the state before each step
// stay in registers between the exchange and the gradients; x and dy are read
// from shared memory again, 1 - a^2 is computed again.
#include "gated_scan.cuh"

namespace ssm {
namespace gated_bwd {
using namespace gated;

constexpr int kStages = 2;

template <typename T>
struct BwdArgs {
    const T *in[3];             // x, gate_r, gate_i
    const float *lam;
    float c;
    const uint8_t *reset;
    const T *dy;
    const float *dh_final;
    Kept kept;
    T *dx, *dr, *di;
    float *part, *dh0;          // part (Bs * cluster, ED): sums of G
    int L, ED, cluster;
    int64_t rows;               // Bs * L
    int pair_stores;
};

// One stage of a warp's ring: rows of x, gate_r, gate_i (of type K: T, or
// int8 with their 24 scales), then of dy.
template <typename T, typename K, int W>
struct Stage {
    static constexpr int kIn = kSteps * kPitch<K, W>, kDy = 3 * kIn, kScales = kDy + kSteps * kPitch<T, W>;
    static constexpr int kBytes = kScales + (sizeof(K) == 1 ? 128 : 0);
};

struct Pieces {
    float4 warp[2][kWarps][32];              // A of two channels, state of two channels
    float2 adjoint[2][kWarps][32];
    float4 block[2][kMaxCluster][32];        // A, adjoint; written by the cluster's blocks
    uint32_t cuts[2][kWarps], block_cut[2][kMaxCluster];
};

template <typename T, typename K, int W>
__device__ __forceinline__ float2 input(const uint8_t *stage, int k, int j, int64_t row, int ED) {
    using S = Stage<T, K, W>;
    const float2 v = pair_at<K, W>(stage + k * S::kIn + j * kPitch<K, W>, shift_of<K, W>(row + j, ED));
    if constexpr (sizeof(K) != 1) return v;
    return mul2(v, both(reinterpret_cast<const float *>(stage + S::kScales)[k * kSteps + j]));
}
template <typename T, typename K, int W>
__device__ __forceinline__ float2 upstream(const uint8_t *stage, int j, int64_t row, int ED) {
    return pair_at<T, W>(stage + Stage<T, K, W>::kDy + j * kPitch<T, W>, shift_of<T, W>(row + j, ED));
}

// GENERAL: decays may be fast, steps may drop the state (bit j of cut) or lie
// behind the end (j >= n).
template <typename T, typename K, int W, bool GENERAL>
__device__ __forceinline__ void pieces(const uint8_t *stage, int64_t row0, int ED, float2 rate, uint32_t cut, int n,
                                       float2 (&a)[kSteps], float2 (&b)[kSteps], float2 (&sr)[kSteps],
                                       float2 (&si)[kSteps], float2 &A, float2 &H, float2 &U) {
    constexpr bool ACC = sizeof(T) == 4;
    A = both(1.0f);
    H = both(0.0f);
    U = both(0.0f);
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
        sr[j] = sigmoid2<ACC>(input<T, K, W>(stage, 1, j, row0, ED));
        si[j] = sigmoid2<ACC>(input<T, K, W>(stage, 2, j, row0, ED));
        float2 w;
        decay2<ACC, GENERAL>(mul2(rate, sr[j]), a[j], w);
        const float2 in = mul2(si[j], input<T, K, W>(stage, 0, j, row0, ED));
        const float2 v = one_minus_square(w);
        b[j] = mul2(mul2(v, rsqrt2<ACC>(v)), in);
        if (GENERAL && j >= n) a[j] = both(1.0f), b[j] = both(0.0f);
        if (GENERAL && (cut >> j & 1)) {
            a[j] = both(0.0f);
            b[j] = in;
            A = both(0.0f);
            H = in;
        } else {
            A = mul2(A, a[j]);
            H = fma2(a[j], H, b[j]);
        }
    }
#pragma unroll
    for (int j = kSteps - 1; j >= 0; --j) {
        U = mul2(a[j], add2(upstream<T, K, W>(stage, j, row0, ED), U));
        if (GENERAL && (cut >> j & 1)) U = both(0.0f);
        if (GENERAL && j >= n) U = both(0.0f);
    }
}

template <typename T, typename K, int W, bool GENERAL>
__device__ __forceinline__ void gradients(const BwdArgs<T> &p, const uint8_t *stage, int64_t row0, float2 rate,
                                          uint32_t cut, int n, const float2 (&a)[kSteps], const float2 (&before)[kSteps],
                                          const float2 (&sr)[kSteps], const float2 (&si)[kSteps], float2 u, int e,
                                          bool in0, bool in1, float2 &sum) {
    constexpr bool ACC = sizeof(T) == 4;
    const int64_t at = row0 * p.ED + e;
#pragma unroll
    for (int j = kSteps - 1; j >= 0; --j) {
        if (GENERAL && j >= n) continue;
        const bool dropped = GENERAL && (cut >> j & 1);
        const float2 g = add2(upstream<T, K, W>(stage, j, row0, p.ED), u);
        const float2 x = input<T, K, W>(stage, 0, j, row0, p.ED);
        const float2 t = mul2(rate, sr[j]);
        float2 w = slow_loss(t);
        if (GENERAL) {
            if (t.x >= kSlow) w.x = 1.0f - a[j].x;
            if (t.y >= kSlow) w.y = 1.0f - a[j].y;
        }
        const float2 v = one_minus_square(w), over = rsqrt2<ACC>(v);
        const float2 in = mul2(si[j], x);
        float2 gm = mul2(g, mul2(v, over));
        // la (a h - (a^2 / m) s_i x) = t a ((a / m) s_i x - h)
        float2 G = mul2(mul2(mul2(t, a[j]), g),
                        fma2(mul2(a[j], over), in, mul2(before[j], both(-1.0f))));
        if (dropped) gm = g, G = both(0.0f);
        const float2 dx = mul2(gm, si[j]), q = mul2(dx, x);
        put_pair(p.dx + at + int64_t(j) * p.ED, dx, p.pair_stores, in0, in1);
        put_pair(p.di + at + int64_t(j) * p.ED, fma2(mul2(q, both(-1.0f)), si[j], q), p.pair_stores, in0, in1);
        put_pair(p.dr + at + int64_t(j) * p.ED, fma2(mul2(G, both(-1.0f)), sr[j], G), p.pair_stores, in0, in1);
        sum = add2(sum, G);
        u = mul2(a[j], g);
        if (dropped) u = both(0.0f);
    }
}

template <typename T, typename K, int W, bool RESET>
__global__ void __launch_bounds__(kThreads, 2)
gated_bwd_kernel(const __grid_constant__ BwdArgs<T> p) {
    using S = Stage<T, K, W>;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ Pieces sh;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int C = p.cluster, rank = C > 1 ? int(cluster_rank()) : 0;
    const int e0 = int(blockIdx.x) / C * 64, e = e0 + 2 * lane;
    const int64_t b = blockIdx.y;
    const int tiles = (p.L + kBlock - 1) / kBlock, turns = (tiles + C - 1) / C;
    const bool in0 = e < p.ED, in1 = e + 1 < p.ED;

    uint8_t *mine = ring + warp * kStages * S::kBytes;
    auto fetch = [&](int turn) {
        const int t = (turn * C + rank) * kBlock + warp * kSteps;
        const int n = min(kSteps, p.L - t);
        if (turn >= 0 && n > 0) {
            uint8_t *to = mine + turn % kStages * S::kBytes;
            const int64_t row0 = b * p.L + t;
            if constexpr (sizeof(K) == 1) {
                const int8_t *q[3] = {p.kept.x_q, p.kept.r_q, p.kept.i_q};
#pragma unroll
                for (int k = 0; k < 3; ++k) copy_rows<int8_t, W>(to + k * S::kIn, q[k], row0, n, e0, p.ED);
                if (lane < 3 * kSteps) {
                    const float *s = lane < kSteps ? p.kept.x_s : lane < 2 * kSteps ? p.kept.r_s : p.kept.i_s;
                    const bool in = lane % kSteps < n;
                    cp_async4(to + S::kScales + 4 * lane,
                              in ? s + (e0 / kGroup) * p.rows + row0 + lane % kSteps : s, in ? 4 : 0);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 3; ++k) copy_rows<T, W>(to + k * S::kIn, p.in[k], row0, n, e0, p.ED);
            }
            copy_rows<T, W>(to + S::kDy, p.dy, row0, n, e0, p.ED);
        }
        cp_async_commit();
    };
    auto reset_of = [&](int turn) -> uint32_t {
        const int t = (turn * C + rank) * kBlock + warp * kSteps + lane;
        return lane < kSteps && t < p.L && turn >= 0 ? p.reset[b * p.L + t] : 0;
    };
    auto kept_of = [&](int turn) {
        const int tile = turn * C + rank;
        if (turn < 0 || tile >= tiles) return both(0.0f);
        const float *k = p.kept.states + (b * tiles + tile) * p.ED + e;
        return make_float2(in0 ? k[0] : 0.0f, in1 ? k[1] : 0.0f);
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(turns - 1 - k);
    uint32_t next_cut = RESET ? reset_of(turns - 1) : 0;
    float2 next_h = kept_of(turns - 1);
    if (C > 1) cluster_sync();     // every block runs before another writes to its shared memory

    const float2 rate = make_float2(in0 ? decay_rate(p.lam[e], p.c) : 0.0f, in1 ? decay_rate(p.lam[e + 1], p.c) : 0.0f);
    const bool wide = __any_sync(0xffffffffu, !(fmaxf(rate.x, rate.y) < kSlow));
    float2 carry = both(0.0f), sum = both(0.0f);     // the adjoint that enters the cluster's next tiles from behind
    if (p.dh_final) carry = make_float2(in0 ? p.dh_final[b * p.ED + e] : 0.0f, in1 ? p.dh_final[b * p.ED + e + 1] : 0.0f);

    for (int turn = turns - 1; turn >= 0; --turn) {
        const int t0 = (turn * C + rank) * kBlock + warp * kSteps, buf = turn & 1;
        const int n = min(kSteps, p.L - t0);      // <= 0 behind the end
        const int64_t row0 = b * p.L + t0;
        fetch(turn - (kStages - 1));
        cp_async_wait<kStages - 1>();
        __syncwarp();
        const uint8_t *stage = mine + turn % kStages * S::kBytes;
        uint32_t cut = 0;
        if (RESET) {
            cut = __ballot_sync(0xffffffffu, next_cut != 0);
            next_cut = reset_of(turn - 1);
        }
        float2 h = next_h;
        next_h = kept_of(turn - 1);

        float2 a[kSteps], s[kSteps], sr[kSteps], si[kSteps], A, H, U;
        const bool general = wide || n < kSteps || (RESET && cut);
        if (general)
            pieces<T, K, W, true>(stage, row0, p.ED, rate, cut, n, a, s, sr, si, A, H, U);
        else
            pieces<T, K, W, false>(stage, row0, p.ED, rate, 0, kSteps, a, s, sr, si, A, H, U);

        sh.warp[buf][warp][lane] = make_float4(A.x, A.y, H.x, H.y);
        sh.adjoint[buf][warp][lane] = U;
        if (RESET && lane == 0) sh.cuts[buf][warp] = cut;
        __syncthreads();

        // the state that enters this warp's steps, the adjoint that enters them from behind
        float2 u = carry, all = carry, Ab = both(1.0f), A1 = Ab;
        uint32_t cut0 = 0, cut1 = 0;
        if (C > 1) all = both(0.0f), u = both(0.0f);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            if (k == warp) break;
            const float4 v = sh.warp[buf][k][lane];
            const float2 on = fma2(make_float2(v.x, v.y), h, make_float2(v.z, v.w));
            h = RESET && sh.cuts[buf][k] ? make_float2(v.z, v.w) : on;
        }
#pragma unroll
        for (int k = kWarps - 1; k >= 0; --k) {
            if (k == warp) u = all, Ab = A1, cut0 = cut1;
            const float4 v = sh.warp[buf][k][lane];
            const float2 w = sh.adjoint[buf][k][lane];
            const float2 on = fma2(make_float2(v.x, v.y), all, w);
            all = RESET && sh.cuts[buf][k] ? w : on;
            if (C > 1) {
                A1 = mul2(A1, make_float2(v.x, v.y));
                if (RESET) cut1 |= sh.cuts[buf][k];
            }
        }
        if (C > 1) {
            if (warp < C) {
                put_remote(&sh.block[buf][rank][lane], warp, make_float4(A1.x, A1.y, all.x, all.y));
                if (RESET && lane == 0) put_remote_u32(&sh.block_cut[buf][rank], warp, cut1);
            }
            cluster_sync();
            float2 behind = carry;
            all = carry;
            for (int k = C - 1; k >= 0; --k) {
                if (k == rank) behind = all;
                const float4 v = sh.block[buf][k][lane];
                const float2 on = fma2(make_float2(v.x, v.y), all, make_float2(v.z, v.w));
                all = RESET && sh.block_cut[buf][k] ? make_float2(v.z, v.w) : on;
            }
            const float2 on = fma2(Ab, behind, u);
            u = RESET && cut0 ? u : on;
        }
        carry = all;

#pragma unroll
        for (int j = 0; j < kSteps; ++j) {      // s: from the steps' inputs to the states before them
            const float2 on = fma2(a[j], h, s[j]), at = h;
            h = RESET && (cut >> j & 1) ? s[j] : on;
            s[j] = at;
        }
        if (general)
            gradients<T, K, W, true>(p, stage, row0, rate, cut, n, a, s, sr, si, u, e, in0, in1, sum);
        else
            gradients<T, K, W, false>(p, stage, row0, rate, 0, kSteps, a, s, sr, si, u, e, in0, in1, sum);
        __syncwarp();      // all lanes have read before any lane copies over this stage
    }
    cp_async_wait<0>();
    if (p.dh0 && warp == 0 && rank == 0) {
        if (in0) p.dh0[b * p.ED + e] = carry.x;
        if (in1) p.dh0[b * p.ED + e + 1] = carry.y;
    }
    __syncthreads();
    float2 *sums = reinterpret_cast<float2 *>(&sh.warp[0][0][0]);
    sums[warp * 32 + lane] = sum;
    __syncthreads();
    if (warp == 0) {
        float2 s = both(0.0f);
        for (int k = 0; k < kWarps; ++k) s = add2(s, sums[k * 32 + lane]);
        float *part = p.part + (b * C + rank) * p.ED + e;
        if (in0) part[0] = s.x;
        if (in1) part[1] = s.y;
    }
    if (C > 1) cluster_sync();     // no block leaves while another may still write to it
}

// dlam from the blocks' sums, in their order.
__global__ void __launch_bounds__(256)
dlam_kernel(const float *__restrict__ part, const float *__restrict__ lam, float *__restrict__ dlam,
            int64_t n, int64_t ED) {
    const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (e >= ED) return;
    float s = 0.0f;
    for (int64_t b = 0; b < n; ++b) s += part[b * ED + e];
    // dla/dlam over la, with la's sign in G
    dlam[e] = s * dlog_decay_over(lam[e]);
}

template <typename T, typename K, int W, bool RESET>
static cudaError_t start(const BwdArgs<T> &p, int64_t Bs, cudaStream_t st) {
    auto kern = gated_bwd_kernel<T, K, W, RESET>;
    const int smem = kWarps * kStages * Stage<T, K, W>::kBytes;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned((p.ED + 63) / 64 * p.cluster), unsigned(Bs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {unsigned(p.cluster), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename T, typename K>
static cudaError_t start(const BwdArgs<T> &p, int W, int64_t Bs, cudaStream_t st) {
    if (W == 16) return p.reset ? start<T, K, 16, true>(p, Bs, st) : start<T, K, 16, false>(p, Bs, st);
    if (W == 4) return p.reset ? start<T, K, 4, true>(p, Bs, st) : start<T, K, 4, false>(p, Bs, st);
    if constexpr (sizeof(K) < 4)
        return p.reset ? start<T, K, 1, true>(p, Bs, st) : start<T, K, 1, false>(p, Bs, st);
    return cudaErrorInvalidValue;      // fp32 is aligned to its 4 bytes
}

template <typename T>
cudaError_t launch(const T *x, const T *gr, const T *gi, const float *lam, float c,
                   const uint8_t *reset, const T *dy, const float *dh_final, const Kept &kept, T *dx,
                   T *dr, T *di, float *dlam, float *dh0, int64_t Bs, int64_t L, int64_t ED,
                   int num_sms, cudaStream_t st) {
    auto at = [](const void *q) { return reinterpret_cast<uintptr_t>(q); };
    BwdArgs<T> p{{x, gr, gi}, lam, c, reset, dy, dh_final, kept, dx, dr, di, nullptr, dh0,
                 int(L), int(ED), cluster_for(Bs, L, ED, num_sms), Bs * L, 0};
    p.pair_stores = ED % 2 == 0 && (at(dx) | at(dr) | at(di)) % (2 * sizeof(T)) == 0;
    cudaError_t err = cudaMallocAsync(&p.part, size_t(Bs * p.cluster * ED) * sizeof(float), st);
    if (err != cudaSuccess) return err;
    if (kept.x_q)
        err = start<T, int8_t>(p, min(widest_copy<int8_t>(at(kept.x_q) | at(kept.r_q) | at(kept.i_q), ED),
                                      widest_copy<T>(at(dy), ED)),
                               Bs, st);
    else
        err = start<T, T>(p, widest_copy<T>(at(x) | at(gr) | at(gi) | at(dy), ED), Bs, st);
    if (err == cudaSuccess) {
        dlam_kernel<<<unsigned((ED + 255) / 256), 256, 0, st>>>(p.part, lam, dlam, Bs * p.cluster, ED);
        err = cudaGetLastError();
    }
    const cudaError_t e2 = cudaFreeAsync(p.part, st);
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
