// gated_scan_bwd.cu -- gradients of the gated linear recurrence.
//
// With g_t = dL/dh_t:  g_t = dy_t + u_{t+1},  u_t = a_t g_t,  u_L = dh_final
//   dx = g m s_i            dgate_i = g m x s_i (1 - s_i)
//   G  = la g (a h_{t-1} - (a^2 / m) s_i x)     (0 at a reset)
//   dgate_r = G (1 - s_r)   dlam = sum of G, times sigmoid(lam) / softplus(lam)
//
// Tiles of 64 steps x 64 channels (8 warps of 8 steps), walked from the end.
// A warp's piece of the time axis has two results, that of its states and
// that of its adjoints u; one exchange a tile carries both.  The states of a
// tile start from the kept one, so only the adjoint passes between tiles, and
// between the blocks of a cluster.  a, m, s_r, s_i and the state before each
// step stay in registers between the exchange and the gradients; x and dy are
// read from shared memory again.
//
// 14 bytes an element (bf16).  At Bs=8 L=2048 ED=1536 (bytes: 52 us): one
// thread a channel 2072 us; tiles 117; boxes 98; one warp folding the pieces
// 92; m kept instead of computed twice 86; dlam's sum launched early 84 (4.2
// TB/s, 62 % of the measured copy rate).  Left out, the folds of the exchange
// save 11 us, the copies in 9, those out 7, all three 29: no single one of them
// bounds it.  856 instructions for 8 x 32 lanes of two elements issue in 33
// us; 16 warps an SM (128 registers) cover them to 46 %, the rest is waiting at
// the two barriers of a tile (a quarter) and for results.  Doing the work that
// does not need the adjoint while it travels was measured slower (88 us), and
// so was taking the adjoint's sum forwards (86).  Bs=16 L=1000 ED=2560 (bytes:
// 85 us): 126 us in whole rounds, 113 with the last sequence in clusters of
// four; from the 8-bit checkpoint (bytes: 68 us) 139 and 125, bound by
// instructions (980, the unpacking of bytes among them).
#include "gated_scan.cuh"

#include <algorithm>
#include <float.h>

namespace ssm {
namespace gated_bwd {
using namespace gated;

constexpr int kWarps = 8, kSteps = kBlock / kWarps, kThreads = 32 * kWarps;
// Tiles of a warp's rows in flight or in use.  With fp32 one, so that two
// blocks fit an SM.
template <typename T>
constexpr int kStages = sizeof(T) == 4 ? 1 : 2;

__device__ unsigned int g_device_error;

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
    float *part, *dh0;          // part (sequences' clusters' blocks, ED): sums of G
    int L, ED;
    int64_t rows;               // Bs * L
    Share share;
};

// One stage of a warp's ring: rows of x, gate_r, gate_i (of type K: T, or
// int8 with their 24 scales), then of dy.  Boxes of outputs (W = 16) take the
// places of the three inputs, or of their own behind the ring where those are
// narrower.
template <typename T, typename K, int W>
struct Stage {
    static constexpr int kIn = kSteps * kPitch<K, W>, kDy = 3 * kIn, kScales = kDy + kSteps * kPitch<T, W>;
    static constexpr int kBytes = kScales + (sizeof(K) == 1 ? 128 : 0);
    static constexpr int kOut = kSteps * kPitch<T, W>, kOwnOut = W == 16 && sizeof(K) < sizeof(T) ? 3 * kOut : 0;
    static constexpr int kDepth = kStages<T>, kWarpBytes = kDepth * kBytes + kOwnOut;
};

// Boxes of 64 channels x kSteps rows (W = 16).
struct BwdMaps {
    CUtensorMap in[3], dy, out[3];
};

struct Shared {
    float4 warp[kWarps][32];        // a piece's A of two channels, state of two channels
    float2 adjoint[kWarps][32];     // its adjoint, then the adjoint that enters it
    float2 state[kWarps][32];       // the state that enters it
    uint64_t full[kWarps][2];       // a warp's copies have arrived (W = 16)
    Exchange ex;
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
                                       float2 (&a)[kSteps], float2 (&b)[kSteps], float2 (&nsr)[kSteps],
                                       float2 (&nsi)[kSteps], float2 (&nm)[kSteps], float2 &A, float2 &H, float2 &U) {
    constexpr bool ACC = sizeof(T) == 4;
    A = both(1.0f);
    H = both(0.0f);
    U = both(0.0f);
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
        nsr[j] = nsigmoid2<ACC>(input<T, K, W>(stage, 1, j, row0, ED));
        nsi[j] = nsigmoid2<ACC>(input<T, K, W>(stage, 2, j, row0, ED));
        float2 em;
        decay2<ACC, GENERAL>(mul2(rate, nsr[j]), a[j], em);
        const float2 nin = mul2(nsi[j], input<T, K, W>(stage, 0, j, row0, ED));
        const float2 v = square_less_one(a[j], em);
        nm[j] = mul2(v, rsqrt_of_minus<ACC>(v));
        b[j] = mul2(nm[j], nin);
        if (GENERAL && j >= n) a[j] = both(1.0f), b[j] = both(0.0f);
        if (GENERAL && (cut >> j & 1)) {
            a[j] = both(0.0f);
            b[j] = mul2(nin, both(-1.0f));
            A = both(-0.0f);
            H = b[j];
        } else {
            A = mul2(A, a[j]);
            H = fma2(a[j], H, b[j]);
        }
    }
    // again, since a NaN gate behind the drop makes it NaN; here alone, and in
    // both channels, costs registers (Bs=8 L=2048 ED=1537 143 -> 149 us)
    if (GENERAL && cut) A.x = -0.0f;
#pragma unroll
    for (int j = kSteps - 1; j >= 0; --j) {
        U = mul2(a[j], add2(upstream<T, K, W>(stage, j, row0, ED), U));
        if (GENERAL && (j >= n || (cut >> j & 1))) U = both(0.0f);
    }
}

template <typename T, typename K, int W, bool GENERAL>
__device__ __forceinline__ void gradients(const BwdArgs<T> &p, const uint8_t *stage, uint8_t *out, int64_t row0, float2 rate,
                                          uint32_t cut, int n, const float2 (&a)[kSteps], const float2 (&before)[kSteps],
                                          const float2 (&nsr)[kSteps], const float2 (&nsi)[kSteps], const float2 (&nm)[kSteps], float2 u, int e,
                                          bool in0, bool in1, float2 &sum) {
    const int64_t at = row0 * p.ED + e;
#pragma unroll
    for (int j = kSteps - 1; j >= 0; --j) {
        if (GENERAL && j >= n) continue;
        const bool dropped = GENERAL && (cut >> j & 1);
        const float2 g = add2(upstream<T, K, W>(stage, j, row0, p.ED), u);
        const float2 x = input<T, K, W>(stage, 0, j, row0, p.ED);
        const float2 la = mul2(rate, nsr[j]);
        // m's reciprocal; G = la a g (h - (a / m) s_i x)
        const float2 over = reciprocal_of_minus<sizeof(T) == 4>(nm[j]);
        float2 ngm = mul2(g, nm[j]);
        float2 G = mul2(mul2(mul2(la, a[j]), g), fma2(mul2(a[j], over), mul2(nsi[j], x), before[j]));
        if (dropped) ngm = mul2(g, both(-1.0f)), G = both(0.0f);
        const float2 dx = mul2(ngm, nsi[j]), q = mul2(dx, x);
        float2 dr = fma2(G, nsr[j], G);
        const float2 di = fma2(q, nsi[j], q);
        if (dropped) dr = both(0.0f);      // the gate was not used, it may be NaN
        if constexpr (W == 16) {
            // over the lane's own elements of the inputs
            T *o = reinterpret_cast<T *>(out + j * kPitch<T, W>) + 2 * (threadIdx.x % 32);
            put2(o, dx);
            put2(o + Stage<T, K, W>::kOut / sizeof(T), dr);
            put2(o + 2 * Stage<T, K, W>::kOut / sizeof(T), di);
        } else {
            put_pair<W>(p.dx + at + int64_t(j) * p.ED, dx, in0, in1);
            put_pair<W>(p.dr + at + int64_t(j) * p.ED, dr, in0, in1);
            put_pair<W>(p.di + at + int64_t(j) * p.ED, di, in0, in1);
        }
        sum = add2(sum, G);
        u = mul2(a[j], g);
        if (dropped) u = both(0.0f);
    }
}

template <typename T, typename K, int W, bool RESET>
__global__ void __launch_bounds__(kThreads, 2)
gated_bwd_kernel(const __grid_constant__ BwdArgs<T> p, const __grid_constant__ BwdMaps maps) {
    using S = Stage<T, K, W>;
    constexpr int kDepth = S::kDepth;
    extern __shared__ __align__(128) uint8_t ring[];
    Shared &sh = *reinterpret_cast<Shared *>(ring + kWarps * S::kWarpBytes);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int C = p.share.cluster, rank = C > 1 ? int(cluster_rank()) : 0;
    const int e0 = int(blockIdx.x) / C * 64, e = e0 + first_channel<W>();
    const int64_t b = p.share.first + blockIdx.y;
    const int tiles = (p.L + kBlock - 1) / kBlock, turns = (tiles + C - 1) / C;
    const bool in0 = e < p.ED, in1 = e + kNext<W> < p.ED;

    uint8_t *mine = ring + warp * S::kWarpBytes;
    let_next_start();      // the rest, or dlam_kernel
    if (threadIdx.x == 0) {
        if (C > 1) sh.ex.init();
        sh.ex.abort = 0;
    }
    if (W == 16) {
        if (lane == 0) {
            for (int k = 0; k < kDepth; ++k) tc::mbar_init(&sh.full[warp][k], 1);
            tc::mbar_fence_init();
            tc::fence_proxy_async_smem();
        }
    } else if (e0 + 64 > p.ED) {
        clear_ring(mine, kDepth * S::kBytes);
    }
    __syncthreads();

    auto fetch = [&](int turn) {
        const int t = (turn * C + rank) * kBlock + warp * kSteps;
        const int n = min(kSteps, p.L - t);
        const int64_t row0 = b * p.L + t;
        if (turn >= 0 && n > 0) {
            uint8_t *to = mine + turn % kDepth * S::kBytes;
            if constexpr (W == 16) {
                if (lane == 0 && !aborted(&sh.ex.abort)) {
                    uint64_t *bar = &sh.full[warp][turn % kDepth];
                    tc::mbar_arrive_expect_tx(bar, uint32_t(S::kScales));
#pragma unroll
                    for (int k = 0; k < 3; ++k) tc::tma_load_3d(to + k * S::kIn, &maps.in[k], bar, e0, t, int(b));
                    tc::tma_load_3d(to + S::kDy, &maps.dy, bar, e0, t, int(b));
                }
            } else {
                if constexpr (sizeof(K) == 1) {
                    const int8_t *q[3] = {p.kept.x_q, p.kept.r_q, p.kept.i_q};
#pragma unroll
                    for (int k = 0; k < 3; ++k) copy_rows<int8_t, W, kSteps>(to + k * S::kIn, q[k], row0, n, e0, p.ED);
                } else {
#pragma unroll
                    for (int k = 0; k < 3; ++k) copy_rows<T, W, kSteps>(to + k * S::kIn, p.in[k], row0, n, e0, p.ED);
                }
                copy_rows<T, W, kSteps>(to + S::kDy, p.dy, row0, n, e0, p.ED);
            }
            if constexpr (sizeof(K) == 1) {
                if (lane < 3 * kSteps && lane % kSteps < n) {
                    const float *s = lane < kSteps ? p.kept.x_s : lane < 2 * kSteps ? p.kept.r_s : p.kept.i_s;
                    cp_async4(to + S::kScales + 4 * lane, s + (e0 / kGroup) * p.rows + row0 + lane % kSteps, 4);
                }
            }
        }
        if (W != 16 || sizeof(K) == 1) cp_async_commit();
    };
    auto reset_of = [&](int turn) -> uint32_t {
        const int t = (turn * C + rank) * kBlock + warp * kSteps + lane;
        return lane < kSteps && t < p.L && turn >= 0 ? p.reset[b * p.L + t] : 0;
    };
    auto kept_of = [&](int turn) {
        const int tile = turn * C + rank;
        if (turn < 0 || tile >= tiles || warp != 1) return both(0.0f);      // warp 1 folds the states
        return get_pair<W>(p.kept.states + (b * tiles + tile) * p.ED + e, in0, in1);
    };
#pragma unroll
    for (int k = 0; k < (kDepth > 1 ? kDepth - 1 : 1); ++k) fetch(turns - 1 - k);
    uint32_t next_cut = RESET ? reset_of(turns - 1) : 0;
    float2 next_h = kept_of(turns - 1);
    if (C > 1) cluster_sync();     // every block runs before another writes to its shared memory

    const float2 rate = make_float2(in0 ? decay_rate(p.lam[e], p.c) : 0.0f,
                                    in1 ? decay_rate(p.lam[e + kNext<W>], p.c) : 0.0f);
    const bool wide = __any_sync(0xffffffffu, !(fmaxf(rate.x, rate.y) < kSlow));
    float2 carry = both(0.0f), sum = both(0.0f);     // the adjoint that enters the cluster's next tiles from behind
    if (p.dh_final) carry = get_pair<W>(p.dh_final + b * p.ED + e, in0, in1);

    uint32_t phases = 0;           // bit k: the parity that stage k's next copies complete

    for (int turn = turns - 1; turn >= 0; --turn) {
        const int t0 = (turn * C + rank) * kBlock + warp * kSteps, buf = turn & 1;
        const int n = min(kSteps, p.L - t0);      // <= 0 behind the end
        const int64_t row0 = b * p.L + t0;
        uint8_t *stage = mine + turn % kDepth * S::kBytes;
        if (W == 16 && n > 0) {
            const int k = turn % kDepth;
            wait_or_abort(&sh.full[warp][k], phases >> k & 1, &sh.ex.abort, &g_device_error);
            phases ^= 1u << k;
        }
        if (W != 16 || sizeof(K) == 1) {
            cp_async_wait<(kDepth > 1 ? kDepth - 2 : 0)>();
            __syncwarp();
        }
        uint32_t cut = 0;
        if (RESET) {
            cut = __ballot_sync(0xffffffffu, next_cut != 0);
            next_cut = reset_of(turn - 1);
        }
        float2 h = next_h;
        next_h = kept_of(turn - 1);

        float2 a[kSteps], s[kSteps], nsr[kSteps], nsi[kSteps], nm[kSteps], A, H, U;
        const bool general = wide || n < kSteps || (RESET && cut);
        if (general)
            pieces<T, K, W, true>(stage, row0, p.ED, rate, cut, n, a, s, nsr, nsi, nm, A, H, U);
        else
            pieces<T, K, W, false>(stage, row0, p.ED, rate, 0, kSteps, a, s, nsr, nsi, nm, A, H, U);

        sh.warp[warp][lane] = make_float4(A.x, A.y, H.x, H.y);
        sh.adjoint[warp][lane] = U;
        if (kDepth > 1) {
            // the stage that the next rows go to was read, and its outputs stored from, a turn ago
            if (W == 16 && lane == 0) tc::bulk_wait_read0();
            __syncwarp();
            fetch(turn - (kDepth - 1));
        }
        __syncthreads();

        // Two warps find what enters each warp's steps: warp 1 the states from
        // the kept one, warp 0 the adjoints from behind (through the blocks
        // behind where they form a cluster).  One warp each, because a fold of
        // eight pieces in every warp was 1/7 of all instructions.
        if (warp == 1) {
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                sh.state[k][lane] = h;
                if (k + 1 < kWarps) h = after<RESET>(sh.warp[k][lane], h);
            }
        }
        if (warp == 0) {
            auto behind = [&](int k) {
                const float4 v = sh.warp[k][lane];
                const float2 w = sh.adjoint[k][lane];
                return make_float4(v.x, v.y, w.x, w.y);
            };
            float2 all = carry;
            if (C > 1) {
                float4 sum = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
#pragma unroll
                for (int k = kWarps - 1; k >= 0; --k) sum = joined<RESET>(sum, behind(k));
                if (lane == 0) sh.ex.expect(buf, C);
                for (int k = 0; k < C; ++k)
                    if (k != rank) sh.ex.send(buf, C, rank, k, sum);
                sh.ex.wait(buf, (turns - 1 - turn) >> 1 & 1, &g_device_error);
                for (int k = C - 1; k > rank; --k) all = after<RESET>(sh.ex.piece(buf, C, rank, k)[lane], all);
                float2 u = all;
                all = after<RESET>(sum, all);
                for (int k = rank - 1; k >= 0; --k) all = after<RESET>(sh.ex.piece(buf, C, rank, k)[lane], all);
                carry = all;
                all = u;
            }
#pragma unroll
            for (int k = kWarps - 1; k >= 0; --k) {
                const float2 w = all;
                all = after<RESET>(behind(k), all);
                sh.adjoint[k][lane] = w;     // in the place of the piece that was read
            }
            if (C == 1) carry = all;
        }
        __syncthreads();
        h = sh.state[warp][lane];
        const float2 u = sh.adjoint[warp][lane];

#pragma unroll
        for (int j = 0; j < kSteps; ++j) {      // s: from the steps' inputs to the states before them
            const float2 on = fma2(a[j], h, s[j]), at = h;
            h = RESET && (cut >> j & 1) ? s[j] : on;
            s[j] = at;
        }
        uint8_t *out = S::kOwnOut ? mine + kDepth * S::kBytes : stage;
        if (general)
            gradients<T, K, W, true>(p, stage, out, row0, rate, cut, n, a, s, nsr, nsi, nm, u, e, in0, in1, sum);
        else
            gradients<T, K, W, false>(p, stage, out, row0, rate, 0, kSteps, a, s, nsr, nsi, nm, u, e, in0, in1, sum);
        if (W == 16) {
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && n > 0) {
                for (int k = 0; k < 3; ++k) tma_store_3d(&maps.out[k], out + k * S::kOut, e0, t0, int(b));
                tc::bulk_commit();
            }
        }
        if (kDepth == 1) {
            if (W == 16 && lane == 0) tc::bulk_wait_read0();
            __syncwarp();
            fetch(turn - 1);
        }
    }
    if (W == 16) {
        if (lane == 0) tc::bulk_wait_read0();
    }
    cp_async_wait<0>();
    if (p.dh0 && warp == 0 && rank == 0) put_pair<W>(p.dh0 + b * p.ED + e, carry, in0, in1);
    __syncthreads();
    float2 *sums = reinterpret_cast<float2 *>(&sh.warp[0][0]);
    sums[warp * 32 + lane] = sum;
    __syncthreads();
    if (warp == 0) {
        float2 s = both(0.0f);
        for (int k = 0; k < kWarps; ++k) s = add2(s, sums[k * 32 + lane]);
        put_pair<W>(p.part + (p.share.sums + int64_t(blockIdx.y) * C + rank) * p.ED + e, s, in0, in1);
    }
    if (C > 1) cluster_sync();     // no block leaves while another may still write to it
    if (aborted(&sh.ex.abort)) linger();
    wait_for_first(p.share);
}

__global__ void __launch_bounds__(32) __cluster_dims__(2, 1, 1) run_out_kernel(bool for_copy) {
    run_out(for_copy, &g_device_error);
}
cudaError_t probe_wait_timeout(bool for_copy, cudaStream_t st) {
    run_out_kernel<<<2, 32, 0, st>>>(for_copy);
    return cudaGetLastError();
}

// Read and clear this unit's device error word (host side, synchronous).
cudaError_t take_device_error(unsigned int *out) {
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_error, sizeof(v));
    if (e != cudaSuccess) return e;
    if (v) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof(zero));
    }
    *out = v;
    return e;
}

// A sum and what its roundings have lost.  One sum of fp32 over the rows of
// 30000 like sequences was off by 4e-4 of their terms' size: each rounding
// goes the same way.
struct Sum {
    float s = 0.0f, lost = 0.0f;
    __device__ __forceinline__ void add(float v) {
        const float t = s + v, took = t - s;
        lost += (s - (t - took)) + (v - took);
        s = t;
    }
    // infinite or NaN sums have lost nothing that could be told
    __device__ __forceinline__ float value() const { return fabsf(s) <= FLT_MAX ? s + lost : s; }
};

// dlam from the blocks' sums: 32 channels a block, each warp adds every
// kSumWarps-th row, and their sums are joined in their order.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(32 * kSumWarps)
dlam_kernel(const float *__restrict__ part, const float *__restrict__ lam, float *__restrict__ dlam,
            int64_t n, int64_t ED) {
    __shared__ Sum sums[kSumWarps][32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t e = int64_t(blockIdx.x) * 32 + lane;
    // dla/dlam over la, with la's sign in G
    const float factor = e < ED && warp == 0 ? dlog_decay_over(lam[e]) : 0.0f;
    wait_for_launch();
    Sum sum;
    if (e < ED) {
#pragma unroll 8
        for (int64_t b = warp; b < n; b += kSumWarps) sum.add(part[b * ED + e]);
    }
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp != 0 || e >= ED) return;
    for (int k = 1; k < kSumWarps; ++k) {
        sum.add(sums[k][lane].s);
        sum.lost += sums[k][lane].lost;
    }
    dlam[e] = sum.value() * factor;
}

template <typename T, typename K, int W, bool RESET>
static cudaError_t start(const BwdArgs<T> &p, const BwdMaps &maps, int64_t Bs, int num_sms, int64_t *sums, cudaStream_t st) {
    constexpr int kSmem = kWarps * Stage<T, K, W>::kWarpBytes + int(sizeof(Shared));
    auto kern = gated_bwd_kernel<T, K, W, RESET>;
    static_assert(kSmem + exchange_bytes(kMaxCluster) <= 227 * 1024, "shared memory of one block exceeds 227 KB");
    static Places places;
    // Fitted to measured passes.  fp32's exchange and hop keep a chain in fewer
    // blocks: with twice bf16's shared time, its exchange and its hop (0.45,
    // 0.1) Bs=3 L=1001 ED=1537 took 55.9 us (now 49.8), 8 x 512 x 1536 54.9
    // (50.9), 16 x 300 x 640 39.6 (33.5), and eleven other shapes within 2 us;
    // its start only fits the short passes' times (3 gave the same split for
    // all 14).  8-bit checkpoints take their tensors' type's turns: with turns
    // longer by a seventh, as their instructions are, nine shapes had the same
    // split.
    const Turn turn = sizeof(T) == 4 ? Turn{3.9, 0.85, 1.3, 0.2, 8.0} : Turn{1.95, 0.92, 0.45, 0.1, 3.0};
    const Split how = best_split(kern, kSmem, kWarps, kBlock, turn, Bs, p.L, p.ED, num_sms, places);
    if (how.err != cudaSuccess) return how.err;
    if (how.warps == 0) return cudaErrorInvalidConfiguration;
    *sums = how.first * how.cluster + (Bs - how.first) * how.rest_cluster;
    return start_split(kern, kSmem, how, Bs, p.ED, p, maps, st);
}

template <typename T, typename K>
static cudaError_t start(const BwdArgs<T> &p, int W, int64_t Bs, int num_sms, int64_t *sums, cudaStream_t st) {
    BwdMaps maps{};
    if (W == 16) {
        const K *in[3];
        if constexpr (sizeof(K) == 1)
            in[0] = p.kept.x_q, in[1] = p.kept.r_q, in[2] = p.kept.i_q;
        else
            in[0] = p.in[0], in[1] = p.in[1], in[2] = p.in[2];
        T *const out[3] = {p.dx, p.dr, p.di};
        for (int k = 0; k < 3; ++k)
            if (!rows_map(&maps.in[k], in[k], Bs, p.L, p.ED, kSteps) ||
                !rows_map(&maps.out[k], out[k], Bs, p.L, p.ED, kSteps))
                return cudaErrorInvalidValue;
        if (!rows_map(&maps.dy, p.dy, Bs, p.L, p.ED, kSteps)) return cudaErrorInvalidValue;
        return p.reset ? start<T, K, 16, true>(p, maps, Bs, num_sms, sums, st)
                       : start<T, K, 16, false>(p, maps, Bs, num_sms, sums, st);
    }
    if (W == 8) return p.reset ? start<T, K, 8, true>(p, maps, Bs, num_sms, sums, st)
                               : start<T, K, 8, false>(p, maps, Bs, num_sms, sums, st);
    return p.reset ? start<T, K, 1, true>(p, maps, Bs, num_sms, sums, st)
                       : start<T, K, 1, false>(p, maps, Bs, num_sms, sums, st);
}

template <typename T>
cudaError_t launch(const T *x, const T *gr, const T *gi, const float *lam, float c,
                   const uint8_t *reset, const T *dy, const float *dh_final, const Kept &kept, T *dx,
                   T *dr, T *di, float *dlam, float *dh0, float *scratch, int64_t Bs, int64_t L,
                   int64_t ED, int num_sms, cudaStream_t st) {
    auto at = [](const void *q) { return reinterpret_cast<uintptr_t>(q); };
    BwdArgs<T> p{{x, gr, gi}, lam, c, reset, dy, dh_final, kept, dx, dr, di, scratch, dh0,
                 int(L), int(ED), Bs * L, {}};
    int64_t sums = 0;
    int W = widest_copy<T>(at(dy), ED);
    if (W == 16 && (at(dx) | at(dr) | at(di)) % 16 != 0) W = 8;
    cudaError_t err;
    if (kept.x_q)
        err = start<T, int8_t>(p, std::min(W, widest_copy<int8_t>(at(kept.x_q) | at(kept.r_q) | at(kept.i_q), ED)), Bs, num_sms,
                               &sums, st);
    else
        err = start<T, T>(p, std::min(W, widest_copy<T>(at(x) | at(gr) | at(gi), ED)), Bs, num_sms,
                               &sums, st);
    if (err == cudaSuccess) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(unsigned((ED + 31) / 32));
        cfg.blockDim = dim3(32 * kSumWarps);
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        err = cudaLaunchKernelEx(&cfg, dlam_kernel, static_cast<const float *>(p.part), lam, dlam, sums, ED);
    }
    return err;
}

#define SSM_GATED_BWD_INSTANTIATE(T)                                                              \
    template cudaError_t launch<T>(const T *, const T *, const T *, const float *, float,         \
                                   const uint8_t *, const T *, const float *, const Kept &, T *,  \
                                   T *, T *, float *, float *, float *, int64_t, int64_t, int64_t, \
                                   int, cudaStream_t);
SSM_GATED_BWD_INSTANTIATE(float)
SSM_GATED_BWD_INSTANTIATE(__nv_bfloat16)

}  // namespace gated_bwd
}  // namespace ssm
