// gated_scan.cu -- the gated linear recurrence, forward and one token.
//
// h_t = a_t h_{t-1} + b_t is joined from pieces of the time axis: a piece is
// the map h -> A h + H with A the product of its decays and H its result from
// 0.  A warp owns 8 steps of 64 channels (two a lane) and keeps its a_t, b_t
// in registers; the eight warps of a block form a tile of 64 steps.  Their
// pieces meet in shared memory, every warp folds those before its own, and
// then runs its 8 steps again from the state that enters them -- one read of
// the inputs, one write of the outputs, and no state in between leaves the
// SM.  Blocks walk along the time axis; where the channels alone cannot fill
// the GPU, a cluster of blocks takes neighbouring tiles of a sequence at
// once and its blocks exchange their tiles' pieces through distributed
// shared memory.
//
// Each warp copies its own rows ahead of their use (cp.async, kStages tiles),
// so that loads need no barrier; one barrier a tile exchanges the pieces.
#include "gated_scan.cuh"

#include <algorithm>

namespace ssm {
namespace gated {

constexpr int kStages = 3;

template <typename T, int W>
constexpr int kStageBytes = 3 * kSteps * kPitch<T, W>;

template <typename T>
struct FwdArgs {
    const T *in[3];             // x, gate_r, gate_i
    const float *lam;
    float c;
    const uint8_t *reset;
    const float *h0;
    T *y;
    float *h_final;
    Kept kept;
    int L, ED, cluster;
    int64_t rows;               // Bs * L
    int pair_stores;            // y's rows take stores of two elements
};

struct Pieces {
    float4 warp[2][kWarps][32];              // A of two channels, H of two channels
    float4 block[2][kMaxCluster][32];        // written by the cluster's blocks
    uint32_t cuts[2][kWarps], block_cut[2][kMaxCluster];
};

// a_t and b_t of a warp's 8 steps, and their piece (A, H).  bit j of `cut`:
// step j drops the state before it.
template <typename T, int W, bool WIDE, bool CUT>
__device__ __forceinline__ void coefficients(const uint8_t *rows, int64_t row0, int ED, float2 rate, uint32_t cut,
                                             float2 (&a)[kSteps], float2 (&b)[kSteps], float2 &A, float2 &H) {
    constexpr bool ACC = sizeof(T) == 4;
    A = both(1.0f);
    H = both(0.0f);
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
        const uint32_t o = shift_of<T, W>(row0 + j, ED);
        const float2 x = pair_at<T, W>(rows + j * kPitch<T, W>, o);
        const float2 sr = sigmoid2<ACC>(pair_at<T, W>(rows + (kSteps + j) * kPitch<T, W>, o));
        const float2 si = sigmoid2<ACC>(pair_at<T, W>(rows + (2 * kSteps + j) * kPitch<T, W>, o));
        float2 w;
        decay2<ACC, WIDE>(mul2(rate, sr), a[j], w);
        const float2 in = mul2(si, x);
        const float2 v = one_minus_square(w);
        b[j] = mul2(mul2(v, rsqrt2<ACC>(v)), in);
        if (CUT && (cut >> j & 1)) {
            a[j] = both(0.0f);
            b[j] = in;
            A = both(0.0f);
            H = in;
        } else {
            A = mul2(A, a[j]);
            H = fma2(a[j], H, b[j]);
        }
    }
}

// Keeps a warp's 8 rows of the three tensors in 8 bits.  The tops of the 24
// groups end up one in each lane, so that the division is done once.
template <typename T, int W>
__device__ __forceinline__ void keep_8bit(const uint8_t *rows, const Kept &kept, int64_t row0,
                                          int n_rows, int e0, int ED, int64_t all_rows) {
    const int lane = threadIdx.x % 32;
    uint32_t mine = 0;
#pragma unroll
    for (int g = 0; g < 3 * kSteps; ++g) {
        const float2 v = pair_at<T, W>(rows + g * kPitch<T, W>, shift_of<T, W>(row0 + g % kSteps, ED));
        // the order of the bit patterns of |v| is that of the values, NaN on top
        const uint32_t top = __reduce_max_sync(0xffffffffu, max(__float_as_uint(v.x) & 0x7fffffffu,
                                                                __float_as_uint(v.y) & 0x7fffffffu));
        if (lane == g) mine = top;
    }
    const float top = __uint_as_float(mine), inv = inverse_of(top);
    if (lane < 3 * kSteps && lane % kSteps < n_rows) {
        float *s = lane < kSteps ? kept.x_s : lane < 2 * kSteps ? kept.r_s : kept.i_s;
        s[(e0 / kGroup) * all_rows + row0 + lane % kSteps] = scale_of(top);
    }
    const int e = e0 + 2 * lane;
#pragma unroll
    for (int g = 0; g < 3 * kSteps; ++g) {
        const int j = g % kSteps;
        const float2 v = pair_at<T, W>(rows + g * kPitch<T, W>, shift_of<T, W>(row0 + j, ED));
        const float k = __shfl_sync(0xffffffffu, inv, g);
        const uint32_t n0 = quantised(v.x, k), n1 = quantised(v.y, k);
        if (j < n_rows && e < ED) {
            int8_t *q = (g < kSteps ? kept.x_q : g < 2 * kSteps ? kept.r_q : kept.i_q) + (row0 + j) * ED + e;
            if (W == 16) {
                *reinterpret_cast<uint16_t *>(q) =
                    uint16_t(__byte_perm(n0, n1, 0x0040));
            } else {
                q[0] = int8_t(n0);
                if (e + 1 < ED) q[1] = int8_t(n1);
            }
        }
    }
}

template <typename T, int W, bool RESET, bool SAVE8>
__global__ void __launch_bounds__(kThreads)
gated_fwd_kernel(const __grid_constant__ FwdArgs<T> p) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ Pieces sh;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int C = p.cluster, rank = C > 1 ? int(cluster_rank()) : 0;
    const int e0 = int(blockIdx.x) / C * 64, e = e0 + 2 * lane;
    const int64_t b = blockIdx.y;
    const int tiles = (p.L + kBlock - 1) / kBlock, turns = (tiles + C - 1) / C;
    const bool in0 = e < p.ED, in1 = e + 1 < p.ED;

    uint8_t *mine = ring + warp * kStages * kStageBytes<T, W>;
    auto fetch = [&](int turn) {
        const int t = (turn * C + rank) * kBlock + warp * kSteps;
        const int n = min(kSteps, p.L - t);
        if (turn < turns && n > 0) {
            uint8_t *to = mine + turn % kStages * kStageBytes<T, W>;
#pragma unroll
            for (int k = 0; k < 3; ++k)
                copy_rows<T, W>(to + k * kSteps * kPitch<T, W>, p.in[k], b * p.L + t, n, e0, p.ED);
        }
        cp_async_commit();
    };
    auto reset_of = [&](int turn) -> uint32_t {
        const int t = (turn * C + rank) * kBlock + warp * kSteps + lane;
        return lane < kSteps && t < p.L && turn < turns ? p.reset[b * p.L + t] : 0;
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(k);
    if (C > 1) cluster_sync();     // every block runs before another writes to its shared memory
    uint32_t next_cut = RESET ? reset_of(0) : 0;

    const float2 rate = make_float2(in0 ? decay_rate(p.lam[e], p.c) : 0.0f, in1 ? decay_rate(p.lam[e + 1], p.c) : 0.0f);
    const bool wide = __any_sync(0xffffffffu, !(fmaxf(rate.x, rate.y) < kSlow));
    float2 carry = both(0.0f);     // the state that enters the cluster's next tiles
    if (p.h0) carry = make_float2(in0 ? p.h0[b * p.ED + e] : 0.0f, in1 ? p.h0[b * p.ED + e + 1] : 0.0f);

    for (int turn = 0; turn < turns; ++turn) {
        const int tile = turn * C + rank, t0 = tile * kBlock + warp * kSteps, buf = turn & 1;
        const int n = min(kSteps, p.L - t0);      // <= 0 behind the end
        const int64_t row0 = b * p.L + t0;
        fetch(turn + kStages - 1);
        cp_async_wait<kStages - 1>();
        __syncwarp();
        const uint8_t *rows = mine + turn % kStages * kStageBytes<T, W>;
        uint32_t cut = 0;
        if (RESET) {
            cut = __ballot_sync(0xffffffffu, next_cut != 0);
            next_cut = reset_of(turn + 1);
        }
        if (SAVE8 && n > 0) keep_8bit<T, W>(rows, p.kept, row0, n, e0, p.ED, p.rows);

        // steps behind the end leave their piece wrong; nothing after them reads it
        float2 a[kSteps], s[kSteps], A, H;
        if (wide || (RESET && cut))
            coefficients<T, W, true, RESET>(rows, row0, p.ED, rate, cut, a, s, A, H);
        else
            coefficients<T, W, false, false>(rows, row0, p.ED, rate, 0, a, s, A, H);
        __syncwarp();      // all lanes have read before any lane copies over these rows

        sh.warp[buf][warp][lane] = make_float4(A.x, A.y, H.x, H.y);
        if (RESET && lane == 0) sh.cuts[buf][warp] = cut;
        __syncthreads();

        // the pieces before this warp's in its block, and the whole block's
        float2 h = carry, all = carry;
        if (C == 1) {
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                if (k == warp) h = all;
                const float4 v = sh.warp[buf][k][lane];
                const bool dropped = RESET && sh.cuts[buf][k];
                const float2 on = fma2(make_float2(v.x, v.y), all, make_float2(v.z, v.w));
                all = dropped ? make_float2(v.z, v.w) : on;
            }
        } else {
            float2 A0 = both(1.0f), H0 = both(0.0f), A1 = A0, H1 = H0;
            uint32_t cut0 = 0, cut1 = 0;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                if (k == warp) A0 = A1, H0 = H1, cut0 = cut1;
                const float4 v = sh.warp[buf][k][lane];
                const bool dropped = RESET && sh.cuts[buf][k];
                const float2 on = fma2(make_float2(v.x, v.y), H1, make_float2(v.z, v.w));
                A1 = mul2(A1, make_float2(v.x, v.y));
                H1 = dropped ? make_float2(v.z, v.w) : on;
                if (RESET) cut1 |= sh.cuts[buf][k];
            }
            if (warp < C) {
                put_remote(&sh.block[buf][rank][lane], warp, make_float4(A1.x, A1.y, H1.x, H1.y));
                if (RESET && lane == 0) put_remote_u32(&sh.block_cut[buf][rank], warp, cut1);
            }
            cluster_sync();
            for (int k = 0; k < C; ++k) {
                if (k == rank) h = all;
                const float4 v = sh.block[buf][k][lane];
                const bool dropped = RESET && sh.block_cut[buf][k];
                const float2 on = fma2(make_float2(v.x, v.y), all, make_float2(v.z, v.w));
                all = dropped ? make_float2(v.z, v.w) : on;
            }
            if (p.kept.states && warp == 0 && tile < tiles) carry = h;      // entering the tile
            const float2 on = fma2(A0, h, H0);
            h = RESET && cut0 ? H0 : on;
        }
        if (p.kept.states && warp == 0 && tile < tiles) {
            float *k = p.kept.states + (b * tiles + tile) * p.ED + e;
            if (in0) k[0] = carry.x;
            if (in1) k[1] = carry.y;
        }
        carry = all;

#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            const float2 on = fma2(a[j], h, s[j]);
            h = RESET && (cut >> j & 1) ? s[j] : on;
            s[j] = h;
        }
        T *y = p.y + row0 * p.ED + e;
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
            if (j < n) put_pair(y + int64_t(j) * p.ED, s[j], p.pair_stores, in0, in1);
        if (p.h_final) {
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
                if (t0 + j == p.L - 1) {
                    if (in0) p.h_final[b * p.ED + e] = s[j].x;
                    if (in1) p.h_final[b * p.ED + e + 1] = s[j].y;
                }
        }
    }
    cp_async_wait<0>();
    if (C > 1) cluster_sync();     // no block leaves while another may still write to it
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
    const float2 s = sigmoid2<ACC>(make_float2(to_f32(gr[at]), to_f32(gi[at])));
    float2 a, w;
    decay2<ACC, true>(both(decay_rate(lam[e], c) * s.x), a, w);
    const float2 v = one_minus_square(w);
    const float h = fmaf(a.x, states[page * ED + e], v.x * rsqrt2<ACC>(v).x * s.y * to_f32(x[at]));
    states[page * ED + e] = h;
    put(y + at, h);
}

template <typename T, int W, bool RESET, bool SAVE8>
static cudaError_t start_fwd(const FwdArgs<T> &p, int64_t Bs, cudaStream_t st) {
    auto kern = gated_fwd_kernel<T, W, RESET, SAVE8>;
    const int smem = kWarps * kStages * kStageBytes<T, W>;
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

template <typename T, int W>
static cudaError_t start_fwd(const FwdArgs<T> &p, int64_t Bs, cudaStream_t st) {
    if (p.kept.x_q) return p.reset ? start_fwd<T, W, true, true>(p, Bs, st) : start_fwd<T, W, false, true>(p, Bs, st);
    return p.reset ? start_fwd<T, W, true, false>(p, Bs, st) : start_fwd<T, W, false, false>(p, Bs, st);
}

template <typename T>
cudaError_t launch_fwd(const T *x, const T *gr, const T *gi, const float *lam, float c,
                       const uint8_t *reset, const float *h0, T *y, float *h_final,
                       const Kept &kept, int64_t Bs, int64_t L, int64_t ED, int num_sms,
                       cudaStream_t st) {
    FwdArgs<T> p{{x, gr, gi}, lam, c, reset, h0, y, h_final, kept, int(L), int(ED), 1, Bs * L, 0};
    const uintptr_t in = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(gr) |
                         reinterpret_cast<uintptr_t>(gi);
    p.pair_stores = ED % 2 == 0 && reinterpret_cast<uintptr_t>(y) % (2 * sizeof(T)) == 0;
    p.cluster = cluster_for(Bs, L, ED, num_sms);
    const uintptr_t q = reinterpret_cast<uintptr_t>(kept.x_q) | reinterpret_cast<uintptr_t>(kept.r_q) |
                        reinterpret_cast<uintptr_t>(kept.i_q);
    const int W = widest_copy<T>(in, ED);
    if (W == 16 && q % 2 == 0) return start_fwd<T, 16>(p, Bs, st);
    if (W >= 4) return start_fwd<T, 4>(p, Bs, st);
    if constexpr (sizeof(T) == 2) return start_fwd<T, 1>(p, Bs, st);
    return cudaErrorInvalidValue;      // fp32 is aligned to its 4 bytes
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
