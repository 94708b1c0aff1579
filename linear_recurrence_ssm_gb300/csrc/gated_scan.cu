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

constexpr int kWarps = 8, kSteps = kBlock / kWarps, kThreads = 32 * kWarps;
constexpr int kStages = 3;
constexpr int kMaxCluster = 8;

// Bytes from one copied row of 64 channels to the next: words that start one
// element early (loads of 4 bytes of bf16 rows) need one word more.
template <typename T, int W>
constexpr int kPitch = 64 * int(sizeof(T)) + (W == 4 && sizeof(T) == 2 ? 16 : 0);
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

// Copies one warp's 8 rows of 64 channels from row0 on, of one tensor.  W is
// the widest copy that every row's start allows; 2 stands for plain loads of
// elements, which wait for their data.
template <typename T, int W>
__device__ __forceinline__ void copy_rows(uint8_t *to, const T *from, int64_t row0, int n_rows, int e0, int ED) {
    const int lane = threadIdx.x % 32;
    if constexpr (W == 16 || (W == 4 && sizeof(T) == 4)) {
        constexpr int kChunks = 64 * int(sizeof(T)) / W, kPer = W / int(sizeof(T));
#pragma unroll
        for (int i = 0; i < kSteps * kChunks / 32; ++i) {
            const int row = (i * 32 + lane) / kChunks, e = (i * 32 + lane) % kChunks * kPer;
            const bool in = row < n_rows && e0 + e < ED;
            const T *src = in ? from + (row0 + row) * ED + e0 + e : from;
            uint8_t *dst = to + row * kPitch<T, W> + e * int(sizeof(T));
            if constexpr (W == 16)
                cp_async16(dst, src, in ? 16 : 0);
            else
                cp_async4(dst, src, in ? 4 : 0);
        }
    } else if constexpr (W == 4) {
        // rows of an odd number of bf16: words from the one that holds the row's first element
#pragma unroll
        for (int row = 0; row < kSteps; ++row) {
            const int64_t first = (row0 + row) * ED + e0;
            const int64_t end = (row0 + row) * ED + ED;     // past the row's last element
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int word = lane + 32 * k;
                if (word > 32) continue;
                const int64_t e = (first & ~int64_t(1)) + 2 * word;
                const bool in = row < n_rows && e < end;
                // the tensor's last element may be the first half of its word
                const int bytes = !in ? 0 : (e + 1 < end ? 4 : 2);
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
                *reinterpret_cast<T *>(to + row * kPitch<T, W> + e * int(sizeof(T))) = v;
            }
    }
}

// The lane's two channels of a copied row.
template <typename T, int W>
__device__ __forceinline__ float2 pair_at(const uint8_t *row, uint32_t odd) {
    const int lane = threadIdx.x % 32;
    if constexpr (sizeof(T) == 4) return *reinterpret_cast<const float2 *>(row + 8 * lane);
    uint32_t w = *reinterpret_cast<const uint32_t *>(row + 4 * lane);
    if (W == 4 && odd) w = __funnelshift_r(w, *reinterpret_cast<const uint32_t *>(row + 4 * lane + 4), 16);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ void put2(float *p, float2 v) { *reinterpret_cast<float2 *>(p) = v; }
__device__ __forceinline__ void put2(__nv_bfloat16 *p, float2 v) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __float22bfloat162_rn(v);
}

struct Pieces {
    float4 warp[2][kWarps][32];              // A of two channels, H of two channels
    float4 block[2][kMaxCluster][32];        // written by the cluster's blocks
    uint32_t cuts[2][kWarps], block_cut[2][kMaxCluster];
};

// a_t and b_t of a warp's 8 steps, and their piece (A, H).  bit j of `cut`:
// step j drops the state before it.
template <typename T, int W, bool WIDE, bool CUT>
__device__ __forceinline__ void coefficients(const uint8_t *rows, uint32_t odd, float2 rate, uint32_t cut,
                                             float2 (&a)[kSteps], float2 (&b)[kSteps], float2 &A, float2 &H) {
    constexpr bool ACC = sizeof(T) == 4;
    A = both(1.0f);
    H = both(0.0f);
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
        const uint32_t o = odd >> j & 1;
        const float2 x = pair_at<T, W>(rows + j * kPitch<T, W>, o);
        const float2 sr = sigmoid2<ACC>(pair_at<T, W>(rows + (kSteps + j) * kPitch<T, W>, o));
        const float2 si = sigmoid2<ACC>(pair_at<T, W>(rows + (2 * kSteps + j) * kPitch<T, W>, o));
        float2 w;
        decay2<ACC, WIDE>(mul2(rate, sr), a[j], w);
        const float2 in = mul2(si, x);
        b[j] = mul2(root2<ACC>(one_minus_square(w)), in);
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
__device__ __forceinline__ void keep_8bit(const uint8_t *rows, uint32_t odd, const Kept &kept, int64_t row0,
                                          int n_rows, int e0, int ED, int64_t all_rows) {
    const int lane = threadIdx.x % 32;
    uint32_t mine = 0;
#pragma unroll
    for (int g = 0; g < 3 * kSteps; ++g) {
        const float2 v = pair_at<T, W>(rows + g * kPitch<T, W>, odd >> (g % kSteps) & 1);
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
        const float2 v = pair_at<T, W>(rows + g * kPitch<T, W>, odd >> j & 1);
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
        uint32_t cut = 0, odd = 0;
        if (RESET) {
            cut = __ballot_sync(0xffffffffu, next_cut != 0);
            next_cut = reset_of(turn + 1);
        }
        // which rows start in the second half of a word: all of them or none, or every second one
        if (sizeof(T) == 2 && W == 4) odd = (p.ED & 1) ? (row0 & 1 ? 0x55u : 0xaau) : 0u;

        if (SAVE8 && n > 0) keep_8bit<T, W>(rows, odd, p.kept, row0, n, e0, p.ED, p.rows);

        // steps behind the end leave their piece wrong; nothing after them reads it
        float2 a[kSteps], s[kSteps], A, H;
        if (wide || (RESET && cut))
            coefficients<T, W, true, RESET>(rows, odd, rate, cut, a, s, A, H);
        else
            coefficients<T, W, false, false>(rows, odd, rate, 0, a, s, A, H);
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
        if (p.pair_stores) {
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
                if (j < n && in0) put2(y + int64_t(j) * p.ED, s[j]);
        } else {
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
                if (j < n && in0) put(y + int64_t(j) * p.ED, s[j].x);
                if (j < n && in1) put(y + int64_t(j) * p.ED + 1, s[j].y);
            }
        }
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
    const float m = root2<ACC>(one_minus_square(w)).x;
    const float h = fmaf(a.x, states[page * ED + e], m * s.y * to_f32(x[at]));
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
    // Blocks of a cluster share the time axis: as many as fill the GPU with
    // two blocks an SM, none with less than two tiles.
    const int64_t chains = (ED + 63) / 64 * Bs, tiles = (L + kBlock - 1) / kBlock;
    while (p.cluster < kMaxCluster && chains * p.cluster * 2 <= 3 * num_sms && p.cluster * 2 <= tiles) p.cluster *= 2;
    const bool q_words = !kept.x_q || (reinterpret_cast<uintptr_t>(kept.x_q) | reinterpret_cast<uintptr_t>(kept.r_q) |
                                       reinterpret_cast<uintptr_t>(kept.i_q)) % 2 == 0;
    if (ED * int64_t(sizeof(T)) % 16 == 0 && in % 16 == 0 && q_words) return start_fwd<T, 16>(p, Bs, st);
    if (in % 4 == 0) return start_fwd<T, 4>(p, Bs, st);
    if constexpr (sizeof(T) == 2) return start_fwd<T, 2>(p, Bs, st);
    return cudaErrorInvalidValue;
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
