// gated_scan.cu -- the gated linear recurrence, forward and one token.
//
// h_t = a_t h_{t-1} + b_t is joined from pieces of the time axis: a piece is
// the map h -> A h + H with A the product of its decays and H its result from
// 0.  A warp owns 16 steps of 64 channels (two a lane) and keeps its a_t, b_t
// in registers; the 4 or 8 warps of a block form a tile.  Their pieces meet in
// shared memory, every warp folds those before its own, and then runs its
// steps again from the state that enters them -- one read of the inputs, one
// write of the outputs, and no state in between leaves the SM.  Blocks walk
// along the time axis; where the channels alone cannot fill the GPU, a cluster
// of blocks takes neighbouring tiles of a sequence at once and its blocks
// exchange their tiles' pieces through distributed shared memory.
//
// Each warp copies its own rows ahead of their use (tensor copies of 16 x 64
// boxes where rows are multiples of 16 bytes), so that loads need no block
// barrier, and stores its outputs as a box from the place of x's rows; one
// barrier a tile exchanges the pieces.
//
// An element costs 8 bytes (bf16) and 3 exponentials' worth of special
// functions, so that bytes, instruction issue and the special-function unit
// lie close together.  What carried it, at Bs=8 L=2048 ED=1536 (bytes: 30 us):
// one thread a channel 1386 us; tiles joined in shared memory 85; pieces sent
// by asynchronous stores instead of cluster barriers 60; boxes and 16 steps a
// warp 48; all four blocks on an SM and clusters of three 43; one root for the
// gate and the input's factor 41 (4.9 TB/s, 73 % of the measured copy rate).
// What is left: 576 blocks of 608 places, a start of 3 us and issue slots
// (997 instructions for 16 steps of 64 channels, 3.5 warps a scheduler).
// More chains than fit at a time, Bs=16 L=1000 ED=2560 (bytes: 49 us): 68 us
// in whole rounds, 62 with the last sequence in clusters of four; with the
// 8-bit checkpoint (bytes: 68 us) 111, 91 and, read in 16-byte pieces, 84.
// Bs=1 L=65536 ED=2560 with resets: 312 us for 198 us of bytes; 40 chains fill
// 10.5 of 16 warps an SM, more blocks a cluster wait for a second round.
#include "gated_scan.cuh"

#include <algorithm>

namespace ssm {
namespace gated {

constexpr int kSteps = 16;
// Tiles of a warp's rows in flight or in use.  With fp32 one, so that four
// blocks of 4 warps fit an SM instead of two; they wait for copies in turn.
template <typename T>
constexpr int kStages = sizeof(T) == 4 ? 1 : 2;

__device__ unsigned int g_device_error;

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
    int L, ED;
    int64_t rows;               // Bs * L
    float one;                  // 1
    Share share;
};

// Boxes of 64 channels x kSteps rows of x, gate_r, gate_i, y and the three
// checkpoints (W = 16).
struct FwdMaps {
    CUtensorMap in[3], y, q[3];
};

// Behind the ring in shared memory; the pieces of ex follow.
template <int WARPS>
struct Shared {
    float4 warp[2][WARPS][32];     // A of two channels, H of two channels
    uint64_t full[WARPS][2];       // a warp's copies have arrived (W = 16)
    float tops[WARPS][3 * kSteps]; // of the 8-bit groups
    Exchange ex;
};

// a_t and b_t of a warp's steps, and their piece (A, H).  bit j of `cut`:
// step j drops the state before it.
//
// Special functions bound this as much as instructions do (a reciprocal or
// root takes the unit twice as long as an exponential).  With bf16 tensors and
// slow decays r = (1 + e^-gate_r)^(-1/2) gives both s_r = r^2 and m =
// (c softplus(lam))^(1/2) r (1 - a^2)^(1/2) / (-la)^(1/2), whose last factor is
// smooth: one root instead of a reciprocal and a root.
template <typename T, int W, bool WIDE, bool CUT>
__device__ __forceinline__ void coefficients(const uint8_t *rows, int64_t row0, int ED, float2 rate, float2 root_rate,
                                             uint32_t cut, float2 (&a)[kSteps], float2 (&b)[kSteps], float2 &A,
                                             float2 &H) {
    constexpr bool ACC = sizeof(T) == 4;
    A = both(1.0f);
    H = both(0.0f);
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
        const uint32_t o = shift_of<T, W>(row0 + j, ED);
        const float2 gr = pair_at<T, W>(rows + (kSteps + j) * kPitch<T, W>, o);
        const float2 nsi = nsigmoid2<ACC>(pair_at<T, W>(rows + (2 * kSteps + j) * kPitch<T, W>, o));
        const float2 nin = mul2(nsi, pair_at<T, W>(rows + j * kPitch<T, W>, o));
        float2 em;
        if constexpr (ACC || WIDE) {
            decay2<ACC, WIDE>(mul2(rate, nsigmoid2<ACC>(gr)), a[j], em);
            const float2 v = square_less_one(a[j], em);
            b[j] = mul2(mul2(v, rsqrt_of_minus<ACC>(v)), nin);
        } else {
            const float2 s = mul2(gr, both(-SSM_LOG2E));
            const float2 d = add2(make_float2(ex2(s.x), ex2(s.y)), both(1.0f));
            const float2 u = mul2(root_rate, make_float2(rsqrt_fast(d.x), rsqrt_fast(d.y)));   // -(-la)^(1/2)
            const float2 la = mul2(u, mul2(u, both(-1.0f)));
            decay2<ACC, WIDE>(la, a[j], em);
            b[j] = mul2(mul2(u, slow_root(la)), nin);
        }
        if (CUT && (cut >> j & 1)) {
            a[j] = both(0.0f);
            b[j] = mul2(nin, both(-1.0f));
            H = b[j];
        } else {
            A = mul2(A, a[j]);
            H = fma2(a[j], H, b[j]);
        }
    }
    if (CUT && cut) A = both(-0.0f);      // here, since a NaN gate behind the drop would make it NaN
}

// The largest of N values over lanes that differ in the bits below 2 * BIT, to
// three values a lane: while there are more, a lane passes half of them on and
// keeps the other half, from `first` on.  u16x2 or u32, by type.
template <typename T>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    if (sizeof(T) == 4) return max(a, b);
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <typename T, int N, int BIT>
__device__ __forceinline__ void largest(uint32_t *v, int &first) {
    if constexpr (BIT > 0) {
        constexpr int kKeep = N > 3 ? N / 2 : N;
        const bool high = threadIdx.x & BIT;
#pragma unroll
        for (int n = 0; n < kKeep; ++n) {
            const uint32_t own = N > 3 && high ? v[n + kKeep] : v[n], pass = N > 3 && !high ? v[n + kKeep] : v[n];
            v[n] = larger<T>(own, __shfl_xor_sync(0xffffffffu, pass, BIT));
        }
        if (N > 3 && high) first += kKeep;
        largest<T, kKeep, BIT / 2>(v, first);
    }
}

// Where the bytes of x, gate_r and gate_i (k = 0, 1, 2) wait as boxes of 64 a
// row, in the place of rows that are not needed any more: gate_i's and
// gate_r's in gate_i's rows, x's in gate_r's (x's own rows will hold y).
template <typename T>
__device__ __forceinline__ uint8_t *box_8bit(uint8_t *rows, int k) {
    constexpr int kIn = kSteps * kPitch<T, 16>;
    return k == 0 ? rows + kIn : k == 1 ? rows + 2 * kIn + 64 * kSteps : rows + 2 * kIn;
}

// Keeps a warp's rows of x, gate_r and gate_i in 8 bits.  The tops of its 3
// kSteps groups go through `tops`, so that one lane divides by each, once.
// Rows that are boxes are read in 16-byte pieces, 8 or 16 lanes a row, and the
// bytes go to boxes; others are read two channels a lane, and the bytes go to
// global memory.  At Bs=16 L=1000 ED=2560, two channels a lane and a warp's
// reduction for each of the 48 tops made it 91 us, pieces make it 84.
template <typename T, int W>
__device__ __forceinline__ void keep_8bit(uint8_t *rows, float *tops, const Kept &kept, int64_t row0, int n_rows,
                                          int e0, int ED, int64_t all_rows, float one) {
    const int lane = threadIdx.x % 32, e = e0 + first_channel<W>();
    constexpr int kLanes = 64 * int(sizeof(T)) / 16, kRows = 32 / kLanes;      // of a row; of one load
    auto piece = [&](int i) { return *reinterpret_cast<const uint4 *>(rows + 512 * i + 16 * lane); };
    auto value = [&](int g) {
        return pair_at<T, W>(rows + g * kPitch<T, W>, shift_of<T, W>(row0 + g % kSteps, ED));
    };
    // the order of the bit patterns of |v| is that of the values, NaN on top
    if constexpr (W == 16) {
        constexpr int kLoads = 3 * kSteps / kRows, kValues = sizeof(T) == 4 ? kLoads : kLoads / 2;
        constexpr uint32_t kAbs = sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu;
        uint32_t v[kValues];
        auto top_of = [&](int i) {
            const uint4 w = piece(i);
            return larger<T>(larger<T>(w.x & kAbs, w.y & kAbs), larger<T>(w.z & kAbs, w.w & kAbs));
        };
#pragma unroll
        for (int i = 0; i < kValues; ++i) {
            if (sizeof(T) == 4) {
                v[i] = top_of(i);
            } else {      // those of two loads in the halves of a word
                const uint32_t a = top_of(2 * i), b = top_of(2 * i + 1);
                v[i] = larger<T>(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
            }
        }
        int first = 0;
        largest<T, kValues, kLanes / 2>(v, first);
        constexpr int kEqual = sizeof(T) == 4 ? 2 : 4;      // lanes with the same three values
#pragma unroll
        for (int n = 0; n < 3; ++n) {
            if (lane % kEqual != n % kEqual) continue;
            if (sizeof(T) == 4) {
                tops[(first + n) * kRows + lane / kLanes] = __uint_as_float(v[n]);
            } else {
                float *to = tops + 2 * (first + n) * kRows + lane / kLanes;
                to[0] = __uint_as_float(v[n] << 16);
                to[kRows] = __uint_as_float(v[n] & 0xffff0000u);
            }
        }
    } else {
#pragma unroll 1
        for (int g = 0; g < 3 * kSteps; g += 4) {      // four at a time, for their latency
            float4 top;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = value(g + i);
                float m;
                asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(fabsf(v.x)), "f"(fabsf(v.y)));
                (&top.x)[i] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
            }
            if (lane == 0) *reinterpret_cast<float4 *>(tops + g) = top;
        }
    }
    __syncwarp();
#pragma unroll
    for (int g = lane; g < 3 * kSteps; g += 32) {
        const float top = tops[g];
        float *s = g < kSteps ? kept.x_s : g < 2 * kSteps ? kept.r_s : kept.i_s;
        if (g % kSteps < n_rows) s[(e0 / kGroup) * all_rows + row0 + g % kSteps] = scale_of(top);
        tops[g] = inverse_of(top);
    }
    __syncwarp();
    // x inv rounded, then to an integer (ties to even) by the addition of
    // 1.5 2^23: as a multiply-add with a 1 that the compiler does not know, so
    // that it cannot join it to the product
    auto quantised2 = [&](float2 v, float inv) {
        const float2 n = fma2(mul2(v, both(inv)), both(one), both(12582912.0f));
        return __byte_perm(__float_as_uint(n.x), __float_as_uint(n.y), 0x0040);
    };
    if constexpr (W == 16) {
        constexpr int kLoads = kSteps / kRows;
#pragma unroll
        for (int k = 2; k >= 0; --k) {
            uint8_t *box = box_8bit<T>(rows, k);
#pragma unroll
            for (int i = 0; i < kLoads; i += 2) {
                uint32_t q[2][2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint4 w = piece(k * kLoads + i + j);
                    const float inv = tops[k * kSteps + (i + j) * kRows + lane / kLanes];
                    if constexpr (sizeof(T) == 4) {
                        auto two = [&](uint32_t a, uint32_t b) {
                            return quantised2(make_float2(__uint_as_float(a), __uint_as_float(b)), inv);
                        };
                        q[j][0] = __byte_perm(two(w.x, w.y), two(w.z, w.w), 0x5410);
                    } else {
                        auto two = [&](uint32_t a) {
                            return quantised2(make_float2(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u)), inv);
                        };
                        q[j][0] = __byte_perm(two(w.x), two(w.y), 0x5410);
                        q[j][1] = __byte_perm(two(w.z), two(w.w), 0x5410);
                    }
                }
                __syncwarp();      // a load's bytes lie over the same load's rows or earlier ones'
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint8_t *to = box + 64 * kRows * (i + j);
                    if (sizeof(T) == 4)
                        *reinterpret_cast<uint32_t *>(to + 4 * lane) = q[j][0];
                    else
                        *reinterpret_cast<uint2 *>(to + 8 * lane) = make_uint2(q[j][0], q[j][1]);
                }
            }
        }
    } else {
#pragma unroll 1
        for (int k = 0; k < 3; ++k) {
            int8_t *q = (k == 0 ? kept.x_q : k == 1 ? kept.r_q : kept.i_q) + row0 * ED + e;
#pragma unroll 1
            for (int j = 0; j < kSteps; j += 4) {
                const float4 inv = *reinterpret_cast<const float4 *>(tops + k * kSteps + j);
                uint32_t n[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) n[i] = quantised2(value(k * kSteps + j + i), (&inv.x)[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i, q += ED) {
                    if (j + i < n_rows && e < ED) q[0] = int8_t(n[i]);
                    if (j + i < n_rows && e + kNext<W> < ED) q[kNext<W>] = int8_t(n[i] >> 8);
                }
            }
        }
    }
}

template <typename T, int W, int WARPS, bool RESET, bool SAVE8>
__global__ void __launch_bounds__(32 * WARPS, 16 / WARPS)
gated_fwd_kernel(const __grid_constant__ FwdArgs<T> p, const __grid_constant__ FwdMaps maps) {
    constexpr int kTile = WARPS * kSteps, kDepth = kStages<T>;
    extern __shared__ __align__(128) uint8_t ring[];
    Shared<WARPS> &sh = *reinterpret_cast<Shared<WARPS> *>(ring + WARPS * kDepth * kStageBytes<T, W>);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int C = p.share.cluster, rank = C > 1 ? int(cluster_rank()) : 0;
    const int e0 = int(blockIdx.x) / C * 64, e = e0 + first_channel<W>();
    const int64_t b = p.share.first + blockIdx.y;
    const int turns = (p.L + kTile * C - 1) / (kTile * C);
    const bool in0 = e < p.ED, in1 = e + kNext<W> < p.ED;

    uint8_t *mine = ring + warp * kDepth * kStageBytes<T, W>;
    if (p.share.order == 1) let_next_start();
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
        clear_ring(mine, kDepth * kStageBytes<T, W>);
    }
    __syncthreads();

    auto fetch = [&](int turn) {
        const int t = (turn * C + rank) * kTile + warp * kSteps;
        const int n = min(kSteps, p.L - t);
        uint8_t *to = mine + turn % kDepth * kStageBytes<T, W>;
        if constexpr (W == 16) {
            if (lane == 0 && turn < turns && n > 0 && !aborted(&sh.ex.abort)) {
                uint64_t *bar = &sh.full[warp][turn % kDepth];
                tc::mbar_arrive_expect_tx(bar, uint32_t(kStageBytes<T, W>));
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    tc::tma_load_3d(to + k * kSteps * kPitch<T, W>, &maps.in[k], bar, e0, t, int(b));
            }
        } else {
            if (turn < turns && n > 0) {
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    copy_rows<T, W, kSteps>(to + k * kSteps * kPitch<T, W>, p.in[k], b * p.L + t, n, e0, p.ED);
            }
            cp_async_commit();
        }
    };
    auto reset_of = [&](int turn) -> uint32_t {
        const int t = (turn * C + rank) * kTile + warp * kSteps + lane;
        return lane < kSteps && t < p.L && turn < turns ? p.reset[b * p.L + t] : 0;
    };
#pragma unroll
    for (int k = 0; k < (kDepth > 1 ? kDepth - 1 : 1); ++k) fetch(k);
    uint32_t next_cut = RESET ? reset_of(0) : 0;

    const float2 rate = make_float2(in0 ? decay_rate(p.lam[e], p.c) : 0.0f,
                                    in1 ? decay_rate(p.lam[e + kNext<W>], p.c) : 0.0f);
    const bool wide = __any_sync(0xffffffffu, !(fmaxf(rate.x, rate.y) < kSlow));
    const float2 root_rate = make_float2(-sqrtf(rate.x), -sqrtf(rate.y));
    float2 carry = both(0.0f);     // the state that enters the cluster's next tiles
    if (p.h0) carry = get_pair<W>(p.h0 + b * p.ED + e, in0, in1);
    if (C > 1) cluster_sync();     // every block runs before another writes to its shared memory

    for (int turn = 0; turn < turns; ++turn) {
        const int t0 = (turn * C + rank) * kTile + warp * kSteps, buf = turn & 1;
        const int n = min(kSteps, p.L - t0);      // <= 0 behind the end
        const int64_t row0 = b * p.L + t0;
        uint8_t *rows = mine + turn % kDepth * kStageBytes<T, W>;
        if constexpr (W == 16) {
            if (n > 0) wait_or_abort(&sh.full[warp][turn % kDepth], turn / kDepth & 1, &sh.ex.abort, &g_device_error);
        } else {
            cp_async_wait<(kDepth > 1 ? kDepth - 2 : 0)>();
            __syncwarp();
        }
        uint32_t cut = 0;
        if (RESET) {
            cut = __ballot_sync(0xffffffffu, next_cut != 0);
            next_cut = reset_of(turn + 1);
        }
        // steps behind the end leave their piece wrong; nothing after them reads it
        float2 a[kSteps], s[kSteps], A, H;
        if (wide || (RESET && cut))
            coefficients<T, W, true, RESET>(rows, row0, p.ED, rate, root_rate, cut, a, s, A, H);
        else
            coefficients<T, W, false, false>(rows, row0, p.ED, rate, root_rate, 0, a, s, A, H);
        sh.warp[buf][warp][lane] = make_float4(A.x, A.y, H.x, H.y);
        if (kDepth > 1) {
            // the stage that the next rows go to was read, and its outputs stored from, a turn ago
            if (W == 16 && lane == 0) tc::bulk_wait_read0();
            __syncwarp();
            fetch(turn + kDepth - 1);
        }
        __syncthreads();

        auto keep = [&] {
            if (!SAVE8 || n <= 0) return;
            keep_8bit<T, W>(rows, sh.tops[warp], p.kept, row0, n, e0, p.ED, p.rows, p.one);
            if (W == 16) {
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    for (int k = 0; k < 3; ++k) tma_store_3d(&maps.q[k], box_8bit<T>(rows, k), e0, t0, int(b));
                    tc::bulk_commit();
                }
            }
        };
        // The state that enters this warp's steps: the pieces before its own,
        // in its block (from 0 with their product where blocks form a cluster),
        // then in the blocks before.
        float2 h = carry, all = carry;
        if (C == 1) {
            keep();
#pragma unroll
            for (int k = 0; k < WARPS; ++k) {
                if (k == warp) h = all;
                all = after<RESET>(sh.warp[buf][k][lane], all);
            }
        } else {
            float4 before = make_float4(1.0f, 1.0f, 0.0f, 0.0f), sum = before;
#pragma unroll
            for (int k = 0; k < WARPS; ++k) {
                if (k == warp) before = sum;
                sum = joined<RESET>(sum, sh.warp[buf][k][lane]);
            }
            if (threadIdx.x == 0) sh.ex.expect(buf, C);
            for (int k = warp; k < C; k += WARPS)
                if (k != rank) sh.ex.send(buf, C, rank, k, sum);
            keep();      // while the pieces travel
            sh.ex.wait(buf, turn >> 1 & 1, &g_device_error);
            for (int k = 0; k < rank; ++k) all = after<RESET>(sh.ex.piece(buf, C, rank, k)[lane], all);
            h = all;
            all = after<RESET>(sum, all);
            for (int k = rank + 1; k < C; ++k) all = after<RESET>(sh.ex.piece(buf, C, rank, k)[lane], all);
            h = after<RESET>(before, h);
        }
        carry = all;
        if (p.kept.states && n > 0 && t0 % kBlock == 0) {
            put_pair<W>(p.kept.states + (b * ((p.L + kBlock - 1) / kBlock) + t0 / kBlock) * p.ED + e, h, in0, in1);
        }

#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            const float2 on = fma2(a[j], h, s[j]);
            h = RESET && (cut >> j & 1) ? s[j] : on;
            s[j] = h;
        }
        if constexpr (W == 16) {
            // over the lane's own elements of x, and from there as one box
#pragma unroll
            for (int j = 0; j < kSteps; ++j) put2(reinterpret_cast<T *>(rows + j * kPitch<T, W>) + 2 * lane, s[j]);
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && n > 0) {
                tma_store_3d(&maps.y, rows, e0, t0, int(b));
                tc::bulk_commit();
            }
        } else {
            T *y = p.y + row0 * p.ED + e;
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
                if (j < n) put_pair<W>(y + int64_t(j) * p.ED, s[j], in0, in1);
        }
        if (kDepth == 1) {
            if (W == 16 && lane == 0) tc::bulk_wait_read0();
            __syncwarp();
            fetch(turn + 1);
        }
        if (p.h_final && t0 < p.L && t0 + kSteps >= p.L) {
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
                if (t0 + j == p.L - 1) put_pair<W>(p.h_final + b * p.ED + e, s[j], in0, in1);
        }
    }
    if (W == 16) {
        if (lane == 0) tc::bulk_wait_read0();
    } else {
        cp_async_wait<0>();
    }
    if (C > 1) cluster_sync();     // no block leaves while another may still write to it
    if (aborted(&sh.ex.abort)) linger();
    wait_for_first(p.share);
}

// One token.  A thread takes two channels of kStepRows rows, so that a
// channel's decay rate is computed once for them and their loads are in
// flight together; bound by latency (page number, then state) up to some
// hundred rows.  With 2560 channels and the start of a launch, bf16: 256 rows
// 10 us, 1024 18 us (bytes: 6), 16384 166 us (bytes: 99); fp32: 1024 16 us
// (bytes: 9), 16384 150 us (bytes: 148).  PAIRS: rows start on pairs of elements.
constexpr int kStepRows = 4, kStepThreads = 128;
__device__ __forceinline__ float2 get2(const float *p) { return *reinterpret_cast<const float2 *>(p); }
__device__ __forceinline__ float2 get2(const __nv_bfloat16 *p) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(p));
}
template <typename T, bool PAIRS>
__global__ void __launch_bounds__(kStepThreads)
gated_step_kernel(const T *__restrict__ x, const T *__restrict__ gr, const T *__restrict__ gi,
                  const float *__restrict__ lam, float c, float *__restrict__ states,
                  const int32_t *__restrict__ pages, T *__restrict__ y, int64_t Bs, int64_t ED, int64_t num_pages) {
    constexpr bool ACC = sizeof(T) == 4;
    const int64_t e = (int64_t(blockIdx.x) * kStepThreads + threadIdx.x) * 2, b0 = int64_t(blockIdx.y) * kStepRows;
    if (e >= ED) return;
    const bool in1 = PAIRS || e + 1 < ED;
    auto get = [&](const auto *p) { return PAIRS ? get2(p) : make_float2(to_f32(p[0]), in1 ? to_f32(p[1]) : 0.0f); };
    auto set = [&](auto *p, float2 v) {
        if (PAIRS) {
            put2(p, v);
        } else {
            put(p, v.x);
            if (in1) put(p + 1, v.y);
        }
    };
    float2 v[kStepRows], r[kStepRows], i[kStepRows], h[kStepRows];
    int64_t at[kStepRows];      // of the state; -1: an idle row, -2: no row
#pragma unroll
    for (int k = 0; k < kStepRows; ++k) {
        at[k] = -2;
        if (b0 + k >= Bs) continue;
        const int64_t page = pages ? pages[b0 + k] : b0 + k;
        at[k] = page >= 0 && page < num_pages ? page * ED + e : -1;
        const int64_t in = (b0 + k) * ED + e;
        v[k] = get(x + in), r[k] = get(gr + in), i[k] = get(gi + in);
    }
#pragma unroll
    for (int k = 0; k < kStepRows; ++k) h[k] = at[k] >= 0 ? get(states + at[k]) : both(0.0f);
    const float2 rate = make_float2(decay_rate(lam[e], c), in1 ? decay_rate(lam[e + 1], c) : 0.0f);
#pragma unroll
    for (int k = 0; k < kStepRows; ++k) {
        if (at[k] == -2) continue;
        float2 out = both(0.0f);
        if (at[k] >= 0) {
            float2 a, em;
            decay2<ACC, true>(mul2(rate, nsigmoid2<ACC>(r[k])), a, em);
            const float2 q = square_less_one(a, em);
            out = fma2(a, h[k], mul2(mul2(q, rsqrt_of_minus<ACC>(q)), mul2(nsigmoid2<ACC>(i[k]), v[k])));
            set(states + at[k], out);
        }
        set(y + (b0 + k) * ED + e, out);
    }
}

template <typename T, int W, int WARPS>
constexpr int kSmem = WARPS * kStages<T> * kStageBytes<T, W> + int(sizeof(Shared<WARPS>));

// The split goes by the sizes and the type alone (the plain kernel's measured
// turns), so that y is the same, bit for bit, whatever is kept.  (A reset sends
// all 16 steps of its warp through the general form of the coefficients, so
// that steps beside it may differ in their last bits from those without it.)
// Rows off 16 bytes take the split counted for boxes as well, although their
// wider pitch lets fewer blocks on an SM: in bf16 three of 4 warps instead of
// four, one of 8 instead of two, so part of a counted round waits for another.
template <typename T>
static Split split_for(int64_t Bs, int64_t L, int64_t ED, int num_sms) {
    static Places places4, places8;
    const double by = sizeof(T) == 4 ? 2.0 : 1.0;
    const Turn of4{1.5 * by, 0.39 * by, 0.3, 0.05, 3.0}, of8{2.0 * by, 0.85 * by, 0.3, 0.1, 3.0};
    const Split with4 = best_split(gated_fwd_kernel<T, 16, 4, false, false>, kSmem<T, 16, 4>, 4, 64, of4, Bs, L, ED,
                                   num_sms, places4);
    const Split with8 = best_split(gated_fwd_kernel<T, 16, 8, false, false>, kSmem<T, 16, 8>, 8, 128, of8, Bs, L, ED,
                                   num_sms, places8);
    if (with4.err != cudaSuccess || with8.err != cudaSuccess) return with4.err != cudaSuccess ? with4 : with8;
    return with8.warps != 0 && (with4.warps == 0 || with8.us < with4.us) ? with8 : with4;
}

template <typename T, int W, bool RESET, bool SAVE8>
static cudaError_t start_fwd(const FwdArgs<T> &p, const FwdMaps &maps, int64_t Bs, int num_sms, cudaStream_t st) {
    static_assert(kSmem<T, W, 4> + exchange_bytes(kMaxCluster) <= 227 * 1024 &&
                      kSmem<T, W, 8> + exchange_bytes(kMaxCluster) <= 227 * 1024,
                  "shared memory of one block exceeds 227 KB");
    const Split how = split_for<T>(Bs, p.L, p.ED, num_sms);
    if (how.err != cudaSuccess) return how.err;
    if (how.warps == 0) return cudaErrorInvalidConfiguration;
    if (how.warps == 8)
        return start_split(gated_fwd_kernel<T, W, 8, RESET, SAVE8>, kSmem<T, W, 8>, how, Bs, p.ED, p, maps, st);
    return start_split(gated_fwd_kernel<T, W, 4, RESET, SAVE8>, kSmem<T, W, 4>, how, Bs, p.ED, p, maps, st);
}

template <typename T, int W>
static cudaError_t start_fwd(const FwdArgs<T> &p, int64_t Bs, int num_sms, cudaStream_t st) {
    FwdMaps maps{};
    if (W == 16) {
        for (int k = 0; k < 3; ++k)
            if (!rows_map(&maps.in[k], p.in[k], Bs, p.L, p.ED, kSteps)) return cudaErrorInvalidValue;
        if (!rows_map(&maps.y, p.y, Bs, p.L, p.ED, kSteps)) return cudaErrorInvalidValue;
        int8_t *const q[3] = {p.kept.x_q, p.kept.r_q, p.kept.i_q};
        for (int k = 0; k < 3 && q[0]; ++k)
            if (!rows_map(&maps.q[k], q[k], Bs, p.L, p.ED, kSteps)) return cudaErrorInvalidValue;
    }
    if (p.kept.x_q)
        return p.reset ? start_fwd<T, W, true, true>(p, maps, Bs, num_sms, st)
                       : start_fwd<T, W, false, true>(p, maps, Bs, num_sms, st);
    return p.reset ? start_fwd<T, W, true, false>(p, maps, Bs, num_sms, st)
                   : start_fwd<T, W, false, false>(p, maps, Bs, num_sms, st);
}

template <typename T>
cudaError_t launch_fwd(const T *x, const T *gr, const T *gi, const float *lam, float c,
                       const uint8_t *reset, const float *h0, T *y, float *h_final,
                       const Kept &kept, int64_t Bs, int64_t L, int64_t ED, int num_sms,
                       cudaStream_t st) {
    auto at = [](const void *q) { return reinterpret_cast<uintptr_t>(q); };
    FwdArgs<T> p{{x, gr, gi}, lam, c, reset, h0, y, h_final, kept, int(L), int(ED), Bs * L, 1.0f, {}};
    const int W = widest_copy<T>(at(x) | at(gr) | at(gi), ED);
    const bool boxes = W == 16 && at(y) % 16 == 0 &&
                       (!kept.x_q || widest_copy<int8_t>(at(kept.x_q) | at(kept.r_q) | at(kept.i_q), ED) == 16);
    if (boxes) return start_fwd<T, 16>(p, Bs, num_sms, st);
    return W >= 8 ? start_fwd<T, 8>(p, Bs, num_sms, st) : start_fwd<T, 1>(p, Bs, num_sms, st);
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

template <typename T>
cudaError_t launch_step(const T *x, const T *gr, const T *gi, const float *lam, float c,
                        float *states, const int32_t *pages, T *y, int64_t Bs, int64_t ED,
                        int64_t num_pages, cudaStream_t st) {
    auto at = [](const void *q) { return reinterpret_cast<uintptr_t>(q); };
    const dim3 grid(unsigned((ED + 2 * kStepThreads - 1) / (2 * kStepThreads)), unsigned((Bs + kStepRows - 1) / kStepRows));
    const bool pairs = ED % 2 == 0 && (at(x) | at(gr) | at(gi) | at(y)) % (2 * sizeof(T)) == 0 && at(states) % 8 == 0;
    auto kern = pairs ? gated_step_kernel<T, true> : gated_step_kernel<T, false>;
    kern<<<grid, kStepThreads, 0, st>>>(x, gr, gi, lam, c, states, pages, y, Bs, ED, num_pages);
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
