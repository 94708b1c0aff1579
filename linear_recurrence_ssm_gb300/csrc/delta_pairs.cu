// delta_pairs.cu -- what the gated delta rule's chains need of each block of
// 64 steps, apart from the state: the inverse of the block's system and the
// decayed products of queries and keys (delta_mma.cuh says how it is kept).
//
// All blocks at once, a thread block each.  Made apart from the chains, these
// are shared by the slices of a head's values and by both passes of a long
// sequence; made by extra warps of the chains' own thread blocks they held the
// chains up (6.5 us a block of 64 steps instead of the chain's own time).  8192
// blocks of K = 128 take 139 us, with P's second term 149: shared memory's
// accesses, 57 % of what it can serve, and the solves' barriers.
#include "delta_mma.cuh"

namespace ssm {
namespace delta {
namespace mma {

// K, Q and the system; the record is put together where K and Q were.
template <int KP>
struct PairLayout {
    static constexpr int tile = kBlock * KP * 2;
    static constexpr int system = 2 * tile > kBothRecord ? 2 * tile : (kBothRecord + 15) / 16 * 16;
    static constexpr int bytes = system + kBlock * kPairStride * 4;
};

struct PairMaps {
    CUtensorMap q, k;
};
__device__ unsigned int g_device_error;

template <int KP>
__global__ void __launch_bounds__(kPairThreads, 4)
pairs_kernel(const Shape s, const __grid_constant__ PairMaps maps, const bf *g, const bf *beta, unsigned char *records,
             const bool both, bf *states) {
    extern __shared__ __align__(1024) unsigned char mem[];
    __shared__ Decays d;
    __shared__ Factors f;
    __shared__ int found, abort;
    __shared__ __align__(8) uint64_t full;
    using L = PairLayout<KP>;
    let_next_begin();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int head = int(blockIdx.x % s.H), group = head / (s.H / s.G);
    const int64_t slot = blockIdx.x / s.H;
    const int seq = sequence_of(s, slot, &found);
    if (seq < 0) {
        if (states) clear_state(s, slot, head, states);
        return;
    }
    const Span span = span_of(s, seq);
    const int c = int(slot - span.slot), rows = min(kBlock, span.len - c * kBlock);
    const int64_t row = span.first + int64_t(c) * kBlock;
    const uint32_t base = smem_u32(mem);
    if (tid == 32) {
        abort = 0;
        tc::mbar_init(&full, 1);
        tc::mbar_fence_init();
        tc::mbar_arrive_expect_tx(&full, 2 * L::tile);
        boxes<KP>(base, &maps.k, &full, group, int(row));
        boxes<KP>(base + L::tile, &maps.q, &full, group, int(row));
    }
    float *system = reinterpret_cast<float *>(mem + L::system);
    if (warp == 0) {
        load_decays(d, g + row * s.H + head, beta + row * s.H + head, s.H, rows);
        __syncwarp();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int t = 32 * half + lane;
            const float start = d.start(t);
            f.start[t] = start;
            f.start_scaled[t] = s.scale * start;
            f.end[t] = d.end(t);
            f.beta[t] = d.beta[t];
            if (t == kBlock - 1) f.last = start;
        }
    }
    __syncthreads();
    wait_for(&full, 0, &abort, &g_device_error);
    if (*reinterpret_cast<volatile int *>(&abort)) {
        linger();           // copies may still be on their way
        return;
    }
    if (rows < kBlock) {
        clear_rows<KP>(base, rows, tid, kPairThreads);
        clear_rows<KP>(base + L::tile, rows, tid, kPairThreads);
        __syncthreads();
    }
    // rows 16 j of K K^T and 16 (3 - j) of Q K^T have five blocks of 16 x 16 together
    pair_products<KP>(base, base, warp, d, [&](int, int, int t, int r, float x, float y) {
        *reinterpret_cast<float2 *>(system + t * kPairStride + r) = make_float2(r < t ? x : 0.0f, r + 1 < t ? y : 0.0f);
    });
    uint32_t hi[4][4], lo[4][4];
    pair_products<KP>(base + L::tile, base, 3 - warp, d, [&](int n, int h, int t, int r, float x, float y) {
        split(r <= t ? s.scale * x : 0.0f, r + 1 <= t ? s.scale * y : 0.0f, hi[n][h], lo[n][h]);
    });
    __syncthreads();
    {
        const int t = 16 * (3 - warp) + lane / 4, c2 = lane % 4 * 2;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (n > 3 - warp) break;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                unsigned char *at = mem + place<64>(0, t + h % 2 * 8, 16 * n + h / 2 * 8) + c2 * 2;
                *reinterpret_cast<uint32_t *>(at + 2 * kTile) = hi[n][h];
                if (both) *reinterpret_cast<uint32_t *>(at + kRecord) = lo[n][h];
            }
        }
        for (int i = tid; i < int(sizeof(Factors)) / 16; i += kPairThreads)
            reinterpret_cast<uint4 *>(mem + 3 * kTile)[i] = reinterpret_cast<const uint4 *>(&f)[i];
    }
    lower_solve(system, d.beta, tid);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = i * kPairThreads + tid, t = at / 8, r = at % 8 * 8;
        uint32_t h[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const int s0 = r + 2 * e;
            const float4 v = *reinterpret_cast<const float4 *>(system + t * kPairStride + s0);
            split(s0 < t ? -v.x : 0.0f, s0 + 1 < t ? -v.y : 0.0f, h[e], l[e]);
            split(s0 + 2 < t ? -v.z : 0.0f, s0 + 3 < t ? -v.w : 0.0f, h[e + 1], l[e + 1]);
        }
        unsigned char *out = mem + place<64>(0, t, r);
        *reinterpret_cast<uint4 *>(out) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4 *>(out + kTile) = make_uint4(l[0], l[1], l[2], l[3]);
    }
    __syncthreads();
    const int size = both ? kBothRecord : kRecord;
    uint4 *to = reinterpret_cast<uint4 *>(records + (slot * s.H + head) * size);
    const uint4 *from = reinterpret_cast<const uint4 *>(mem);
    for (int i = tid; i < size / 16; i += kPairThreads) to[i] = from[i];
}

template <int KP>
static cudaError_t go(const Shape &s, const PairMaps &maps, const bf *g, const bf *beta, unsigned char *records, bool both,
                      bf *states, cudaStream_t st) {
    const int64_t grid = s.slots() * s.H;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    constexpr int bytes = PairLayout<KP>::bytes;
    if (cudaError_t e = allow<pairs_kernel<KP>>(bytes)) return e;
    pairs_kernel<KP><<<unsigned(grid), kPairThreads, bytes, st>>>(s, maps, g, beta, records, both, states);
    return cudaGetLastError();
}

cudaError_t make_pairs(const Shape &s, const CUtensorMap &q, const CUtensorMap &k, const bf *g, const bf *beta,
                       unsigned char *records, bool both, bf *states, cudaStream_t st) {
    const PairMaps maps{q, k};
    return s.K <= 64 ? go<64>(s, maps, g, beta, records, both, states, st)
                     : go<128>(s, maps, g, beta, records, both, states, st);
}

cudaError_t take_device_error(unsigned int *out) { return take_error(g_device_error, out); }

}  // namespace mma
}  // namespace delta
}  // namespace ssm
