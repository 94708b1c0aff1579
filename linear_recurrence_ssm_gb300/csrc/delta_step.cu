// delta_step.cu -- one token of the gated delta rule for each row of a batch,
// on states kept in pages, updated in place.
//
// A state is read and written once (8 K V bytes a head), which is all the time
// of a large batch.  A row of S needs its products with k and q; both come
// from the row as it was, since y = a S.q + u (k.q), so a row is read, reduced
// once over its lanes, and written.  A row takes the lanes of a warp that its
// 16-byte vectors need (32 for K = 128, 16 for 64), a lane holds kRows rows in
// flight: 256 rows of 32 heads of 64 x 128 take 82 us, 98 % of the copy
// bandwidth for the states' 0.54 GB alone.  Vectors of one element where rows
// of the states do not start on 16 bytes.
#include "delta_rule.cuh"

namespace ssm {
namespace delta {
namespace step {

constexpr int kWarps = 4, kRows = 8;

template <typename T>
struct Args {
    const T *q, *k, *v, *g, *beta;
    float *states;
    const int32_t *pages;
    T *y;
    int64_t num_pages;
    int Bs, G, H, K, V, tiles;
    float scale;
};

// LANES lanes share a row of S; VEC elements an access, CHUNKS accesses a row.
template <typename T, int LANES, int VEC, int CHUNKS>
__global__ void __launch_bounds__(32 * kWarps) kernel(const Args<T> p) {
    constexpr int per_warp = 32 / LANES * kRows;
    const int lane = threadIdx.x % 32, in_row = lane % LANES, warp = threadIdx.x / 32;
    const int tile = int(blockIdx.x % p.tiles), head = int(blockIdx.x / p.tiles % p.H);
    const int64_t b = blockIdx.x / p.tiles / p.H;
    const int v0 = (tile * kWarps + warp) * per_warp + lane / LANES;      // this lane's rows: v0 + i 32 / LANES
    const int64_t page = p.pages ? p.pages[b] : b;
    T *y = p.y + (b * p.H + head) * p.V;
    if (page < 0 || page >= p.num_pages) {
        if (in_row == 0)
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                if (v0 + i * (32 / LANES) < p.V) put(y + v0 + i * (32 / LANES), 0.0f);
        return;
    }
    float *S = p.states + (page * p.H + head) * int64_t(p.V) * p.K;
    float w[kRows][CHUNKS][VEC];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int v = v0 + i * (32 / LANES);
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            const int k = (c * LANES + in_row) * VEC;
            const bool in = v < p.V && k < p.K;
            if (VEC == 4) {
                float4 x = make_float4(0, 0, 0, 0);
                if (in) x = __ldcs(reinterpret_cast<const float4 *>(S + int64_t(v) * p.K + k));
                w[i][c][0] = x.x, w[i][c][VEC > 1 ? 1 : 0] = x.y, w[i][c][VEC > 2 ? 2 : 0] = x.z, w[i][c][VEC > 3 ? 3 : 0] = x.w;
            } else {
                w[i][c][0] = in ? S[int64_t(v) * p.K + k] : 0.0f;
            }
        }
    }
    const int64_t from = (b * p.G + head / (p.H / p.G)) * p.K;
    float kk[CHUNKS][VEC], qq[CHUNKS][VEC], kq = 0.0f;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int k = (c * LANES + in_row) * VEC + e;
            kk[c][e] = k < p.K ? to_f32(p.k[from + k]) : 0.0f;
            qq[c][e] = k < p.K ? to_f32(p.q[from + k]) : 0.0f;
            kq += kk[c][e] * qq[c][e];
        }
    const float g = to_f32(p.g[b * p.H + head]), beta = to_f32(p.beta[b * p.H + head]);
    const float a = g < kCut ? 0.0f : expf(g);
    float sk[kRows], sq[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        sk[i] = sq[i] = 0.0f;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                // a decay of 0 drops the state, whatever it holds
                w[i][c][e] = a == 0.0f ? 0.0f : a * w[i][c][e];
                sk[i] += w[i][c][e] * kk[c][e];
                sq[i] += w[i][c][e] * qq[c][e];
            }
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o /= 2) {
        kq += __shfl_xor_sync(0xffffffffu, kq, o);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            sk[i] += __shfl_xor_sync(0xffffffffu, sk[i], o);
            sq[i] += __shfl_xor_sync(0xffffffffu, sq[i], o);
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int v = v0 + i * (32 / LANES);
        if (v >= p.V) break;
        const float u = beta * (to_f32(p.v[(b * p.H + head) * p.V + v]) - sk[i]);
        if (in_row == 0) put(y + v, p.scale * (sq[i] + u * kq));
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            const int k = (c * LANES + in_row) * VEC;
            if (k >= p.K) continue;
            float *out = S + int64_t(v) * p.K + k;
            if (VEC == 4)
                __stcs(reinterpret_cast<float4 *>(out),
                       make_float4(w[i][c][0] + u * kk[c][0], w[i][c][VEC > 1 ? 1 : 0] + u * kk[c][VEC > 1 ? 1 : 0],
                                   w[i][c][VEC > 2 ? 2 : 0] + u * kk[c][VEC > 2 ? 2 : 0],
                                   w[i][c][VEC > 3 ? 3 : 0] + u * kk[c][VEC > 3 ? 3 : 0]));
            else
                *out = w[i][c][0] + u * kk[c][0];
        }
    }
}

template <typename T, int LANES, int VEC, int CHUNKS>
static cudaError_t go(Args<T> a, cudaStream_t st) {
    constexpr int rows = kWarps * (32 / LANES) * kRows;
    a.tiles = (a.V + rows - 1) / rows;
    const int64_t grid = int64_t(a.Bs) * a.H * a.tiles;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    kernel<T, LANES, VEC, CHUNKS><<<unsigned(grid), 32 * kWarps, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch(const T *q, const T *k, const T *v, const T *g, const T *beta, float scale, float *states,
                   const int32_t *pages, T *y, int64_t Bs, int64_t G, int64_t H, int64_t K, int64_t V,
                   int64_t num_pages, cudaStream_t st) {
    const Args<T> a{q, k, v, g, beta, states, pages, y, num_pages, int(Bs), int(G), int(H), int(K), int(V), 0, scale};
    // 16-byte vectors where every row of the states starts on one
    if (K % 4 == 0 && reinterpret_cast<uintptr_t>(states) % 16 == 0) {
        if (K <= 32) return go<T, 8, 4, 1>(a, st);
        if (K <= 64) return go<T, 16, 4, 1>(a, st);
        if (K <= 128) return go<T, 32, 4, 1>(a, st);
        return go<T, 32, 4, 2>(a, st);
    }
    if (K <= 64) return go<T, 32, 1, 2>(a, st);
    return go<T, 32, 1, 8>(a, st);
}

template cudaError_t launch<float>(const float *, const float *, const float *, const float *, const float *, float,
                                   float *, const int32_t *, float *, int64_t, int64_t, int64_t, int64_t, int64_t,
                                   int64_t, cudaStream_t);
template cudaError_t launch<__nv_bfloat16>(const __nv_bfloat16 *, const __nv_bfloat16 *, const __nv_bfloat16 *,
                                           const __nv_bfloat16 *, const __nv_bfloat16 *, float, float *,
                                           const int32_t *, __nv_bfloat16 *, int64_t, int64_t, int64_t, int64_t,
                                           int64_t, int64_t, cudaStream_t);

}  // namespace step
}  // namespace delta
}  // namespace ssm
