// delta_general.cu -- the gated delta rule on CUDA cores, in fp32 throughout,
// for every type and head size (K, V up to 256): the path for fp32 inputs and
// for sizes without a tensor-core form.
//
// pairs_kernel takes all blocks of 64 steps at once and solves each one's
// system, N with (I + Ab beta) N = Ab, 16 rows at a time; a thread block of the
// chains takes one head of one sequence and 32 rows of its state (the rows are
// independent of one another) with the state in shared memory, and has matrix
// products left: W = V - Gam K S^T, X = W - N (beta W) and so on.  With the
// systems solved inside the chain a block of 64 steps took 40 us of it.  A chain
// alone is latency: a head of 64 x 64 takes 6.6 us a block forward and 12 back
// (30217 steps: 3.1 and 5.7 ms), of loads for the block that wait for the one
// before and of operands from shared memory (8.8 us a block forward before K and Q
// shared the reads of the state and N and P were read by 16 bytes).
#include "delta_rule.cuh"

namespace ssm {
namespace delta {
namespace general {

constexpr int kSlice = 32, kThreads = 256;
constexpr int kPairs = kBlock + 4, kRow = kSlice + 4;      // row strides, in floats
// Rows of the state that a thread block of the chains has, SL: 32, or 16 where
// that leaves SMs without one (a block of 64 steps takes about half as long).

__host__ __device__ inline int padded(int K) { return (K + 3) / 4 * 4; }
__host__ __device__ inline int stride_of(int K) { return padded(K) + 4; }

__device__ __forceinline__ void fma4(float4 &o, float a, const float4 &b) {
    o.x += a * b.x, o.y += a * b.y, o.z += a * b.z, o.w += a * b.w;
}

// What load_tile, load_pairs and load_made asked for has come, for this thread.
__device__ __forceinline__ void arrived() {
    cp_async_commit();
    cp_async_wait<0>();
}

// Four elements of a row, `left` of them there.
template <typename T>
__device__ __forceinline__ float4 four_of(const T *p, int left, bool vectors) {
    if (vectors && left >= 4) return to_f32x4(p);
    return make_float4(left > 0 ? to_f32(p[0]) : 0.0f, left > 1 ? to_f32(p[1]) : 0.0f, left > 2 ? to_f32(p[2]) : 0.0f,
                       left > 3 ? to_f32(p[3]) : 0.0f);
}
template <typename T>
__device__ __forceinline__ bool on_vectors(const T *p, int64_t step) {
    return reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0 && step % 4 == 0;
}

// `rows` rows of `width` elements, `step` elements apart, as floats; zeros up
// to 64 x `cols` (a multiple of 4).  Sixteen threads take a row.
template <typename T>
__device__ __forceinline__ void load_tile(float *tile, int stride, const T *src, int64_t step, int rows, int width,
                                          int cols) {
    const bool vectors = on_vectors(src, step);
    const int col = threadIdx.x % 16 * 4;
    if constexpr (sizeof(T) == 4)
        if (vectors && width % 4 == 0) {        // asynchronous: the caller waits
            for (int c = col; c < cols; c += 64)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = threadIdx.x / 16 + 16 * i;
                    const bool in = t < rows && c < width;
                    cp_async16(tile + t * stride + c, in ? src + t * step + c : src, in ? 16 : 0);
                }
            return;
        }
    float4 v[4];
    for (int c = col; c < cols; c += 64) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = threadIdx.x / 16 + 16 * i;
            v[i] = t < rows ? four_of(src + t * step + c, width - c, vectors) : make_float4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4 *>(tile + (threadIdx.x / 16 + 16 * i) * stride + c) = v[i];
    }
}

// The 4 x 4 products of this thread's rows ty + 16 i of `a` and tx + 16 j of `b`.
__device__ __forceinline__ void products(float (&out)[4][4], const float *a, const float *b, int stride, int Kp) {
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
    for (int i = 0; i < 16; ++i) out[i / 4][i % 4] = 0.0f;
    for (int k = 0; k < Kp; k += 4) {
        float4 u[4], w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u[i] = *reinterpret_cast<const float4 *>(a + (ty + 16 * i) * stride + k);
            w[i] = *reinterpret_cast<const float4 *>(b + (tx + 16 * i) * stride + k);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                out[i][j] += u[i].x * w[j].x + u[i].y * w[j].y + u[i].z * w[j].z + u[i].w * w[j].w;
    }
}

// Where row v of the state lies: a thread reads four neighbours, and the eight
// threads beside it the next ones, which so lie in different banks.
template <int SL>
__device__ __forceinline__ int lies(int v) { return v % 4 * (SL / 4) + v / 4; }

// Rows t (and t + 32 of 32-row slices) of each of N matrices times four rows v..
// of the state: out[n][i][j] = a[n]_(t + 32 i) . S_(v + j).
template <int SL, int R, int N>
__device__ __forceinline__ void through_state(float (&out)[N][R][4], const float *const (&a)[N], const float *S, int stride,
                                              int Kp, int t, int v) {
#pragma unroll
    for (int i = 0; i < 4 * R * N; ++i) out[i / (4 * R)][i / 4 % R][i % 4] = 0.0f;
#pragma unroll 2
    for (int k = 0; k < Kp; k += 4) {
        float4 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const float4 *>(S + (j * (SL / 4) + v / 4) * stride + k);
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float4 u = *reinterpret_cast<const float4 *>(a[n] + (t + 32 * i) * stride + k);
#pragma unroll
                for (int j = 0; j < 4; ++j) out[n][i][j] += u.x * w[j].x + u.y * w[j].y + u.z * w[j].z + u.w * w[j].w;
            }
    }
}

// Four rows of the state and this many of its columns are a thread's in the
// state's sums: as many threads for 16 rows as for 32.
template <int SL>
constexpr int kColumns = SL / 8;
template <int N>
__device__ __forceinline__ void get(float (&v)[N], const float *p) {
    if constexpr (N == 4) {
        const float4 w = *reinterpret_cast<const float4 *>(p);
        v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
    } else {
        const float2 w = *reinterpret_cast<const float2 *>(p);
        v[0] = w.x, v[1] = w.y;
    }
}
template <int N>
__device__ __forceinline__ void set(float *p, const float (&v)[N]) {
    if constexpr (N == 4) *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
}
// o += u_t k_t^T
template <int N>
__device__ __forceinline__ void outer(float (&o)[4][N], const float4 &u, const float *k) {
    float kk[N];
    get(kk, k);
#pragma unroll
    for (int e = 0; e < N; ++e) o[0][e] += u.x * kk[e], o[1][e] += u.y * kk[e], o[2][e] += u.z * kk[e], o[3][e] += u.w * kk[e];
}

// What the chains need of a block, in floats: N, P (with the scale), and the
// decays.
struct Made {
    float n[kBlock * kBlock], p[kBlock * kBlock];
    Decays d;
};

struct Layout {
    int stride, q, k, s, a, p, w, x, words;
};
__host__ __device__ inline Layout layout_of(int K) {
    Layout l;
    l.stride = stride_of(K);
    l.q = 0;
    l.k = l.q + kBlock * l.stride;
    l.s = l.k + kBlock * l.stride;
    l.a = l.s + kSlice * l.stride;
    l.p = l.a + kBlock * kPairs;
    l.w = l.p + kBlock * kPairs;
    l.x = l.w + kBlock * kRow;
    l.words = l.x + kBlock * kRow;
    return l;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) pairs_kernel(const Shape s, const T *q, const T *k, const T *g, const T *beta,
                                                         Made *made, T *states) {
    extern __shared__ __align__(16) float mem[];
    __shared__ Decays d;
    __shared__ int found;
    const int Kp = padded(s.K), stride = stride_of(s.K), tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const int wide = stride > kPairs ? stride : kPairs;
    float *Q = mem, *Kt = Q + kBlock * stride, *A = mem + 2 * kBlock * wide;
    const int head = int(blockIdx.x % s.H), group = head / (s.H / s.G);
    const int64_t slot = blockIdx.x / s.H;
    const int seq = sequence_of(s, slot, &found);
    if (seq < 0) {
        if (states) clear_state(s, slot, head, states);
        return;
    }
    const Span span = span_of(s, seq);
    const int c = int(slot - span.slot), rows = min(kBlock, span.len - c * kBlock);
    const int64_t row = span.first + int64_t(c) * kBlock, step = int64_t(s.G) * s.K;
    Made &out = made[slot * s.H + head];
    load_tile(Q, stride, q + row * step + int64_t(group) * s.K, step, rows, s.K, Kp);
    load_tile(Kt, stride, k + row * step + int64_t(group) * s.K, step, rows, s.K, Kp);
    if (tid < 32) load_decays(d, g + row * s.H + head, beta + row * s.H + head, s.H, rows);
    arrived();
    __syncthreads();
    for (int i = tid; i < int(sizeof(Decays) / 4); i += kThreads)
        reinterpret_cast<float *>(&out.d)[i] = reinterpret_cast<const float *>(&d)[i];
    float m[4][4];
    products(m, Q, Kt, stride, Kp);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int t = ty + 16 * (i / 4), r = tx + 16 * (i % 4);
        out.p[t * kBlock + r] = r <= t ? s.scale * m[i / 4][i % 4] * d.between(t, r) : 0.0f;
    }
    products(m, Kt, Kt, stride, Kp);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int t = ty + 16 * (i / 4), r = tx + 16 * (i % 4);
        A[t * kPairs + r] = r < t ? m[i / 4][i % 4] * d.between(t, r) : 0.0f;
    }
    __syncthreads();
    // N in A's place, a thread a column: N_t = A_t - sum over s < t of A_ts beta_s N_s.  The rows below a block of 16
    // are brought up to date by all threads; column j of N is 0 down to row j, where A is.
    float *N = mem;      // in the tiles' place
    for (int b = 0; b < kBlock; b += 16) {
        if (tid < kBlock) {
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[i] = b == 0 ? A[i * kPairs + tid] : N[(b + i) * kPairs + tid];
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (j < i) x[i] -= A[(b + i) * kPairs + b + j] * (d.beta[b + j] * x[j]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) N[(b + i) * kPairs + tid] = x[i];
        }
        __syncthreads();
        // four columns of a row
        for (int i = tid + (b + 16) * 16; i < kBlock * 16; i += kThreads) {
            const int t = i / 16, r = i % 16 * 4;
            float4 o = *reinterpret_cast<const float4 *>((b == 0 ? A : N) + t * kPairs + r);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                fma4(o, -A[t * kPairs + b + j] * d.beta[b + j], *reinterpret_cast<const float4 *>(N + (b + j) * kPairs + r));
            *reinterpret_cast<float4 *>(N + t * kPairs + r) = o;
        }
        __syncthreads();
    }
    for (int i = tid; i < kBlock * kBlock; i += kThreads) {
        const int t = i / kBlock, r = i % kBlock;
        out.n[i] = r < t ? N[t * kPairs + r] : 0.0f;
    }
}

// N (or P) and the decays of a block, into shared memory.
__device__ __forceinline__ void load_pairs(float *tile, const float *from) {
    for (int i = threadIdx.x; i < kBlock * kBlock / 4; i += kThreads)
        cp_async16(tile + i / 16 * kPairs + i % 16 * 4, from + 4 * i, 16);
}
__device__ __forceinline__ void load_made(Decays &d, const Decays &from) {
    for (int i = threadIdx.x; i < int(sizeof(Decays) / 16); i += kThreads)
        cp_async16(reinterpret_cast<float4 *>(&d) + i, reinterpret_cast<const float4 *>(&from) + i, 16);
}


// The first step that reaches step t: the last cut at or before it, or 0.  What
// lies before a cut takes no part in any sum, so that 0 times a NaN never enters.
__device__ __forceinline__ int behind_cut(const Decays &d, int t) {
    if (d.cut[t] == 0) return 0;
    while (t > 0 && d.cut[t - 1] == d.cut[t]) --t;
    return t;
}

// o += sign sum over r from `from` up to (not with) `to` of a_r x_r; a starts on 16 bytes.
template <int SIGN>
__device__ __forceinline__ void add_rows(float4 &o, const float *a, const float *x, int from, int to) {
    int r = from;
    for (; r < to && r % 4; ++r) fma4(o, SIGN * a[r], *reinterpret_cast<const float4 *>(x + r * kRow));
#pragma unroll 4
    for (; r + 4 <= to; r += 4) {
        const float4 w = *reinterpret_cast<const float4 *>(a + r);
        fma4(o, SIGN * w.x, *reinterpret_cast<const float4 *>(x + r * kRow));
        fma4(o, SIGN * w.y, *reinterpret_cast<const float4 *>(x + (r + 1) * kRow));
        fma4(o, SIGN * w.z, *reinterpret_cast<const float4 *>(x + (r + 2) * kRow));
        fma4(o, SIGN * w.w, *reinterpret_cast<const float4 *>(x + (r + 3) * kRow));
    }
    for (; r < to; ++r) fma4(o, SIGN * a[r], *reinterpret_cast<const float4 *>(x + r * kRow));
}

// Which head, sequence and rows of the state a thread block has.
struct Work {
    int seq, head, group, v0, width;
};
template <int SL>
__device__ __forceinline__ Work work_of(const Shape &s) {
    const int slices = (s.V + SL - 1) / SL;
    const int64_t at = blockIdx.x;
    Work w;
    w.v0 = int(at % slices) * SL;
    w.head = int(at / slices % s.H);
    w.seq = int(at / slices / s.H);
    w.group = w.head / (s.H / s.G);
    w.width = min(SL, s.V - w.v0);
    return w;
}

template <typename T, int SL>
__global__ void __launch_bounds__(kThreads) fwd_kernel(const FwdArgs<T> p) {
    extern __shared__ __align__(16) float mem[];
    __shared__ Decays d;
    const Shape &s = p.s;
    const Layout l = layout_of(s.K);
    float *Q = mem + l.q, *Kt = mem + l.k, *S = mem + l.s, *A = mem + l.a, *P = mem + l.p, *W = mem + l.w;
    const int Kp = padded(s.K), tid = threadIdx.x;
    const Work w = work_of<SL>(s);
    constexpr int R = SL / 16;      // rows of a thread: t0, t0 + 32
    const Span span = span_of(s, w.seq);
    const int64_t qk_step = int64_t(s.G) * s.K, v_step = int64_t(s.H) * s.V;
    const int64_t state_at = (int64_t(w.seq) * s.H + w.head) * s.V * s.K + int64_t(w.v0) * s.K;

    for (int v = tid / 32; v < SL; v += kThreads / 32)
        for (int k = tid % 32; k < Kp; k += 32)
            S[lies<SL>(v) * l.stride + k] = p.h0 && v < w.width && k < s.K ? p.h0[state_at + int64_t(v) * s.K + k] : 0.0f;
    const int t0 = tid / (SL / 4), v4 = tid % (SL / 4) * 4;
    for (int c = 0; c < span.blocks; ++c) {
        const int rows = min(kBlock, span.len - c * kBlock);
        const int64_t row = span.first + int64_t(c) * kBlock;
        __syncthreads();
        load_tile(Q, l.stride, p.q + row * qk_step + int64_t(w.group) * s.K, qk_step, rows, s.K, Kp);
        load_tile(Kt, l.stride, p.k + row * qk_step + int64_t(w.group) * s.K, qk_step, rows, s.K, Kp);
        load_tile(W, kRow, p.v + row * v_step + int64_t(w.head) * s.V + w.v0, v_step, rows, w.width, SL);
        const Made &made = reinterpret_cast<const Made *>(p.scratch)[(span.slot + c) * s.H + w.head];
        load_made(d, made.d);
        load_pairs(A, made.n);
        load_pairs(P, made.p);
        arrived();
        __syncthreads();
        if (p.states) {
            T *out = p.states + ((span.slot + c) * s.H + w.head) * int64_t(s.V) * s.K + int64_t(w.v0) * s.K;
            for (int v = tid / 32; v < w.width; v += kThreads / 32)
                for (int k = tid % 32; k < s.K; k += 32) put(out + v * s.K + k, S[lies<SL>(v) * l.stride + k]);
        }
        float both[2][R][4];
        through_state<SL, R, 2>(both, {Kt, Q}, S, l.stride, Kp, t0, v4);
        float(&from)[R][4] = both[0], (&y)[R][4] = both[1];
        // W, and beta W beside it
        float *U = mem + l.x;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int t = t0 + 32 * i;
            const float start = d.start(t), beta = d.beta[t];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // a cut drops the state before it, whatever that holds
                const float v = W[t * kRow + v4 + j] - (start == 0.0f ? 0.0f : start * from[i][j]);
                from[i][j] = v;
                U[t * kRow + v4 + j] = beta * v;
                y[i][j] = start == 0.0f ? 0.0f : s.scale * start * y[i][j];
            }
        }
        __syncthreads();
        // X
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int t = t0 + 32 * i;
            float4 o = make_float4(from[i][0], from[i][1], from[i][2], from[i][3]);
            add_rows<-1>(o, A + t * kPairs, U + v4, behind_cut(d, t), t);
            *reinterpret_cast<float4 *>(W + t * kRow + v4) = o;
        }
        __syncthreads();
        if (p.errors) {
            T *out = p.errors + row * v_step + int64_t(w.head) * s.V + w.v0;
            for (int t = tid / 32; t < rows; t += kThreads / 32)
                if (tid % 32 < w.width) put(out + t * v_step + tid % 32, W[t * kRow + tid % 32]);
            __syncthreads();
        }
        for (int i = tid; i < kBlock * SL; i += kThreads) W[i / SL * kRow + i % SL] *= d.beta[i / SL];
        __syncthreads();
        // outputs of rows t0 and t0 + 32, four columns
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int t = t0 + 32 * i;
            float4 o = make_float4(y[i][0], y[i][1], y[i][2], y[i][3]);
            add_rows<1>(o, P + t * kPairs, W + v4, behind_cut(d, t), t + 1);
            if (t < rows) {
                T *out = p.y + (row + t) * v_step + int64_t(w.head) * s.V + w.v0 + v4;
                const float v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (v4 + j < w.width) put(out + j, v[j]);
            }
        }
        const float last = d.start(kBlock - 1);
        const int first = behind_cut(d, kBlock - 1);
        __syncthreads();
        for (int i = tid; i < kBlock * SL; i += kThreads) W[i / SL * kRow + i % SL] *= d.end(i / SL);
        __syncthreads();
        for (int i = tid; i < SL / 4 * (Kp / kColumns<SL>); i += kThreads) {
            const int v = i % (SL / 4) * 4, k = i / (SL / 4) * kColumns<SL>;
            float o[4][kColumns<SL>];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                get(o[j], S + lies<SL>(v + j) * l.stride + k);
#pragma unroll
                for (int e = 0; e < kColumns<SL>; ++e) o[j][e] = last == 0.0f ? 0.0f : last * o[j][e];
            }
#pragma unroll 4
            for (int t = first; t < rows; ++t) outer(o, *reinterpret_cast<const float4 *>(W + t * kRow + v), Kt + t * l.stride + k);
#pragma unroll
            for (int j = 0; j < 4; ++j) set(S + lies<SL>(v + j) * l.stride + k, o[j]);
        }
    }
    __syncthreads();
    if (p.h_final)
        for (int v = tid / 32; v < w.width; v += kThreads / 32)
            for (int k = tid % 32; k < s.K; k += 32) p.h_final[state_at + v * s.K + k] = S[lies<SL>(v) * l.stride + k];
    clear_uncovered(s, w.seq, p.y + int64_t(w.head) * s.V + w.v0, v_step, w.width);
    if (p.errors) clear_uncovered(s, w.seq, p.errors + int64_t(w.head) * s.V + w.v0, v_step, w.width);
}

// Back along a sequence: dv, the shares of dbeta, the adjoint of every
// block's last state (into the scratch) and of the first one.
template <typename T, int SL>
__global__ void __launch_bounds__(kThreads) back_kernel(const BwdArgs<T> p) {
    extern __shared__ __align__(16) float mem[];
    __shared__ Decays d;
    const Shape &s = p.s;
    const Layout l = layout_of(s.K);
    float *Q = mem + l.q, *Kt = mem + l.k, *S = mem + l.s, *A = mem + l.a, *P = mem + l.p, *Y = mem + l.w,
          *Z = mem + l.x;
    const int Kp = padded(s.K), tid = threadIdx.x;
    const Work w = work_of<SL>(s);
    constexpr int R = SL / 16;      // rows of a thread: t0, t0 + 32
    const Span span = span_of(s, w.seq);
    const int64_t qk_step = int64_t(s.G) * s.K, v_step = int64_t(s.H) * s.V;
    const int64_t state_at = (int64_t(w.seq) * s.H + w.head) * s.V * s.K + int64_t(w.v0) * s.K;
    const int64_t rows_all = s.offsets ? s.L : s.L * s.n;
    float *part = p.dbeta_part + int64_t(w.v0 / SL) * rows_all * s.H + w.head;

    for (int v = tid / 32; v < SL; v += kThreads / 32)
        for (int k = tid % 32; k < Kp; k += 32)
            S[lies<SL>(v) * l.stride + k] =
                p.dh_final && v < w.width && k < s.K ? p.dh_final[state_at + int64_t(v) * s.K + k] : 0.0f;
    const int t0 = tid / (SL / 4), v4 = tid % (SL / 4) * 4;
    for (int c = span.blocks - 1; c >= 0; --c) {
        const int rows = min(kBlock, span.len - c * kBlock);
        const int64_t row = span.first + int64_t(c) * kBlock;
        __syncthreads();
        load_tile(Q, l.stride, p.q + row * qk_step + int64_t(w.group) * s.K, qk_step, rows, s.K, Kp);
        load_tile(Kt, l.stride, p.k + row * qk_step + int64_t(w.group) * s.K, qk_step, rows, s.K, Kp);
        load_tile(Y, kRow, p.dy + row * v_step + int64_t(w.head) * s.V + w.v0, v_step, rows, w.width, SL);
        const Made &made = reinterpret_cast<const Made *>(p.records)[(span.slot + c) * s.H + w.head];
        load_made(d, made.d);
        load_pairs(A, made.n);
        load_pairs(P, made.p);
        arrived();
        __syncthreads();
        T *ds = p.ds + ((span.slot + c) * s.H + w.head) * int64_t(s.V) * s.K + int64_t(w.v0) * s.K;
        for (int v = tid / 32; v < w.width; v += kThreads / 32)
            for (int k = tid % 32; k < s.K; k += 32) put(ds + v * s.K + k, S[lies<SL>(v) * l.stride + k]);
        float of_keys[1][R][4];
        through_state<SL, R, 1>(of_keys, {Kt}, S, l.stride, Kp, t0, v4);
        const float(&from)[R][4] = of_keys[0];
        // dU, and beta dU beside it
        float4 du[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int t = t0 + 32 * i;
            const float end = d.end(t), beta = d.beta[t];
            float4 o = end == 0.0f ? make_float4(0, 0, 0, 0)
                                   : make_float4(end * from[i][0], end * from[i][1], end * from[i][2], end * from[i][3]);
#pragma unroll 4
            for (int r = t; r < rows; ++r) fma4(o, P[r * kPairs + t], *reinterpret_cast<const float4 *>(Y + r * kRow + v4));
            du[i] = o;
            *reinterpret_cast<float4 *>(Z + t * kRow + v4) = make_float4(beta * o.x, beta * o.y, beta * o.z, beta * o.w);
        }
        __syncthreads();
        // Z
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int t = t0 + 32 * i;
#pragma unroll 4
            for (int r = t + 1; r < rows; ++r)
                fma4(du[i], -A[r * kPairs + t], *reinterpret_cast<const float4 *>(Z + r * kRow + v4));
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < R; ++i) *reinterpret_cast<float4 *>(Z + (t0 + 32 * i) * kRow + v4) = du[i];
        __syncthreads();
        // a warp takes a row at a time: dbeta's share, dv, and beta Z in Z's place
        {
            const int lane = tid % 32;
            const T *x = p.errors + row * v_step + int64_t(w.head) * s.V + w.v0;
            T *dv = p.dv + row * v_step + int64_t(w.head) * s.V + w.v0;
            for (int t = tid / 32; t < kBlock; t += kThreads / 32) {
                const float z = Z[t * kRow + lane], bz = d.beta[t] * z;
                float sum = t < rows && lane < w.width ? z * to_f32(x[t * v_step + lane]) : 0.0f;
#pragma unroll
                for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (t < rows) {
                    if (lane < w.width) put(dv + t * v_step + lane, bz);
                    if (lane == 0) part[(row + t) * s.H] = sum;
                }
                const float start = d.start(t);
                Z[t * kRow + lane] = -start * bz;
                Y[t * kRow + lane] *= s.scale * start;
            }
        }
        const float last = d.start(kBlock - 1);
        __syncthreads();
        for (int i = tid; i < SL / 4 * (Kp / kColumns<SL>); i += kThreads) {
            const int v = i % (SL / 4) * 4, k = i / (SL / 4) * kColumns<SL>;
            float o[4][kColumns<SL>];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                get(o[j], S + lies<SL>(v + j) * l.stride + k);
#pragma unroll
                for (int e = 0; e < kColumns<SL>; ++e) o[j][e] = last == 0.0f ? 0.0f : last * o[j][e];
            }
#pragma unroll 4
            for (int t = 0; t < rows; ++t) {
                outer(o, *reinterpret_cast<const float4 *>(Y + t * kRow + v), Q + t * l.stride + k);
                outer(o, *reinterpret_cast<const float4 *>(Z + t * kRow + v), Kt + t * l.stride + k);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) set(S + lies<SL>(v + j) * l.stride + k, o[j]);
        }
    }
    __syncthreads();
    if (p.dh0)
        for (int v = tid / 32; v < w.width; v += kThreads / 32)
            for (int k = tid % 32; k < s.K; k += 32) p.dh0[state_at + v * s.K + k] = S[lies<SL>(v) * l.stride + k];
    clear_uncovered(s, w.seq, p.dv + int64_t(w.head) * s.V + w.v0, v_step, w.width);
    if (w.v0 == 0) {
        clear_uncovered(s, w.seq, p.dg + w.head, s.H, 1);
        clear_uncovered(s, w.seq, p.dbeta + w.head, s.H, 1);
        if (w.head < s.G) {
            clear_uncovered(s, w.seq, p.dq + int64_t(w.head) * s.K, qk_step, s.K);
            clear_uncovered(s, w.seq, p.dk + int64_t(w.head) * s.K, qk_step, s.K);
        }
    }
}

struct GradLayout {
    int stride, q, k, dp, da, m, y, u, z, s0, s1, words;
};
__host__ __device__ inline GradLayout grad_layout_of(int K) {
    GradLayout l;
    l.stride = stride_of(K);
    l.q = 0;
    l.k = l.q + kBlock * l.stride;
    l.dp = l.k + kBlock * l.stride;
    l.da = l.dp + kBlock * kPairs;
    l.y = l.da + kBlock * kPairs;
    l.u = l.y + kBlock * kRow;
    l.z = l.u + kBlock * kRow;
    l.s0 = l.z + kBlock * kRow;
    l.s1 = l.s0 + kSlice * kPairs;
    l.words = l.s1 + kSlice * kPairs;
    l.m = l.y;                  // after the slices are done with; 64 x 65
    return l;
}

// dq, dk, dg and dbeta of one block of one head.
template <typename T>
__global__ void __launch_bounds__(kThreads) grads_kernel(const BwdArgs<T> p, const int shares) {
    extern __shared__ __align__(16) float mem[];
    __shared__ Decays d;
    __shared__ int found;
    __shared__ float row_term[kBlock], col_term[kBlock], both_term[kThreads / 32];
    const Shape &s = p.s;
    const GradLayout l = grad_layout_of(s.K);
    float *Q = mem + l.q, *Kt = mem + l.k, *dP = mem + l.dp, *dA = mem + l.da, *Y = mem + l.y, *U = mem + l.u,
          *Z = mem + l.z, *S0 = mem + l.s0, *S1 = mem + l.s1, *M = mem + l.m;
    const int Kp = padded(s.K), tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const int head = int(blockIdx.x % s.H), group = head / (s.H / s.G);
    const int64_t slot = blockIdx.x / s.H;
    const int seq = sequence_of(s, slot, &found);
    if (seq < 0) return;
    const Span span = span_of(s, seq);
    const int c = int(slot - span.slot), rows = min(kBlock, span.len - c * kBlock);
    const int64_t row = span.first + int64_t(c) * kBlock, rows_all = s.offsets ? s.L : s.L * s.n;
    const int64_t qk_step = int64_t(s.G) * s.K, v_step = int64_t(s.H) * s.V;
    load_tile(Q, l.stride, p.q + row * qk_step + int64_t(group) * s.K, qk_step, rows, s.K, Kp);
    load_tile(Kt, l.stride, p.k + row * qk_step + int64_t(group) * s.K, qk_step, rows, s.K, Kp);
    if (tid < 32) load_decays(d, p.g + row * s.H + head, p.beta + row * s.H + head, s.H, rows);
    if (tid < kBlock) row_term[tid] = col_term[tid] = 0.0f;
    arrived();
    const T *st0 = p.states + (slot * s.H + head) * int64_t(s.V) * s.K;
    const T *st1 = p.ds + (slot * s.H + head) * int64_t(s.V) * s.K;

    // a slice of dY, U = beta x and beta Z = dv
    const auto load_slice = [&](int v0) {
        const int width = min(kSlice, s.V - v0);
        const int64_t at = row * v_step + int64_t(head) * s.V + v0;
        for (int i = tid; i < kBlock * kSlice; i += kThreads) {
            const int t = i / kSlice, v = i % kSlice;
            const bool in = t < rows && v < width;
            const int64_t o = at + t * v_step + v;
            Y[t * kRow + v] = in ? s.scale * to_f32(p.dy[o]) : 0.0f;
            U[t * kRow + v] = in ? d.beta[t] * to_f32(p.errors[o]) : 0.0f;
            Z[t * kRow + v] = in ? to_f32(p.dv[o]) : 0.0f;
        }
    };
    float gp[4][4] = {}, ga[4][4] = {};
    for (int v0 = 0; v0 < s.V; v0 += kSlice) {
        __syncthreads();
        load_slice(v0);
        __syncthreads();
        float m[4][4];
        products(m, Y, U, kRow, kSlice);
#pragma unroll
        for (int i = 0; i < 16; ++i) gp[i / 4][i % 4] += m[i / 4][i % 4];
        products(m, Z, U, kRow, kSlice);
#pragma unroll
        for (int i = 0; i < 16; ++i) ga[i / 4][i % 4] -= m[i / 4][i % 4];
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int t = ty + 16 * (i / 4), r = tx + 16 * (i % 4);
        const float D = d.between(t, r);
        dP[t * kPairs + r] = r <= t ? gp[i / 4][i % 4] * D : 0.0f;
        dA[t * kPairs + r] = r < t ? ga[i / 4][i % 4] * D : 0.0f;
    }
    float both = 0.0f;
    // 64 columns of K at a time: what goes through the states, then through the pairs
    for (int k0 = 0; k0 < Kp; k0 += kBlock) {
        const int wide = min(kBlock, s.K - k0);
        float dq[4][4] = {}, dr[4][4] = {}, dc[4][4] = {};      // rows ty + 16 i, columns tx + 16 j
        for (int v0 = 0; v0 < s.V; v0 += kSlice) {
            const int width = min(kSlice, s.V - v0);
            __syncthreads();
            load_slice(v0);
            for (int i = tid; i < kSlice * kBlock; i += kThreads) {
                const int v = i / kBlock, k = i % kBlock;
                const bool in = v < width && k < wide;
                const float a = in ? to_f32(st0[int64_t(v0 + v) * s.K + k0 + k]) : 0.0f;
                const float b = in ? to_f32(st1[int64_t(v0 + v) * s.K + k0 + k]) : 0.0f;
                S0[v * kPairs + k] = a;
                S1[v * kPairs + k] = b;
                both += a * b;
            }
            __syncthreads();
            for (int v = 0; v < width; ++v) {
                float a[4], b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) a[j] = S0[v * kPairs + tx + 16 * j], b[j] = S1[v * kPairs + tx + 16 * j];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = ty + 16 * i;
                    const float y = Y[t * kRow + v], u = U[t * kRow + v], z = Z[t * kRow + v];
#pragma unroll
                    for (int j = 0; j < 4; ++j) dq[i][j] += y * a[j], dr[i][j] -= z * a[j], dc[i][j] += u * b[j];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = ty + 16 * i;
            const float start = d.start(t), end = d.end(t);
            float rt = 0.0f, ct = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = tx + 16 * j;
                const float qv = k < wide ? Q[t * l.stride + k0 + k] : 0.0f, kv = k < wide ? Kt[t * l.stride + k0 + k] : 0.0f;
                dq[i][j] = start == 0.0f ? 0.0f : start * dq[i][j];
                dr[i][j] = start == 0.0f ? 0.0f : start * dr[i][j];
                dc[i][j] = end == 0.0f ? 0.0f : end * dc[i][j];
                rt += dq[i][j] * qv + dr[i][j] * kv;
                ct += dc[i][j] * kv;
                dr[i][j] += dc[i][j];
            }
#pragma unroll
            for (int o = 8; o > 0; o /= 2) {
                rt += __shfl_xor_sync(0xffffffffu, rt, o);
                ct += __shfl_xor_sync(0xffffffffu, ct, o);
            }
            if (tx == 0) row_term[t] += rt, col_term[t] += ct;
        }
        for (int r = 0; r < rows; ++r) {
            float kr[4], qr[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = tx + 16 * j;
                kr[j] = k < wide ? Kt[r * l.stride + k0 + k] : 0.0f;
                qr[j] = k < wide ? Q[r * l.stride + k0 + k] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = ty + 16 * i;
                const float pd = dP[t * kPairs + r], pt = dP[r * kPairs + t];
                const float ad = dA[t * kPairs + r] + dA[r * kPairs + t];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    dq[i][j] += pd * kr[j];
                    dr[i][j] += pt * qr[j] + ad * kr[j];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int t = ty + 16 * (i / 4), k = tx + 16 * (i % 4);
            if (t >= rows || k >= wide) continue;
            if (s.H > s.G) {
                const int64_t o = ((row + t) * s.H + head) * s.K + k0 + k;
                p.dq_head[o] = dq[i / 4][i % 4];
                p.dk_head[o] = dr[i / 4][i % 4];
            } else {
                const int64_t o = ((row + t) * s.H + head) * s.K + k0 + k;
                put(p.dq + o, dq[i / 4][i % 4]);
                put(p.dk + o, dr[i / 4][i % 4]);
            }
        }
    }
    // dg: the pairs' products, their sums along rows up to each step, then down the columns
#pragma unroll
    for (int o = 16; o > 0; o /= 2) both += __shfl_xor_sync(0xffffffffu, both, o);
    if (tid % 32 == 0) both_term[tid / 32] = both;
    float mk[4][4], mq[4][4];
    products(mq, Q, Kt, l.stride, Kp);
    products(mk, Kt, Kt, l.stride, Kp);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int t = ty + 16 * (i / 4), r = tx + 16 * (i % 4);
        M[t * (kBlock + 1) + r] =
            r < t ? dP[t * kPairs + r] * mq[i / 4][i % 4] + dA[t * kPairs + r] * mk[i / 4][i % 4] : 0.0f;
    }
    __syncthreads();
    if (tid < kBlock) {
        float sum = 0.0f;
        for (int r = 0; r < kBlock; ++r) {
            const float v = M[tid * (kBlock + 1) + r];
            M[tid * (kBlock + 1) + r] = sum;        // pairs of row tid before step r
            sum += v;
        }
    }
    __syncthreads();
    if (tid < rows) {
        float sum = 0.0f;
        for (int i = 0; i < kThreads / 32; ++i) sum += both_term[i];
        const float last = d.start(kBlock - 1);
        sum = last == 0.0f ? 0.0f : last * sum;
        for (int r = tid; r < rows; ++r) sum += row_term[r] + M[r * (kBlock + 1) + tid];
        for (int r = 0; r < tid; ++r) sum += col_term[r];
        put(p.dg + (row + tid) * s.H + head, sum);
        float b = 0.0f;
        for (int i = 0; i < shares; ++i) b += p.dbeta_part[(int64_t(i) * rows_all + row + tid) * s.H + head];
        put(p.dbeta + (row + tid) * s.H + head, b);
    }
}

// dq and dk of a group: the sum of its heads', in their order.  Rows that no
// sequence covers are 0 (back_kernel) and stay.
template <typename T>
__global__ void __launch_bounds__(kThreads) fold_kernel(const BwdArgs<T> p) {
    const Shape &s = p.s;
    const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x, row = i / (s.G * s.K);
    int64_t a = 0, b = s.L * s.n;
    if (s.offsets) {
        const Span last = span_of(s, s.n - 1);
        a = span_of(s, 0).first, b = last.first + last.len;
    }
    if (row < a || row >= b) return;
    const int at = int(i % (s.G * s.K)), group = at / s.K, k = at % s.K, per = s.H / s.G;
    const int64_t from = (row * s.H + group * per) * s.K + k;
    float q = 0.0f, kk = 0.0f;
    for (int h = 0; h < per; ++h) q += p.dq_head[from + int64_t(h) * s.K], kk += p.dk_head[from + int64_t(h) * s.K];
    put(p.dq + i, q);
    put(p.dk + i, kk);
}

static int slices(const Shape &s, int rows) { return (s.V + rows - 1) / rows; }
// 16 rows a thread block where 32 would leave some of a GB300's 152 SMs idle (3 x 333
// steps of 5 heads of 40 x 96, forward and back: 284 us with 32, 257 with 16; with
// the SMs full, 32 rows read K and Q half as often).
static int rows_of(const Shape &s) { return int64_t(s.n) * s.H * slices(s, 32) < 152 ? 16 : 32; }
int64_t shares(const Shape &s) { return slices(s, rows_of(s)) * s.rows() * s.H; }

template <typename K>
static cudaError_t room(K kernel, int words) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, words * 4);
}

int64_t made_bytes(const Shape &s) { return s.slots() * s.H * int64_t(sizeof(Made)); }

template <typename T>
static cudaError_t make_pairs(const Shape &s, const T *q, const T *k, const T *g, const T *beta, unsigned char *made,
                              T *states, cudaStream_t st) {
    const int64_t grid = s.slots() * s.H;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const auto words = [](int K) { return 2 * kBlock * (stride_of(K) > kPairs ? stride_of(K) : kPairs) + kBlock * kPairs; };
    if (cudaError_t e = room(pairs_kernel<T>, words(256))) return e;
    pairs_kernel<T><<<unsigned(grid), kThreads, words(s.K) * 4, st>>>(s, q, k, g, beta, reinterpret_cast<Made *>(made), states);
    return cudaGetLastError();
}

template <typename T, int SL>
static cudaError_t go(const FwdArgs<T> &a, unsigned grid, cudaStream_t st) {
    // the limit is the largest layout's, whatever this call takes: calls of several threads cannot lower it
    if (cudaError_t e = room(fwd_kernel<T, SL>, layout_of(256).words)) return e;
    fwd_kernel<T, SL><<<grid, kThreads, layout_of(a.s.K).words * 4, st>>>(a);
    return cudaGetLastError();
}
template <typename T>
cudaError_t fwd(const FwdArgs<T> &a, cudaStream_t st) {
    const int each = rows_of(a.s);
    const int64_t grid = int64_t(a.s.n) * a.s.H * slices(a.s, each);
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (cudaError_t e = make_pairs(a.s, a.q, a.k, a.g, a.beta, a.scratch, a.states, st)) return e;
    return each == 16 ? go<T, 16>(a, unsigned(grid), st) : go<T, 32>(a, unsigned(grid), st);
}

template <typename T>
cudaError_t fold(const BwdArgs<T> &a, cudaStream_t st) {
    const int64_t grid = (a.s.rows() * a.s.G * a.s.K + kThreads - 1) / kThreads;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    fold_kernel<T><<<unsigned(grid), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int SL>
static cudaError_t go(const BwdArgs<T> &a, unsigned grid, cudaStream_t st) {
    if (cudaError_t e = room(back_kernel<T, SL>, layout_of(256).words)) return e;
    back_kernel<T, SL><<<grid, kThreads, layout_of(a.s.K).words * 4, st>>>(a);
    return cudaGetLastError();
}
template <typename T>
cudaError_t bwd(const BwdArgs<T> &a, cudaStream_t st) {
    const int each = rows_of(a.s);
    const int64_t grid = int64_t(a.s.n) * a.s.H * slices(a.s, each), blocks = a.s.slots() * a.s.H;
    if (grid > 0x7fffffff || blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (cudaError_t e = make_pairs<T>(a.s, a.q, a.k, a.g, a.beta, a.records, nullptr, st)) return e;
    if (cudaError_t e = room(grads_kernel<T>, grad_layout_of(256).words)) return e;
    if (cudaError_t e = each == 16 ? go<T, 16>(a, unsigned(grid), st) : go<T, 32>(a, unsigned(grid), st)) return e;
    grads_kernel<T><<<unsigned(blocks), kThreads, grad_layout_of(a.s.K).words * 4, st>>>(a, slices(a.s, each));
    if (cudaError_t e = cudaGetLastError()) return e;
    return a.s.H > a.s.G ? fold(a, st) : cudaSuccess;
}

template cudaError_t fold<__nv_bfloat16>(const BwdArgs<__nv_bfloat16> &, cudaStream_t);
template cudaError_t fwd<float>(const FwdArgs<float> &, cudaStream_t);
template cudaError_t fwd<__nv_bfloat16>(const FwdArgs<__nv_bfloat16> &, cudaStream_t);
template cudaError_t bwd<float>(const BwdArgs<float> &, cudaStream_t);
template cudaError_t bwd<__nv_bfloat16>(const BwdArgs<__nv_bfloat16> &, cudaStream_t);

}  // namespace general
}  // namespace delta
}  // namespace ssm
