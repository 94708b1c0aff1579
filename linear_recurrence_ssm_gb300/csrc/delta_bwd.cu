// delta_bwd.cu -- gradients of the gated delta rule, bf16, on tensor cores.
//
// back_kernel walks a sequence from its end with the state's adjoint A (V x K)
// in four warps' accumulators, 16 rows each, as the forward kernel does:
//   dU^T = E (A K^T) + dY^T P,  Z^T = dU^T - (beta dU)^T N,  dV = beta Z
//   A = Gam_C A + (scale Gam dY)^T Q - (Gam beta Z)^T K
// Four more warps form dY^T P and (scale Gam dY)^T Q, which do not depend on
// A, one block ahead.  A's own chain uses operands of two bf16 terms (dh0 comes
// out as the forward pass's final state does); it leaves A of every block, dV and
// shares of dbeta (Z in fp32 times the kept X).
//
// block_kernel then takes all blocks at once: dQ, dK and dg from the kept states,
// the adjoints, dY, X and dV.  Those are bf16, A and dV rounded once for it, and so
// are dP D and dAb D as operands of the last products: up to 2^-8 of a term, as
// dq, dk and dg themselves are rounded (3.4e-3 in the 2-norm where that rounding
// gives 1.7e-3).  Two terms of each would double its products, and A and dV in
// fp32 take half as much memory again.
//
// 4 x 4096 steps of 32 heads of 64 x 128: the chain 267 us (tensor cores 47 %, its
// products wait for one another), the blocks 307 (issue 44 %, shared memory 47 %,
// tensor cores 32 %; barriers are a fifth of the stalls: two thread blocks of eight
// warps are all that a SM's shared memory holds).
#include "delta_mma.cuh"

namespace ssm {
namespace delta {
namespace mma {
namespace bwd {

constexpr int kSlice = 64, kChain = 4, kThreads = 256;

template <int KP>
struct Layout {
    static constexpr int tile = kBlock * KP * 2, v = kBlock * kSlice * 2;
    static constexpr int chain = tile + 2 * kTile + v;              // K, N in two terms, X: two of them
    static constexpr int ahead = tile + v + 2 * kTile;              // Q, dY, P in two terms: two of them
    static constexpr int at_ahead = 2 * chain, handed = at_ahead + 2 * ahead;
    static constexpr int u = 16 * kBlock * 4, s = 16 * KP * 4;      // of a warp: dY^T P and (scale Gam dY)^T Q
    static constexpr int out = handed + kChain * (u + s);
    static constexpr int out_warp = 16 * 128 * 2;
    static constexpr int factors = out + kChain * out_warp;         // two of them, and scale Gam of the blocks ahead
    static constexpr int scaled = factors + 2 * int(sizeof(Factors));
    static constexpr int bars = scaled + 2 * kBlock * 4;            // two barriers, and whether a wait ran out
    static constexpr int bytes = bars + 32;
    static_assert(chain % 1024 == 0 && ahead % 1024 == 0 && bytes <= 232448, "shared memory");
};
struct Maps {
    CUtensorMap q, k, dy, x;
};
__device__ unsigned int g_device_error;

template <int KP>
__global__ void __launch_bounds__(kThreads, 1) back_kernel(const BwdArgs<bf> p, const __grid_constant__ Maps maps) {
    extern __shared__ __align__(1024) unsigned char mem[];
    using L = Layout<KP>;
    let_next_begin();
    const Shape &s = p.s;
    const uint32_t base = smem_u32(mem);
    const int slices = (s.V + kSlice - 1) / kSlice;
    const int slice = int(blockIdx.x % slices), head = int(blockIdx.x / slices % s.H);
    const int seq = int(blockIdx.x / slices / s.H), group = head / (s.H / s.G), v0 = slice * kSlice;
    const Span span = span_of(s, seq);
    const int64_t qk_step = int64_t(s.G) * s.K, v_step = int64_t(s.H) * s.V;
    const int64_t slots = s.offsets ? s.L / kBlock + s.n : (s.L + kBlock - 1) / kBlock * s.n;
    const int tid = threadIdx.x, warp = tid / 32 % kChain, lane = tid % 32;
    const bool chain = tid < 32 * kChain;
    const int g = lane / 4, c2 = lane % 4 * 2, mine = v0 + 16 * warp;
    const int width = s.V - mine;
    const int64_t state_at = (int64_t(seq) * s.H + head) * s.V * s.K;
    const uint32_t hand_u = base + L::handed + warp * (L::u + L::s) + lane * 16, hand_s = hand_u + L::u;

    uint64_t *full = reinterpret_cast<uint64_t *>(mem + L::bars);
    int *abort = reinterpret_cast<int *>(full + 2);
    // One thread asks for a turn's copies: what the warps ahead need of block blocks - 1 - turn, the chain of the one behind.
    const auto copy = [&](int turn) {
        const int ahead = span.blocks - 1 - turn, behind = ahead + 1, stage = turn % 2;
        uint64_t *bar = &full[stage];
        const auto record = [&](int c) { return p.records + ((span.slot + c) * s.H + head) * kBothRecord; };
        constexpr int for_ahead = L::ahead + kBlock * 4, for_chain = L::chain + int(sizeof(Factors));
        tc::mbar_arrive_expect_tx(bar, (ahead >= 0 ? for_ahead : 0) + (turn > 0 ? for_chain : 0));
        if (ahead >= 0) {
            const uint32_t to = base + L::at_ahead + stage * L::ahead;
            const int row = int(span.first + int64_t(ahead) * kBlock);
            boxes<KP>(to, &maps.q, bar, group, row);
            box(to + L::tile, &maps.dy, bar, v0, head, row);
            bulk(to + L::tile + L::v, record(ahead) + 2 * kTile, kTile, bar);
            bulk(to + L::tile + L::v + kTile, record(ahead) + kRecord, kTile, bar);
            bulk(base + L::scaled + stage * kBlock * 4, record(ahead) + 3 * kTile + offsetof(Factors, start_scaled), kBlock * 4, bar);
        }
        if (turn > 0) {
            const uint32_t to = base + stage * L::chain;
            const int row = int(span.first + int64_t(behind) * kBlock);
            boxes<KP>(to, &maps.k, bar, group, row);
            bulk(to + L::tile, record(behind), 2 * kTile, bar);
            box(to + L::tile + 2 * kTile, &maps.x, bar, v0, head, row);
            bulk(base + L::factors + stage * int(sizeof(Factors)), record(behind) + 3 * kTile, int(sizeof(Factors)), bar);
        }
    };
    const bool asks = tid == 32 * kChain;
    if (asks) {
        *abort = 0;
        tc::mbar_init(&full[0], 1), tc::mbar_init(&full[1], 1);
        tc::mbar_fence_init();
    }
    __syncthreads();
    float st[KP / 8][4], w[8][4];       // the adjoint and dU; of the warps ahead, what they hand over
#pragma unroll
    for (int n = 0; n < KP / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int v = g + e / 2 * 8, k = 8 * n + c2 + e % 2;
            st[n][e] = chain && p.dh_final && v < width && k < s.K ? p.dh_final[state_at + int64_t(mine + v) * s.K + k] : 0.0f;
        }
    wait_for_last();
    const int turns = span.blocks > 0 ? span.blocks + 1 : 0;
    if (asks && turns > 0) copy(0);
    for (int i = 0; i < turns; ++i) {
        wait_for(&full[i % 2], i / 2 & 1, abort, &g_device_error);
        const int rows_last = span.len - (span.blocks - 1) * kBlock;
        if (rows_last < kBlock && i < 2) {
            // the last block: it is ahead in the first turn, the chain's in the second
            if (i == 0) {
                clear_rows<KP>(base + L::at_ahead, rows_last, tid, kThreads);
                clear_rows<64>(base + L::at_ahead + L::tile, rows_last, tid, kThreads);
            } else {
                clear_rows<KP>(base + L::chain, rows_last, tid, kThreads);
                clear_rows<64>(base + L::chain + L::tile + 2 * kTile, rows_last, tid, kThreads);
            }
            tc::fence_proxy_async_smem();
        }
        __syncthreads();
        if (*reinterpret_cast<volatile int *>(abort)) break;
        if (asks && i + 1 < turns) copy(i + 1);
        if (!chain) {
            if (i > 0) {
#pragma unroll
                for (int n = 0; n < 8; ++n) put_values(hand_u + n * 512, w[n]);
#pragma unroll
                for (int n = 0; n < KP / 8; ++n) put_values(hand_s + n * 512, st[n]);
                asm volatile("bar.arrive 1, 256;" ::: "memory");
            }
            if (i == span.blocks) break;
            const int from = L::at_ahead + i % 2 * L::ahead;
            const uint32_t at = base + from, pairs = at + L::tile + L::v;
            const float *by = reinterpret_cast<const float *>(mem + L::scaled) + i % 2 * kBlock;
            uint32_t y[4][4];
#pragma unroll
            for (int t = 0; t < 4; ++t) load4t(y[t], four_across<64>(at + L::tile, 16 * t, 16 * warp));
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) w[n][e] = 0.0f;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                uint32_t b[4][4], rest[4][4];
#pragma unroll
                for (int r = 0; r <= t; ++r) {
                    load4t(b[r], four<64>(pairs, 16 * t, 16 * r));
                    load4t(rest[r], four<64>(pairs + kTile, 16 * t, 16 * r));
                }
                across_to(w, y[t], b, t);
                across_to(w, y[t], rest, t);
            }
            uint32_t hi[4][4], lo[4][4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 f = *reinterpret_cast<const float2 *>(by + 16 * t + 8 * h + c2);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        split(f.x * low(y[t][2 * h + e]), f.y * high(y[t][2 * h + e]), hi[t][2 * h + e], lo[t][2 * h + e]);
                }
#pragma unroll
            for (int n = 0; n < KP / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) st[n][e] = 0.0f;
            add_outer<KP>(st, hi, lo, at);
        } else if (i > 0) {
            const int c = span.blocks - i, rows = min(kBlock, span.len - c * kBlock);
            const int64_t row = span.first + int64_t(c) * kBlock;
            const int from = i % 2 * L::chain;
            const uint32_t at = base + from, room = base + L::out + warp * L::out_warp;
            const Factors &f = reinterpret_cast<const Factors *>(mem + L::factors)[i % 2];
            // A K^T
            through_tile<KP>(w, st, at, [&](int k, const uint32_t(&hi)[4]) { store4(four<KP, 16>(room, 0, 16 * k), hi); });
            __syncwarp();
            {
                bf *out = p.ds + ((span.slot + c) * s.H + head) * int64_t(s.V) * s.K + int64_t(mine) * s.K;
#pragma unroll
                for (int j = 0; j < 16 * KP / 8 / 32; ++j) {
                    const int v = (j * 32 + lane) / (KP / 8), k = (j * 32 + lane) % (KP / 8) * 8;
                    const uint4 x = load16(place<KP, 16>(room, v, k));
                    if (v < width && k < s.K) *reinterpret_cast<uint4 *>(out + int64_t(v) * s.K + k) = x;
                }
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
            // dU, and beta dU as two terms
            uint32_t hi[4][4], lo[4][4];
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                const float2 end = *reinterpret_cast<const float2 *>(f.end + 8 * n + c2);
                const float2 beta = *reinterpret_cast<const float2 *>(f.beta + 8 * n + c2);
                const float4 more = get_values(hand_u + n * 512);
                w[n][0] = kept(end.x, w[n][0]) + more.x, w[n][1] = kept(end.y, w[n][1]) + more.y;
                w[n][2] = kept(end.x, w[n][2]) + more.z, w[n][3] = kept(end.y, w[n][3]) + more.w;
                split(beta.x * w[n][0], beta.y * w[n][1], hi[n / 2][n % 2 * 2], lo[n / 2][n % 2 * 2]);
                split(beta.x * w[n][2], beta.y * w[n][3], hi[n / 2][n % 2 * 2 + 1], lo[n / 2][n % 2 * 2 + 1]);
            }
            // Z
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                uint32_t n[4][4], rest[4][4];
#pragma unroll
                for (int r = 0; r <= t; ++r) {
                    load4t(n[r], four<64>(at + L::tile, 16 * t, 16 * r));
                    load4t(rest[r], four<64>(at + L::tile + kTile, 16 * t, 16 * r));
                }
                across_to(w, hi[t], n, t);
                across_to(w, lo[t], n, t);
                across_to(w, hi[t], rest, t);
            }
            // shares of dbeta, dV, and -Gam beta Z
            float *part = p.dbeta_part + (((int64_t(slice) * kChain + warp) * slots + span.slot + c) * s.H + head) * kBlock;
            float sums[8][2];
            __syncwarp();
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                uint32_t x[4];
                load4t(x, four_across<64>(at + L::tile + 2 * kTile, 16 * t, 16 * warp));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int n = 2 * t + h;
                    sums[n][0] = w[n][0] * low(x[2 * h]) + w[n][2] * low(x[2 * h + 1]);
                    sums[n][1] = w[n][1] * high(x[2 * h]) + w[n][3] * high(x[2 * h + 1]);
                    const float2 beta = *reinterpret_cast<const float2 *>(f.beta + 8 * n + c2);
                    const float2 start = *reinterpret_cast<const float2 *>(f.start + 8 * n + c2);
                    w[n][0] *= beta.x, w[n][1] *= beta.y, w[n][2] *= beta.x, w[n][3] *= beta.y;
                    split(kept(-start.x, w[n][0]), kept(-start.y, w[n][1]), hi[t][2 * h], lo[t][2 * h]);
                    split(kept(-start.x, w[n][2]), kept(-start.y, w[n][3]), hi[t][2 * h + 1], lo[t][2 * h + 1]);
                }
                store_turned(room, t, w);
            }
            // of the columns' sums over eight lanes each lane keeps those of one n
#pragma unroll
            for (int half = 4; half > 0; half /= 2) {
                const bool upper = (g & half) != 0;
#pragma unroll
                for (int n = 0; n < half; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float give = upper ? sums[n][e] : sums[n + half][e];
                        sums[n][e] = (upper ? sums[n + half][e] : sums[n][e]) + __shfl_xor_sync(0xffffffffu, give, 4 * half);
                    }
            }
            *reinterpret_cast<float2 *>(part + 8 * g + c2) = make_float2(sums[0][0], sums[0][1]);
            __syncwarp();
            write_turned(p.dv + row * v_step + int64_t(head) * s.V + mine, v_step, rows, width, room);
            __syncwarp();
            // A
            const float last = f.last;
#pragma unroll
            for (int n = 0; n < KP / 8; ++n) {
                const float4 more = get_values(hand_s + n * 512);
                st[n][0] = kept(last, st[n][0]) + more.x, st[n][1] = kept(last, st[n][1]) + more.y;
                st[n][2] = kept(last, st[n][2]) + more.z, st[n][3] = kept(last, st[n][3]) + more.w;
            }
            add_outer<KP>(st, hi, lo, at);
        }
    }
    if (*reinterpret_cast<volatile int *>(abort)) {
        if (asks) linger();         // copies may still be on their way
        return;
    }
    if (chain && p.dh0)
#pragma unroll
        for (int n = 0; n < KP / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int v = g + e / 2 * 8, k = 8 * n + c2 + e % 2;
                if (v < width && k < s.K) p.dh0[state_at + int64_t(mine + v) * s.K + k] = st[n][e];
            }
    clear_uncovered(s, seq, p.dv + int64_t(head) * s.V + v0, v_step, min(kSlice, s.V - v0));
    if (slice == 0) {
        clear_uncovered(s, seq, p.dg + head, s.H, 1);
        clear_uncovered(s, seq, p.dbeta + head, s.H, 1);
        if (head < s.G) {
            clear_uncovered(s, seq, p.dq + int64_t(head) * s.K, qk_step, s.K);
            clear_uncovered(s, seq, p.dk + int64_t(head) * s.K, qk_step, s.K);
        }
    }
}

// ---- dQ, dK, dg of a block -------------------------------------------------------------
template <int KP, int VP>
struct BlockLayout {
    static constexpr int qk = kBlock * KP * 2, v = kBlock * 64 * 2, values = VP / 64 * v;
    static constexpr int states = VP * KP * 2;
    static constexpr int q = 0, k = q + qk, y = k + qk, x = y + values, dv = x + values, s0 = dv + values, s1 = s0 + states;
    static constexpr int dp = s1 + states, da = dp + kTile, bytes = da + kTile;
};

struct BlockMaps {
    CUtensorMap q, k, dy, x, dv, s0, s1;
};

// Warp 2 j + h: rows 16 j; of the pairs, those of the queries (h = 0) or of the
// keys (h = 1); of dQ and dK, columns h KP / 2 to (h + 1) KP / 2.
//
// dg needs, of the pairs' products M = dP P + dAb Ab, the sums over r >= t > s:
// a row's sums up to each column (over four lanes and the blocks of 16 columns),
// and those of the rows from t on.  Pairs on one side of step t never enter:
// differences of whole rows' and columns' sums would leave their rounding, 2^-24
// of everything in the block, where little or nothing crosses a step.
template <int KP, int VP>
__global__ void __launch_bounds__(256, VP == 64 ? 2 : 1)
block_kernel(const BwdArgs<bf> p, const __grid_constant__ BlockMaps maps, const int parts) {
    extern __shared__ __align__(1024) unsigned char mem[];
    __shared__ Decays d;
    __shared__ int found, abort;
    __shared__ __align__(8) uint64_t full[2];       // the block's rows; the states
    __shared__ float row_term[2][kBlock], col_term[2][kBlock], both_term[8];
    __shared__ float across_sum[8][kBlock];
    using L = BlockLayout<KP, VP>;
    let_next_begin();
    const Shape &s = p.s;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, c2 = lane % 4 * 2;
    const int head = int(blockIdx.x % s.H), group = head / (s.H / s.G);
    const int64_t slot = blockIdx.x / s.H;
    const int seq = sequence_of(s, slot, &found);
    if (seq < 0) {
        wait_for_last();        // or this grid could end before the one ahead of it
        return;
    }
    const Span span = span_of(s, seq);
    const int c = int(slot - span.slot), rows = min(kBlock, span.len - c * kBlock);
    const int64_t row = span.first + int64_t(c) * kBlock;
    const uint32_t base = smem_u32(mem);
    const int j = warp / 2, h = warp % 2;

    const auto ask_rows = [&](int tile, const CUtensorMap *map) {
#pragma unroll
        for (int v0 = 0; v0 < VP; v0 += 64) box(base + tile + v0 / 64 * L::v, map, &full[0], v0, head, int(row));
    };
    const auto ask_states = [&](int tile, const CUtensorMap *map) {
#pragma unroll
        for (int v0 = 0; v0 < VP; v0 += 64)
#pragma unroll
            for (int k = 0; k < KP; k += 64)
                box(base + tile + v0 * KP * 2 + k * kBlock * 2, map, &full[1], k, v0, int(slot * s.H + head));
    };
    if (tid == 32) {
        abort = 0;
        tc::mbar_init(&full[0], 1), tc::mbar_init(&full[1], 1);
        tc::mbar_fence_init();
        tc::mbar_arrive_expect_tx(&full[0], 2 * L::qk + 3 * L::values);
        tc::mbar_arrive_expect_tx(&full[1], 2 * L::states);
        boxes<KP>(base + L::q, &maps.q, &full[0], group, int(row));
        boxes<KP>(base + L::k, &maps.k, &full[0], group, int(row));
        ask_rows(L::y, &maps.dy);
        ask_rows(L::x, &maps.x);
        ask_states(L::s0, &maps.s0);
        // what the chain has written
        wait_for_last();
        ask_rows(L::dv, &maps.dv);
        ask_states(L::s1, &maps.s1);
    } else {
        wait_for_last();
    }
    if (warp == 0) load_decays(d, p.g + row * s.H + head, p.beta + row * s.H + head, s.H, rows);
    // dbeta: the shares of the chain's warps
    float share = 0.0f;
    if (tid >= 64 && tid < 128) {
        const int64_t slots = s.offsets ? s.L / kBlock + s.n : (s.L + kBlock - 1) / kBlock * s.n;
        for (int i = 0; i < parts; ++i) share += p.dbeta_part[((i * slots + slot) * s.H + head) * kBlock + tid - 64];
    }
    __syncthreads();
    wait_for(&full[0], 0, &abort, &g_device_error);
    if (rows < kBlock) {
        clear_rows<KP>(base + L::q, rows, tid, 256);
        clear_rows<KP>(base + L::k, rows, tid, 256);
        for (int v0 = 0; v0 < VP; v0 += 64) {
            clear_rows<64>(base + L::y + v0 / 64 * L::v, rows, tid, 256);
            clear_rows<64>(base + L::x + v0 / 64 * L::v, rows, tid, 256);
            clear_rows<64>(base + L::dv + v0 / 64 * L::v, rows, tid, 256);
        }
        __syncthreads();
    }
    // pairs: scale beta_s dY_t.x_s D with q_t.k_s, or -beta_s dV_t.x_s D with k_t.k_s
    {
        const uint32_t left = base + (h == 0 ? L::y : L::dv), key = base + (h == 0 ? L::q : L::k);
        const uint32_t out = base + (h == 0 ? L::dp : L::da);
        const float by = h == 0 ? s.scale : -1.0f;
        uint32_t fv[VP / 16][4], fk[KP / 16][4];
#pragma unroll
        for (int v = 0; v < VP / 16; ++v) load4(fv[v], four<64>(left + v / 4 * L::v, 16 * j, v % 4 * 16));
#pragma unroll
        for (int k = 0; k < KP / 16; ++k) load4(fk[k], four<KP>(key, 16 * j, 16 * k));
        const int t = 16 * j + g;
        const float hi0 = d.hi[t], lo0 = d.lo[t], hi1 = d.hi[t + 8], lo1 = d.lo[t + 8];
        const int cut0 = d.cut[t], cut1 = d.cut[t + 8];
        float before0 = 0.0f, before1 = 0.0f;       // of rows t and t + 8, M's columns up to here
#pragma unroll 1
        for (int n = 0; n <= j; ++n) {
            float a[2][4] = {}, m[2][4] = {}, down[4];
#pragma unroll
            for (int v = 0; v < VP / 16; ++v) {
                uint32_t b[4];
                load4(b, four_across<64>(base + L::x + v / 4 * L::v, 16 * n, v % 4 * 16));
                product(a[0], fv[v], b[0], b[1]);
                product(a[1], fv[v], b[2], b[3]);
            }
#pragma unroll
            for (int k = 0; k < KP / 16; ++k) {
                uint32_t b[4];
                load4(b, four_across<KP>(base + L::k, 16 * n, 16 * k));
                product(m[0], fk[k], b[0], b[1]);
                product(m[1], fk[k], b[2], b[3]);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 16 * n + 8 * e + c2;
                const float2 hi = *reinterpret_cast<const float2 *>(d.hi + r), lo = *reinterpret_cast<const float2 *>(d.lo + r);
                const float2 beta = *reinterpret_cast<const float2 *>(d.beta + r);
                const int2 cut = *reinterpret_cast<const int2 *>(d.cut + r);
                // below the diagonal; of the queries, on it as well
                const float x0 = t >= r + h && cut0 == cut.x ? by * beta.x * a[e][0] * ex2((hi0 - hi.x) + (lo0 - lo.x)) : 0.0f;
                const float x1 = t >= r + 1 + h && cut0 == cut.y ? by * beta.y * a[e][1] * ex2((hi0 - hi.y) + (lo0 - lo.y)) : 0.0f;
                const float x2 = t + 8 >= r + h && cut1 == cut.x ? by * beta.x * a[e][2] * ex2((hi1 - hi.x) + (lo1 - lo.x)) : 0.0f;
                const float x3 = t + 8 >= r + 1 + h && cut1 == cut.y ? by * beta.y * a[e][3] * ex2((hi1 - hi.y) + (lo1 - lo.y)) : 0.0f;
                const float m0 = t > r ? x0 * m[e][0] : 0.0f, m1 = t > r + 1 ? x1 * m[e][1] : 0.0f;
                const float m2 = t + 8 > r ? x2 * m[e][2] : 0.0f, m3 = t + 8 > r + 1 ? x3 * m[e][3] : 0.0f;
                // what the lanes before this one have in their two columns, and what all four have
                float up0 = m0 + m1, up1 = m2 + m3, left0 = 0.0f, left1 = 0.0f;
#pragma unroll
                for (int o = 1; o < 4; o *= 2) {
                    const float x = __shfl_xor_sync(0xffffffffu, up0, o), y = __shfl_xor_sync(0xffffffffu, up1, o);
                    if (lane & o) left0 += x, left1 += y;
                    up0 += x, up1 += y;
                }
                left0 += before0, left1 += before1;
                down[2 * e] = (t >= r ? left0 : 0.0f) + (t + 8 >= r ? left1 : 0.0f);
                down[2 * e + 1] = (t > r ? left0 + m0 : 0.0f) + (t + 8 > r ? left1 + m2 : 0.0f);
                before0 += up0, before1 += up1;
                const uint32_t w0 = pack(x0, x1), w1 = pack(x2, x3);
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(place<64>(out, t, r & ~7) + (r & 7) * 2), "r"(w0) : "memory");
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(place<64>(out, t + 8, r & ~7) + (r & 7) * 2), "r"(w1) : "memory");
            }
            // of the four columns' sums over the rows, each lane keeps one
            const bool upper = (g & 4) != 0, odd = (g & 2) != 0;
            const float of0 = (upper ? down[2] : down[0]) + __shfl_xor_sync(0xffffffffu, upper ? down[0] : down[2], 16);
            const float of1 = (upper ? down[3] : down[1]) + __shfl_xor_sync(0xffffffffu, upper ? down[1] : down[3], 16);
            float sum = (odd ? of1 : of0) + __shfl_xor_sync(0xffffffffu, odd ? of0 : of1, 8);
            sum += __shfl_xor_sync(0xffffffffu, sum, 4);
            if (g % 2 == 0) across_sum[warp][16 * n + 8 * upper + c2 + odd] = sum;
        }
        for (int r = 16 * (j + 1) + lane; r < kBlock; r += 32) across_sum[warp][r] = 0.0f;
    }
    wait_for(&full[1], 0, &abort, &g_device_error);
    __syncthreads();
    if (*reinterpret_cast<volatile int *>(&abort)) {
        linger();           // copies may still be on their way
        return;
    }
    // <S0, dS>
    {
        float both = 0.0f;
        for (int i = tid; i < VP * KP / 8; i += 256) {
            const int v = i / (KP / 8), k = i % (KP / 8) * 8;
            const uint32_t at = v / kBlock * (kBlock * KP * 2);
            const uint4 a = load16(place<KP>(base + L::s0 + at, v % kBlock, k)), b = load16(place<KP>(base + L::s1 + at, v % kBlock, k));
            both += low(a.x) * low(b.x) + high(a.x) * high(b.x) + low(a.y) * low(b.y) + high(a.y) * high(b.y) +
                    low(a.z) * low(b.z) + high(a.z) * high(b.z) + low(a.w) * low(b.w) + high(a.w) * high(b.w);
        }
#pragma unroll
        for (int o = 16; o > 0; o /= 2) both += __shfl_xor_sync(0xffffffffu, both, o);
        if (lane == 0) both_term[warp] = both;
    }
    const int t0 = 16 * j + g, t1 = t0 + 8;
    const float start0 = d.start(t0), start1 = d.start(t1), end0 = d.end(t0), end1 = d.end(t1);
    float rt0 = 0.0f, rt1 = 0.0f, ct0 = 0.0f, ct1 = 0.0f;
    constexpr int wide = KP / 2 < 64 ? KP / 2 : 64, tiles = wide / 8;      // columns at a time
#pragma unroll 1
    for (int k0 = h * (KP / 2); k0 < (h + 1) * (KP / 2); k0 += wide) {
        float dq[tiles][4] = {}, dk[tiles][4] = {};
        // through the state before the block
#pragma unroll 2
        for (int v = 0; v < VP / 16; ++v) {
            uint32_t a[4], z[4], b[tiles / 2][4];
            load4(a, four<64>(base + L::y + v / 4 * L::v, 16 * j, v % 4 * 16));
            load4(z, four<64>(base + L::dv + v / 4 * L::v, 16 * j, v % 4 * 16));
#pragma unroll
            for (int n = 0; n < tiles / 2; ++n) load4t(b[n], four<KP>(base + L::s0 + v / 4 * (kBlock * KP * 2), v % 4 * 16, k0 + 16 * n));
#pragma unroll
            for (int n = 0; n < tiles / 2; ++n) {
                product(dq[2 * n], a, b[n][0], b[n][1]);
                product(dq[2 * n + 1], a, b[n][2], b[n][3]);
                product(dk[2 * n], z, b[n][0], b[n][1]);
                product(dk[2 * n + 1], z, b[n][2], b[n][3]);
            }
        }
#pragma unroll
        for (int m = 0; m < tiles / 2; ++m) {
            uint32_t qs[4], ks[4];      // rows t0 and t1, columns c2 of tiles 2 m and 2 m + 1
            load4(qs, four<KP>(base + L::q, 16 * j, k0 + 16 * m));
            load4(ks, four<KP>(base + L::k, 16 * j, k0 + 16 * m));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = 2 * m + e;
                const uint32_t q0 = qs[2 * e], q1 = qs[2 * e + 1], e0 = ks[2 * e], e1 = ks[2 * e + 1];
                dq[n][0] = kept(s.scale * start0, dq[n][0]), dq[n][1] = kept(s.scale * start0, dq[n][1]);
                dq[n][2] = kept(s.scale * start1, dq[n][2]), dq[n][3] = kept(s.scale * start1, dq[n][3]);
                dk[n][0] = kept(-start0, dk[n][0]), dk[n][1] = kept(-start0, dk[n][1]);
                dk[n][2] = kept(-start1, dk[n][2]), dk[n][3] = kept(-start1, dk[n][3]);
                rt0 += dq[n][0] * low(q0) + dq[n][1] * high(q0) + dk[n][0] * low(e0) + dk[n][1] * high(e0);
                rt1 += dq[n][2] * low(q1) + dq[n][3] * high(q1) + dk[n][2] * low(e1) + dk[n][3] * high(e1);
            }
        }
        // through the pairs: dQ += (dP D) K, dK += (dAb D) K + (dAb D)^T K + (dP D)^T Q
#pragma unroll 1
        for (int r = 0; r < 4; ++r) {
            uint32_t b[tiles / 2][4];
#pragma unroll
            for (int n = 0; n < tiles / 2; ++n) load4t(b[n], four<KP>(base + L::k, 16 * r, k0 + 16 * n));
            if (r <= j) {
                uint32_t a[4], z[4];
                load4(a, four<64>(base + L::dp, 16 * j, 16 * r));
                load4(z, four<64>(base + L::da, 16 * j, 16 * r));
#pragma unroll
                for (int n = 0; n < tiles / 2; ++n) {
                    product(dq[2 * n], a, b[n][0], b[n][1]);
                    product(dq[2 * n + 1], a, b[n][2], b[n][3]);
                    product(dk[2 * n], z, b[n][0], b[n][1]);
                    product(dk[2 * n + 1], z, b[n][2], b[n][3]);
                }
            }
            if (r >= j) {
                uint32_t a[4], z[4];
                load4t(z, four_across<64>(base + L::da, 16 * r, 16 * j));
                load4t(a, four_across<64>(base + L::dp, 16 * r, 16 * j));
#pragma unroll
                for (int n = 0; n < tiles / 2; ++n) {
                    product(dk[2 * n], z, b[n][0], b[n][1]);
                    product(dk[2 * n + 1], z, b[n][2], b[n][3]);
                }
#pragma unroll
                for (int n = 0; n < tiles / 2; ++n) load4t(b[n], four<KP>(base + L::q, 16 * r, k0 + 16 * n));
#pragma unroll
                for (int n = 0; n < tiles / 2; ++n) {
                    product(dk[2 * n], a, b[n][0], b[n][1]);
                    product(dk[2 * n + 1], a, b[n][2], b[n][3]);
                }
            }
        }
        // two tiles at a time: a lane takes two of its columns and two of its neighbour's, so
        // that 32 bytes of a row are one access
        const auto write = [&](bf *whole, float *of_head, const float (&v)[tiles][4]) {
            const bool odd = lane % 2 != 0;
#pragma unroll
            for (int m = 0; m < tiles / 2; ++m)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = t0 + 8 * e, k = k0 + 16 * m;
                    const int64_t o = ((row + t) * s.H + head) * s.K;
                    const float *a = v[2 * m] + 2 * e, *b = v[2 * m + 1] + 2 * e;
                    if (s.H > s.G) {
                        if (t < rows && k + c2 < s.K) *reinterpret_cast<float2 *>(of_head + o + k + c2) = make_float2(a[0], a[1]);
                        if (t < rows && k + 8 + c2 < s.K) *reinterpret_cast<float2 *>(of_head + o + k + 8 + c2) = make_float2(b[0], b[1]);
                        continue;
                    }
                    const uint32_t even = pack(a[0], a[1]), next = pack(b[0], b[1]);
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? even : next, 1);
                    const int at = k + 8 * odd + (c2 & 4);
                    if (t < rows && at < s.K) *reinterpret_cast<uint2 *>(whole + o + at) = odd ? make_uint2(got, next) : make_uint2(even, got);
                }
        };
        write(p.dq, p.dq_head, dq);
        // through the adjoint of the state behind the block, in dQ's place
#pragma unroll
        for (int n = 0; n < tiles; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) dq[n][e] = 0.0f;
#pragma unroll 2
        for (int v = 0; v < VP / 16; ++v) {
            uint32_t a[4], b[tiles / 2][4];
            load4(a, four<64>(base + L::x + v / 4 * L::v, 16 * j, v % 4 * 16));
#pragma unroll
            for (int n = 0; n < tiles / 2; ++n) load4t(b[n], four<KP>(base + L::s1 + v / 4 * (kBlock * KP * 2), v % 4 * 16, k0 + 16 * n));
#pragma unroll
            for (int n = 0; n < tiles / 2; ++n) {
                product(dq[2 * n], a, b[n][0], b[n][1]);
                product(dq[2 * n + 1], a, b[n][2], b[n][3]);
            }
        }
        const float by0 = end0 * d.beta[t0], by1 = end1 * d.beta[t1];
#pragma unroll
        for (int m = 0; m < tiles / 2; ++m) {
            uint32_t ks[4];
            load4(ks, four<KP>(base + L::k, 16 * j, k0 + 16 * m));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = 2 * m + e;
                const uint32_t e0 = ks[2 * e], e1 = ks[2 * e + 1];
                const float a = kept(by0, dq[n][0]), b = kept(by0, dq[n][1]), x = kept(by1, dq[n][2]), y = kept(by1, dq[n][3]);
                ct0 += a * low(e0) + b * high(e0);
                ct1 += x * low(e1) + y * high(e1);
                dk[n][0] += a, dk[n][1] += b, dk[n][2] += x, dk[n][3] += y;
            }
        }
        write(p.dk, p.dk_head, dk);
    }
#pragma unroll
    for (int o = 1; o < 4; o *= 2) {
        rt0 += __shfl_xor_sync(0xffffffffu, rt0, o), rt1 += __shfl_xor_sync(0xffffffffu, rt1, o);
        ct0 += __shfl_xor_sync(0xffffffffu, ct0, o), ct1 += __shfl_xor_sync(0xffffffffu, ct1, o);
    }
    if (lane % 4 == 0) {
        row_term[h][t0] = rt0, row_term[h][t1] = rt1;
        col_term[h][t0] = ct0, col_term[h][t1] = ct1;
    }
    __syncthreads();
    // one warp, steps 2 lane and 2 lane + 1: sums over the steps behind and before each
    if (warp == 0) {
        float both = both_term[lane % 8];
#pragma unroll
        for (int o = 4; o > 0; o /= 2) both += __shfl_xor_sync(0xffffffffu, both, o);
        both = kept(d.start(kBlock - 1), both);
        float behind[2], before[2], crossing[2];        // this step's terms
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            crossing[e] = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) crossing[e] += across_sum[i][t];
            behind[e] = row_term[0][t] + row_term[1][t];
            before[e] = col_term[0][t] + col_term[1][t];
        }
        float up = behind[0] + behind[1], down = before[0] + before[1];
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const float x = __shfl_down_sync(0xffffffffu, up, o), y = __shfl_up_sync(0xffffffffu, down, o);
            if (lane + o < 32) up += x;
            if (lane >= o) down += y;
        }
        float first = __shfl_up_sync(0xffffffffu, down, 1), last = __shfl_down_sync(0xffffffffu, up, 1);
        if (lane == 0) first = 0.0f;
        if (lane == 31) last = 0.0f;
        const float at[2] = {crossing[0] + up + first, crossing[1] + behind[1] + last + first + before[0]};
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (2 * lane + e < rows) put(p.dg + (row + 2 * lane + e) * s.H + head, both + at[e]);
    }
    if (tid >= 64 && tid - 64 < rows) put(p.dbeta + (row + tid - 64) * s.H + head, share);
}

static bool on16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

bool fits(const BwdArgs<bf> &a) {
    return fits_bwd(a.s) && on16(a.q) && on16(a.k) && on16(a.dy) && on16(a.states) && on16(a.errors) && on16(a.dv) &&
           reinterpret_cast<uintptr_t>(a.dq) % 8 == 0 && reinterpret_cast<uintptr_t>(a.dk) % 8 == 0;
}

template <int KP>
static cudaError_t back(const BwdArgs<bf> &a, const Maps &maps, cudaStream_t st) {
    const int64_t grid = int64_t(a.s.n) * a.s.H * ((a.s.V + kSlice - 1) / kSlice);
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    constexpr int bytes = Layout<KP>::bytes;
    if (cudaError_t e = allow<back_kernel<KP>>(bytes)) return e;
    return launch_behind(back_kernel<KP>, unsigned(grid), kThreads, bytes, st, a, maps);
}
template <int KP, int VP>
static cudaError_t blocks(const BwdArgs<bf> &a, const BlockMaps &maps, cudaStream_t st) {
    const int64_t grid = a.s.slots() * a.s.H;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    constexpr int bytes = BlockLayout<KP, VP>::bytes;
    if (cudaError_t e = allow<block_kernel<KP, VP>>(bytes)) return e;
    return launch_behind(block_kernel<KP, VP>, unsigned(grid), 256, bytes, st, a, maps, dbeta_parts(a.s));
}

cudaError_t launch(const BwdArgs<bf> &a, cudaStream_t st) {
    Maps maps;
    if (!map_of(&maps.q, a.q, a.s.rows(), a.s.G, a.s.K) || !map_of(&maps.k, a.k, a.s.rows(), a.s.G, a.s.K) ||
        !map_of(&maps.dy, a.dy, a.s.rows(), a.s.H, a.s.V) || !map_of(&maps.x, a.errors, a.s.rows(), a.s.H, a.s.V))
        return cudaErrorInvalidValue;
    if (cudaError_t e = make_pairs(a.s, maps.q, maps.k, a.g, a.beta, a.records, true, nullptr, st)) return e;
    if (cudaError_t e = a.s.K <= 64 ? back<64>(a, maps, st) : back<128>(a, maps, st)) return e;
    BlockMaps of;
    of.q = maps.q, of.k = maps.k, of.dy = maps.dy, of.x = maps.x;
    const int64_t states = a.s.slots() * a.s.H;
    if (!map_of(&of.dv, a.dv, a.s.rows(), a.s.H, a.s.V) || !map_of(&of.s0, a.states, states, a.s.V, a.s.K, true) ||
        !map_of(&of.s1, a.ds, states, a.s.V, a.s.K, true))
        return cudaErrorInvalidValue;
    const cudaError_t e = a.s.K <= 64 ? (a.s.V <= 64 ? blocks<64, 64>(a, of, st) : blocks<64, 128>(a, of, st))
                                      : (a.s.V <= 64 ? blocks<128, 64>(a, of, st) : blocks<128, 128>(a, of, st));
    if (e) return e;
    return a.s.H > a.s.G ? general::fold(a, st) : cudaSuccess;
}

cudaError_t take_device_error(unsigned int *out) { return take_error(g_device_error, out); }

}  // namespace bwd
}  // namespace mma
}  // namespace delta
}  // namespace ssm
