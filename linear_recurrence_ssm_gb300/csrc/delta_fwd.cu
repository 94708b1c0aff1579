// delta_fwd.cu -- the gated delta rule, forward, bf16, on tensor cores.
//
// A thread block takes one head of one sequence and 64 rows of its state, and
// walks the sequence 64 steps at a time.  Four warps hold 16 rows each, as
// accumulators in fp32, from the first step to the last:
//   W^T = V^T - Gam (S K^T),  X^T = W^T - (beta W)^T N^T,  U = beta X
//   S = Gam_C S + (E U)^T K
// and hand S and U to four more warps, which form the block's outputs while
// the chain is at the next one:
//   Y^T = scale Gam (S Q^T) + U^T P^T.
// N and P come from pairs_kernel.  One thread asks for the tensor copies of the
// next block: memory takes its 64 KB slower than warps can ask for them piece by
// piece (a chain that did so stood still for 1000 of 6300 cycles, its outputs
// for 3500).  4 x 4096 steps of 32 heads of 64 x 128 take 201 us, 3.1 a block of
// 64 steps: the tensor cores are busy 51 % of it, and the rest is the chain's
// dependent products (S K^T, N beta W, E U K) waiting for one another.
//
// Operands of the state's own chain (S, beta W, N, E U) go into the tensor
// cores as two bf16 terms, 16 bits, without the low terms' product: 2^-17 of an
// operand.  States of 200 steps come out within 1.4e-5 of the 64-bit ones for
// beta up to 1, also where keys are all the same; for beta near 2 and keys alike,
// where sums over N cancel, within 3e-5 (beta 1.9, keys 0.2 apart) and 1.3e-4
// (beta 2, keys all the same; fp32 there 7e-6).  All 24 bits would cost twice
// the chain's products.  K and Q are bf16 as given.
// What y alone sees (S in S Q^T, U and P in U P) is one term, rounded by up to
// 2^-8 of itself as y is: y comes out within 3.4e-3 to 4e-3 in the 2-norm where
// its own rounding gives 1.7e-3, and two terms would double the outputs' products.
// What is kept for the gradients (S before a block, x) is rounded once to the
// inputs' type, half of what fp32 would have to be kept and read.
#include "delta_mma.cuh"

namespace ssm {
namespace delta {
namespace mma {
namespace fwd {

constexpr int kSlice = 64, kChain = 4, kThreads = 256;

template <int KP, bool CARRY>
struct Layout {
    static constexpr int tile = kBlock * KP * 2, v = kBlock * kSlice * 2;
    static constexpr int chain = tile + v + 2 * kTile;              // K, V, N in two terms: two of them
    static constexpr int outputs = 2 * chain, output = tile + kTile + 2048;      // Q, P, the factors: three of them
    static constexpr int handed = outputs + 3 * output;
    static constexpr int state = 16 * KP * 2, u = 16 * kBlock * 2;  // of a warp
    static constexpr int hand = kChain * (state + 2 * u);           // S, U, X: two of them
    static constexpr int bytes = CARRY ? 2 * chain + 2 * 2048 : handed + 2 * hand;
    static_assert(sizeof(Factors) <= 2048 && chain % 1024 == 0 && output % 1024 == 0 && bytes <= 232448 - 1024, "shared memory");
};

// CARRY: no outputs, only what a part adds to a state and what it makes of one
// (its rows of the identity: 64 rows of K more slices), by the four warps of
// the chain alone.
struct Maps {
    CUtensorMap q, k, v;
};
__device__ unsigned int g_device_error;

template <int KP, bool CARRY>
__global__ void __launch_bounds__(CARRY ? 32 * kChain : kThreads, CARRY ? 2 : 1)
fwd_kernel(const FwdArgs<bf> p, const __grid_constant__ Maps maps) {
    extern __shared__ __align__(1024) unsigned char mem[];
    __shared__ int found, abort;
    __shared__ __align__(8) uint64_t full[3];
    using L = Layout<KP, CARRY>;
    constexpr int threads = CARRY ? 32 * kChain : kThreads;
    let_next_begin();
    const Shape &s = p.s;
    const uint32_t base = smem_u32(mem);
    const int of_values = (s.V + kSlice - 1) / kSlice, slices = CARRY ? of_values + (s.K + kSlice - 1) / kSlice : of_values;
    const int slice = int(blockIdx.x % slices), head = int(blockIdx.x / slices % s.H);
    const int group = head / (s.H / s.G);
    const bool turning = CARRY && slice >= of_values;
    const int height = turning ? s.K : s.V, v0 = (turning ? slice - of_values : slice) * kSlice;
    const int64_t index = blockIdx.x / slices / s.H;        // of the sequence, or of the part's place
    int seq = int(index), part = 0;
    // A grid may not end before the one ahead of it, since the next one waits for
    // this one alone: blocks without work wait too.
    if (p.part) {
        seq = part_sequence_of(s, index, p.part, &found);
        if (seq < 0) {
            wait_for_last();
            return;
        }
    }
    Span span = span_of(s, seq);
    bool last_part = true;
    if (p.part) {
        part = int(index - first_part(s, span, seq, p.part));
        last_part = part + 1 == parts_of(span, p.part);
        if (CARRY && (last_part || (turning && part == 0 && !p.h0))) {
            wait_for_last();
            return;
        }
        const int first = part * p.part;
        span.first += int64_t(first) * kBlock;
        span.slot += first;
        span.len = min(span.len - first * kBlock, p.part * kBlock);
        span.blocks = min(span.blocks - first, p.part);
    }
    const float *entering = part == 0 ? p.h0 : p.entering;
    const int64_t entering_at = ((part == 0 ? int64_t(seq) : index) * s.H + head) * s.V * s.K;
    const int64_t v_step = int64_t(s.H) * s.V;
    const int tid = threadIdx.x, warp = tid / 32 % kChain, lane = tid % 32;
    const bool chain = tid < 32 * kChain;
    const int g = lane / 4, c2 = lane % 4 * 2, mine = v0 + 16 * warp;       // rows mine + g, mine + g + 8 of the state
    const int width = height - mine;                                        // of them, may be below 1 or above 16

    // One thread asks for what block c needs: K, V and N for the chain, Q, P and the factors for the outputs.
    const auto copy = [&](int c) {
        const int row = int(span.first + int64_t(c) * kBlock);
        const uint32_t to = base + c % 2 * L::chain;
        const uint32_t out = base + L::outputs + (CARRY ? c % 2 * 2048 : c % 3 * L::output);
        const unsigned char *record = p.scratch + ((span.slot + c) * s.H + head) * kRecord;
        uint64_t *bar = &full[c % 3];
        constexpr int factors = int(sizeof(Factors));
        tc::mbar_arrive_expect_tx(bar, L::tile + (turning ? 0 : L::v) + 2 * kTile + (CARRY ? 0 : L::tile + kTile) + factors);
        boxes<KP>(to, &maps.k, bar, group, row);
        if (!turning) box(to + L::tile, &maps.v, bar, v0, head, row);
        bulk(to + L::tile + L::v, record, 2 * kTile, bar);
        if (CARRY) {
            bulk(out, record + 3 * kTile, factors, bar);
        } else {
            boxes<KP>(out, &maps.q, bar, group, row);
            bulk(out + L::tile, record + 2 * kTile, kTile + factors, bar);
        }
    };
    const bool asks = tid == (CARRY ? 0 : 32 * kChain);
    if (asks) {
        abort = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i) tc::mbar_init(&full[i], 1);
        tc::mbar_fence_init();
    }
    // no values of a part's identity: they are zeros from here on
    if (turning)
#pragma unroll
        for (int i = 0; i < 2; ++i) clear_rows<64>(base + i * L::chain + L::tile, 0, tid, threads);
    __syncthreads();
    wait_for_last();
    float st[KP / 8][4];
    if (chain) {
#pragma unroll
        for (int n = 0; n < KP / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int v = g + e / 2 * 8, k = 8 * n + c2 + e % 2;
                if (CARRY) st[n][e] = turning && mine + v == k ? 1.0f : 0.0f;
                else st[n][e] = entering && v < width && k < s.K ? entering[entering_at + int64_t(mine + v) * s.K + k] : 0.0f;
            }
    }
    if (asks && span.blocks > 0) copy(0);
    // the chain is at block c, the outputs at the one before
    for (int c = 0; c < span.blocks + (CARRY ? 0 : 1); ++c) {
        if (c < span.blocks) {
            wait_for(&full[c % 3], c / 3 & 1, &abort, &g_device_error);
            const int rows = span.len - c * kBlock;
            if (rows < kBlock) {
                const uint32_t to = base + c % 2 * L::chain;
                clear_rows<KP>(to, rows, tid, threads);
                clear_rows<64>(to + L::tile, rows, tid, threads);
                if (!CARRY) clear_rows<KP>(base + L::outputs + c % 3 * L::output, rows, tid, threads);
            }
        }
        __syncthreads();
        if (*reinterpret_cast<volatile int *>(&abort)) break;
        if (asks && c + 1 < span.blocks) copy(c + 1);
        if (chain) {
            if (c == span.blocks) break;
            const uint32_t at = base + c % 2 * L::chain, hand = base + L::handed + c % 2 * L::hand;
            const uint32_t hand_u = hand + kChain * L::state + warp * L::u, hand_x = hand_u + kChain * L::u;
            const Factors &f = *reinterpret_cast<const Factors *>(
                mem + L::outputs + (CARRY ? c % 2 * 2048 : c % 3 * L::output + L::tile + kTile));
            float w[8][4];
            through_tile<KP>(w, st, at, [&](int k, const uint32_t(&hi)[4]) {
                if (!CARRY) store4(four<KP, 16>(hand + warp * L::state, 0, 16 * k), hi);
            });
            // from here on the tensor cores have room for the outputs
            if (!CARRY && c > 0) asm volatile("bar.arrive 1, 256;" ::: "memory");
            // W, beta W as two terms, and X in W's place
            uint32_t hi[4][4], lo[4][4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                uint32_t v[4];
                load4t(v, four_across<64>(at + L::tile, 16 * t, 16 * warp));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 by = *reinterpret_cast<const float2 *>(f.start + 16 * t + 8 * h + c2);
                    const float2 beta = *reinterpret_cast<const float2 *>(f.beta + 16 * t + 8 * h + c2);
                    float(&x)[4] = w[2 * t + h];
                    x[0] = low(v[2 * h]) - kept(by.x, x[0]);
                    x[1] = high(v[2 * h]) - kept(by.y, x[1]);
                    x[2] = low(v[2 * h + 1]) - kept(by.x, x[2]);
                    x[3] = high(v[2 * h + 1]) - kept(by.y, x[3]);
                    split(beta.x * x[0], beta.y * x[1], hi[t][2 * h], lo[t][2 * h]);
                    split(beta.x * x[2], beta.y * x[3], hi[t][2 * h + 1], lo[t][2 * h + 1]);
                }
            }
            // of a block with a cut: what is not finite in the state stays out of the steps behind it
            const float last = f.last;
            unsigned bad = 0;
            if (last == 0.0f && (bad = not_finite(st)) != 0) {
#pragma unroll
                for (int t = 0; t < 4; ++t) drop(hi[t], bad, f.start + 16 * t), drop(lo[t], bad, f.start + 16 * t);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                uint32_t n[4][4], rest[4][4];
#pragma unroll
                for (int t = r; t < 4; ++t) {
                    load4(n[t], four_across<64>(at + L::tile + L::v, 16 * t, 16 * r));
                    load4(rest[t], four_across<64>(at + L::tile + L::v + kTile, 16 * t, 16 * r));
                }
                across(w, hi[r], n, r);
                across(w, lo[r], n, r);
                across(w, hi[r], rest, r);
            }
            // U for the outputs, E U for the state, X to be kept
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                uint32_t u[4];
                if (!CARRY && p.errors) store_turned(hand_x, t, w);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 beta = *reinterpret_cast<const float2 *>(f.beta + 16 * t + 8 * h + c2);
                    const float2 end = *reinterpret_cast<const float2 *>(f.end + 16 * t + 8 * h + c2);
                    const float(&x)[4] = w[2 * t + h];
                    const float a = beta.x * x[0], b = beta.y * x[1], d = beta.x * x[2], e = beta.y * x[3];
                    u[2 * h] = pack(a, b);
                    u[2 * h + 1] = pack(d, e);
                    split(kept(end.x, a), kept(end.y, b), hi[t][2 * h], lo[t][2 * h]);
                    split(kept(end.x, d), kept(end.y, e), hi[t][2 * h + 1], lo[t][2 * h + 1]);
                }
                if (!CARRY) store4(four<64, 16>(hand_u, 0, 16 * t), u);
            }
            if (!CARRY && __any_sync(0xffffffffu, bad)) {
                __syncwarp();
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    uint32_t u[4];
                    load4(u, four<64, 16>(hand_u, 0, 16 * t));
                    drop(u, bad, f.start + 16 * t);
                    store4(four<64, 16>(hand_u, 0, 16 * t), u);
                }
            }
            // S
#pragma unroll
            for (int n = 0; n < KP / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) st[n][e] = kept(last, st[n][e]);
            add_outer<KP>(st, hi, lo, at);
        } else if (!CARRY && c > 0) {
            const int rows = min(kBlock, span.len - (c - 1) * kBlock);
            const int64_t row = span.first + int64_t(c - 1) * kBlock;
            const int from = L::outputs + (c - 1) % 3 * L::output;
            const uint32_t at = base + from;
            const uint32_t hand = base + L::handed + (c - 1) % 2 * L::hand, hand_s = hand + warp * L::state;
            const uint32_t hand_u = hand + kChain * L::state + warp * L::u, hand_x = hand_u + kChain * L::u;
            const Factors &f = *reinterpret_cast<const Factors *>(mem + from + L::tile + kTile);
            const int64_t out_at = row * v_step + int64_t(head) * s.V + mine;
            if (p.states) {
                bf *out = p.states + ((span.slot + c - 1) * s.H + head) * int64_t(s.V) * s.K + int64_t(mine) * s.K;
#pragma unroll
                for (int i = 0; i < 16 * KP / 8 / 32; ++i) {
                    const int v = (i * 32 + lane) / (KP / 8), k = (i * 32 + lane) % (KP / 8) * 8;
                    const uint4 w = load16(place<KP, 16>(hand_s, v, k));
                    if (v < width && k < s.K) *reinterpret_cast<uint4 *>(out + int64_t(v) * s.K + k) = w;
                }
                write_turned(p.errors + out_at, v_step, rows, width, hand_x);
                __syncwarp();
            }
            // not before the chain is through its first products, which all else waits for
            if (c < span.blocks) asm volatile("bar.sync 1, 256;" ::: "memory");
            float y[8][4] = {};
            {
                uint32_t b[2][4][4], a[2][4];
                load4(a[0], four<KP, 16>(hand_s, 0, 0));
#pragma unroll
                for (int t = 0; t < 4; ++t) load4(b[0][t], four_across<KP>(at, 16 * t, 0));
#pragma unroll
                for (int k = 0; k < KP / 16; ++k) {
                    if (k + 1 < KP / 16) {
                        load4(a[(k + 1) % 2], four<KP, 16>(hand_s, 0, 16 * (k + 1)));
#pragma unroll
                        for (int t = 0; t < 4; ++t) load4(b[(k + 1) % 2][t], four_across<KP>(at, 16 * t, 16 * (k + 1)));
                    }
                    across(y, a[k % 2], b[k % 2]);
                }
            }
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float2 by = *reinterpret_cast<const float2 *>(f.start_scaled + 8 * t + c2);
                y[t][0] = kept(by.x, y[t][0]), y[t][1] = kept(by.y, y[t][1]);
                y[t][2] = kept(by.x, y[t][2]), y[t][3] = kept(by.y, y[t][3]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                uint32_t u[4], b[4][4];
                load4(u, four<64, 16>(hand_u, 0, 16 * r));
#pragma unroll
                for (int t = r; t < 4; ++t) load4(b[t], four_across<64>(at + L::tile, 16 * t, 16 * r));
                across(y, u, b, r);
            }
            // through shared memory, where X was: 32 bytes of a row are one access
#pragma unroll
            for (int t = 0; t < 4; ++t) store_turned(hand_x, t, y);
            __syncwarp();
            write_turned(p.y + out_at, v_step, rows, width, hand_x);
        }
    }
    if (*reinterpret_cast<volatile int *>(&abort)) {
        // copies may still be on their way to this block's shared memory
        if (asks) linger();
        return;
    }
    float *out = CARRY ? (turning ? p.turned : p.added) : last_part ? p.h_final : nullptr;
    if (chain && out) {
        out += ((CARRY ? index : int64_t(seq)) * s.H + head) * height * s.K;
#pragma unroll
        for (int n = 0; n < KP / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int v = g + e / 2 * 8, k = 8 * n + c2 + e % 2;
                if (v < width && k < s.K) out[int64_t(mine + v) * s.K + k] = st[n][e];
            }
    }
    if (!CARRY && part == 0) {
        clear_uncovered(s, seq, p.y + int64_t(head) * s.V + v0, v_step, min(kSlice, s.V - v0));
        if (p.errors) clear_uncovered(s, seq, p.errors + int64_t(head) * s.V + v0, v_step, min(kSlice, s.V - v0));
    }
}

// The states that enter a sequence's parts: S_(i + 1) = S_i T_i + B_i, four
// rows of one head a thread block.  Rows are independent; T is read from L2, a
// quarter of its rows by each quarter of the threads.
constexpr int kJoinRows = 4, kJoinSplit = 4;
__global__ void __launch_bounds__(128 * kJoinSplit) join_kernel(const FwdArgs<bf> p) {
    __shared__ float S[kJoinRows][128], shares[kJoinSplit][kJoinRows][128];
    let_next_begin();
    wait_for_last();
    const Shape &s = p.s;
    const int tiles = (s.V + kJoinRows - 1) / kJoinRows, k = threadIdx.x % 128, quarter = threadIdx.x / 128;
    const int v0 = int(blockIdx.x % tiles) * kJoinRows, head = int(blockIdx.x / tiles % s.H), seq = int(blockIdx.x / tiles / s.H);
    const Span span = span_of(s, seq);
    const int parts = parts_of(span, p.part), rows = min(kJoinRows, s.V - v0);
    const int64_t first = first_part(s, span, seq, p.part);
    const bool in = k < s.K;
    // this thread's row, column of the result
    const int mine = quarter;
    const bool has = in && mine < rows;
    S[mine][k] = p.h0 && has ? p.h0[((int64_t(seq) * s.H + head) * s.V + v0 + mine) * s.K + k] : 0.0f;
    for (int i = 0; i + 1 < parts; ++i) {
        const int64_t at = (first + i) * s.H + head;
        const float added = has ? p.added[(at * s.V + v0 + mine) * s.K + k] : 0.0f;
        const float *turned = p.turned + at * s.K * s.K + k;
        float sum[kJoinRows] = {};
        uint32_t any = 0;
        __syncthreads();
        // the first part starts from h0: nothing was made of it, unless there is one
        if (in && (i > 0 || p.h0)) {
            const int each = (s.K + kJoinSplit - 1) / kJoinSplit, to = min((quarter + 1) * each, s.K);
            for (int m = quarter * each; m < to; m += 16) {
                float t[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) t[j] = m + j < to ? turned[int64_t(m + j) * s.K] : 0.0f;
#pragma unroll
                for (int j = 0; j < 16; ++j) any |= __float_as_uint(t[j]) << 1;
#pragma unroll
                for (int j = 0; j < 16; ++j)
#pragma unroll
                    for (int v = 0; v < kJoinRows; ++v) sum[v] += S[v][min(m + j, 127)] * t[j];
            }
        }
#pragma unroll
        for (int v = 0; v < kJoinRows; ++v) shares[quarter][v][k] = sum[v];
        // a part that makes nothing of a state (a step in it has no decay left) drops it, whatever it holds
        const bool reaches = __syncthreads_or(any != 0);
        float all = added;
        if (reaches) {
#pragma unroll
            for (int j = 0; j < kJoinSplit; ++j) all += shares[j][mine][k];
        }
        S[mine][k] = all;
        if (has) p.entering[((at + s.H) * s.V + v0 + mine) * s.K + k] = all;
    }
}
static_assert(kJoinRows == kJoinSplit, "a row a quarter");

template <int KP, bool CARRY>
static cudaError_t go(const FwdArgs<bf> &a, const Maps &maps, int64_t places, cudaStream_t st) {
    const int64_t slices = (a.s.V + kSlice - 1) / kSlice + (CARRY ? (a.s.K + kSlice - 1) / kSlice : 0);
    const int64_t grid = places * a.s.H * slices;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    constexpr int bytes = Layout<KP, CARRY>::bytes;
    if (cudaError_t e = allow<fwd_kernel<KP, CARRY>>(bytes)) return e;
    return launch_behind(fwd_kernel<KP, CARRY>, unsigned(grid), CARRY ? 32 * kChain : kThreads, bytes, st, a, maps);
}

static bool on16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Rows that 16-byte copies can take.
bool fits(const FwdArgs<bf> &a) {
    return mma::fits(a.s) && on16(a.q) && on16(a.k) && on16(a.v) && on16(a.y) && on16(a.states) && on16(a.errors);
}

cudaError_t launch(FwdArgs<bf> a, cudaStream_t st) {
    Maps maps;
    if (!map_of(&maps.q, a.q, a.s.rows(), a.s.G, a.s.K) || !map_of(&maps.k, a.k, a.s.rows(), a.s.G, a.s.K) ||
        !map_of(&maps.v, a.v, a.s.rows(), a.s.H, a.s.V))
        return cudaErrorInvalidValue;
    if (cudaError_t e = make_pairs(a.s, maps.q, maps.k, a.g, a.beta, a.scratch, false, a.states, st)) return e;
    const FwdScratch at = fwd_scratch(a.s);
    const bool wide = a.s.K > 64;
    a.part = at.part;
    if (!a.part) return wide ? go<128, false>(a, maps, a.s.n, st) : go<64, false>(a, maps, a.s.n, st);
    a.added = reinterpret_cast<float *>(a.scratch + at.added);
    a.turned = reinterpret_cast<float *>(a.scratch + at.turned);
    a.entering = reinterpret_cast<float *>(a.scratch + at.entering);
    const int64_t places = part_places(a.s, a.part);
    if (cudaError_t e = wide ? go<128, true>(a, maps, places, st) : go<64, true>(a, maps, places, st)) return e;
    if (cudaError_t e = launch_behind(join_kernel, unsigned((a.s.V + kJoinRows - 1) / kJoinRows * a.s.H * a.s.n),
                                      128 * kJoinSplit, 0, st, a))
        return e;
    return wide ? go<128, false>(a, maps, places, st) : go<64, false>(a, maps, places, st);
}

// Self-test of the wait: for a copy that was never asked for.
__global__ void __launch_bounds__(32) run_out_kernel() {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int abort;
    if (threadIdx.x == 0) {
        abort = 0;
        tc::mbar_init(&bar, 1);
        tc::mbar_fence_init();
    }
    __syncthreads();
    wait_for(&bar, 0, &abort, &g_device_error, 20000000ull);
    __syncthreads();
    // what a kernel then does in its remaining turns: it has to wait no more
    if (*reinterpret_cast<volatile int *>(&abort)) return;
    linger();
}
cudaError_t probe_wait_timeout(cudaStream_t st) {
    run_out_kernel<<<1, 32, 0, st>>>();
    return cudaGetLastError();
}

cudaError_t take_device_error(unsigned int *out) { return take_error(g_device_error, out); }

}  // namespace fwd
}  // namespace mma
}  // namespace delta
}  // namespace ssm
