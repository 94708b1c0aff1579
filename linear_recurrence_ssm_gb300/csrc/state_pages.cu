// state_pages.cu -- pages of a state cache: copied, forked, freed, compacted.
//
// A pool holds (layers, pages, page bytes); page p of every layer belongs to
// one sequence (a recurrent state is overwritten at every token, so forked
// sequences cannot share a page).  `used` has one byte for each page.
//
// fork and compact are two launches: one block plans (prefix sums over the
// bytes, 16 pages a thread), then all SMs copy.  The copy is launched early
// and waits for the plan on the device.  Bound by the copy's bytes: 100 pages
// of 1 MB in 4 layers, 839 MB, 118 us (7.1 TB/s); 500 of 2048 pages of 10 KB
// in 24 layers, 251 MB, 37 us (6.8 TB/s); the plans take 5 and 9 us.  Pages
// that are no multiples of 16 bytes are copied in words of 4, or of 1: 500 pages
// of 10 KB in 24 layers, 246 MB (bytes: 36 us), with the start of the launch 45
// us in words of 16 bytes, 61 of 4 (fp32, 2561 elements), 143 of 1 (bf16, 5121).
#include "ssm_common.cuh"

#include <algorithm>

namespace ssm {
namespace pages {

constexpr int kPlan = 1024;   // threads of the planning kernels' one block
constexpr int kEach = 16;     // pages a thread looks at in one sweep

// Exclusive prefix sum of v over the block, and the total.
__device__ __forceinline__ int block_prefix(int v, int *warp_sums, int *total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int s = v;
    for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += o;
    }
    __syncthreads();          // the sums of the sweep before have been read
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    int w = warp_sums[lane];  // kPlan / 32 = 32 warps
    for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += o;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) % 32);
    return (warp ? before : 0) + s - v;
}

// Bit i: page p0 + i is in use; bits behind the pool's end are 0.
__device__ __forceinline__ uint32_t use_bits(const uint8_t *used, int64_t p0, int64_t num_pages) {
    uint32_t bits = 0;
    if (p0 + kEach <= num_pages && reinterpret_cast<uintptr_t>(used + p0) % 16 == 0) {
        const uint4 w = *reinterpret_cast<const uint4 *>(used + p0);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            for (int k = 0; k < 4; ++k) bits |= uint32_t((u[i] >> (8 * k) & 0xff) != 0) << (4 * i + k);
    } else {
        for (int i = 0; i < kEach && p0 + i < num_pages; ++i) bits |= uint32_t(used[p0 + i] != 0) << i;
    }
    return bits;
}
// The bits of the pages that the pool has.
__device__ __forceinline__ uint32_t real_bits(int64_t p0, int64_t num_pages) {
    const int64_t n = num_pages - p0;
    return n >= kEach ? (1u << kEach) - 1 : n <= 0 ? 0 : (1u << n) - 1;
}

// dst[k] for every request: the r-th valid one takes the r-th lowest free page.
// dst holds the free pages in their order first.  The requests are then
// answered from the last to the first: r <= k, so nothing is overwritten that
// is still to be read.
__global__ void __launch_bounds__(kPlan)
fork_plan_kernel(uint8_t *used, const int32_t *__restrict__ src, int32_t *dst, int64_t n, int64_t num_pages) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ int sums[kPlan / 32];
    int64_t found = 0;
    for (int64_t s0 = 0; s0 < num_pages && found < n; s0 += kPlan * kEach) {
        const int64_t p0 = s0 + int64_t(threadIdx.x) * kEach;
        uint32_t bits = real_bits(p0, num_pages);
        if (bits) bits &= ~use_bits(used, p0, num_pages);
        int all;
        int64_t at = found + block_prefix(__popc(bits), sums, &all);
        for (; bits && at < n; bits &= bits - 1) dst[at++] = int32_t(p0 + __ffs(bits) - 1);
        found += all;
    }
    auto valid = [&](int64_t k) {
        const int s = k < n ? src[k] : -2;
        return int(s == -1 || (s >= 0 && s < num_pages && used[s] != 0));
    };
    int mine = 0, all;
    for (int64_t k = threadIdx.x; k < n; k += kPlan) mine += valid(k);
    block_prefix(mine, sums, &all);
    int64_t left = all;       // valid requests up to this chunk's end
    for (int64_t k0 = (n - 1) / kPlan * kPlan; k0 >= 0; k0 -= kPlan) {
        const int64_t k = k0 + threadIdx.x;
        const int v = valid(k), at = block_prefix(v, sums, &all);
        left -= all;
        const int page = v && left + at < found ? dst[left + at] : -1;
        __syncthreads();
        if (k < n) dst[k] = page;
    }
    __syncthreads();
    for (int64_t k = threadIdx.x; k < n; k += kPlan)
        if (dst[k] >= 0) used[dst[k]] = 1;
}

// moved[p]: where page p's content is afterwards, -1 for a free page; the
// moves' number, sources and targets in list[0], list + 2 and list + 2 + pages.
__global__ void __launch_bounds__(kPlan)
compact_plan_kernel(uint8_t *used, int32_t *moved, int32_t *list, int32_t *pages, int64_t n, int64_t num_pages) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ int sums[kPlan / 32];
    const int64_t per_sweep = int64_t(kPlan) * kEach;
    int mine = 0, all;
    for (int64_t p0 = int64_t(threadIdx.x) * kEach; p0 < num_pages; p0 += per_sweep)
        mine += __popc(use_bits(used, p0, num_pages));
    block_prefix(mine, sums, &all);
    const int64_t live = all;
    int32_t *from = list + 2, *to = list + 2 + num_pages;
    int64_t holes = 0, movers = 0;
    for (int64_t s0 = 0; s0 < num_pages; s0 += per_sweep) {
        const int64_t p0 = s0 + int64_t(threadIdx.x) * kEach;
        const uint32_t real = real_bits(p0, num_pages), low = real_bits(p0, live);
        const uint32_t in_use = real ? use_bits(used, p0, num_pages) : 0;
        uint32_t hole = low & ~in_use, mover = in_use & ~low;
        // both counts of a sweep fit 16 bits
        const int at = block_prefix(__popc(hole) << 16 | __popc(mover), sums, &all);
        int64_t h = holes + (at >> 16), m = movers + (at & 0xffff);
        for (; hole; hole &= hole - 1) to[h++] = int32_t(p0 + __ffs(hole) - 1);
        for (uint32_t left = mover; left; left &= left - 1) from[m++] = int32_t(p0 + __ffs(left) - 1);
        for (int i = 0; i < kEach && p0 + i < num_pages; ++i) {
            moved[p0 + i] = in_use >> i & 1 ? int32_t(p0 + i) : -1;
            used[p0 + i] = low >> i & 1;
        }
        holes += all >> 16;
        movers += all & 0xffff;
    }
    __syncthreads();
    if (threadIdx.x == 0) list[0] = int32_t(movers);
    for (int64_t k = threadIdx.x; k < movers; k += kPlan) moved[from[k]] = to[k];
    __syncthreads();
    for (int64_t k = threadIdx.x; k < n; k += kPlan) {
        const int p = pages[k];
        if (p >= 0) pages[k] = p < num_pages ? moved[p] : -1;
    }
}

// Copies page from[k] to page to[k] of every layer; from -1 writes zeros.
// `count` (device) or `n` says how many.  A warp copies 128 words at a time,
// four loads in flight a lane; the warps walk along a page, then the list,
// then the layers.
template <typename V>
__global__ void __launch_bounds__(256)
copy_kernel(V *pool, const int32_t *from, const int32_t *to, const int32_t *count, int64_t n, int64_t layers,
            int64_t num_pages, int64_t words) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (count) n = *count;
    const int lane = threadIdx.x % 32;
    const int64_t parts = (words + 127) / 128, total = parts * n * layers;
    for (int64_t u = int64_t(blockIdx.x) * 8 + threadIdx.x / 32; u < total; u += int64_t(gridDim.x) * 8) {
        int64_t rest, w0, k, layer;
        if (total <= 0xffffffffll) {      // 32-bit divisions
            const uint32_t r = uint32_t(u) / uint32_t(parts);
            rest = r, w0 = int64_t(uint32_t(u) - r * uint32_t(parts)) * 128 + lane;
            layer = r / uint32_t(n), k = rest - layer * n;
        } else {
            rest = u / parts, w0 = u % parts * 128 + lane, layer = rest / n, k = rest % n;
        }
        const int64_t f = from[k], t = to[k];
        if (t < 0 || t >= num_pages || f < -1 || f >= num_pages) continue;
        const V *src = pool + (layer * num_pages + f) * words;
        V *dst = pool + (layer * num_pages + t) * words;
        V v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = V{};
            if (f >= 0 && w0 + 32 * i < words) v[i] = src[w0 + 32 * i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (w0 + 32 * i < words) dst[w0 + 32 * i] = v[i];
    }
}

__global__ void __launch_bounds__(256)
free_kernel(uint8_t *__restrict__ used, const int32_t *__restrict__ pages, int64_t n, int64_t num_pages) {
    const int64_t k = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (k >= n) return;
    const int p = pages[k];
    if (p >= 0 && p < num_pages) used[p] = 0;
}

// `most`: how many pages there can be to copy.  `after_plan`: the kernel
// before it on the stream is a plan, whose end the copy waits for by itself.
template <typename V>
static cudaError_t start_copy(void *pool, const int32_t *from, const int32_t *to, const int32_t *count, int64_t n,
                              int64_t most, int64_t layers, int64_t num_pages, int64_t bytes, int num_sms,
                              bool after_plan, cudaStream_t st) {
    const int64_t words = bytes / int64_t(sizeof(V));
    const int64_t units = (words + 127) / 128 * most * layers;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(std::min<int64_t>((units + 7) / 8, int64_t(num_sms) * 8)));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = after_plan ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, copy_kernel<V>, static_cast<V *>(pool), from, to, count, n, layers, num_pages,
                              words);
}

static cudaError_t run_copy(void *pool, const int32_t *from, const int32_t *to, const int32_t *count, int64_t n,
                            int64_t most, int64_t layers, int64_t num_pages, int64_t bytes, int num_sms,
                            bool after_plan, cudaStream_t st) {
    const uintptr_t all = reinterpret_cast<uintptr_t>(pool) | uintptr_t(bytes);
    auto start = all % 16 == 0 ? start_copy<uint4> : all % 4 == 0 ? start_copy<uint32_t> : start_copy<uint8_t>;
    return start(pool, from, to, count, n, most, layers, num_pages, bytes, num_sms, after_plan, st);
}

cudaError_t copy(void *pool, const int32_t *src, const int32_t *dst, int64_t n, int64_t layers,
                 int64_t num_pages, int64_t bytes, int num_sms, cudaStream_t st) {
    return run_copy(pool, src, dst, nullptr, n, n, layers, num_pages, bytes, num_sms, false, st);
}

cudaError_t fork(void *pool, uint8_t *used, const int32_t *src, int32_t *dst, int64_t n, int64_t layers,
                 int64_t num_pages, int64_t bytes, int num_sms, cudaStream_t st) {
    fork_plan_kernel<<<1, kPlan, 0, st>>>(used, src, dst, n, num_pages);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    return run_copy(pool, src, dst, nullptr, n, n, layers, num_pages, bytes, num_sms, true, st);
}

cudaError_t free_pages(uint8_t *used, const int32_t *pages, int64_t n, int64_t num_pages, cudaStream_t st) {
    free_kernel<<<unsigned((n + 255) / 256), 256, 0, st>>>(used, pages, n, num_pages);
    return cudaGetLastError();
}

cudaError_t compact(void *pool, uint8_t *used, int32_t *moved, int32_t *pages, int32_t *scratch, int64_t n,
                    int64_t layers, int64_t num_pages, int64_t bytes, int num_sms, cudaStream_t st) {
    compact_plan_kernel<<<1, kPlan, 0, st>>>(used, moved, scratch, pages, n, num_pages);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    return run_copy(pool, scratch + 2, scratch + 2 + num_pages, scratch, 0, num_pages / 2 + 1, layers, num_pages, bytes,
                    num_sms, true, st);
}

}  // namespace pages
}  // namespace ssm
