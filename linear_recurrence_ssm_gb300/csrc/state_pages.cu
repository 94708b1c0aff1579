// state_pages.cu -- pages of a state cache: copied, forked, freed, compacted.
//
// A pool holds (layers, pages, page bytes); page p of every layer belongs to
// one sequence (a recurrent state is overwritten at every token, so forked
// sequences cannot share a page).  `used` has one byte for each page.
#include "ssm_common.cuh"

namespace ssm {
namespace pages {

constexpr int kPlan = 1024;   // threads of the planning kernels' one block

// Exclusive prefix sum of v over the block, and the total.
__device__ __forceinline__ int block_prefix(int v, int *warp_sums, int *total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int s = v;
    for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += o;
    }
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kPlan / 32; ++w) {
        if (w < warp) before += warp_sums[w];
        all += warp_sums[w];
    }
    __syncthreads();
    *total = all;
    return before + s - v;
}

// dst[k] for every request: the k-th valid one takes the k-th lowest free
// page.  The free pages' numbers go through `list` (pages entries).
__global__ void __launch_bounds__(kPlan)
fork_plan_kernel(uint8_t *__restrict__ used, const int32_t *__restrict__ src, int32_t *__restrict__ dst,
                 int32_t *__restrict__ list, int64_t n, int64_t num_pages) {
    __shared__ int sums[kPlan / 32];
    int64_t found = 0;
    for (int64_t p0 = 0; p0 < num_pages; p0 += kPlan) {
        const int64_t p = p0 + threadIdx.x;
        const int is_free = p < num_pages && used[p] == 0;
        int all;
        const int at = block_prefix(is_free, sums, &all);
        if (is_free) list[found + at] = int32_t(p);
        found += all;
    }
    __syncthreads();
    int64_t taken = 0;
    for (int64_t k0 = 0; k0 < n; k0 += kPlan) {
        const int64_t k = k0 + threadIdx.x;
        const int s = k < n ? src[k] : -2;
        const int valid = s == -1 || (s >= 0 && s < num_pages && used[s] != 0);
        int all;
        const int at = block_prefix(valid, sums, &all);
        if (k < n) dst[k] = valid && taken + at < found ? list[taken + at] : -1;
        taken += all;
    }
    __syncthreads();
    for (int64_t k = threadIdx.x; k < min(taken, found); k += kPlan) used[list[k]] = 1;
}

// moved[p]: where page p's content is afterwards, -1 for a free page; the
// moves as (from, to) pairs and their number in list.
__global__ void __launch_bounds__(kPlan)
compact_plan_kernel(uint8_t *__restrict__ used, int32_t *__restrict__ moved, int32_t *__restrict__ list,
                    int32_t *__restrict__ pages, int64_t n, int64_t num_pages) {
    __shared__ int sums[kPlan / 32];
    int64_t live = 0;
    for (int64_t p0 = 0; p0 < num_pages; p0 += kPlan) {
        const int64_t p = p0 + threadIdx.x;
        int all;
        block_prefix(p < num_pages && used[p] != 0, sums, &all);
        live += all;
    }
    int32_t *from = list + 2, *to = list + 2 + num_pages;
    int64_t holes = 0, movers = 0;
    for (int64_t p0 = 0; p0 < num_pages; p0 += kPlan) {
        const int64_t p = p0 + threadIdx.x;
        const bool in_use = p < num_pages && used[p] != 0;
        const int hole = p < live && !in_use, mover = p >= live && in_use;
        int all;
        int at = block_prefix(hole, sums, &all);
        if (hole) to[holes + at] = int32_t(p);
        holes += all;
        at = block_prefix(mover, sums, &all);
        if (mover) from[movers + at] = int32_t(p);
        movers += all;
        if (p < num_pages) moved[p] = in_use ? int32_t(p) : -1;
    }
    __syncthreads();
    if (threadIdx.x == 0) list[0] = int32_t(movers);
    for (int64_t k = threadIdx.x; k < movers; k += kPlan) moved[from[k]] = to[k];
    __syncthreads();
    for (int64_t p = threadIdx.x; p < num_pages; p += kPlan) used[p] = p < live;
    for (int64_t k = threadIdx.x; k < n; k += kPlan) {
        const int p = pages[k];
        if (p >= 0) pages[k] = p < num_pages ? moved[p] : -1;
    }
}

// Copies page from[k] to page to[k] of every layer; from -1 writes zeros.
// `count` (device) or `n` says how many.
template <typename V>
__global__ void __launch_bounds__(256)
copy_kernel(V *__restrict__ pool, const int32_t *__restrict__ from, const int32_t *__restrict__ to,
            const int32_t *__restrict__ count, int64_t n, int64_t layers, int64_t num_pages, int64_t words) {
    if (count) n = *count;
    const int64_t total = n * layers * words;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) {
        const int64_t w = i % words, k = i / words % n, layer = i / words / n;
        const int64_t f = from[k], t = to[k];
        if (t < 0 || t >= num_pages || f < -1 || f >= num_pages) continue;
        V v{};
        if (f >= 0) v = pool[(layer * num_pages + f) * words + w];
        pool[(layer * num_pages + t) * words + w] = v;
    }
}

__global__ void __launch_bounds__(256)
free_kernel(uint8_t *__restrict__ used, const int32_t *__restrict__ pages, int64_t n, int64_t num_pages) {
    const int64_t k = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (k >= n) return;
    const int p = pages[k];
    if (p >= 0 && p < num_pages) used[p] = 0;
}

static cudaError_t run_copy(void *pool, const int32_t *from, const int32_t *to, const int32_t *count,
                            int64_t n, int64_t layers, int64_t num_pages, int64_t bytes, int num_sms,
                            cudaStream_t st) {
    const unsigned grid = unsigned(num_sms * 8);
    if (bytes % 16 == 0 && reinterpret_cast<uintptr_t>(pool) % 16 == 0)
        copy_kernel<uint4><<<grid, 256, 0, st>>>(static_cast<uint4 *>(pool), from, to, count, n, layers,
                                                 num_pages, bytes / 16);
    else
        copy_kernel<uint8_t><<<grid, 256, 0, st>>>(static_cast<uint8_t *>(pool), from, to, count, n, layers,
                                                   num_pages, bytes);
    return cudaGetLastError();
}

cudaError_t copy(void *pool, const int32_t *src, const int32_t *dst, int64_t n, int64_t layers,
                 int64_t num_pages, int64_t bytes, int num_sms, cudaStream_t st) {
    return run_copy(pool, src, dst, nullptr, n, layers, num_pages, bytes, num_sms, st);
}

cudaError_t fork(void *pool, uint8_t *used, const int32_t *src, int32_t *dst, int64_t n, int64_t layers,
                 int64_t num_pages, int64_t bytes, int num_sms, cudaStream_t st) {
    int32_t *list = nullptr;
    cudaError_t err = cudaMallocAsync(&list, size_t(num_pages) * 4, st);
    if (err != cudaSuccess) return err;
    fork_plan_kernel<<<1, kPlan, 0, st>>>(used, src, dst, list, n, num_pages);
    err = cudaGetLastError();
    if (err == cudaSuccess) err = run_copy(pool, src, dst, nullptr, n, layers, num_pages, bytes, num_sms, st);
    const cudaError_t e2 = cudaFreeAsync(list, st);
    return err != cudaSuccess ? err : e2;
}

cudaError_t free_pages(uint8_t *used, const int32_t *pages, int64_t n, int64_t num_pages, cudaStream_t st) {
    free_kernel<<<unsigned((n + 255) / 256), 256, 0, st>>>(used, pages, n, num_pages);
    return cudaGetLastError();
}

cudaError_t compact(void *pool, uint8_t *used, int32_t *moved, int32_t *pages, int64_t n, int64_t layers,
                    int64_t num_pages, int64_t bytes, int num_sms, cudaStream_t st) {
    int32_t *list = nullptr;
    cudaError_t err = cudaMallocAsync(&list, size_t(num_pages) * 8 + 8, st);
    if (err != cudaSuccess) return err;
    compact_plan_kernel<<<1, kPlan, 0, st>>>(used, moved, list, pages, n, num_pages);
    err = cudaGetLastError();
    if (err == cudaSuccess)
        err = run_copy(pool, list + 2, list + 2 + num_pages, list, 0, layers, num_pages, bytes, num_sms, st);
    const cudaError_t e2 = cudaFreeAsync(list, st);
    return err != cudaSuccess ? err : e2;
}

}  // namespace pages
}  // namespace ssm
