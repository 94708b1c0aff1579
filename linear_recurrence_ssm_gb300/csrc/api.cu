// api.cu -- the C ABI of libssmscan.so: argument validation, device checks
// and dispatch to the kernels.  See include/ssm_scan.h for the contract.
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include <float.h>
#include <limits.h>
#include <algorithm>
#include <mutex>

#include "delta_mma.cuh"
#include "gated_scan.cuh"
#include "ssm_common.cuh"

namespace ssm {
namespace diag {
template <typename Tin>
cudaError_t launch(const Tin *x, const Tin *dlt, const float *A, const Tin *Bm, const Tin *Cm,
                   const float *D, float *y, int64_t Bs, int64_t L, int64_t ED, int64_t N,
                   int num_sms, cudaStream_t st);
template <typename Tin>
cudaError_t launch_ext(const Tin *x, const Tin *dlt, const float *A, const Tin *Bm, const Tin *Cm,
                       const float *D, float *y, int64_t Bs, int64_t L, int64_t ED, int64_t N,
                       int num_sms, const ScanOpts &ex, cudaStream_t st);
struct Plan {
    int S, G, K, seg_len;
};
Plan plan_for(int64_t Bs, int64_t L, int64_t ED, int64_t N, int esz, int num_sms);
}  // namespace diag
namespace diag_bwd {
template <typename Tin>
cudaError_t launch_bwd(const Tin *x, const Tin *dlt, const float *A, const Tin *Bm, const Tin *Cm,
                       const float *D, const float *dy, float *dx, float *ddelta, float *dA,
                       float *dB, float *dC, float *dD, int64_t Bs, int64_t L, int64_t ED,
                       int64_t N, int num_sms, cudaStream_t st);
}
namespace ssd_bwd {
bool supported(int64_t P, int64_t N);
template <typename Tin>
cudaError_t launch(const Tin *x, const Tin *dt, const float *A_head, const Tin *Bm, const Tin *Cm,
                   const float *D, const float *dy, float *dx, float *ddt, float *dA, float *dB,
                   float *dC, float *dD, int64_t Bs, int64_t L, int64_t H, int64_t P, int64_t N,
                   int64_t G, bool bidir, cudaStream_t st);
}
namespace diag_bwd_ex {
template <typename Tin>
cudaError_t launch(const Tin *x, const Tin *dlt, const float *A, const Tin *Bm, const Tin *Cm,
                   const float *D, const float *dy, float *dx, float *ddelta, float *dA, float *dB,
                   float *dC, float *dD, float *dz, float *ddt_bias, float *dh0, int64_t Bs,
                   int64_t L, int64_t ED, int64_t N, const ScanOpts &o, int num_sms,
                   cudaStream_t st);
}
namespace ssd_bwd_ex {
template <typename Tin>
cudaError_t launch(const Tin *x, const Tin *dt, const float *A_head, const Tin *Bm, const Tin *Cm,
                   const float *D, const float *dy, float *dx, float *ddt, float *dA, float *dB,
                   float *dC, float *dD, float *dz, float *ddt_bias, float *dh0, int64_t Bs,
                   int64_t L, int64_t H, int64_t P, int64_t N, int64_t G, bool bidir,
                   const ScanOpts &o, int num_sms, cudaStream_t st);
}
namespace ssd_general {
bool supported(int64_t P, int64_t N);
template <typename Tin>
cudaError_t launch(const Tin *x, const Tin *dt, const float *A_head, const Tin *Bm, const Tin *Cm,
                   const float *D, float *y, int64_t Bs, int64_t L, int64_t H, int64_t P,
                   int64_t N, bool bidir, int num_sms, const ScanOpts *opt, cudaStream_t st);
}
namespace gated {
template <typename T>
cudaError_t launch_fwd(const T *x, const T *gr, const T *gi, const float *lam, float c,
                       const uint8_t *reset, const float *h0, T *y, float *h_final,
                       const Kept &kept, int64_t Bs, int64_t L, int64_t ED, int num_sms,
                       cudaStream_t st);
template <typename T>
cudaError_t launch_step(const T *x, const T *gr, const T *gi, const float *lam, float c,
                        float *states, const int32_t *pages, T *y, int64_t Bs, int64_t ED,
                        int64_t num_pages, cudaStream_t st);
cudaError_t take_device_error(unsigned int *out);
cudaError_t probe_wait_timeout(bool for_copy, cudaStream_t st);
}
namespace gated_bwd {
template <typename T>
cudaError_t launch(const T *x, const T *gr, const T *gi, const float *lam, float c,
                   const uint8_t *reset, const T *dy, const float *dh_final,
                   const gated::Kept &kept, T *dx, T *dr, T *di, float *dlam, float *dh0,
                   float *scratch, int64_t Bs, int64_t L, int64_t ED, int num_sms,
                   cudaStream_t st);
cudaError_t take_device_error(unsigned int *out);
cudaError_t probe_wait_timeout(bool for_copy, cudaStream_t st);
}
namespace ckpt8 {
template <typename T>
cudaError_t save(const T *x, int8_t *q, float *scale, int64_t rows, int64_t cols, cudaStream_t st);
template <typename T>
cudaError_t load(const int8_t *q, const float *scale, T *x, int64_t rows, int64_t cols,
                 cudaStream_t st);
}
namespace pages {
cudaError_t copy(void *pool, const int32_t *src, const int32_t *dst, int64_t n, int64_t layers,
                 int64_t num_pages, int64_t bytes, int num_sms, cudaStream_t st);
cudaError_t fork(void *pool, uint8_t *used, const int32_t *src, int32_t *dst, int64_t n,
                 int64_t layers, int64_t num_pages, int64_t bytes, int num_sms, cudaStream_t st);
cudaError_t free_pages(uint8_t *used, const int32_t *pages, int64_t n, int64_t num_pages,
                       cudaStream_t st);
cudaError_t compact(void *pool, uint8_t *used, int32_t *moved, int32_t *pages, int32_t *scratch,
                    int64_t n, int64_t layers, int64_t num_pages, int64_t bytes, int num_sms,
                    cudaStream_t st);
}
namespace delta {
namespace general {
template <typename T>
cudaError_t fwd(const FwdArgs<T> &a, cudaStream_t st);
template <typename T>
cudaError_t bwd(const BwdArgs<T> &a, cudaStream_t st);
}
namespace mma {
namespace fwd {
cudaError_t probe_wait_timeout(cudaStream_t st);
cudaError_t take_device_error(unsigned int *out);
bool fits(const FwdArgs<__nv_bfloat16> &a);
cudaError_t launch(FwdArgs<__nv_bfloat16> a, cudaStream_t st);
}
namespace bwd {
cudaError_t take_device_error(unsigned int *out);
bool fits(const BwdArgs<__nv_bfloat16> &a);
cudaError_t launch(const BwdArgs<__nv_bfloat16> &a, cudaStream_t st);
}
}
namespace step {
template <typename T>
cudaError_t launch(const T *q, const T *k, const T *v, const T *g, const T *beta, float scale,
                   float *states, const int32_t *pages, T *y, int64_t Bs, int64_t G, int64_t H,
                   int64_t K, int64_t V, int64_t num_pages, cudaStream_t st);
}
}
namespace norm {
template <typename T>
cudaError_t launch_fwd(const T *x, const T *residual, const float *weight, float eps, T *sum, T *y,
                       int8_t *q, float *scale, float *rstd, int64_t rows, int64_t cols,
                       cudaStream_t st);
template <typename T>
cudaError_t launch_bwd(const T *dy, const T *s, const T *residual, const float *weight,
                       const float *rstd, const T *ds, T *dx, float *dweight, float *scratch, int64_t rows, int64_t cols,
                       cudaStream_t st);
}
namespace bidir {
cudaError_t take_device_error(unsigned int *out);
}
namespace ssd {
cudaError_t launch(const __nv_bfloat16 *x, const __nv_bfloat16 *dt, const float *A_head,
                   const __nv_bfloat16 *Bm, const __nv_bfloat16 *Cm, const float *D, float *y,
                   int64_t Bs, int64_t L, int64_t H, int64_t P, int64_t N, int64_t chunk,
                   bool bidirectional, int num_sms, cudaStream_t st, const ScanOpts *opt);
cudaError_t take_device_error(unsigned int *out);
cudaError_t probe_wait_timeout(cudaStream_t st);
size_t noalloc_scratch_needed(int64_t Bs, int64_t L, int64_t H, int64_t N, bool bidirectional);
cudaError_t launch_noalloc(const __nv_bfloat16 *x, const __nv_bfloat16 *dt, const float *A_head,
                           const __nv_bfloat16 *Bm, const __nv_bfloat16 *Cm, const float *D,
                           float *y, int64_t Bs, int64_t L, int64_t H, int64_t P, int64_t N,
                           bool bidirectional, cudaStream_t stream);
}
}  // namespace ssm

namespace {

constexpr int kMaxDevices = 64;

struct DeviceInfo {
    bool ok = false;
    int num_sms = 0;
};

std::mutex g_dev_mutex;
bool g_dev_known[kMaxDevices];   // set only once the attribute queries succeeded
DeviceInfo g_dev[kMaxDevices];

// Device attributes, kept per device once a query has succeeded.  A device that is not
// compute capability 10.3 cannot run this library's sm_103a code.
ssm_status_t current_device(DeviceInfo *out) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return SSM_ERR_NO_DEVICE;
    }
    {
        // a failed query is not kept: the next call asks again
        std::lock_guard<std::mutex> lock(g_dev_mutex);
        if (!g_dev_known[dev]) {
            int major = 0, minor = 0, sms = 0;
            if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
                cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
                cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
                return SSM_ERR_NO_DEVICE;
            g_dev[dev].ok = major == 10 && minor == 3;
            g_dev[dev].num_sms = sms;
            g_dev_known[dev] = true;
        }
        *out = g_dev[dev];
    }
    return out->ok ? SSM_OK : SSM_ERR_NO_DEVICE;
}

bool mul_ok(int64_t a, int64_t b, int64_t *out) {
    if (a < 0 || b < 0) return false;
    if (a != 0 && b > INT64_MAX / a) return false;
    *out = a * b;
    return true;
}

// Every size >= 1 and the product of all of them fits in int64.
bool sizes_ok(std::initializer_list<int64_t> dims) {
    int64_t prod = 1;
    for (int64_t d : dims) {
        if (d < 1) return false;
        if (!mul_ok(prod, d, &prod)) return false;
    }
    return true;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

ssm_status_t from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return SSM_OK;
    if (e == cudaErrorNoKernelImageForDevice || e == cudaErrorNoDevice ||
        e == cudaErrorInsufficientDriver)
        return SSM_ERR_NO_DEVICE;
    if (e == cudaErrorInvalidConfiguration) return SSM_ERR_UNSUPPORTED;
    return SSM_ERR_CUDA;
}

// Options present, and their pointers aligned to `zsize` (z) / 4 bytes.
ssm_status_t check_options(const ssm_scan_options_t *o, size_t zsize) {
    if (!o) return SSM_OK;
    if ((o->z && !aligned(o->z, zsize)) || (o->dt_bias && !aligned(o->dt_bias, 4)) ||
        (o->h0 && !aligned(o->h0, 4)) || (o->h_final && !aligned(o->h_final, 4)))
        return SSM_ERR_ALIGNMENT;
    return SSM_OK;
}

template <typename Tin>
ssm_status_t diag_entry(const Tin *x, const Tin *delta, const float *A, const Tin *B, const Tin *C,
                        const float *D, float *y, int64_t Bs, int64_t L, int64_t ED, int64_t N,
                        void *stream, const ssm_scan_options_t *opts = nullptr) {
    if (!x || !delta || !A || !B || !C || !y) return SSM_ERR_INVALID_ARG;
    if (!sizes_ok({Bs, L, ED}) || !sizes_ok({Bs, L, N}) || !sizes_ok({ED, N}))
        return SSM_ERR_INVALID_ARG;
    if (N > 256) return SSM_ERR_UNSUPPORTED;
    if (L > INT_MAX || ED > INT_MAX) return SSM_ERR_UNSUPPORTED;
    const size_t es = sizeof(Tin);
    if (!aligned(x, es) || !aligned(delta, es) || !aligned(B, es) || !aligned(C, es) ||
        !aligned(A, 4) || !aligned(y, 4) || (D && !aligned(D, 4)))
        return SSM_ERR_ALIGNMENT;
    if (opts && opts->ngroups > 1) return SSM_ERR_UNSUPPORTED;   // groups: SSD only
    ssm_status_t s = check_options(opts, es);
    if (s != SSM_OK) return s;
    DeviceInfo dev;
    s = current_device(&dev);
    if (s != SSM_OK) return s;
    // the plain kernels unless an option is on
    if (opts && (opts->dt_bias || opts->dt_softplus || opts->dt_limit || opts->z || opts->h0 ||
                 opts->h_final)) {
        const ssm::ScanOpts ex{opts->dt_bias, opts->z, opts->h0, opts->h_final,
                               opts->dt_min, opts->dt_max, opts->dt_softplus, opts->dt_limit, 1};
        return from_cuda(ssm::diag::launch_ext<Tin>(x, delta, A, B, C, D, y, Bs, L, ED, N,
                                                    dev.num_sms, ex,
                                                    static_cast<cudaStream_t>(stream)));
    }
    return from_cuda(ssm::diag::launch<Tin>(x, delta, A, B, C, D, y, Bs, L, ED, N, dev.num_sms,
                                            static_cast<cudaStream_t>(stream)));
}


// The chunked scan: validation, then the tensor-core kernel (bf16, P = 64,
// N in {64, 128}) or the CUDA-core kernel (every other supported shape and
// fp32 inputs).  `noalloc`: the reverse states' scratch comes from the fixed
// module array (the CUDA-core kernel needs none).
ssm_status_t ssd_entry(const void *x, const void *dt, const float *A_head, const void *B,
                       const void *C, const float *D, float *y, int64_t Bs, int64_t L, int64_t H,
                       int64_t P, int64_t N, int64_t chunk, int bidirectional, int input_bf16,
                       const ssm_scan_options_t *opts, void *stream, bool noalloc) {
    if (!x || !dt || !A_head || !B || !C || !y) return SSM_ERR_INVALID_ARG;
    if (!sizes_ok({Bs, L, H, P}) || !sizes_ok({Bs, L, N}) || chunk < 1) return SSM_ERR_INVALID_ARG;
    const bool tc = input_bf16 && P == 64 && (N == 64 || N == 128);
    if (!tc && !ssm::ssd_general::supported(P, N)) return SSM_ERR_UNSUPPORTED;
    if (chunk != 64 && chunk != 128 && chunk != 256) return SSM_ERR_UNSUPPORTED;
    if (L > INT_MAX || H > 65535 || Bs > INT_MAX) return SSM_ERR_UNSUPPORTED;
    if (opts) {
        if (bidirectional && (opts->h0 || opts->h_final)) return SSM_ERR_UNSUPPORTED;
        if (opts->ngroups < 0 || (opts->ngroups > 1 && H % opts->ngroups != 0))
            return SSM_ERR_INVALID_ARG;
        if (opts->ngroups > 1 && !sizes_ok({Bs, L, opts->ngroups, N})) return SSM_ERR_INVALID_ARG;
    }
    if (tc && noalloc &&
        ssm::ssd::noalloc_scratch_needed(Bs, L, H, N, bidirectional != 0) > SSM_NOALLOC_SCRATCH_BYTES)
        return SSM_ERR_UNSUPPORTED;
    const size_t es = input_bf16 ? 2 : 4;
    if (!aligned(x, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(y, 16) ||
        !aligned(dt, es) || !aligned(A_head, 4) || (D && !aligned(D, 4)))
        return SSM_ERR_ALIGNMENT;
    ssm_status_t s = check_options(opts, 16);
    if (s != SSM_OK) return s;
    DeviceInfo dev;
    s = current_device(&dev);
    if (s != SSM_OK) return s;
    using bf = __nv_bfloat16;
    ssm::ScanOpts o{};
    if (opts)
        o = ssm::ScanOpts{opts->dt_bias, opts->z, opts->h0, opts->h_final, opts->dt_min,
                          opts->dt_max, opts->dt_softplus, opts->dt_limit, opts->ngroups};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!tc) {
        if (input_bf16)
            return from_cuda(ssm::ssd_general::launch<bf>(
                static_cast<const bf *>(x), static_cast<const bf *>(dt), A_head,
                static_cast<const bf *>(B), static_cast<const bf *>(C), D, y, Bs, L, H, P, N,
                bidirectional != 0, dev.num_sms, opts ? &o : nullptr, st));
        return from_cuda(ssm::ssd_general::launch<float>(
            static_cast<const float *>(x), static_cast<const float *>(dt), A_head,
            static_cast<const float *>(B), static_cast<const float *>(C), D, y, Bs, L, H, P, N,
            bidirectional != 0, dev.num_sms, opts ? &o : nullptr, st));
    }
    if (noalloc)
        return from_cuda(ssm::ssd::launch_noalloc(static_cast<const bf *>(x),
                                                  static_cast<const bf *>(dt), A_head,
                                                  static_cast<const bf *>(B),
                                                  static_cast<const bf *>(C), D, y, Bs, L, H, P, N,
                                                  bidirectional != 0, st));
    return from_cuda(ssm::ssd::launch(static_cast<const bf *>(x), static_cast<const bf *>(dt),
                                      A_head, static_cast<const bf *>(B),
                                      static_cast<const bf *>(C), D, y, Bs, L, H, P, N, chunk,
                                      bidirectional != 0, dev.num_sms, st, opts ? &o : nullptr));
}

bool pages_ok(int64_t n, int64_t num_pages) {
    return n >= 0 && n <= INT_MAX && num_pages >= 1;
}

// What a gated forward call writes and a backward call reads; `need` says
// whether the states must be there.
ssm_status_t check_saved(const gated_scan_saved_t *saved, bool need, ssm::gated::Kept *out) {
    *out = ssm::gated::Kept{};
    if (!saved) return need ? SSM_ERR_INVALID_ARG : SSM_OK;
    const gated_scan_saved_t &k = *saved;
    if (!k.states) return SSM_ERR_INVALID_ARG;
    const bool any = k.x_q || k.r_q || k.i_q || k.x_s || k.r_s || k.i_s;
    if (any && !(k.x_q && k.r_q && k.i_q && k.x_s && k.r_s && k.i_s)) return SSM_ERR_INVALID_ARG;
    if (!aligned(k.states, 4) || !aligned(k.x_s, 4) || !aligned(k.r_s, 4) || !aligned(k.i_s, 4))
        return SSM_ERR_ALIGNMENT;
    *out = ssm::gated::Kept{k.states, k.x_q, k.r_q, k.i_q, k.x_s, k.r_s, k.i_s};
    return SSM_OK;
}

ssm_status_t check_gated_sizes(int64_t Bs, int64_t L, int64_t ED, float c) {
    if (!sizes_ok({Bs, L, ED, 4}) || !(c > 0.0f) || c > FLT_MAX) return SSM_ERR_INVALID_ARG;
    // room for the tiles behind the end
    if (Bs > 65535 || L > INT_MAX - 4096 || ED > INT_MAX - 4096)
        return SSM_ERR_UNSUPPORTED;
    return SSM_OK;
}

template <typename T>
ssm_status_t gated_fwd_entry(const void *x, const void *gr, const void *gi, const float *lam,
                             float c, const uint8_t *reset, const float *h0, void *y,
                             float *h_final, const gated_scan_saved_t *saved, int64_t Bs,
                             int64_t L, int64_t ED, void *stream) {
    if (!x || !gr || !gi || !lam || !y) return SSM_ERR_INVALID_ARG;
    ssm_status_t s = check_gated_sizes(Bs, L, ED, c);
    if (s != SSM_OK) return s;
    if (!aligned(x, sizeof(T)) || !aligned(gr, sizeof(T)) || !aligned(gi, sizeof(T)) ||
        !aligned(y, sizeof(T)) || !aligned(lam, 4) || !aligned(h0, 4) || !aligned(h_final, 4))
        return SSM_ERR_ALIGNMENT;
    ssm::gated::Kept kept;
    s = check_saved(saved, false, &kept);
    if (s != SSM_OK) return s;
    DeviceInfo dev;
    s = current_device(&dev);
    if (s != SSM_OK) return s;
    return from_cuda(ssm::gated::launch_fwd<T>(
        static_cast<const T *>(x), static_cast<const T *>(gr), static_cast<const T *>(gi), lam, c,
        reset, h0, static_cast<T *>(y), h_final, kept, Bs, L, ED, dev.num_sms,
        static_cast<cudaStream_t>(stream)));
}

template <typename T>
ssm_status_t gated_bwd_entry(const void *x, const void *gr, const void *gi, const float *lam,
                             float c, const uint8_t *reset, const void *dy, const float *dh_final,
                             const gated_scan_saved_t *saved, void *dx, void *dr, void *di,
                             float *dlam, float *dh0, float *scratch, int64_t Bs, int64_t L,
                             int64_t ED, void *stream) {
    ssm::gated::Kept kept;
    ssm_status_t s = check_saved(saved, true, &kept);
    if (s != SSM_OK) return s;
    if ((!kept.x_q && (!x || !gr || !gi)) || !lam || !dy || !dx || !dr || !di || !dlam ||
        !scratch)
        return SSM_ERR_INVALID_ARG;
    s = check_gated_sizes(Bs, L, ED, c);
    if (s != SSM_OK) return s;
    const size_t es = sizeof(T);
    if (!aligned(x, es) || !aligned(gr, es) || !aligned(gi, es) || !aligned(dy, es) ||
        !aligned(dx, es) || !aligned(dr, es) || !aligned(di, es) || !aligned(lam, 4) ||
        !aligned(dh_final, 4) || !aligned(dlam, 4) || !aligned(dh0, 4) || !aligned(scratch, 4))
        return SSM_ERR_ALIGNMENT;
    DeviceInfo dev;
    s = current_device(&dev);
    if (s != SSM_OK) return s;
    return from_cuda(ssm::gated_bwd::launch<T>(
        static_cast<const T *>(x), static_cast<const T *>(gr), static_cast<const T *>(gi), lam, c,
        reset, static_cast<const T *>(dy), dh_final, kept, static_cast<T *>(dx),
        static_cast<T *>(dr), static_cast<T *>(di), dlam, dh0, scratch, Bs, L, ED, dev.num_sms,
        static_cast<cudaStream_t>(stream)));
}

template <typename T>
ssm_status_t gated_step_entry(const void *x, const void *gr, const void *gi, const float *lam,
                              float c, float *states, const int32_t *pages, void *y, int64_t Bs,
                              int64_t ED, int64_t num_pages, void *stream) {
    if (!x || !gr || !gi || !lam || !states || !y) return SSM_ERR_INVALID_ARG;
    ssm_status_t s = check_gated_sizes(Bs, 1, ED, c);
    if (s != SSM_OK) return s;
    if (!pages_ok(Bs, num_pages) || !sizes_ok({num_pages, ED, 4}) || (!pages && num_pages < Bs))
        return SSM_ERR_INVALID_ARG;
    if (num_pages > SSM_MAX_PAGES) return SSM_ERR_UNSUPPORTED;
    if (!aligned(x, sizeof(T)) || !aligned(gr, sizeof(T)) || !aligned(gi, sizeof(T)) ||
        !aligned(y, sizeof(T)) || !aligned(lam, 4) || !aligned(states, 4) || !aligned(pages, 4))
        return SSM_ERR_ALIGNMENT;
    DeviceInfo dev;
    s = current_device(&dev);
    if (s != SSM_OK) return s;
    return from_cuda(ssm::gated::launch_step<T>(
        static_cast<const T *>(x), static_cast<const T *>(gr), static_cast<const T *>(gi), lam, c,
        states, pages, static_cast<T *>(y), Bs, ED, num_pages, static_cast<cudaStream_t>(stream)));
}

ssm_status_t check_ckpt8(const void *x, const void *q, const float *scale, int64_t rows,
                         int64_t cols, size_t es) {
    if (!x || !q || !scale || !sizes_ok({rows, cols, 4})) return SSM_ERR_INVALID_ARG;
    if (rows > INT_MAX || cols > INT_MAX - 64) return SSM_ERR_UNSUPPORTED;
    return aligned(x, es) && aligned(scale, 4) ? SSM_OK : SSM_ERR_ALIGNMENT;
}

// Arguments of the calls on a pool and a list of n pages.
ssm_status_t check_pool(const void *pool, int64_t n, int64_t layers, int64_t num_pages,
                        int64_t page_bytes, DeviceInfo *dev) {
    if (!pool || !pages_ok(n, num_pages) || !sizes_ok({layers, num_pages, page_bytes}))
        return SSM_ERR_INVALID_ARG;
    if (num_pages > SSM_MAX_PAGES) return SSM_ERR_UNSUPPORTED;
    return current_device(dev);
}
// The sizes of a call of the gated delta rule; `packed` sequences share one
// row of the batch.
ssm_status_t check_delta_sizes(int64_t Bs, int64_t L, int64_t G, int64_t H, int64_t K, int64_t V,
                               int64_t n_seq, float scale) {
    if (!sizes_ok({Bs, L, H, V, 4}) || !sizes_ok({Bs, L, G, K, 4}) || !sizes_ok({Bs, L, H, K, 4}) ||
        !sizes_ok({Bs, H, K, V, 4}) || n_seq < 0 || (n_seq > 0 && Bs != 1) || H % G != 0 ||
        !(scale >= -FLT_MAX && scale <= FLT_MAX))
        return SSM_ERR_INVALID_ARG;
    if (n_seq > 0 && !sizes_ok({n_seq, H, K, V, 4})) return SSM_ERR_INVALID_ARG;
    // room for the steps behind the end; a block a head and 64 steps in the grid
    if (K > 256 || V > 256 || L > INT_MAX - 4096 || Bs > INT_MAX / 2 || n_seq > INT_MAX / 2 || H > INT_MAX / 2)
        return SSM_ERR_UNSUPPORTED;
    const int64_t slots = n_seq > 0 ? L / 64 + n_seq : Bs * ((L + 63) / 64);
    if (!sizes_ok({slots, H, K, V, 4})) return SSM_ERR_INVALID_ARG;
    return slots * H > INT_MAX ? SSM_ERR_UNSUPPORTED : SSM_OK;
}

ssm::delta::Shape delta_shape(const int32_t *offsets, int64_t Bs, int64_t L, int64_t G, int64_t H,
                              int64_t K, int64_t V, int64_t n_seq, float scale) {
    ssm::delta::Shape s{};
    s.offsets = offsets;
    s.L = L;
    s.n = int(offsets ? n_seq : Bs);
    s.G = int(G), s.H = int(H), s.K = int(K), s.V = int(V);
    s.scale = scale;
    return s;
}

// The scratch of the gradients holds what either path needs.
ssm::delta::Scratch delta_scratch(const ssm::delta::Shape &s, int elem) {
    int64_t shares = ssm::delta::general::shares(s), records = ssm::delta::general::made_bytes(s);
    if (elem == 2 && ssm::delta::mma::fits_bwd(s)) {
        const int64_t blocks = s.slots() * s.H;
        shares = std::max(shares, blocks * ssm::delta::kBlock * ssm::delta::mma::dbeta_parts(s));
        records = std::max(records, blocks * ssm::delta::mma::kBothRecord);
    }
    return ssm::delta::scratch_of(s, elem, shares, records);
}

template <typename T>
ssm_status_t delta_fwd_entry(const void *q, const void *k, const void *v, const void *g,
                             const void *beta, float scale, const int32_t *offsets,
                             const float *h0, void *y, float *h_final, void *states, void *errors,
                             void *scratch, int64_t Bs, int64_t L, int64_t G, int64_t H, int64_t K, int64_t V,
                             int64_t n_seq, void *stream) {
    if (!q || !k || !v || !g || !beta || !y || !states != !errors || (n_seq > 0) != (offsets != nullptr))
        return SSM_ERR_INVALID_ARG;
    ssm_status_t s = check_delta_sizes(Bs, L, G, H, K, V, n_seq, scale);
    if (s != SSM_OK) return s;
    if (!scratch) return SSM_ERR_INVALID_ARG;       // of no size for sizes that are refused
    const size_t e = sizeof(T);
    for (const void *p : {q, k, v, g, beta, static_cast<const void *>(y), static_cast<const void *>(states),
                          static_cast<const void *>(errors)})
        if (!aligned(p, e)) return SSM_ERR_ALIGNMENT;
    if (!aligned(offsets, 4) || !aligned(h0, 4) || !aligned(h_final, 4) || !aligned(scratch, 16))
        return SSM_ERR_ALIGNMENT;
    DeviceInfo dev;
    s = current_device(&dev);
    if (s != SSM_OK) return s;
    const ssm::delta::FwdArgs<T> a{delta_shape(offsets, Bs, L, G, H, K, V, n_seq, scale),
                                   static_cast<const T *>(q), static_cast<const T *>(k),
                                   static_cast<const T *>(v), static_cast<const T *>(g),
                                   static_cast<const T *>(beta), h0, static_cast<T *>(y), h_final,
                                   static_cast<T *>(states), static_cast<T *>(errors),
                                   static_cast<unsigned char *>(scratch), 0, nullptr, nullptr, nullptr};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if constexpr (sizeof(T) == 2)
        if (ssm::delta::mma::fwd::fits(a)) return from_cuda(ssm::delta::mma::fwd::launch(a, st));
    return from_cuda(ssm::delta::general::fwd(a, st));
}

template <typename T>
ssm_status_t delta_bwd_entry(const void *q, const void *k, const void *g, const void *beta,
                             float scale, const int32_t *offsets, const void *dy,
                             const float *dh_final, const void *states, const void *errors,
                             void *dq, void *dk, void *dv, void *dg, void *dbeta, float *dh0,
                             void *scratch, int64_t Bs, int64_t L, int64_t G, int64_t H, int64_t K,
                             int64_t V, int64_t n_seq, void *stream) {
    if (!q || !k || !g || !beta || !dy || !states || !errors || !dq || !dk || !dv || !dg || !dbeta ||
        (n_seq > 0) != (offsets != nullptr))
        return SSM_ERR_INVALID_ARG;
    ssm_status_t s = check_delta_sizes(Bs, L, G, H, K, V, n_seq, scale);
    if (s != SSM_OK) return s;
    if (!scratch) return SSM_ERR_INVALID_ARG;
    const size_t e = sizeof(T);
    for (const void *p : {q, k, g, beta, dy, states, errors, static_cast<const void *>(dq),
                          static_cast<const void *>(dk), static_cast<const void *>(dv),
                          static_cast<const void *>(dg), static_cast<const void *>(dbeta)})
        if (!aligned(p, e)) return SSM_ERR_ALIGNMENT;
    if (!aligned(offsets, 4) || !aligned(dh_final, 4) || !aligned(dh0, 4) || !aligned(scratch, 16))
        return SSM_ERR_ALIGNMENT;
    DeviceInfo dev;
    s = current_device(&dev);
    if (s != SSM_OK) return s;
    const ssm::delta::Shape shape = delta_shape(offsets, Bs, L, G, H, K, V, n_seq, scale);
    const ssm::delta::Scratch at = delta_scratch(shape, int(e));
    char *mem = static_cast<char *>(scratch);
    const ssm::delta::BwdArgs<T> a{shape, static_cast<const T *>(q), static_cast<const T *>(k),
                                   static_cast<const T *>(g), static_cast<const T *>(beta),
                                   static_cast<const T *>(dy), dh_final, static_cast<const T *>(states),
                                   static_cast<const T *>(errors), static_cast<T *>(dq),
                                   static_cast<T *>(dk), static_cast<T *>(dv), static_cast<T *>(dg),
                                   static_cast<T *>(dbeta), dh0, reinterpret_cast<T *>(mem + at.ds),
                                   reinterpret_cast<float *>(mem + at.dbeta),
                                   reinterpret_cast<float *>(mem + at.dq),
                                   reinterpret_cast<float *>(mem + at.dk),
                                   reinterpret_cast<unsigned char *>(mem + at.records)};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if constexpr (sizeof(T) == 2)
        if (ssm::delta::mma::bwd::fits(a)) return from_cuda(ssm::delta::mma::bwd::launch(a, st));
    return from_cuda(ssm::delta::general::bwd(a, st));
}

template <typename T>
ssm_status_t delta_step_entry(const void *q, const void *k, const void *v, const void *g,
                              const void *beta, float scale, float *states, const int32_t *pages,
                              void *y, int64_t Bs, int64_t G, int64_t H, int64_t K, int64_t V,
                              int64_t num_pages, void *stream) {
    if (!q || !k || !v || !g || !beta || !states || !y) return SSM_ERR_INVALID_ARG;
    ssm_status_t s = check_delta_sizes(Bs, 1, G, H, K, V, 0, scale);
    if (s != SSM_OK) return s;
    if (!sizes_ok({num_pages, H, K, V, 4}) || (!pages && num_pages < Bs)) return SSM_ERR_INVALID_ARG;
    if (num_pages > SSM_MAX_PAGES) return SSM_ERR_UNSUPPORTED;
    const size_t e = sizeof(T);
    for (const void *p : {q, k, v, g, beta, static_cast<const void *>(y)})
        if (!aligned(p, e)) return SSM_ERR_ALIGNMENT;
    if (!aligned(states, 4) || !aligned(pages, 4)) return SSM_ERR_ALIGNMENT;
    DeviceInfo dev;
    s = current_device(&dev);
    if (s != SSM_OK) return s;
    return from_cuda(ssm::delta::step::launch(static_cast<const T *>(q), static_cast<const T *>(k),
                                              static_cast<const T *>(v), static_cast<const T *>(g),
                                              static_cast<const T *>(beta), scale, states, pages,
                                              static_cast<T *>(y), Bs, G, H, K, V, num_pages,
                                              static_cast<cudaStream_t>(stream)));
}

ssm_status_t check_norm(const void *a, const void *b, float eps, int64_t rows, int64_t cols) {
    if (!a || !b || !sizes_ok({rows, cols, 4}) || !(eps >= 0.0f) || eps > FLT_MAX) return SSM_ERR_INVALID_ARG;
    return rows > INT_MAX || cols > INT_MAX - 4096 ? SSM_ERR_UNSUPPORTED : SSM_OK;
}

template <typename T>
ssm_status_t norm_fwd_entry(const void *x, const void *residual, const float *weight, float eps,
                            void *sum, void *y, int8_t *y_q, float *y_scale, float *rstd,
                            int64_t rows, int64_t cols, void *stream) {
    if (!residual != !sum || !y_q != !y_scale || !y == !y_q) return SSM_ERR_INVALID_ARG;
    ssm_status_t s = check_norm(x, y ? y : y_q, eps, rows, cols);
    if (s != SSM_OK) return s;
    const size_t e = sizeof(T);
    if (!aligned(x, e) || !aligned(residual, e) || !aligned(sum, e) || !aligned(y, e) || !aligned(weight, 4) ||
        !aligned(y_scale, 4) || !aligned(rstd, 4))
        return SSM_ERR_ALIGNMENT;
    DeviceInfo dev;
    s = current_device(&dev);
    if (s != SSM_OK) return s;
    return from_cuda(ssm::norm::launch_fwd(static_cast<const T *>(x), static_cast<const T *>(residual), weight,
                                           eps, static_cast<T *>(sum), static_cast<T *>(y), y_q, y_scale, rstd,
                                           rows, cols, static_cast<cudaStream_t>(stream)));
}

template <typename T>
ssm_status_t norm_bwd_entry(const void *dy, const void *x, const void *residual, const float *weight, const float *rstd,
                            const void *dsum, void *dx, float *dweight, float *scratch, int64_t rows,
                            int64_t cols, void *stream) {
    if (!x || !rstd || (dweight && !scratch)) return SSM_ERR_INVALID_ARG;
    ssm_status_t s = check_norm(dy, dx, 0.0f, rows, cols);
    if (s != SSM_OK) return s;
    const size_t e = sizeof(T);
    if (!aligned(dy, e) || !aligned(x, e) || !aligned(residual, e) || !aligned(dsum, e) || !aligned(dx, e) || !aligned(weight, 4) ||
        !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(scratch, 4))
        return SSM_ERR_ALIGNMENT;
    DeviceInfo dev;
    s = current_device(&dev);
    if (s != SSM_OK) return s;
    return from_cuda(ssm::norm::launch_bwd(static_cast<const T *>(dy), static_cast<const T *>(x),
                                           static_cast<const T *>(residual), weight, rstd,
                                           static_cast<const T *>(dsum), static_cast<T *>(dx), dweight, scratch,
                                           rows, cols, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

ssm_status_t ssm_scan_fwd(const float *x, const float *delta, const float *A, const float *B,
                          const float *C, const float *D, float *y, int64_t Bs, int64_t L,
                          int64_t ED, int64_t N, void *stream) {
    return diag_entry<float>(x, delta, A, B, C, D, y, Bs, L, ED, N, stream);
}

ssm_status_t ssm_scan_fwd_bf16(const void *x, const void *delta, const float *A, const void *B,
                               const void *C, const float *D, float *y, int64_t Bs, int64_t L,
                               int64_t ED, int64_t N, void *stream) {
    using bf = __nv_bfloat16;
    return diag_entry<bf>(static_cast<const bf *>(x), static_cast<const bf *>(delta), A,
                          static_cast<const bf *>(B), static_cast<const bf *>(C), D, y, Bs, L, ED,
                          N, stream);
}

ssm_status_t ssd_chunk_scan_fwd(const void *x, const void *dt, const float *A_head, const void *B,
                                const void *C, const float *D, float *y, int64_t Bs, int64_t L,
                                int64_t H, int64_t P, int64_t N, int64_t chunk, int bidirectional,
                                void *stream) {
    return ssd_entry(x, dt, A_head, B, C, D, y, Bs, L, H, P, N, chunk, bidirectional, 1, nullptr,
                     stream, false);
}

ssm_status_t ssd_chunk_scan_fwd_noalloc(const void *x, const void *dt, const float *A_head,
                                        const void *B, const void *C, const float *D, float *y,
                                        int64_t Bs, int64_t L, int64_t H, int64_t P, int64_t N,
                                        int64_t chunk, int bidirectional, void *stream) {
    return ssd_entry(x, dt, A_head, B, C, D, y, Bs, L, H, P, N, chunk, bidirectional, 1, nullptr,
                     stream, true);
}

ssm_status_t ssm_scan_fwd_ex(const void *x, const void *delta, const float *A, const void *B,
                             const void *C, const float *D, float *y, int64_t Bs, int64_t L,
                             int64_t ED, int64_t N, int input_bf16,
                             const ssm_scan_options_t *opts, void *stream) {
    using bf = __nv_bfloat16;
    if (input_bf16)
        return diag_entry<bf>(static_cast<const bf *>(x), static_cast<const bf *>(delta), A,
                              static_cast<const bf *>(B), static_cast<const bf *>(C), D, y, Bs, L,
                              ED, N, stream, opts);
    return diag_entry<float>(static_cast<const float *>(x), static_cast<const float *>(delta), A,
                             static_cast<const float *>(B), static_cast<const float *>(C), D, y, Bs,
                             L, ED, N, stream, opts);
}

ssm_status_t ssd_chunk_scan_fwd_ex(const void *x, const void *dt, const float *A_head,
                                   const void *B, const void *C, const float *D, float *y,
                                   int64_t Bs, int64_t L, int64_t H, int64_t P, int64_t N,
                                   int64_t chunk, int bidirectional, int input_bf16,
                                   const ssm_scan_options_t *opts, void *stream) {
    return ssd_entry(x, dt, A_head, B, C, D, y, Bs, L, H, P, N, chunk, bidirectional, input_bf16,
                     opts, stream, false);
}

ssm_status_t ssm_scan_bwd(const void *x, const void *delta, const float *A, const void *B,
                          const void *C, const float *D, const float *dy, float *dx,
                          float *ddelta, float *dA, float *dB, float *dC, float *dD, int64_t Bs,
                          int64_t L, int64_t ED, int64_t N, int input_bf16, void *stream) {
    if (!x || !delta || !A || !B || !C || !dy || !dx || !ddelta || !dA || !dB || !dC)
        return SSM_ERR_INVALID_ARG;
    if (!sizes_ok({Bs, L, ED}) || !sizes_ok({Bs, L, N}) || !sizes_ok({ED, N}))
        return SSM_ERR_INVALID_ARG;
    if (N > 256 || Bs > 65535 || L > INT_MAX || ED > INT_MAX) return SSM_ERR_UNSUPPORTED;
    const size_t es = input_bf16 ? 2 : 4;
    if (!aligned(x, es) || !aligned(delta, es) || !aligned(B, es) || !aligned(C, es) ||
        !aligned(A, 4) || (D && !aligned(D, 4)) || !aligned(dy, 4) || !aligned(dx, 4) ||
        !aligned(ddelta, 4) || !aligned(dA, 4) || !aligned(dB, 4) || !aligned(dC, 4) ||
        (dD && !aligned(dD, 4)))
        return SSM_ERR_ALIGNMENT;
    DeviceInfo dev;
    ssm_status_t s = current_device(&dev);
    if (s != SSM_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    using bf = __nv_bfloat16;
    if (input_bf16)
        return from_cuda(ssm::diag_bwd::launch_bwd<bf>(
            static_cast<const bf *>(x), static_cast<const bf *>(delta), A,
            static_cast<const bf *>(B), static_cast<const bf *>(C), D, dy, dx, ddelta, dA, dB, dC,
            dD, Bs, L, ED, N, dev.num_sms, st));
    return from_cuda(ssm::diag_bwd::launch_bwd<float>(
        static_cast<const float *>(x), static_cast<const float *>(delta), A,
        static_cast<const float *>(B), static_cast<const float *>(C), D, dy, dx, ddelta, dA, dB,
        dC, dD, Bs, L, ED, N, dev.num_sms, st));
}

ssm_status_t ssm_scan_bwd_ex(const void *x, const void *delta, const float *A, const void *B,
                             const void *C, const float *D, const float *dy, float *dx,
                             float *ddelta, float *dA, float *dB, float *dC, float *dD, float *dz,
                             float *ddt_bias, float *dh0, int64_t Bs, int64_t L, int64_t ED,
                             int64_t N, int input_bf16, const ssm_scan_options_t *opts,
                             void *stream) {
    if (!x || !delta || !A || !B || !C || !dy || !dx || !ddelta || !dA || !dB || !dC)
        return SSM_ERR_INVALID_ARG;
    if (!sizes_ok({Bs, L, ED}) || !sizes_ok({Bs, L, N}) || !sizes_ok({ED, N}))
        return SSM_ERR_INVALID_ARG;
    if (opts && opts->h_final) return SSM_ERR_INVALID_ARG;       // an output of the forward only
    if (opts && opts->z && !dz) return SSM_ERR_INVALID_ARG;
    if (opts && opts->ngroups > 1) return SSM_ERR_UNSUPPORTED;  // groups: SSD only
    if (N > 256 || Bs > 65535 || L > INT_MAX || ED > INT_MAX) return SSM_ERR_UNSUPPORTED;
    const size_t es = input_bf16 ? 2 : 4;
    if (!aligned(x, es) || !aligned(delta, es) || !aligned(B, es) || !aligned(C, es) ||
        !aligned(A, 4) || (D && !aligned(D, 4)) || !aligned(dy, 4) || !aligned(dx, 4) ||
        !aligned(ddelta, 4) || !aligned(dA, 4) || !aligned(dB, 4) || !aligned(dC, 4) ||
        (dD && !aligned(dD, 4)) || (dz && !aligned(dz, 4)) || (ddt_bias && !aligned(ddt_bias, 4)) ||
        (dh0 && !aligned(dh0, 4)))
        return SSM_ERR_ALIGNMENT;
    ssm_status_t s = check_options(opts, es);
    if (s != SSM_OK) return s;
    DeviceInfo dev;
    s = current_device(&dev);
    if (s != SSM_OK) return s;
    ssm::ScanOpts o{};
    if (opts)
        o = ssm::ScanOpts{opts->dt_bias, opts->z, opts->h0, nullptr, opts->dt_min,
                          opts->dt_max, opts->dt_softplus, opts->dt_limit, 1};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    using bf = __nv_bfloat16;
    float *dzo = o.z ? dz : nullptr;
    float *dbo = o.dt_bias ? ddt_bias : nullptr;
    float *dho = o.h0 ? dh0 : nullptr;
    if (input_bf16)
        return from_cuda(ssm::diag_bwd_ex::launch<bf>(
            static_cast<const bf *>(x), static_cast<const bf *>(delta), A,
            static_cast<const bf *>(B), static_cast<const bf *>(C), D, dy, dx, ddelta, dA, dB, dC,
            dD, dzo, dbo, dho, Bs, L, ED, N, o, dev.num_sms, st));
    return from_cuda(ssm::diag_bwd_ex::launch<float>(
        static_cast<const float *>(x), static_cast<const float *>(delta), A,
        static_cast<const float *>(B), static_cast<const float *>(C), D, dy, dx, ddelta, dA, dB,
        dC, dD, dzo, dbo, dho, Bs, L, ED, N, o, dev.num_sms, st));
}

ssm_status_t ssd_chunk_scan_bwd(const void *x, const void *dt, const float *A_head, const void *B,
                                const void *C, const float *D, const float *dy, float *dx,
                                float *ddt, float *dA_head, float *dB, float *dC, float *dD,
                                int64_t Bs, int64_t L, int64_t H, int64_t P, int64_t N,
                                int64_t ngroups, int bidirectional, int input_bf16, void *stream) {
    if (!x || !dt || !A_head || !B || !C || !dy || !dx || !ddt || !dA_head || !dB || !dC)
        return SSM_ERR_INVALID_ARG;
    if (ngroups < 1 || !sizes_ok({Bs, L, H, P}) || !sizes_ok({Bs, L, ngroups, N}) ||
        !sizes_ok({Bs, H, L, P, N}))
        return SSM_ERR_INVALID_ARG;
    if (!ssm::ssd_bwd::supported(P, N) || H % ngroups != 0 || Bs * H > INT_MAX || L > INT_MAX)
        return SSM_ERR_UNSUPPORTED;
    const size_t es = input_bf16 ? 2 : 4;
    if (!aligned(x, es) || !aligned(dt, es) || !aligned(B, es) || !aligned(C, es) ||
        !aligned(A_head, 4) || (D && !aligned(D, 4)) || !aligned(dy, 4) || !aligned(dx, 4) ||
        !aligned(ddt, 4) || !aligned(dA_head, 4) || !aligned(dB, 4) || !aligned(dC, 4) ||
        (dD && !aligned(dD, 4)))
        return SSM_ERR_ALIGNMENT;
    DeviceInfo dev;
    ssm_status_t s = current_device(&dev);
    if (s != SSM_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    using bf = __nv_bfloat16;
    if (input_bf16)
        return from_cuda(ssm::ssd_bwd::launch<bf>(
            static_cast<const bf *>(x), static_cast<const bf *>(dt), A_head,
            static_cast<const bf *>(B), static_cast<const bf *>(C), D, dy, dx, ddt, dA_head, dB,
            dC, dD, Bs, L, H, P, N, ngroups, bidirectional != 0, st));
    return from_cuda(ssm::ssd_bwd::launch<float>(
        static_cast<const float *>(x), static_cast<const float *>(dt), A_head,
        static_cast<const float *>(B), static_cast<const float *>(C), D, dy, dx, ddt, dA_head, dB,
        dC, dD, Bs, L, H, P, N, ngroups, bidirectional != 0, st));
}

ssm_status_t ssd_chunk_scan_bwd_ex(const void *x, const void *dt, const float *A_head,
                                   const void *B, const void *C, const float *D, const float *dy,
                                   float *dx, float *ddt, float *dA_head, float *dB, float *dC,
                                   float *dD, float *dz, float *ddt_bias, float *dh0, int64_t Bs,
                                   int64_t L, int64_t H, int64_t P, int64_t N, int bidirectional,
                                   int input_bf16, const ssm_scan_options_t *opts, void *stream) {
    if (!x || !dt || !A_head || !B || !C || !dy || !dx || !ddt || !dA_head || !dB || !dC)
        return SSM_ERR_INVALID_ARG;
    const int64_t G = (opts && opts->ngroups > 1) ? opts->ngroups : 1;
    if ((opts && opts->ngroups < 0) || !sizes_ok({Bs, L, H, P}) || !sizes_ok({Bs, L, G, N}) ||
        !sizes_ok({Bs, H, L, P, N}))
        return SSM_ERR_INVALID_ARG;
    if (opts && opts->h_final) return SSM_ERR_INVALID_ARG;       // an output of the forward only
    if (opts && opts->z && !dz) return SSM_ERR_INVALID_ARG;
    if (bidirectional && opts && opts->h0) return SSM_ERR_UNSUPPORTED;
    if (!ssm::ssd_bwd::supported(P, N) || H % G != 0 || Bs * H > INT_MAX || L > INT_MAX)
        return SSM_ERR_UNSUPPORTED;
    const size_t es = input_bf16 ? 2 : 4;
    if (!aligned(x, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(dt, es) ||
        !aligned(A_head, 4) || (D && !aligned(D, 4)) || !aligned(dy, 4) || !aligned(dx, 4) ||
        !aligned(ddt, 4) || !aligned(dA_head, 4) || !aligned(dB, 4) || !aligned(dC, 4) ||
        (dD && !aligned(dD, 4)) || (dz && !aligned(dz, 4)) || (ddt_bias && !aligned(ddt_bias, 4)) ||
        (dh0 && !aligned(dh0, 4)))
        return SSM_ERR_ALIGNMENT;
    ssm_status_t s = check_options(opts, es);
    if (s != SSM_OK) return s;
    DeviceInfo dev;
    s = current_device(&dev);
    if (s != SSM_OK) return s;
    ssm::ScanOpts o{};
    if (opts)
        o = ssm::ScanOpts{opts->dt_bias, opts->z, opts->h0, nullptr, opts->dt_min,
                          opts->dt_max, opts->dt_softplus, opts->dt_limit, opts->ngroups};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    using bf = __nv_bfloat16;
    float *dzo = o.z ? dz : nullptr;
    float *dbo = o.dt_bias ? ddt_bias : nullptr;
    float *dho = o.h0 ? dh0 : nullptr;
    if (input_bf16)
        return from_cuda(ssm::ssd_bwd_ex::launch<bf>(
            static_cast<const bf *>(x), static_cast<const bf *>(dt), A_head,
            static_cast<const bf *>(B), static_cast<const bf *>(C), D, dy, dx, ddt, dA_head, dB, dC,
            dD, dzo, dbo, dho, Bs, L, H, P, N, G, bidirectional != 0, o, dev.num_sms, st));
    return from_cuda(ssm::ssd_bwd_ex::launch<float>(
        static_cast<const float *>(x), static_cast<const float *>(dt), A_head,
        static_cast<const float *>(B), static_cast<const float *>(C), D, dy, dx, ddt, dA_head, dB,
        dC, dD, dzo, dbo, dho, Bs, L, H, P, N, G, bidirectional != 0, o, dev.num_sms, st));
}

ssm_status_t ssm_scan_fwd_plan(int64_t Bs, int64_t L, int64_t ED, int64_t N, int input_bf16,
                               int32_t *states_per_thread, int32_t *lanes_per_channel,
                               int32_t *time_segments) {
    if (!states_per_thread || !lanes_per_channel || !time_segments) return SSM_ERR_INVALID_ARG;
    if (!sizes_ok({Bs, L, ED}) || !sizes_ok({Bs, L, N}) || !sizes_ok({ED, N}))
        return SSM_ERR_INVALID_ARG;
    if (N > 256) return SSM_ERR_UNSUPPORTED;
    if (L > INT_MAX || ED > INT_MAX) return SSM_ERR_UNSUPPORTED;
    DeviceInfo dev;
    ssm_status_t s = current_device(&dev);
    if (s != SSM_OK) return s;
    const ssm::diag::Plan p = ssm::diag::plan_for(Bs, L, ED, N, input_bf16 ? 2 : 4, dev.num_sms);
    *states_per_thread = p.S;
    *lanes_per_channel = p.G;
    *time_segments = p.K;
    return SSM_OK;
}

ssm_status_t gated_scan_fwd(const void *x, const void *gate_r, const void *gate_i, const float *lam,
                            float c, const uint8_t *reset, const float *h0, void *y, float *h_final,
                            const gated_scan_saved_t *saved, int64_t Bs, int64_t L, int64_t ED,
                            int input_bf16, void *stream) {
    return input_bf16 ? gated_fwd_entry<__nv_bfloat16>(x, gate_r, gate_i, lam, c, reset, h0, y,
                                                       h_final, saved, Bs, L, ED, stream)
                      : gated_fwd_entry<float>(x, gate_r, gate_i, lam, c, reset, h0, y, h_final,
                                               saved, Bs, L, ED, stream);
}

ssm_status_t gated_scan_bwd(const void *x, const void *gate_r, const void *gate_i, const float *lam,
                            float c, const uint8_t *reset, const void *dy, const float *dh_final,
                            const gated_scan_saved_t *saved, void *dx, void *dgate_r,
                            void *dgate_i, float *dlam, float *dh0, float *scratch, int64_t Bs,
                            int64_t L, int64_t ED, int io_bf16, void *stream) {
    return io_bf16 ? gated_bwd_entry<__nv_bfloat16>(x, gate_r, gate_i, lam, c, reset, dy, dh_final,
                                                    saved, dx, dgate_r, dgate_i, dlam, dh0, scratch,
                                                    Bs, L, ED, stream)
                   : gated_bwd_entry<float>(x, gate_r, gate_i, lam, c, reset, dy, dh_final, saved,
                                            dx, dgate_r, dgate_i, dlam, dh0, scratch, Bs, L, ED,
                                            stream);
}

ssm_status_t gated_scan_step(const void *x, const void *gate_r, const void *gate_i, const float *lam,
                             float c, float *states, const int32_t *pages, void *y, int64_t Bs,
                             int64_t ED, int64_t num_pages, int input_bf16, void *stream) {
    return input_bf16 ? gated_step_entry<__nv_bfloat16>(x, gate_r, gate_i, lam, c, states, pages, y,
                                                        Bs, ED, num_pages, stream)
                      : gated_step_entry<float>(x, gate_r, gate_i, lam, c, states, pages, y, Bs, ED,
                                                num_pages, stream);
}

ssm_status_t ckpt8_save(const void *x, int8_t *q, float *scale, int64_t rows, int64_t cols,
                        int input_bf16, void *stream) {
    ssm_status_t s = check_ckpt8(x, q, scale, rows, cols, input_bf16 ? 2 : 4);
    if (s != SSM_OK) return s;
    DeviceInfo dev;
    s = current_device(&dev);
    if (s != SSM_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return from_cuda(input_bf16 ? ssm::ckpt8::save(static_cast<const __nv_bfloat16 *>(x), q, scale,
                                                   rows, cols, st)
                                : ssm::ckpt8::save(static_cast<const float *>(x), q, scale, rows,
                                                   cols, st));
}

ssm_status_t ckpt8_load(const int8_t *q, const float *scale, void *x, int64_t rows, int64_t cols,
                        int output_bf16, void *stream) {
    ssm_status_t s = check_ckpt8(x, q, scale, rows, cols, output_bf16 ? 2 : 4);
    if (s != SSM_OK) return s;
    DeviceInfo dev;
    s = current_device(&dev);
    if (s != SSM_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return from_cuda(output_bf16 ? ssm::ckpt8::load(q, scale, static_cast<__nv_bfloat16 *>(x), rows,
                                                    cols, st)
                                 : ssm::ckpt8::load(q, scale, static_cast<float *>(x), rows, cols,
                                                    st));
}

ssm_status_t state_pages_fork(void *pool, uint8_t *used, const int32_t *src, int32_t *dst, int64_t n,
                              int64_t layers, int64_t num_pages, int64_t page_bytes, void *stream) {
    if (!used || (n > 0 && (!src || !dst))) return SSM_ERR_INVALID_ARG;
    if (!aligned(src, 4) || !aligned(dst, 4)) return SSM_ERR_ALIGNMENT;
    DeviceInfo dev;
    const ssm_status_t s = check_pool(pool, n, layers, num_pages, page_bytes, &dev);
    if (s != SSM_OK || n == 0) return s;
    return from_cuda(ssm::pages::fork(pool, used, src, dst, n, layers, num_pages, page_bytes,
                                      dev.num_sms, static_cast<cudaStream_t>(stream)));
}

ssm_status_t state_pages_copy(void *pool, const int32_t *src, const int32_t *dst, int64_t n,
                              int64_t layers, int64_t num_pages, int64_t page_bytes, void *stream) {
    if (n > 0 && (!src || !dst)) return SSM_ERR_INVALID_ARG;
    if (!aligned(src, 4) || !aligned(dst, 4)) return SSM_ERR_ALIGNMENT;
    DeviceInfo dev;
    const ssm_status_t s = check_pool(pool, n, layers, num_pages, page_bytes, &dev);
    if (s != SSM_OK || n == 0) return s;
    return from_cuda(ssm::pages::copy(pool, src, dst, n, layers, num_pages, page_bytes, dev.num_sms,
                                      static_cast<cudaStream_t>(stream)));
}

ssm_status_t state_pages_free(uint8_t *used, const int32_t *pages, int64_t n, int64_t num_pages,
                              void *stream) {
    if (!used || (n > 0 && !pages) || !pages_ok(n, num_pages)) return SSM_ERR_INVALID_ARG;
    if (num_pages > SSM_MAX_PAGES) return SSM_ERR_UNSUPPORTED;
    if (!aligned(pages, 4)) return SSM_ERR_ALIGNMENT;
    DeviceInfo dev;
    const ssm_status_t s = current_device(&dev);
    if (s != SSM_OK || n == 0) return s;
    return from_cuda(ssm::pages::free_pages(used, pages, n, num_pages,
                                            static_cast<cudaStream_t>(stream)));
}

ssm_status_t state_pages_compact(void *pool, uint8_t *used, int32_t *moved, int32_t *pages,
                                 int32_t *scratch, int64_t n, int64_t layers, int64_t num_pages,
                                 int64_t page_bytes, void *stream) {
    if (!used || !moved || !scratch || (n > 0 && !pages)) return SSM_ERR_INVALID_ARG;
    if (!aligned(moved, 4) || !aligned(pages, 4) || !aligned(scratch, 4)) return SSM_ERR_ALIGNMENT;
    DeviceInfo dev;
    const ssm_status_t s = check_pool(pool, n, layers, num_pages, page_bytes, &dev);
    if (s != SSM_OK) return s;
    return from_cuda(ssm::pages::compact(pool, used, moved, pages, scratch, n, layers, num_pages, page_bytes,
                                         dev.num_sms, static_cast<cudaStream_t>(stream)));
}

ssm_status_t delta_rule_fwd(const void *q, const void *k, const void *v, const void *g,
                            const void *beta, float scale, const int32_t *offsets, const float *h0,
                            void *y, float *h_final, void *states, void *errors, void *scratch,
                            int64_t Bs, int64_t L, int64_t G, int64_t H, int64_t K, int64_t V, int64_t n_seq,
                            int input_bf16, void *stream) {
    return input_bf16 ? delta_fwd_entry<__nv_bfloat16>(q, k, v, g, beta, scale, offsets, h0, y, h_final,
                                                       states, errors, scratch, Bs, L, G, H, K, V, n_seq, stream)
                      : delta_fwd_entry<float>(q, k, v, g, beta, scale, offsets, h0, y, h_final, states,
                                               errors, scratch, Bs, L, G, H, K, V, n_seq, stream);
}

int64_t delta_rule_fwd_scratch(int64_t Bs, int64_t L, int64_t G, int64_t H, int64_t K, int64_t V,
                               int64_t n_seq, int input_bf16) {
    if (check_delta_sizes(Bs, L, G, H, K, V, n_seq, 1.0f) != SSM_OK) return 0;
    static const int32_t some = 0;      // only that there are offsets counts
    const ssm::delta::Shape s = delta_shape(n_seq > 0 ? &some : nullptr, Bs, L, G, H, K, V, n_seq, 1.0f);
    const int64_t made = ssm::delta::general::made_bytes(s);
    return input_bf16 && ssm::delta::mma::fits(s) ? std::max(made, ssm::delta::mma::fwd_scratch(s).bytes) : made;
}

int64_t delta_rule_bwd_scratch(int64_t Bs, int64_t L, int64_t G, int64_t H, int64_t K, int64_t V,
                               int64_t n_seq, int io_bf16) {
    if (check_delta_sizes(Bs, L, G, H, K, V, n_seq, 1.0f) != SSM_OK) return 0;
    static const int32_t some = 0;      // only that there are offsets counts
    const ssm::delta::Shape s = delta_shape(n_seq > 0 ? &some : nullptr, Bs, L, G, H, K, V, n_seq, 1.0f);
    return delta_scratch(s, io_bf16 ? 2 : 4).bytes;
}

ssm_status_t delta_rule_bwd(const void *q, const void *k, const void *g, const void *beta, float scale,
                            const int32_t *offsets, const void *dy, const float *dh_final,
                            const void *states, const void *errors, void *dq, void *dk, void *dv,
                            void *dg, void *dbeta, float *dh0, void *scratch, int64_t Bs, int64_t L,
                            int64_t G, int64_t H, int64_t K, int64_t V, int64_t n_seq, int io_bf16,
                            void *stream) {
    return io_bf16 ? delta_bwd_entry<__nv_bfloat16>(q, k, g, beta, scale, offsets, dy, dh_final, states,
                                                    errors, dq, dk, dv, dg, dbeta, dh0, scratch, Bs, L, G,
                                                    H, K, V, n_seq, stream)
                   : delta_bwd_entry<float>(q, k, g, beta, scale, offsets, dy, dh_final, states, errors,
                                            dq, dk, dv, dg, dbeta, dh0, scratch, Bs, L, G, H, K, V, n_seq,
                                            stream);
}

ssm_status_t delta_rule_step(const void *q, const void *k, const void *v, const void *g,
                             const void *beta, float scale, float *states, const int32_t *pages,
                             void *y, int64_t Bs, int64_t G, int64_t H, int64_t K, int64_t V,
                             int64_t num_pages, int input_bf16, void *stream) {
    return input_bf16 ? delta_step_entry<__nv_bfloat16>(q, k, v, g, beta, scale, states, pages, y, Bs, G, H,
                                                        K, V, num_pages, stream)
                      : delta_step_entry<float>(q, k, v, g, beta, scale, states, pages, y, Bs, G, H, K, V,
                                                num_pages, stream);
}

ssm_status_t rms_norm_fwd(const void *x, const void *residual, const float *weight, float eps,
                          void *sum, void *y, int8_t *y_q, float *y_scale, float *rstd, int64_t rows,
                          int64_t cols, int input_bf16, void *stream) {
    return input_bf16 ? norm_fwd_entry<__nv_bfloat16>(x, residual, weight, eps, sum, y, y_q, y_scale, rstd,
                                                      rows, cols, stream)
                      : norm_fwd_entry<float>(x, residual, weight, eps, sum, y, y_q, y_scale, rstd, rows,
                                              cols, stream);
}

ssm_status_t rms_norm_bwd(const void *dy, const void *x, const void *residual, const float *weight, const float *rstd,
                          const void *dsum, void *dx, float *dweight, float *scratch, int64_t rows,
                          int64_t cols, int io_bf16, void *stream) {
    return io_bf16 ? norm_bwd_entry<__nv_bfloat16>(dy, x, residual, weight, rstd, dsum, dx, dweight, scratch, rows,
                                                   cols, stream)
                   : norm_bwd_entry<float>(dy, x, residual, weight, rstd, dsum, dx, dweight, scratch, rows, cols,
                                           stream);
}

ssm_status_t ssm_check_device_errors(void *stream) {
    DeviceInfo dev;
    ssm_status_t s = current_device(&dev);
    if (s != SSM_OK) return s;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return SSM_ERR_CUDA;
    unsigned int flag = 0, flag_bi = 0, flag_g = 0, flag_gb = 0, flag_d = 0, flag_dp = 0, flag_db = 0;
    if (ssm::ssd::take_device_error(&flag) != cudaSuccess) return SSM_ERR_CUDA;
    if (ssm::bidir::take_device_error(&flag_bi) != cudaSuccess) return SSM_ERR_CUDA;
    if (ssm::gated::take_device_error(&flag_g) != cudaSuccess) return SSM_ERR_CUDA;
    if (ssm::gated_bwd::take_device_error(&flag_gb) != cudaSuccess) return SSM_ERR_CUDA;
    if (ssm::delta::mma::fwd::take_device_error(&flag_d) != cudaSuccess) return SSM_ERR_CUDA;
    if (ssm::delta::mma::take_device_error(&flag_dp) != cudaSuccess) return SSM_ERR_CUDA;
    if (ssm::delta::mma::bwd::take_device_error(&flag_db) != cudaSuccess) return SSM_ERR_CUDA;
    return (flag | flag_bi | flag_g | flag_gb | flag_d | flag_dp | flag_db) ? SSM_ERR_DEVICE_TIMEOUT : SSM_OK;
}

ssm_status_t ssm_selftest_wait_timeout(void *stream) {
    DeviceInfo dev;
    ssm_status_t s = current_device(&dev);
    if (s != SSM_OK) return s;
    return from_cuda(ssm::ssd::probe_wait_timeout(static_cast<cudaStream_t>(stream)));
}

ssm_status_t gated_selftest_wait_timeout(int backward, int copy, void *stream) {
    DeviceInfo dev;
    ssm_status_t s = current_device(&dev);
    if (s != SSM_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return from_cuda(backward ? ssm::gated_bwd::probe_wait_timeout(copy != 0, st)
                              : ssm::gated::probe_wait_timeout(copy != 0, st));
}

ssm_status_t delta_selftest_wait_timeout(void *stream) {
    DeviceInfo dev;
    ssm_status_t s = current_device(&dev);
    if (s != SSM_OK) return s;
    return from_cuda(ssm::delta::mma::fwd::probe_wait_timeout(static_cast<cudaStream_t>(stream)));
}

const char *ssm_status_string(ssm_status_t status) {
    switch (status) {
        case SSM_OK: return "SSM_OK";
        case SSM_ERR_INVALID_ARG: return "SSM_ERR_INVALID_ARG: null pointer or size < 1 / overflow";
        case SSM_ERR_UNSUPPORTED: return "SSM_ERR_UNSUPPORTED: size outside the supported set";
        case SSM_ERR_ALIGNMENT: return "SSM_ERR_ALIGNMENT: pointer not aligned as required";
        case SSM_ERR_CUDA: return "SSM_ERR_CUDA: a CUDA call or kernel launch failed";
        case SSM_ERR_DEVICE_TIMEOUT: return "SSM_ERR_DEVICE_TIMEOUT: a bounded device wait ran out";
        case SSM_ERR_NO_DEVICE: return "SSM_ERR_NO_DEVICE: no sm_103 CUDA device is current";
    }
    return "unknown ssm_status_t";
}

int ssm_version(void) { return 100; }

}  // extern "C"
