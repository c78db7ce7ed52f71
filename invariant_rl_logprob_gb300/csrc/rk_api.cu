// rk_api.cu -- the extern "C" entry points declared in include/rk.h:
// argument validation (before any launch), per-device lookups, TMA descriptor
// encoding, and dispatch to the kernels' launchers.
#include <cudaTypedefs.h>

#include <cmath>
#include <cstring>
#include <mutex>

#include "rk.h"
#include "rk_device.cuh"
#include "rk_internal.h"
#include "token_loss.cuh"

// One error word per device (the module is loaded per device context).
__device__ unsigned int g_rk_device_error = 0u;

namespace rk {
namespace {

constexpr int kMaxDevices = 64;

std::mutex g_mu;
DeviceInfo g_dev[kMaxDevices];
bool g_dev_ready[kMaxDevices] = {};

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

thread_local int g_last_cuda_error = 0;

void load_encode() {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
}

bool encode_2d(CUtensorMap *map, CUtensorMapDataType dt, uint32_t esize, const void *base,
               uint64_t inner, uint64_t outer, uint64_t row_stride_bytes, uint32_t box_inner,
               uint32_t box_outer, CUtensorMapSwizzle swizzle) {
    std::call_once(g_encode_once, load_encode);
    if (!g_encode) return false;
    (void)esize;
    cuuint64_t dims[2] = {inner, outer};
    cuuint64_t strides[1] = {row_stride_bytes};
    cuuint32_t box[2] = {box_inner, box_outer};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = g_encode(map, dt, 2, const_cast<void *>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE,
                          swizzle,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

rk_status cuda_fail(cudaError_t e) {
    g_last_cuda_error = (int)e;
    return RK_ERR_CUDA;
}

}  // namespace

bool encode_tmap_bf16_2d(CUtensorMap *map, const void *base, uint64_t inner, uint64_t outer,
                         uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer,
                         bool sw128) {
    return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, inner, outer,
                     row_stride_bytes, box_inner, box_outer,
                     sw128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE);
}

bool encode_tmap_bf16_2d_sw64(CUtensorMap *map, const void *base, uint64_t inner, uint64_t outer,
                              uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer) {
    return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, inner, outer,
                     row_stride_bytes, box_inner, box_outer, CU_TENSOR_MAP_SWIZZLE_64B);
}

void record_cuda_error(int e) { g_last_cuda_error = e; }

cudaError_t current_device_info(DeviceInfo *di) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (g_dev_ready[dev]) {
            *di = g_dev[dev];
            return cudaSuccess;
        }
    }
    DeviceInfo d;
    d.device = dev;
    e = cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    void *p = nullptr;
    e = cudaGetSymbolAddress(&p, g_rk_device_error);
    if (e != cudaSuccess) return e;
    d.err = static_cast<unsigned *>(p);
    std::lock_guard<std::mutex> lk(g_mu);
    g_dev[dev] = d;
    g_dev_ready[dev] = true;
    *di = d;
    return cudaSuccess;
}

}  // namespace rk

using rk::DeviceInfo;

namespace {

// One thread waits on an mbarrier that nothing ever arrives on, through the
// same bounded wait the pipelines use; it gives up after `limit_ns`.
__global__ void selftest_wait_kernel(uint64_t limit_ns, unsigned *err) {
    __shared__ uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        rk::mbar_init(rk::smem_u32(&bar), 1);
        abort_flag = 0;
        rk::fence_mbar_init();
        (void)rk::mbar_wait_limit(rk::smem_u32(&bar), 0, &abort_flag, err, limit_ns);
    }
}

using rk::aligned;
using rk::check_rows;

}  // namespace

extern "C" {

const char *rk_status_string(rk_status s) {
    switch (s) {
        case RK_OK: return "RK_OK";
        case RK_ERR_INVALID_ARG: return "RK_ERR_INVALID_ARG";
        case RK_ERR_UNSUPPORTED: return "RK_ERR_UNSUPPORTED";
        case RK_ERR_WORKSPACE: return "RK_ERR_WORKSPACE";
        case RK_ERR_CUDA: return "RK_ERR_CUDA";
    }
    return "RK_ERR_UNKNOWN";
}

int rk_last_cuda_error(void) { return rk::g_last_cuda_error; }

const char *rk_version(void) { return "rk 0.1.0 sm_103a"; }

size_t rk_linear_logp_workspace_size(int64_t T, int64_t H, int64_t V) {
    (void)H;
    if (T <= 0 || V <= 0) return 0;
    return rk::linear_fwd_workspace_bytes(T, V);
}

rk_status rk_linear_logp(const uint16_t *h, const uint16_t *W, const int64_t *targets,
                         const int32_t *cu_seqlens, int32_t num_seqs, int64_t T, int64_t H,
                         int64_t V, float *logp, float *lse, void *workspace,
                         size_t workspace_bytes, void *stream) {
    if (T < 0 || H <= 0 || V <= 0) return RK_ERR_INVALID_ARG;
    if (T == 0) return RK_OK;
    if (!h || !W || !logp) return RK_ERR_INVALID_ARG;
    rk_status st = check_rows(targets, cu_seqlens, num_seqs);
    if (st != RK_OK) return st;
    if (H % 64 != 0 || H > 65536 || V >= (int64_t(1) << 31) || T >= (int64_t(1) << 31))
        return RK_ERR_UNSUPPORTED;
    if (!aligned(h, 16) || !aligned(W, 16)) return RK_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < rk::linear_fwd_workspace_bytes(T, V))
        return RK_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_linear_fwd(h, W, targets, cu_seqlens, num_seqs, T, H, V, logp, lse, workspace,
                              di, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

rk_status rk_linear_logp_grpo(const uint16_t *h, const uint16_t *W, const int64_t *targets,
                              const int32_t *cu_seqlens, int32_t num_seqs, int64_t T, int64_t H,
                              int64_t V, const float *logp_old, const float *logp_ref,
                              const float *advantages, float eps_low, float eps_high, float beta,
                              float scale, float *logp, float *lse, float *loss, float *grad_logp,
                              float *ratio, float *kl, void *workspace, size_t workspace_bytes,
                              void *stream) {
    if (T < 0 || H <= 0 || V <= 0) return RK_ERR_INVALID_ARG;
    if (T == 0) return RK_OK;
    if (!h || !W || !logp || !logp_old || !advantages || !loss || !grad_logp)
        return RK_ERR_INVALID_ARG;
    rk_status st = check_rows(targets, cu_seqlens, num_seqs);
    if (st != RK_OK) return st;
    if (!(eps_low >= 0.f && eps_low < 1.f) || !(eps_high >= 0.f) || !(beta >= 0.f))
        return RK_ERR_INVALID_ARG;
    if (H % 64 != 0 || H > 65536 || V >= (int64_t(1) << 31) || T >= (int64_t(1) << 31))
        return RK_ERR_UNSUPPORTED;
    if (!aligned(h, 16) || !aligned(W, 16)) return RK_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < rk::linear_fwd_workspace_bytes(T, V))
        return RK_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    const rk::GrpoArgs p{logp_old, logp_ref, advantages, eps_low, eps_high, beta, scale,
                         loss, grad_logp, ratio, kl};
    e = rk::launch_linear_fwd(h, W, targets, cu_seqlens, num_seqs, T, H, V, logp, lse, workspace,
                              di, static_cast<cudaStream_t>(stream), &p);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

size_t rk_linear_logp_saved_size(int64_t T, int64_t H, int64_t V) {
    (void)H;
    if (T <= 0 || V <= 0) return 0;
    return rk::linear_fwd_saved_bytes(T, V);
}

rk_status rk_linear_logp_fwd_saved(const uint16_t *h, const uint16_t *W, const int64_t *targets,
                                   const int32_t *cu_seqlens, int32_t num_seqs, int64_t T,
                                   int64_t H, int64_t V, float *logp, float *lse, void *saved,
                                   size_t saved_bytes, void *stream) {
    if (T < 0 || H <= 0 || V <= 0) return RK_ERR_INVALID_ARG;
    if (T == 0) return RK_OK;
    if (!h || !W || !logp) return RK_ERR_INVALID_ARG;
    rk_status st = check_rows(targets, cu_seqlens, num_seqs);
    if (st != RK_OK) return st;
    if (H % 64 != 0 || H > 65536 || V >= (int64_t(1) << 31) || T >= (int64_t(1) << 31))
        return RK_ERR_UNSUPPORTED;
    if (!aligned(h, 16) || !aligned(W, 16)) return RK_ERR_UNSUPPORTED;
    if (!saved || saved_bytes < rk::linear_fwd_saved_bytes(T, V)) return RK_ERR_WORKSPACE;
    if (!aligned(saved, 256)) return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_linear_fwd_saved(h, W, targets, cu_seqlens, num_seqs, T, H, V, logp, lse, saved,
                                    di, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

size_t rk_linear_logp_bwd_saved_workspace_size(int64_t T, int64_t H, int64_t V) {
    (void)H;
    if (T <= 0 || V <= 0) return 0;
    return rk::linear_bwd_saved_workspace_bytes(T);
}

rk_status rk_linear_logp_bwd_saved(const uint16_t *h, const uint16_t *W, const int64_t *targets,
                                   const int32_t *cu_seqlens, int32_t num_seqs, int64_t T,
                                   int64_t H, int64_t V, const float *lse,
                                   const float *grad_logp, void *saved, size_t saved_bytes,
                                   float *dh, void *workspace, size_t workspace_bytes,
                                   void *stream) {
    if (T < 0 || H <= 0 || V <= 0) return RK_ERR_INVALID_ARG;
    if (T == 0) return RK_OK;
    if (!h || !W || !lse || !grad_logp || !dh) return RK_ERR_INVALID_ARG;
    rk_status st = check_rows(targets, cu_seqlens, num_seqs);
    if (st != RK_OK) return st;
    if (H % 64 != 0 || H > 65536 || V >= (int64_t(1) << 31) || T >= (int64_t(1) << 31))
        return RK_ERR_UNSUPPORTED;
    if ((V + 8191) / 8192 > 65535) return RK_ERR_UNSUPPORTED;
    if (!aligned(h, 16) || !aligned(W, 16) || !aligned(dh, 16)) return RK_ERR_UNSUPPORTED;
    if (!saved || saved_bytes < rk::linear_fwd_saved_bytes(T, V)) return RK_ERR_WORKSPACE;
    if (!aligned(saved, 256)) return RK_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < rk::linear_bwd_saved_workspace_bytes(T))
        return RK_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_linear_bwd_saved(h, W, targets, cu_seqlens, num_seqs, T, H, V, lse, grad_logp,
                                    saved, dh, workspace, di, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

rk_status rk_logp_from_logits(const uint16_t *logits, const int64_t *targets,
                              const int32_t *cu_seqlens, int32_t num_seqs, int64_t T, int64_t V,
                              float *logp, float *lse, void *stream) {
    if (T < 0 || V <= 0) return RK_ERR_INVALID_ARG;
    if (T == 0) return RK_OK;
    if (!logits || !logp) return RK_ERR_INVALID_ARG;
    rk_status st = check_rows(targets, cu_seqlens, num_seqs);
    if (st != RK_OK) return st;
    if (V >= (int64_t(1) << 31)) return RK_ERR_UNSUPPORTED;
    if (!aligned(logits, 2)) return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_logits_logp(logits, targets, cu_seqlens, num_seqs, T, V, logp, lse, di,
                               static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

size_t rk_linear_logp_bwd_workspace_size(int64_t T, int64_t H, int64_t V) {
    (void)H;
    if (T <= 0 || V <= 0) return 0;
    const int64_t q = rk::linear_bwd_chunk_quantum();
    return rk::linear_bwd_chunk_bytes((T + q - 1) / q * q, V);
}

size_t rk_linear_logp_bwd_min_workspace_size(int64_t H, int64_t V) {
    (void)H;
    if (V <= 0) return 0;
    return rk::linear_bwd_chunk_bytes(rk::linear_bwd_chunk_quantum(), V);
}

rk_status rk_linear_logp_bwd(const uint16_t *h, const uint16_t *W, const int64_t *targets,
                             const int32_t *cu_seqlens, int32_t num_seqs, int64_t T, int64_t H,
                             int64_t V, const float *lse, const float *grad_logp, float *dh,
                             void *workspace, size_t workspace_bytes, void *stream) {
    if (T < 0 || H <= 0 || V <= 0) return RK_ERR_INVALID_ARG;
    if (T == 0) return RK_OK;
    if (!h || !W || !lse || !grad_logp || !dh) return RK_ERR_INVALID_ARG;
    rk_status st = check_rows(targets, cu_seqlens, num_seqs);
    if (st != RK_OK) return st;
    if (H % 64 != 0 || H > 65536 || V >= (int64_t(1) << 31) || T >= (int64_t(1) << 31))
        return RK_ERR_UNSUPPORTED;
    if (!aligned(h, 16) || !aligned(W, 16) || !aligned(dh, 16)) return RK_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < rk_linear_logp_bwd_min_workspace_size(H, V))
        return RK_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_linear_bwd(h, W, targets, cu_seqlens, num_seqs, T, H, V, lse, grad_logp, dh,
                              workspace, workspace_bytes, di, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

size_t rk_lm_head_workspace_size(void) { return 256; }

rk_status rk_lm_head(const uint16_t *h, const uint16_t *W, int64_t T, int64_t H, int64_t V,
                     uint16_t *logits, int64_t ld_logits, void *workspace,
                     size_t workspace_bytes, void *stream) {
    if (T < 0 || H <= 0 || V <= 0) return RK_ERR_INVALID_ARG;
    if (T == 0) return RK_OK;
    if (!h || !W || !logits || ld_logits < V) return RK_ERR_INVALID_ARG;
    if (H % 64 != 0 || H > 65536 || V >= (int64_t(1) << 31) || T >= (int64_t(1) << 31))
        return RK_ERR_UNSUPPORTED;
    if (!aligned(h, 16) || !aligned(W, 16) || !aligned(logits, 16) || ld_logits % 8 != 0)
        return RK_ERR_UNSUPPORTED;
    if (workspace && (workspace_bytes < rk_lm_head_workspace_size() || !aligned(workspace, 16)))
        return RK_ERR_WORKSPACE;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_lm_head(h, W, T, H, V, logits, ld_logits, static_cast<unsigned *>(workspace), di,
                           static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

rk_status rk_logp_from_logits_bwd(const uint16_t *logits, const int64_t *targets,
                                  const int32_t *cu_seqlens, int32_t num_seqs, int64_t T,
                                  int64_t V, const float *lse, const float *grad_logp,
                                  float *dlogits, void *stream) {
    if (T < 0 || V <= 0) return RK_ERR_INVALID_ARG;
    if (T == 0) return RK_OK;
    if (!logits || !lse || !grad_logp || !dlogits) return RK_ERR_INVALID_ARG;
    rk_status st = check_rows(targets, cu_seqlens, num_seqs);
    if (st != RK_OK) return st;
    if (V >= (int64_t(1) << 31)) return RK_ERR_UNSUPPORTED;
    if (!aligned(logits, 2) || !aligned(dlogits, 4)) return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_logits_bwd(logits, targets, cu_seqlens, num_seqs, T, V, lse, grad_logp, dlogits,
                              di, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

rk_status rk_grpo_token_loss(const float *logp, const float *logp_old, const float *logp_ref,
                             const float *advantages, const int64_t *targets,
                             const int32_t *cu_seqlens, int32_t num_seqs, int64_t T,
                             float eps_low, float eps_high, float beta, float scale, float *loss,
                             float *grad_logp, float *ratio, float *kl, void *stream) {
    if (T < 0) return RK_ERR_INVALID_ARG;
    if (T == 0) return RK_OK;
    if (!logp || !logp_old || !advantages || !loss || !grad_logp) return RK_ERR_INVALID_ARG;
    rk_status st = check_rows(targets, cu_seqlens, num_seqs);
    if (st != RK_OK) return st;
    if (!(eps_low >= 0.f && eps_low < 1.f) || !(eps_high >= 0.f) || !(beta >= 0.f))
        return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_grpo_token(logp, logp_old, logp_ref, advantages, targets, cu_seqlens, num_seqs,
                              T, eps_low, eps_high, beta, scale, loss, grad_logp, ratio, kl, di,
                              static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

size_t rk_linear_greedy_workspace_size(int64_t T, int64_t H, int64_t V) {
    (void)H;
    if (T <= 0 || V <= 0) return 0;
    return rk::linear_greedy_workspace_bytes(T, V);
}

rk_status rk_linear_greedy(const uint16_t *h, const uint16_t *W, const int32_t *cu_seqlens,
                           int32_t num_seqs, int64_t T, int64_t H, int64_t V, int64_t *token,
                           float *logp, float *lse, void *workspace, size_t workspace_bytes,
                           void *stream) {
    if (T < 0 || H <= 0 || V <= 0) return RK_ERR_INVALID_ARG;
    if (T == 0) return RK_OK;
    if (!h || !W || !token || !logp) return RK_ERR_INVALID_ARG;
    if (cu_seqlens && num_seqs < 0) return RK_ERR_INVALID_ARG;
    if (H % 64 != 0 || H > 65536 || V >= (int64_t(1) << 31) || T >= (int64_t(1) << 31))
        return RK_ERR_UNSUPPORTED;
    if (!aligned(h, 16) || !aligned(W, 16)) return RK_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < rk::linear_greedy_workspace_bytes(T, V))
        return RK_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_linear_greedy(h, W, cu_seqlens, num_seqs, T, H, V, token, logp, lse, workspace,
                                 di, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

size_t rk_linear_logp_dw_workspace_size(int64_t n, int64_t H, int64_t V) {
    if (n <= 0 || H <= 0 || V <= 0) return 0;
    return rk::linear_dw_workspace_bytes(n, H, V);
}

rk_status rk_linear_logp_dw(const uint16_t *h, const uint16_t *W, const int64_t *targets,
                            const int32_t *cu_seqlens, int32_t num_seqs, int64_t T, int64_t H,
                            int64_t V, const float *lse, const float *grad_logp,
                            const int64_t *row_order, int64_t n_order, float *dW,
                            void *workspace, size_t workspace_bytes, void *stream) {
    if (T < 0 || H <= 0 || V <= 0) return RK_ERR_INVALID_ARG;
    if (!dW || !W) return RK_ERR_INVALID_ARG;
    const int64_t n = row_order ? n_order : T;
    if (n < 0) return RK_ERR_INVALID_ARG;
    if (n > 0 && (!h || !lse || !grad_logp)) return RK_ERR_INVALID_ARG;
    rk_status st = check_rows(targets, cu_seqlens, num_seqs);
    if (st != RK_OK && n > 0) return st;
    if (H % 64 != 0 || H > 65536 || V >= (int64_t(1) << 31) || T >= (int64_t(1) << 31) ||
        n >= (int64_t(1) << 31))
        return RK_ERR_UNSUPPORTED;
    if ((h && !aligned(h, 16)) || !aligned(W, 16) || !aligned(dW, 16)) return RK_ERR_UNSUPPORTED;
    if (n > 0 && (!workspace || workspace_bytes < rk::linear_dw_workspace_bytes(n, H, V)))
        return RK_ERR_WORKSPACE;
    if (n > 0 && !aligned(workspace, 16)) return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_linear_dw(h, W, targets, cu_seqlens, num_seqs, T, H, V, lse, grad_logp,
                             row_order, n, dW, workspace, di, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

size_t rk_linear_logp_bwd_full_workspace_size(int64_t n, int64_t H, int64_t V) {
    if (n <= 0 || H <= 0 || V <= 0) return 0;
    return rk::linear_bwd_full_workspace_bytes(n, H, V);
}

rk_status rk_linear_logp_bwd_full(const uint16_t *h, const uint16_t *W, const int64_t *targets,
                                  const int32_t *cu_seqlens, int32_t num_seqs, int64_t T,
                                  int64_t H, int64_t V, const float *lse, const float *grad_logp,
                                  const int64_t *row_order, int64_t n_order, float *dh, float *dW,
                                  void *workspace, size_t workspace_bytes, void *stream) {
    if (T < 0 || H <= 0 || V <= 0) return RK_ERR_INVALID_ARG;
    if (!dW || !W || (T > 0 && !dh)) return RK_ERR_INVALID_ARG;
    const int64_t n = row_order ? n_order : T;
    if (n < 0) return RK_ERR_INVALID_ARG;
    if ((n > 0 || T > 0) && (!h || !lse || !grad_logp)) return RK_ERR_INVALID_ARG;
    if (T > 0 || n > 0) {
        rk_status st = check_rows(targets, cu_seqlens, num_seqs);
        if (st != RK_OK) return st;
    }
    if (H % 64 != 0 || H > 65536 || V >= (int64_t(1) << 31) || T >= (int64_t(1) << 31) ||
        n >= (int64_t(1) << 31))
        return RK_ERR_UNSUPPORTED;
    if ((h && !aligned(h, 16)) || !aligned(W, 16) || !aligned(dW, 16) || (dh && !aligned(dh, 16)))
        return RK_ERR_UNSUPPORTED;
    if (n > 0 && (!workspace || workspace_bytes < rk::linear_bwd_full_workspace_bytes(n, H, V)))
        return RK_ERR_WORKSPACE;
    if (n > 0 && !aligned(workspace, 16)) return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_linear_bwd_full(h, W, targets, cu_seqlens, num_seqs, T, H, V, lse, grad_logp,
                                   row_order, n, dh, dW, workspace, di,
                                   static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

rk_status rk_set_row_blocks(int32_t n) {
    if (n < 0 || n > 2) return RK_ERR_INVALID_ARG;
    rk::set_row_blocks_override((int)n);
    return RK_OK;
}

int32_t rk_last_row_blocks(int32_t gemm) {
    if (gemm != 0 && gemm != 1) return -1;
    return (int32_t)rk::last_row_blocks(gemm == 0 ? rk::RowGemm::kDhGemm : rk::RowGemm::kDwGemm);
}

int32_t rk_last_tile_order(int32_t gemm) {
    if (gemm != 0 && gemm != 1) return -1;
    return (int32_t)rk::last_tile_order(gemm == 0 ? rk::RowGemm::kDhGemm : rk::RowGemm::kDwGemm);
}

rk_status rk_linear_logp_bwd_full_saved(const uint16_t *h, const uint16_t *W,
                                        const int64_t *targets, const int32_t *cu_seqlens,
                                        int32_t num_seqs, int64_t T, int64_t H, int64_t V,
                                        const float *lse, const float *grad_logp,
                                        const void *saved, size_t saved_bytes,
                                        const int64_t *row_order, int64_t n_order, float *dh,
                                        float *dW, void *workspace, size_t workspace_bytes,
                                        void *stream) {
    if (T < 0 || H <= 0 || V <= 0) return RK_ERR_INVALID_ARG;
    if (!dW || !W || (T > 0 && !dh)) return RK_ERR_INVALID_ARG;
    const int64_t n = row_order ? n_order : T;
    if (n < 0) return RK_ERR_INVALID_ARG;
    if ((n > 0 || T > 0) && (!h || !lse || !grad_logp)) return RK_ERR_INVALID_ARG;
    if (T > 0 || n > 0) {
        rk_status st = check_rows(targets, cu_seqlens, num_seqs);
        if (st != RK_OK) return st;
    }
    if (H % 64 != 0 || H > 65536 || V >= (int64_t(1) << 31) || T >= (int64_t(1) << 31) ||
        n >= (int64_t(1) << 31))
        return RK_ERR_UNSUPPORTED;
    if ((V + 8191) / 8192 > 65535 || (V + 63) / 64 > 65535) return RK_ERR_UNSUPPORTED;
    if ((h && !aligned(h, 16)) || !aligned(W, 16) || !aligned(dW, 16) || (dh && !aligned(dh, 16)))
        return RK_ERR_UNSUPPORTED;
    if (T > 0 && (!saved || saved_bytes < rk::linear_fwd_saved_bytes(T, V)))
        return RK_ERR_WORKSPACE;
    if (saved && !aligned(saved, 256)) return RK_ERR_INVALID_ARG;
    if (n > 0 && (!workspace || workspace_bytes < rk::linear_bwd_full_workspace_bytes(n, H, V)))
        return RK_ERR_WORKSPACE;
    if (n > 0 && !aligned(workspace, 16)) return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_linear_bwd_full(h, W, targets, cu_seqlens, num_seqs, T, H, V, lse, grad_logp,
                                   row_order, n, dh, dW, workspace, di,
                                   static_cast<cudaStream_t>(stream), T > 0 ? saved : nullptr);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

static bool good_type(rk_dtype t) { return t == RK_BF16 || t == RK_FP32; }
static int elem_size(rk_dtype t) { return t == RK_E4M3 ? 1 : t == RK_BF16 ? 2 : 4; }
static bool elem_aligned(const void *p, rk_dtype t) { return aligned(p, elem_size(t)); }

// Whether two ranges of memory have a byte in common.
static bool ranges_meet(const void *a, __int128 bytes_a, const void *b, __int128 bytes_b) {
    const __int128 x = (__int128)reinterpret_cast<uintptr_t>(a), y = (__int128)reinterpret_cast<uintptr_t>(b);
    return x < y + bytes_b && y < x + bytes_a;
}

// Whether two [T, V] matrices have no byte in common.  (Rows side by side in one buffer take
// the first branch; the loop is for strides of different lengths in ranges that meet.)
static bool rows_apart(const rk::RulesMatrix &in, const rk::RulesMatrix &out, int64_t T, int64_t V) {
    using i128 = __int128;  // no address or stride takes it past its range
    const i128 size_a = elem_size(in.type), size_b = elem_size(out.type);
    const i128 a = (i128)reinterpret_cast<uintptr_t>(in.p), b = (i128)reinterpret_cast<uintptr_t>(out.p);
    const i128 step_a = in.ld * size_a, step_b = out.ld * size_b;  // bytes from row to row
    const i128 row_a = V * size_a, row_b = V * size_b;             // bytes of a row
    if (!ranges_meet(in.p, (T - 1) * step_a + row_a, out.p, (T - 1) * step_b + row_b)) return true;
    // row i of a meets row j of b if and only if b_j + row_b > a_i and b_j < a_i + row_a: the first j
    // with the former decides
    const auto first_above = [](i128 x, i128 step) {  // the least k with k step > x
        return x >= 0 ? x / step + 1 : -((-x - 1) / step);
    };
    if (step_a == step_b) {  // k = j - i
        i128 k = first_above(a - b - row_b, step_a);
        if (k < 1 - T) k = 1 - T;
        return k > T - 1 || b + k * step_a >= a + row_a;
    }
    for (int64_t i = 0; i < T; ++i) {
        const i128 at = a + i * step_a;
        i128 j = first_above(at - b - row_b, step_b);
        if (j < 0) j = 0;
        if (j < T && b + j * step_b < at + row_a) return false;
    }
    return true;
}

// Whether a [T, V] matrix can be made from another one that other blocks still read: in
// its place, or with no byte of it among the other's.
static bool can_hold(const rk::RulesMatrix &in, const rk::RulesMatrix &out, int64_t T, int64_t V) {
    return (in.p == out.p && in.type == out.type && (in.ld == out.ld || T == 1)) ||
           rows_apart(in, out, T, V);
}

// Argument checks of a rules struct against T rows.
static rk_status check_rules(const rk_logits_rules *r, int64_t T) {
    if (!r) return RK_ERR_INVALID_ARG;
    if (r->num_requests < 0 || r->num_tokens < 0 || r->num_bias < 0 || r->mask_rows < 0)
        return RK_ERR_INVALID_ARG;
    if (r->num_requests >= (int64_t(1) << 31)) return RK_ERR_UNSUPPORTED;
    if (r->num_requests == 0 &&
        (r->temperature || r->repetition || r->frequency || r->presence || r->tokens || r->bias_ids))
        return RK_ERR_INVALID_ARG;
    if (r->tokens && !r->token_offsets) return RK_ERR_INVALID_ARG;
    if (r->prompt_lengths && !r->tokens) return RK_ERR_INVALID_ARG;
    if (r->bias_ids && (!r->bias_values || !r->bias_offsets)) return RK_ERR_INVALID_ARG;
    if (r->num_requests > 0 && !r->row_request && r->num_requests != T) return RK_ERR_INVALID_ARG;
    if (r->mask && !r->row_mask && r->mask_rows != T) return RK_ERR_INVALID_ARG;
    return RK_OK;
}

rk_status rk_logits_rules_apply(const void *logits, rk_dtype logits_type, int64_t ld_logits,
                                const rk_logits_rules *rules, int64_t T, int64_t V, void *out,
                                rk_dtype out_type, int64_t ld_out, void *stream) {
    if (T < 0 || V <= 0 || !good_type(logits_type) || !good_type(out_type)) return RK_ERR_INVALID_ARG;
    if (T == 0) return RK_OK;
    if (!logits || !out || ld_logits < V || ld_out < V) return RK_ERR_INVALID_ARG;
    if (V >= (int64_t(1) << 31) || T >= (int64_t(1) << 31)) return RK_ERR_UNSUPPORTED;
    rk_status st = check_rules(rules, T);
    if (st != RK_OK) return st;
    if (!elem_aligned(logits, logits_type) || !elem_aligned(out, out_type)) return RK_ERR_INVALID_ARG;
    const rk::RulesMatrix from{logits, logits_type, ld_logits}, to{out, out_type, ld_out};
    if (!can_hold(from, to, T, V)) return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_rules_apply(from, *rules, T, V, to, di, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

size_t rk_logp_from_logits_rules_workspace_size(int64_t T, int64_t V) {
    if (T <= 0 || V <= 0) return 0;
    return rk::logp_rules_workspace_bytes(T, V);
}

// rk_logp_from_logits_rules with the log-sum-exp in fp32 or (lse64) in fp64; either may be NULL.
static rk_status logp_rules(const void *logits, rk_dtype logits_type, int64_t ld_logits,
                            const int64_t *targets, const int32_t *cu_seqlens, int32_t num_seqs,
                            const rk_logits_rules *rules, int64_t T, int64_t V, float *logp,
                            float *lse, double *lse64, void *workspace, size_t workspace_bytes,
                            void *stream) {
    if (T < 0 || V <= 0 || !good_type(logits_type)) return RK_ERR_INVALID_ARG;
    if (T == 0) return RK_OK;
    if (!logits || !logp || ld_logits < V) return RK_ERR_INVALID_ARG;
    rk_status st = check_rows(targets, cu_seqlens, num_seqs);
    if (st != RK_OK) return st;
    if (V >= (int64_t(1) << 31) || T >= (int64_t(1) << 31)) return RK_ERR_UNSUPPORTED;
    st = check_rules(rules, T);
    if (st != RK_OK) return st;
    if (!elem_aligned(logits, logits_type)) return RK_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < rk::logp_rules_workspace_bytes(T, V)) return RK_ERR_WORKSPACE;
    if (!aligned(workspace, 16) || !aligned(lse64, 8)) return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_rules_logp({logits, logits_type, ld_logits}, targets, cu_seqlens, num_seqs, *rules,
                              T, V, logp, lse, lse64, workspace, di,
                              static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

rk_status rk_logp_from_logits_rules(const void *logits, rk_dtype logits_type, int64_t ld_logits,
                                    const int64_t *targets, const int32_t *cu_seqlens,
                                    int32_t num_seqs, const rk_logits_rules *rules, int64_t T,
                                    int64_t V, float *logp, float *lse, void *workspace,
                                    size_t workspace_bytes, void *stream) {
    return logp_rules(logits, logits_type, ld_logits, targets, cu_seqlens, num_seqs, rules, T, V, logp,
                      lse, nullptr, workspace, workspace_bytes, stream);
}

rk_status rk_logp_from_logits_rules_lse64(const void *logits, rk_dtype logits_type,
                                          int64_t ld_logits, const int64_t *targets,
                                          const int32_t *cu_seqlens, int32_t num_seqs,
                                          const rk_logits_rules *rules, int64_t T, int64_t V,
                                          float *logp, double *lse, void *workspace,
                                          size_t workspace_bytes, void *stream) {
    return logp_rules(logits, logits_type, ld_logits, targets, cu_seqlens, num_seqs, rules, T, V, logp,
                      nullptr, lse, workspace, workspace_bytes, stream);
}

// rk_logp_from_logits_rules_bwd from a log-sum-exp in fp32 or (lse64) in fp64; one of them is NULL.
static rk_status logp_rules_bwd(const void *logits, rk_dtype logits_type, int64_t ld_logits,
                                const int64_t *targets, const int32_t *cu_seqlens, int32_t num_seqs,
                                const rk_logits_rules *rules, int64_t T, int64_t V, const float *lse,
                                const double *lse64, const float *grad_logp, void *dlogits,
                                rk_dtype dlogits_type, int64_t ld_dlogits, void *stream) {
    if (T < 0 || V <= 0 || !good_type(logits_type) || !good_type(dlogits_type))
        return RK_ERR_INVALID_ARG;
    if (T == 0) return RK_OK;
    if (!logits || (!lse && !lse64) || !grad_logp || !dlogits || ld_logits < V || ld_dlogits < V)
        return RK_ERR_INVALID_ARG;
    rk_status st = check_rows(targets, cu_seqlens, num_seqs);
    if (st != RK_OK) return st;
    if (V >= (int64_t(1) << 31) || T >= (int64_t(1) << 31)) return RK_ERR_UNSUPPORTED;
    st = check_rules(rules, T);
    if (st != RK_OK) return st;
    if (!elem_aligned(logits, logits_type) || !elem_aligned(dlogits, dlogits_type) ||
        !aligned(lse64, 8))
        return RK_ERR_INVALID_ARG;
    const rk::RulesMatrix from{logits, logits_type, ld_logits}, to{dlogits, dlogits_type, ld_dlogits};
    if (!can_hold(from, to, T, V)) return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_rules_bwd(from, targets, cu_seqlens, num_seqs, *rules, T, V, lse, lse64, grad_logp, to,
                             di, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

rk_status rk_logp_from_logits_rules_bwd(const void *logits, rk_dtype logits_type,
                                        int64_t ld_logits, const int64_t *targets,
                                        const int32_t *cu_seqlens, int32_t num_seqs,
                                        const rk_logits_rules *rules, int64_t T, int64_t V,
                                        const float *lse, const float *grad_logp, void *dlogits,
                                        rk_dtype dlogits_type, int64_t ld_dlogits, void *stream) {
    return logp_rules_bwd(logits, logits_type, ld_logits, targets, cu_seqlens, num_seqs, rules, T, V, lse,
                          nullptr, grad_logp, dlogits, dlogits_type, ld_dlogits, stream);
}

rk_status rk_logp_from_logits_rules_bwd_lse64(const void *logits, rk_dtype logits_type,
                                              int64_t ld_logits, const int64_t *targets,
                                              const int32_t *cu_seqlens, int32_t num_seqs,
                                              const rk_logits_rules *rules, int64_t T, int64_t V,
                                              const double *lse, const float *grad_logp,
                                              void *dlogits, rk_dtype dlogits_type,
                                              int64_t ld_dlogits, void *stream) {
    return logp_rules_bwd(logits, logits_type, ld_logits, targets, cu_seqlens, num_seqs, rules, T, V,
                          nullptr, lse, grad_logp, dlogits, dlogits_type, ld_dlogits, stream);
}

rk_status rk_embedding(const int64_t *ids, const int32_t *cu_seqlens, int32_t num_seqs,
                       const void *E, rk_dtype e_type, int64_t T, int64_t H, int64_t V, float scale,
                       void *out, rk_dtype out_type, void *stream) {
    if (T < 0 || H <= 0 || V <= 0 || !good_type(e_type) || !good_type(out_type))
        return RK_ERR_INVALID_ARG;
    if (T == 0) return RK_OK;
    if (!E || !out) return RK_ERR_INVALID_ARG;
    rk_status st = check_rows(ids, cu_seqlens, num_seqs);
    if (st != RK_OK) return st;
    const int64_t lim = int64_t(1) << 31;
    if (V >= lim || T >= lim || H >= lim) return RK_ERR_UNSUPPORTED;
    if (!elem_aligned(E, e_type) || !elem_aligned(out, out_type)) return RK_ERR_INVALID_ARG;
    if (ranges_meet(E, (__int128)V * H * elem_size(e_type), out, (__int128)T * H * elem_size(out_type)))
        return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_embedding(ids, cu_seqlens, num_seqs, E, e_type, T, H, V, scale, out, out_type, di,
                             static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

size_t rk_embedding_bwd_workspace_size(int64_t n, int64_t H, int64_t V) {
    if (n <= 0 || H <= 0 || V <= 0) return 0;
    return rk::embedding_bwd_workspace_bytes(n, H);
}

rk_status rk_embedding_bwd(const void *dout, rk_dtype dout_type, const int64_t *ids,
                           const int32_t *cu_seqlens, int32_t num_seqs, int64_t T, int64_t H,
                           int64_t V, float scale, const int64_t *row_order, int64_t n_order,
                           float *dE, int32_t accumulate, void *workspace, size_t workspace_bytes,
                           void *stream) {
    if (T < 0 || H <= 0 || V <= 0 || !good_type(dout_type)) return RK_ERR_INVALID_ARG;
    if (!dE || (accumulate != 0 && accumulate != 1)) return RK_ERR_INVALID_ARG;
    const int64_t n = row_order ? n_order : T;
    if (n < 0) return RK_ERR_INVALID_ARG;
    if (T > 0 && n > 0) {
        if (!dout) return RK_ERR_INVALID_ARG;
        rk_status st = check_rows(ids, cu_seqlens, num_seqs);
        if (st != RK_OK) return st;
    }
    const int64_t lim = int64_t(1) << 31;
    if (V >= lim - 1 || T >= lim || H >= lim || n >= lim) return RK_ERR_UNSUPPORTED;
    if ((dout && !elem_aligned(dout, dout_type)) || !aligned(dE, 4)) return RK_ERR_INVALID_ARG;
    if (n > 0 && (!workspace || workspace_bytes < rk::embedding_bwd_workspace_bytes(n, H)))
        return RK_ERR_WORKSPACE;
    if (n > 0 && !aligned(workspace, 16)) return RK_ERR_INVALID_ARG;
    if (T > 0 && n > 0 &&
        ranges_meet(dout, (__int128)T * H * elem_size(dout_type), dE, (__int128)V * H * 4))
        return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_embedding_bwd(dout, dout_type, ids, cu_seqlens, num_seqs, T, H, V, scale,
                                 row_order, T > 0 ? n : 0, dE, accumulate != 0, workspace, di,
                                 static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

// Bytes from a [T, H] matrix's first element to its last.
static __int128 span(const rk::RulesMatrix &m, int64_t T, int64_t H) {
    return ((__int128)(T - 1) * m.ld + H) * elem_size(m.type);
}

static bool good_matrix(const rk::RulesMatrix &m, int64_t H) {
    return m.p && m.ld >= H && elem_aligned(m.p, m.type);
}

// The lists that say which rows are active, and in which order: aligned, and apart from a result, which
// some blocks write while others still read them.
struct RowLists {
    const int64_t *targets;
    int64_t T;
    const int32_t *cu;
    int64_t num_seqs;
    const int64_t *order;
    int64_t n;
    bool good() const { return aligned(targets, 8) && aligned(cu, 4) && aligned(order, 8); }
    bool apart(const void *p, __int128 bytes) const {
        return !(targets && ranges_meet(p, bytes, targets, T * 8)) &&
               !(cu && ranges_meet(p, bytes, cu, (num_seqs + 1) * 4)) &&
               !(order && n > 0 && ranges_meet(p, bytes, order, n * 8));
    }
};

rk_status rk_rms_norm(const void *x, rk_dtype x_type, int64_t ld_x, const void *residual,
                      rk_dtype residual_type, int64_t ld_residual, const void *weight,
                      rk_dtype weight_type, float eps, const int64_t *targets,
                      const int32_t *cu_seqlens, int32_t num_seqs, int64_t T, int64_t H,
                      void *residual_out, int64_t ld_residual_out, void *out, rk_dtype out_type,
                      int64_t ld_out, float *scales, int64_t group, void *stream) {
    const bool e4m3 = out_type == RK_E4M3;
    if (T < 0 || H <= 0 || !good_type(x_type) || !good_type(weight_type) ||
        (!good_type(out_type) && !e4m3) || (residual && !good_type(residual_type)))
        return RK_ERR_INVALID_ARG;
    if (!(eps > 0.f && eps < INFINITY) || (cu_seqlens && num_seqs < 0)) return RK_ERR_INVALID_ARG;
    if (e4m3 ? group != 0 && group != 128 : group != 0 || scales) return RK_ERR_INVALID_ARG;
    if (T == 0) return RK_OK;
    const rk::RulesMatrix mx{x, x_type, ld_x}, mr{residual, residual_type, ld_residual},
        mro{residual_out, residual_type, ld_residual_out}, mo{out, out_type, ld_out};
    if (!good_matrix(mx, H) || !good_matrix(mo, H) || !weight || !elem_aligned(weight, weight_type))
        return RK_ERR_INVALID_ARG;
    if (residual ? !good_matrix(mr, H) || !good_matrix(mro, H) : residual_out != nullptr)
        return RK_ERR_INVALID_ARG;
    if (e4m3 && (!scales || !aligned(scales, 4))) return RK_ERR_INVALID_ARG;
    if (T >= (int64_t(1) << 31) || H > rk::kNormMaxColumns) return RK_ERR_UNSUPPORTED;
    const RowLists lists{targets, T, cu_seqlens, num_seqs, nullptr, 0};
    if (!lists.good() || !lists.apart(out, span(mo, T, H)) || (residual && !lists.apart(residual_out, span(mro, T, H))))
        return RK_ERR_INVALID_ARG;
    // results in place of x or residual, or apart from everything
    const int64_t weight_bytes = H * elem_size(weight_type);
    if (!can_hold(mx, mo, T, H) || ranges_meet(weight, weight_bytes, out, span(mo, T, H)))
        return RK_ERR_INVALID_ARG;
    if (residual && (!can_hold(mr, mo, T, H) || !can_hold(mx, mro, T, H) || !can_hold(mr, mro, T, H) ||
                     !rows_apart(mo, mro, T, H) ||
                     ranges_meet(weight, weight_bytes, residual_out, span(mro, T, H))))
        return RK_ERR_INVALID_ARG;
    if (e4m3) {
        const __int128 bytes = (__int128)T * (group ? (H + group - 1) / group : 1) * 4;
        if (!lists.apart(scales, bytes) || ranges_meet(scales, bytes, x, span(mx, T, H)) ||
            ranges_meet(scales, bytes, out, span(mo, T, H)) || ranges_meet(scales, bytes, weight, weight_bytes))
            return RK_ERR_INVALID_ARG;
        if (residual && (ranges_meet(scales, bytes, residual, span(mr, T, H)) ||
                         ranges_meet(scales, bytes, residual_out, span(mro, T, H))))
            return RK_ERR_INVALID_ARG;
    }
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_rms_norm(mx, residual ? &mr : nullptr, weight, weight_type, eps, targets, cu_seqlens,
                            num_seqs, T, H, residual ? &mro : nullptr, mo, scales, (int)group, di,
                            static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

size_t rk_rms_norm_bwd_workspace_size(int64_t T, int64_t n, int64_t H) {
    if (T <= 0 || n < 0 || H <= 0 || H > rk::kNormMaxColumns) return 0;
    return rk::rms_norm_bwd_workspace_bytes(T, n, H);
}

rk_status rk_rms_norm_bwd(const void *dout, rk_dtype dout_type, int64_t ld_dout, const void *r,
                          rk_dtype r_type, int64_t ld_r, const void *weight, rk_dtype weight_type,
                          float eps, const void *dr, rk_dtype dr_type, int64_t ld_dr,
                          const int64_t *targets, const int32_t *cu_seqlens, int32_t num_seqs, int64_t T,
                          int64_t H, const int64_t *row_order, int64_t n_order, void *dx,
                          rk_dtype dx_type, int64_t ld_dx, float *dweight, int32_t accumulate,
                          void *workspace, size_t workspace_bytes, void *stream) {
    if (T < 0 || H <= 0 || !good_type(dout_type) || !good_type(r_type) || !good_type(weight_type) ||
        !good_type(dx_type) || (dr && !good_type(dr_type)))
        return RK_ERR_INVALID_ARG;
    if (!(eps > 0.f && eps < INFINITY) || (cu_seqlens && num_seqs < 0)) return RK_ERR_INVALID_ARG;
    if ((accumulate != 0 && accumulate != 1) || !aligned(dweight, 4)) return RK_ERR_INVALID_ARG;
    const int64_t n = row_order ? n_order : T;
    if (n < 0) return RK_ERR_INVALID_ARG;
    if (T >= (int64_t(1) << 31) || n >= (int64_t(1) << 31) || H > rk::kNormMaxColumns)
        return RK_ERR_UNSUPPORTED;
    const rk::RulesMatrix md{dout, dout_type, ld_dout}, mr{r, r_type, ld_r}, mg{dr, dr_type, ld_dr},
        mx{dx, dx_type, ld_dx};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T > 0) {
        if (!good_matrix(md, H) || !good_matrix(mr, H) || !good_matrix(mx, H) || (dr && !good_matrix(mg, H)) ||
            !weight || !elem_aligned(weight, weight_type))
            return RK_ERR_INVALID_ARG;
        const RowLists lists{targets, T, cu_seqlens, num_seqs, row_order, n};
        if (!lists.good() || !lists.apart(dx, span(mx, T, H)) || (dweight && !lists.apart(dweight, H * 4)))
            return RK_ERR_INVALID_ARG;
        // A row that row_order names twice is read twice: dx is apart from what it is made of.
        const auto fits = row_order ? rows_apart : can_hold;
        if (!fits(md, mx, T, H) || !fits(mr, mx, T, H) || (dr && !fits(mg, mx, T, H)))
            return RK_ERR_INVALID_ARG;
        const int64_t weight_bytes = H * elem_size(weight_type);
        if (ranges_meet(weight, weight_bytes, dx, span(mx, T, H))) return RK_ERR_INVALID_ARG;
        if (dweight && (ranges_meet(dweight, H * 4, weight, weight_bytes) ||
                        ranges_meet(dweight, H * 4, dx, span(mx, T, H)) ||
                        ranges_meet(dweight, H * 4, dout, span(md, T, H)) ||
                        ranges_meet(dweight, H * 4, r, span(mr, T, H)) ||
                        (dr && ranges_meet(dweight, H * 4, dr, span(mg, T, H)))))
            return RK_ERR_INVALID_ARG;
        if (!workspace || workspace_bytes < rk::rms_norm_bwd_workspace_bytes(T, n, H)) return RK_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return RK_ERR_INVALID_ARG;
    }
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    if (T == 0)
        e = dweight && !accumulate ? cudaMemsetAsync(dweight, 0, (size_t)H * 4, st) : cudaSuccess;
    else
        e = rk::launch_rms_norm_bwd(md, mr, weight, weight_type, eps, dr ? &mg : nullptr, targets, cu_seqlens,
                                    num_seqs, T, H, row_order, n, mx, dweight, accumulate != 0, workspace, di, st);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

size_t rk_preference_loss_workspace_size(int64_t num_seqs, int64_t P) {
    if (num_seqs < 0 || P < 0) return 0;
    return rk::preference_workspace_bytes(num_seqs, P);
}

rk_status rk_preference_loss(const float *logp, const float *logp_ref, const int64_t *targets,
                             const int32_t *cu_seqlens, int32_t num_seqs, int64_t T,
                             const int32_t *chosen, const int32_t *rejected, int64_t P,
                             const float *margin, rk_preference kind, float beta,
                             float label_smoothing, int32_t average, float scale, float *loss,
                             float *grad_logp, float *logratio, void *workspace,
                             size_t workspace_bytes, void *stream) {
    if (T < 0 || P < 0 || num_seqs < 0 || !cu_seqlens) return RK_ERR_INVALID_ARG;
    if (kind != RK_PREFERENCE_SIGMOID && kind != RK_PREFERENCE_HINGE && kind != RK_PREFERENCE_IPO)
        return RK_ERR_INVALID_ARG;
    if (!(beta > 0.f && beta < INFINITY) || !(label_smoothing >= 0.f && label_smoothing <= 1.f) ||
        (label_smoothing != 0.f && kind != RK_PREFERENCE_SIGMOID) || (average != 0 && average != 1))
        return RK_ERR_INVALID_ARG;
    if (T == 0 && P == 0 && num_seqs == 0) return RK_OK;
    if (T > 0 && (!logp || !targets || !grad_logp)) return RK_ERR_INVALID_ARG;
    if (P > 0 && (!chosen || !rejected || !loss)) return RK_ERR_INVALID_ARG;
    const int64_t lim = int64_t(1) << 31;
    if (T >= lim || P >= lim) return RK_ERR_UNSUPPORTED;
    if (!aligned(logp, 4) || !aligned(logp_ref, 4) || !aligned(targets, 8) || !aligned(cu_seqlens, 4) ||
        !aligned(chosen, 4) || !aligned(rejected, 4) || !aligned(margin, 4) || !aligned(loss, 4) ||
        !aligned(grad_logp, 4) || !aligned(logratio, 4))
        return RK_ERR_INVALID_ARG;
    // results apart from what is read, and from one another
    const struct { const void *p; int64_t bytes; } in[] = {
        {logp, T * 4}, {logp_ref, T * 4}, {targets, T * 8}, {cu_seqlens, ((int64_t)num_seqs + 1) * 4},
        {chosen, P * 4}, {rejected, P * 4}, {margin, P * 4},
    }, out[] = {{loss, P * 4}, {grad_logp, T * 4}, {logratio, (int64_t)num_seqs * 4}};
    for (int i = 0; i < 3; ++i) {
        if (!out[i].p || !out[i].bytes) continue;
        for (const auto &b : in)
            if (b.p && b.bytes && ranges_meet(out[i].p, out[i].bytes, b.p, b.bytes)) return RK_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (out[j].p && out[j].bytes && ranges_meet(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
                return RK_ERR_INVALID_ARG;
    }
    if (!workspace || workspace_bytes < rk::preference_workspace_bytes(num_seqs, P)) return RK_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_preference(logp, logp_ref, targets, cu_seqlens, num_seqs, T, chosen, rejected, P, margin,
                              (int)kind, beta, label_smoothing, average != 0, scale, loss, grad_logp, logratio,
                              workspace, di, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

rk_status rk_adamw_step(const rk_adamw_tensor *tensors, int64_t count, const rk_adamw_options *options,
                        void *stream) {
    if (count < 0 || !options || (count > 0 && !tensors)) return RK_ERR_INVALID_ARG;
    const rk_adamw_options &o = *options;
    if (!std::isfinite(o.lr) || !(o.beta1 >= 0.0 && o.beta1 < 1.0) || !(o.beta2 >= 0.0 && o.beta2 < 1.0) ||
        !((float)o.eps > 0.f && (float)o.eps < 0x1p100f) || (!o.step_device && o.step < 1) ||
        !aligned(o.lr_device, 4) || !aligned(o.step_device, 8) || !aligned(o.grad_scale, 4))
        return RK_ERR_INVALID_ARG;
    for (int64_t i = 0; i < count; ++i) {
        const rk_adamw_tensor &t = tensors[i];
        if (t.n < 0 || !good_type(t.param_type) || !good_type(t.grad_type) || !std::isfinite(t.lr_scale) ||
            !std::isfinite(t.weight_decay))
            return RK_ERR_INVALID_ARG;
        if ((t.m_scale == nullptr) != (t.v_scale == nullptr) || (t.master && t.param_type == RK_FP32))
            return RK_ERR_INVALID_ARG;
        if (t.n >= (int64_t(1) << 40)) return RK_ERR_UNSUPPORTED;
        if (t.n == 0) continue;
        if (!t.param || !t.grad || !t.m || !t.v) return RK_ERR_INVALID_ARG;
        const int state = t.m_scale ? 1 : 4;
        if (!elem_aligned(t.param, t.param_type) || !elem_aligned(t.grad, t.grad_type) || !aligned(t.master, 4) ||
            !aligned(t.m, state) || !aligned(t.v, state) || !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))
            return RK_ERR_INVALID_ARG;
    }
    if (count == 0) return RK_OK;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = rk::launch_adamw(tensors, count, o, di, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

rk_status rk_selftest_wait_timeout(int64_t limit_ns, void *stream) {
    if (limit_ns <= 0 || limit_ns > 10000000000ll) return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    selftest_wait_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>((uint64_t)limit_ns, di.err);
    e = cudaGetLastError();
    if (e != cudaSuccess) return rk::cuda_fail(e);
    return RK_OK;
}

rk_status rk_get_device_error(void *stream, int32_t *err) {
    if (!err) return RK_ERR_INVALID_ARG;
    DeviceInfo di;
    cudaError_t e = rk::current_device_info(&di);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned v = 0;
    e = cudaMemcpyAsync(&v, di.err, sizeof(v), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    e = cudaMemsetAsync(di.err, 0, sizeof(unsigned), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return rk::cuda_fail(e);
    *err = (int32_t)v;
    return RK_OK;
}

}  // extern "C"
