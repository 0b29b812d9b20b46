// What the translation units of liblce.so share on the host: the device
// record, the status word's address, the launch counter and the last CUDA
// error. Defined in lce_api.cu.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>

#include "lce.h"

namespace lce {

struct HostDev {
    int index = 0;           // device number, below 64
    int sms = 0;
    int *status = nullptr;   // device status word (LCE_DEV_* bits)
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
};

// The current device, checked to be sm_103.
lce_status_t host_device(HostDev *out);

// Records a CUDA error for lce_last_cuda_error(), and clears it in the runtime; LCE_OK on cudaSuccess.
lce_status_t host_cuda(cudaError_t e);

// Counts a launch for lce_launch_count() and returns its error, if any.
lce_status_t host_launched();

// Device scratch of a call: the caller's workspace, or a stream-ordered
// allocation that is freed on the stream when the call returns.
class HostScratch {
  public:
    explicit HostScratch(cudaStream_t s) : s_(s) {}
    HostScratch(const HostScratch &) = delete;
    HostScratch &operator=(const HostScratch &) = delete;
    ~HostScratch() {
        if (owned_) cudaFreeAsync(p_, s_);
    }
    lce_status_t get(void *workspace, size_t have, size_t need, uint8_t **out) {
        if (need == 0) {
            *out = nullptr;
            return LCE_OK;
        }
        if (workspace) {
            if (have < need) return LCE_ERR_WORKSPACE;
            if (reinterpret_cast<uintptr_t>(workspace) & 15u) return LCE_ERR_ALIGN;
            p_ = workspace;
        } else {
            const lce_status_t s = host_cuda(cudaMallocAsync(&p_, need, s_));
            if (s != LCE_OK) return s;
            owned_ = true;
        }
        *out = static_cast<uint8_t *>(p_);
        return LCE_OK;
    }

  private:
    cudaStream_t s_;
    void *p_ = nullptr;
    bool owned_ = false;
};

// Raises a kernel's dynamic shared-memory limit, once per kernel and device.
template <auto kKernel>
lce_status_t host_smem(const HostDev &dev, int bytes) {
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = uint64_t(1) << dev.index;
    if (done.load(std::memory_order_relaxed) & bit) return LCE_OK;
    const lce_status_t s = host_cuda(cudaFuncSetAttribute(reinterpret_cast<const void *>(kKernel),
                                                          cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    if (s == LCE_OK) done.fetch_or(bit, std::memory_order_relaxed);
    return s;
}

// A launch that may begin before the one ahead of it in the stream has ended
// (once all its blocks have allowed it, or ended), and waits in the kernel
// where it reads what that one wrote.
template <typename... P, typename... A>
lce_status_t host_launch_early(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t st, const A &...args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const lce_status_t s = host_cuda(cudaLaunchKernelEx(&cfg, kernel, P(args)...));
    return s != LCE_OK ? s : host_launched();
}

inline bool host_misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// The layout of N rows of d channels in 8 bits, where there are rows.
inline lce_status_t host_check_packed(const void *codes, int64_t ld_codes, const void *exps, int64_t ld_exps, int64_t N, int64_t d) {
    if (!codes || !exps) return LCE_ERR_NULL;
    if (ld_codes < d || ld_exps < N || ld_codes >= (int64_t(1) << 36) || ld_exps >= (int64_t(1) << 36)) return LCE_ERR_SHAPE;
    return host_misaligned(codes) || host_misaligned(exps) || ld_codes % 16 || ld_exps % 16 ? LCE_ERR_ALIGN : LCE_OK;
}

}  // namespace lce
