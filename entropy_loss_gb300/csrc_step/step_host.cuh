// step_host.cuh - host-side pieces that the training-step operators share: launches,
// checks of sizes, pointers and types, and the blocks a kernel keeps resident.
#pragma once
#include "../csrc/host.cuh"
#include "vec.cuh"

namespace flp {  // step.cu

// M rows of H bf16 elements (pitch ld, any alignment) copied to rows of Hp elements, a
// multiple of 8, 16-byte aligned, zeros behind each row.
flp_status align_rows(const void* src, int64_t ld, int64_t M, int64_t H, void* dst, int64_t Hp, cudaStream_t s);

// dW [N, K] (+)= dY^T X for bf16 rows aligned to 16 bytes; the workspace's first word is the
// error word, which the caller has cleared.
flp_status weight_grad_checks(int64_t M, int64_t N, int64_t K, int dw_dtype);
size_t weight_grad_bytes(int64_t M, int64_t N, int64_t K, int dw_dtype, int pairs);
flp_status weight_grad(const void* dY, int64_t ldy, const void* X, int64_t ldx, int64_t M, int64_t N, int64_t K, void* dW,
                       int dw_dtype, int accumulate, uint8_t* ws, int pairs, bool after_kernel, cudaStream_t s);

}  // namespace flp

namespace {

using namespace flp;

constexpr int64_t kMaxRows = INT32_MAX;

// One launch; with `after_kernel` it follows another kernel of the same call
// and may be scheduled while that one finishes (it waits in griddep_wait).
template <typename... KArgs, typename... Args>
flp_status launch_step(void (*kernel)(KArgs...), int64_t grid, int threads, size_t smem, cudaStream_t s,
                       const char* what, bool after_kernel, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = after_kernel ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
    return e == cudaSuccess ? FLP_OK : cuda_fail(e, what);
}

// One launch of one cluster of `blocks` blocks.
template <typename P>
flp_status launch_cluster(void (*kernel)(P), int blocks, int threads, size_t smem, cudaStream_t s, const char* what,
                          const P& p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(blocks);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    return e == cudaSuccess ? FLP_OK : cuda_fail(e, what);
}

// The device is an sm_103 one (no attributes are needed by these kernels).
flp_status step_device(DevInfo** d) {
    const flp_status st = device_info(d, nullptr);
    if (st != FLP_OK) return st;
    if ((*d)->major != 10 || (*d)->minor != 3)
        return fail(FLP_ERR_UNSUPPORTED, "kernels are built for sm_103a (GB300) only");
    return FLP_OK;
}

inline bool is_dtype(int t) { return t == FLP_F32 || t == FLP_BF16; }
inline int64_t elem(int t) { return t == FLP_F32 ? 4 : 2; }
inline bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Whether rows at this base and pitch (in elements) are 16-byte aligned.
inline bool rows16(const void* p, int64_t ld, int dtype) { return aligned16(p) && (ld * elem(dtype)) % 16 == 0; }

// Resident blocks per SM of a kernel with `smem` bytes of dynamic shared memory,
// asked once per kernel, block size and device; the kernel's limit is set to what
// its largest block needs, whichever size comes first.
template <auto* kernel>
flp_status resident_blocks(int threads, size_t smem, size_t largest, int* per_sm) {
    static int8_t known[kMaxDevices][1024 / 32 + 1] = {};
    int dev = 0;
    FLP_CUDA(cudaGetDevice(&dev));  // in range: step_device has run
    std::lock_guard<std::mutex> lk(g_mu);
    int8_t& at = known[dev][threads / 32];
    if (at == 0) {
        FLP_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(largest)));
        int n = 0;
        FLP_CUDA(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem));
        if (n < 1) return fail(FLP_ERR_UNSUPPORTED, "a block of the kernel does not fit an SM");
        at = static_cast<int8_t>(n);
    }
    *per_sm = at;
    return FLP_OK;
}

flp_status row_checks(const void* p, int64_t ld, int64_t H, int dtype, const char* what) {
    if (!p) return fail(FLP_ERR_INVALID_ARG, what);
    if (ld < H || !aligned_to(p, elem(dtype)))
        return fail(FLP_ERR_INVALID_ARG, "row pitch below the width, or a pointer not aligned to its elements");
    return FLP_OK;
}

}  // namespace
