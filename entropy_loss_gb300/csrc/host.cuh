// host.cuh - host-side pieces that the library's translation units share: error
// text, device facts, tensor maps, pointer checks and the launch of CTA pairs.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>
#include <utility>

#include "flp.h"
#include "pair.cuh"

namespace flp {

inline thread_local std::string g_msg;

inline flp_status fail(flp_status st, const char* what) {
    g_msg = what;
    return st;
}

inline flp_status cuda_fail(cudaError_t e, const char* where) {
    char buf[256];
    snprintf(buf, sizeof buf, "%s: %s", where, cudaGetErrorString(e));
    g_msg = buf;
    return FLP_ERR_CUDA;
}

#define FLP_CUDA(call)                                         \
    do {                                                       \
        cudaError_t e_ = (call);                               \
        if (e_ != cudaSuccess) return cuda_fail(e_, #call);    \
    } while (0)

constexpr int kMaxDevices = 64;
constexpr size_t kHeaderBytes = 1024;      // error word, ticket counter; keeps regions 1 KiB aligned
constexpr size_t kTicketOffset = 8;        // 64-bit tile ticket counter of the backward contractions
constexpr int64_t kDefaultChunkRows = 8192;
constexpr unsigned long long kWaitLimitNs = 10ull * 1000 * 1000 * 1000;  // 10 s per wait

struct DevInfo {
    bool init = false;
    cudaError_t err = cudaSuccess;
    int sm_count = 0;
    int major = 0, minor = 0;
    bool attrs_set = false;
    int pairs = 0;  // CTA pairs that can be resident at once (persistent grid size / 2)
};
inline DevInfo g_dev[kMaxDevices];
inline std::mutex g_mu;

inline flp_status device_info(DevInfo** out, int* dev_out) {
    int dev = 0;
    FLP_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= kMaxDevices) return fail(FLP_ERR_UNSUPPORTED, "device index out of range");
    std::lock_guard<std::mutex> lk(g_mu);
    DevInfo& d = g_dev[dev];
    if (!d.init) {
        cudaError_t e = cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d.major, cudaDevAttrComputeCapabilityMajor, dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d.minor, cudaDevAttrComputeCapabilityMinor, dev);
        if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
        d.init = true;
    }
    *out = &d;
    if (dev_out) *dev_out = dev;
    return FLP_OK;
}

inline PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

inline flp_status get_encode(PFN_cuTensorMapEncodeTiled_v12000* fn) {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_encode) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                         cudaEnableDefault, &q);
        if (e != cudaSuccess) return cuda_fail(e, "cudaGetDriverEntryPointByVersion");
        if (q != cudaDriverEntryPointSuccess || !p)
            return fail(FLP_ERR_CUDA, "cuTensorMapEncodeTiled not available from the driver");
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
    *fn = g_encode;
    return FLP_OK;
}

// 2-D tiled tensor map, 128-byte swizzle, zero fill outside the tensor.
inline flp_status tmap_2d(CUtensorMap* tm, CUtensorMapDataType dt, const void* base, uint64_t inner,
                   uint64_t outer, uint64_t row_pitch_bytes, uint32_t box_inner,
                   uint32_t box_outer, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    flp_status st = get_encode(&enc);
    if (st != FLP_OK) return st;
    cuuint64_t dims[2] = {inner, outer};
    cuuint64_t strides[1] = {row_pitch_bytes};
    cuuint32_t box[2] = {box_inner, box_outer};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(tm, dt, 2, const_cast<void*>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        char buf[160];
        snprintf(buf, sizeof buf, "cuTensorMapEncodeTiled failed (%d) dims %llu x %llu pitch %llu",
                 static_cast<int>(r), (unsigned long long)inner, (unsigned long long)outer,
                 (unsigned long long)row_pitch_bytes);
        g_msg = buf;
        return FLP_ERR_CUDA;
    }
    return FLP_OK;
}

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Shared-memory limits of the head's kernels and the number of CTA pairs that can
// be resident, once per device (flp.cu).
flp_status ensure_attrs(DevInfo* d);

inline flp_status check_device(DevInfo** d) {
    flp_status st = device_info(d, nullptr);
    if (st != FLP_OK) return st;
    if ((*d)->major != 10 || (*d)->minor != 3)
        return fail(FLP_ERR_UNSUPPORTED, "kernels are built for sm_103a (GB300) only");
    return ensure_attrs(*d);
}

// A device pointer must live on the device the call launches on (the one
// current on the calling thread); host or managed-elsewhere memory is refused.
inline flp_status check_on_current_device(const void* p, const char* what) {
    if (!p) return FLP_OK;
    int dev = 0;
    FLP_CUDA(cudaGetDevice(&dev));
    cudaPointerAttributes a{};
    cudaError_t e = cudaPointerGetAttributes(&a, p);
    if (e != cudaSuccess) return cuda_fail(e, "cudaPointerGetAttributes");
    if (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged) {
        char buf[160];
        snprintf(buf, sizeof buf, "%s is not device memory", what);
        return fail(FLP_ERR_INVALID_ARG, buf);
    }
    if (a.type == cudaMemoryTypeDevice && a.device != dev) {
        char buf[160];
        snprintf(buf, sizeof buf, "%s lives on device %d but the current device is %d", what, a.device, dev);
        return fail(FLP_ERR_INVALID_ARG, buf);
    }
    return FLP_OK;
}

// Launches `kernel` on `grid` CTAs grouped in clusters of two (the CTA pairs
// that share each tcgen05.mma.cta_group::2 tile).  With `after_kernel` the
// launch follows another of this library's kernels on the stream and uses
// programmatic dependent launch: its CTAs may be scheduled on the SMs the
// previous grid frees while that grid's last tiles finish, run their set-up,
// and wait in griddepcontrol.wait for its results.
template <typename... KArgs, typename... Args>
flp_status launch_pairs_n(void (*kernel)(KArgs...), int grid, int threads, cudaStream_t s, const char* what,
                          bool after_kernel, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = SMEM_ALLOC;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = after_kernel ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, what);
    return FLP_OK;
}

}  // namespace flp
