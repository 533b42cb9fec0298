// Host-side helpers that the library's translation units share: the device query, launch
// attributes and overlap mode, and the row kernels' launch shapes.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <map>
#include <mutex>
#include <set>
#include <tuple>
#include <utility>

#include "w8a8.h"

namespace w8a8 {

constexpr unsigned long long kWaitLimitNs = 2000000000ull; // 2 s per bounded wait
constexpr int kMaxDevices = 64;

struct DeviceInfo {
    int ok = -1; // -1 unknown, 0 unsupported, 1 sm_100
    int num_sms = 0;
};

inline std::mutex g_mu;
inline DeviceInfo g_dev[kMaxDevices];
inline std::set<std::pair<const void *, int>> g_smem_set;
inline PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

inline bool aligned16(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// Current device if it is an sm_100 part; fills its SM count.
inline int current_device(int *dev, int *num_sms)
{
    int d = -1;
    if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= kMaxDevices) {
        cudaGetLastError();
        return W8A8_ERR_NO_DEVICE;
    }
    std::lock_guard<std::mutex> lk(g_mu);
    DeviceInfo &info = g_dev[d];
    if (info.ok < 0) {
        int major = 0, sms = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, d) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, d) != cudaSuccess) {
            cudaGetLastError();
            return W8A8_ERR_NO_DEVICE;
        }
        info.ok = (major == 10) ? 1 : 0;
        info.num_sms = sms;
    }
    if (info.ok != 1)
        return W8A8_ERR_NO_DEVICE;
    if (!g_encode) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess || fn == nullptr) {
            cudaGetLastError();
            return W8A8_ERR_CUDA;
        }
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    *dev = d;
    *num_sms = info.num_sms;
    return W8A8_OK;
}

// cuTensorMapEncodeTiled (of the device that current_device() found). It wants a context bound to
// the calling thread, which a host thread without a call of the runtime so far does not have: the
// threads of PyTorch's backward pass, for one.
template <typename... Args> CUresult encode_tiled(Args... args)
{
    CUresult r = g_encode(args...);
    int dev = -1;
    if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&dev) == cudaSuccess &&
        cudaSetDevice(dev) == cudaSuccess)
        r = g_encode(args...);
    return r;
}

// Once per kernel and device: raise the dynamic shared-memory limit, and ask for the
// largest shared-memory carveout for every kernel of the library, so consecutive launches
// of row kernels and GEMMs never reconfigure the L1/shared split between them.
inline int ensure_smem(const void *kernel, int dev, int bytes)
{
    std::lock_guard<std::mutex> lk(g_mu);
    auto key = std::make_pair(kernel, dev);
    if (g_smem_set.count(key))
        return W8A8_OK;
    if ((bytes > 0 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           bytes) != cudaSuccess) ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared) != cudaSuccess) {
        cudaGetLastError();
        return W8A8_ERR_CUDA;
    }
    g_smem_set.insert(key);
    return W8A8_OK;
}

// Overlap mode (w8a8_set_overlap): 0 plain stream order, 1 programmatic dependent launch,
// 2 dependent launch + weight prefetch before the dependency wait.
inline std::atomic<int> g_overlap{1};

// Launches `kernel`, with programmatic stream serialization when the overlap mode asks for
// it (the kernels call griddepcontrol.wait before touching dependent data either way).
template <typename... KArgs, typename... Args>
int launch_kernel_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                          cudaStream_t st, unsigned cluster_x, Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (g_overlap.load(std::memory_order_relaxed) >= 1) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    if (cluster_x > 0) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster_x;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    if (cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return W8A8_ERR_CUDA;
    }
    return W8A8_OK;
}

template <typename... KArgs, typename... Args>
int launch_kernel(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                  Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    if (g_overlap.load(std::memory_order_relaxed) >= 1) {
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    if (cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return W8A8_ERR_CUDA;
    }
    return W8A8_OK;
}

// The status word of the gradient kernels' translation unit (grad.cu): its asynchronous read on
// a stream, and its reset.
cudaError_t grad_status_read(unsigned int *word, cudaStream_t st);
cudaError_t grad_status_clear();

// ------------------------------------------------------------------ row kernels

struct RowLaunch {
    int nch;
    int threads;
};

// One CTA per row; each thread holds nch vectors of 8 values (nch <= 4, <= 1024 threads).
inline RowLaunch row_launch(int64_t K)
{
    const int64_t nvec = K / 8;
    int nch = static_cast<int>((nvec + 255) / 256);
    nch = nch < 1 ? 1 : (nch > 4 ? 4 : nch);
    if (nch == 3)
        nch = 4;
    int64_t t = (nvec + nch - 1) / nch;
    t = ((t + 31) / 32) * 32;
    return RowLaunch{nch, static_cast<int>(t)};
}

inline int check_row_shape(int64_t M, int64_t K)
{
    if (M < 1 || K < 16)
        return W8A8_ERR_INVALID_ARG;
    if (K % 16 != 0 || K > 32768 || M > 0x7fffffffLL)
        return W8A8_ERR_UNSUPPORTED_SHAPE;
    return W8A8_OK;
}

// Persistent row grid: at most as many CTAs as are resident on the device at once (cached
// per kernel, block size and device), never more than there are rows.
inline unsigned row_grid(const void *kernel, int threads, int64_t M, int dev, int sms)
{
    static std::mutex mu;
    static std::map<std::tuple<const void *, int, int>, int> cache;
    int occ = 0;
    {
        std::lock_guard<std::mutex> lk(mu);
        auto key = std::make_tuple(kernel, threads, dev);
        auto it = cache.find(key);
        if (it != cache.end()) {
            occ = it->second;
        } else {
            if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kernel, threads, 0) !=
                cudaSuccess) {
                cudaGetLastError();
                occ = 1;
            }
            occ = occ < 1 ? 1 : occ;
            cache[key] = occ;
        }
    }
    const int64_t g = static_cast<int64_t>(sms) * occ;
    return static_cast<unsigned>(M < g ? M : g);
}

} // namespace w8a8
