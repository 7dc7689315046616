// Host helpers shared by the C ABI's translation units.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>

namespace kvtc {

// cuTensorMapEncodeTiled through the runtime, or null.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                         cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// Makes a device current for a scope.
struct DeviceGuard {
  int prev = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev != dev) ok = cudaSetDevice(dev) == cudaSuccess;
    if (!ok) cudaGetLastError();  // reported here, not by the next launch
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev)
      cudaSetDevice(prev);
  }
};

inline bool aligned16(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// Let a kernel use `bytes` of shared memory, and `wide` clusters of up to 16
// blocks; set once per device (`ready` holds the devices done, as bits; above
// 64 it is set on every call).
template <class F>
inline cudaError_t allow_smem(F* kernel, int bytes, int device,
                              std::atomic<uint64_t>& ready,
                              bool wide = false) {
  const uint64_t bit = device < 64 ? 1ull << device : 0;
  if (ready.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(
      kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && wide)
    e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launch a kernel; its own status, whatever error an earlier call left
// behind.  `overlap`: it may start while the launch before it on the stream
// still runs, and waits for that launch's end itself (griddepcontrol.wait).
// `cluster`: blocks per cluster, 0 for none.
template <class... A, class... B>
inline cudaError_t launch_kernel(void (*kernel)(A...), dim3 grid, dim3 block,
                                 size_t smem, cudaStream_t st, bool overlap,
                                 int cluster, const B&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute a[2];
  c.attrs = a;
  if (overlap) {
    a[c.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[c.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster) {
    a[c.numAttrs].id = cudaLaunchAttributeClusterDimension;
    a[c.numAttrs].val.clusterDim.x = (unsigned)cluster;
    a[c.numAttrs].val.clusterDim.y = 1;
    a[c.numAttrs++].val.clusterDim.z = 1;
  }
  return cudaLaunchKernelEx(&c, kernel, static_cast<A>(args)...);
}

}  // namespace kvtc
