// Attention of chunks of new tokens over paged K and V pools.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/kvtc.h"
#include "kvtc_hostutil.cuh"
#include "kvtc_internal.cuh"

namespace kvtc {
namespace {

constexpr int kBlock = 16;           // tokens per pool block
constexpr int kMaxReq = 4096;        // requests per call
constexpr int kMaxGroup = 128;       // query heads per KV head
constexpr int kMaxTable = INT32_MAX / kBlock - 1;
constexpr float kMaxScale = 0x1p127f;

struct ChunkParams {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* table;
  const int64_t* cu;
  const int32_t* lens;
  void* out;
  float* lse;
  unsigned* flags;
  int64_t N, q_ld, out_ld, num_blocks;
  float scale;
  int32_t R, heads, kv_heads, max_blocks, sink, window;
};

__device__ __forceinline__ float to_float(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <class T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float x) {
  return __float2bfloat16(x);
}
template <>
__device__ __forceinline__ __half from_float(float x) {
  return __float2half(x);
}

// A block per row, a warp per query head: one token after the other.
template <class T, int HD>
__global__ void __launch_bounds__(256)
    chunk_simple_kernel(const __grid_constant__ ChunkParams p) {
  constexpr int kEach = HD / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  int lo = 0, hi = p.R;               // cu[lo] <= row < cu[hi]
  if (row < p.cu[0] || row >= p.cu[p.R]) {
    if (row == 0 && threadIdx.x == 0 && p.cu[p.R] > p.N && p.flags)
      atomicOr(p.flags, KVTC_FLAG_SPACE);
    return;
  }
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cu[mid] <= row) lo = mid; else hi = mid;
  }
  const int r = lo;
  const int64_t c0 = min(max(p.cu[r], (int64_t)0), p.N);
  const int64_t c1 = min(max(p.cu[r + 1], (int64_t)0), p.N);
  const int64_t most = (int64_t)p.max_blocks * kBlock;
  const int64_t len = min(max((int64_t)p.lens[r], (int64_t)0), most);
  if (p.flags && threadIdx.x == 0 &&
      (p.lens[r] > most || p.cu[r + 1] > p.N))
    atomicOr(p.flags, KVTC_FLAG_SPACE);
  const int64_t pos = len - (c1 - c0) + (row - c0);
  const int group = p.heads / p.kv_heads;
  for (int h = warp; h < p.heads; h += 8) {
    const T* q = static_cast<const T*>(p.q) + row * p.q_ld + h * HD;
    float qv[kEach], o[kEach], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      qv[i] = to_float(q[i * 32 + lane]) * p.scale;
      o[i] = 0.f;
    }
    for (int64_t t = 0; t <= pos; ++t) {
      if (p.window && t >= p.sink && t <= pos - p.window) continue;
      const int64_t id = p.table[(int64_t)r * p.max_blocks + t / kBlock];
      if (id < 0 || id >= p.num_blocks) {
        if (lane == 0 && p.flags) atomicOr(p.flags, KVTC_FLAG_BLOCK);
        continue;
      }
      const int64_t at =
          ((id * kBlock + t % kBlock) * p.kv_heads + h / group) * HD + lane;
      const T* k = static_cast<const T*>(p.k) + at;
      const T* v = static_cast<const T*>(p.v) + at;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        s = fmaf(qv[i], to_float(k[i * 32]), s);
#pragma unroll
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
      if (s == -INFINITY) continue;
      const float top = fmaxf(m, s);
      const float was = expf(m - top), w = expf(s - top);
      m = top;
      l = l * was + w;
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        o[i] = fmaf(w, to_float(v[i * 32]), o[i] * was);
    }
    T* out = static_cast<T*>(p.out) + row * p.out_ld + h * HD;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      out[i * 32 + lane] = from_float<T>(o[i] * inv);
    if (lane == 0 && p.lse)
      p.lse[row * p.heads + h] = l == 0.f ? -INFINITY : m + logf(l);
  }
}

inline bool misaligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

template <class T>
cudaError_t launch(const ChunkParams& p, int head_dim, cudaStream_t st) {
  const unsigned grid = (unsigned)std::max<int64_t>(p.N, 1);
  if (head_dim == 64)
    return launch_kernel(chunk_simple_kernel<T, 64>, grid, 256, 0, st, false,
                         0, p);
  if (head_dim == 128)
    return launch_kernel(chunk_simple_kernel<T, 128>, grid, 256, 0, st, false,
                         0, p);
  return launch_kernel(chunk_simple_kernel<T, 256>, grid, 256, 0, st, false,
                       0, p);
}

}  // namespace
}  // namespace kvtc

using namespace kvtc;

extern "C" {

int64_t kvtc_paged_attend_chunks_workspace_bytes(int cuda_device, int R,
                                                 int64_t N, int heads,
                                                 int kv_heads, int head_dim) {
  if (cuda_device < 0 || R < 0 || R > kMaxReq || N < 0 || N > INT32_MAX ||
      heads <= 0 || kv_heads <= 0 || heads % kv_heads || head_dim <= 0)
    return KVTC_EINVAL;
  if ((head_dim != 64 && head_dim != 128 && head_dim != 256) ||
      (int64_t)kv_heads * head_dim > kMaxD || heads / kv_heads > kMaxGroup)
    return KVTC_ENOTSUP;
  return 256;
}

int kvtc_paged_attend_chunks(
    int cuda_device, int R, int64_t N, int heads, int kv_heads, int head_dim,
    int dtype, const void* q, int64_t q_ld, const void* k_cache,
    const void* v_cache, int64_t num_blocks, int block_size,
    const int32_t* block_table, int max_blocks, const int64_t* cu,
    const int32_t* lens, int sink, int window, float scale, void* out,
    int64_t out_ld, float* lse, void* workspace, int64_t workspace_bytes,
    uint32_t* flags, void* cuda_stream) {
  const int64_t need = kvtc_paged_attend_chunks_workspace_bytes(
      cuda_device, R, N, heads, kv_heads, head_dim);
  if (need < 0) return (int)need;
  if ((dtype != KVTC_DTYPE_BF16 && dtype != KVTC_DTYPE_FP16) || !k_cache ||
      !v_cache || num_blocks <= 0 || num_blocks > INT32_MAX ||
      max_blocks <= 0 || sink < 0 || window < 0 ||
      !(std::fabs(scale) <= kMaxScale) ||      // (nor NaN)
      !workspace || (R && (!block_table || !cu || !lens)) ||
      (R && N && (!q || !out)))
    return KVTC_EINVAL;
  if (block_size != kBlock || max_blocks > kMaxTable) return KVTC_ENOTSUP;
  const int64_t width = (int64_t)heads * head_dim;
  if (q_ld < width || out_ld < width || workspace_bytes < need)
    return KVTC_ESIZE;
  if (q_ld % 8 || out_ld % 8 || !aligned16(q) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned16(out) || !aligned16(workspace) ||
      misaligned(block_table, 4) || misaligned(cu, 8) ||
      misaligned(lens, 4) || misaligned(lse, 4) || misaligned(flags, 4))
    return KVTC_EALIGN;
  if (R == 0 || N == 0) return KVTC_OK;
  DeviceGuard guard(cuda_device);
  if (!guard.ok) return KVTC_ECUDA;
  ChunkParams p;
  p.q = q;
  p.k = k_cache;
  p.v = v_cache;
  p.table = block_table;
  p.cu = cu;
  p.lens = lens;
  p.out = out;
  p.lse = lse;
  p.flags = flags;
  p.N = N;
  p.q_ld = q_ld;
  p.out_ld = out_ld;
  p.num_blocks = num_blocks;
  p.scale = scale;
  p.R = R;
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.max_blocks = max_blocks;
  p.sink = sink;
  p.window = window;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = dtype == KVTC_DTYPE_BF16
                            ? launch<__nv_bfloat16>(p, head_dim, st)
                            : launch<__half>(p, head_dim, st);
  if (e != cudaSuccess) return KVTC_ECUDA;
  count_launch();
  return KVTC_OK;
}

}  // extern "C"
