// Attention of one new token per request over paged K and V pools.
//
// For a query head, s_t = scale q.k_t over the attended tokens; with a
// running maximum m, l = sum e^(s_t - m) and o = sum e^(s_t - m) v_t are
// rescaled by e^(m_old - m_new) when m grows, so the tokens are read once;
// out = o / l, lse = m + ln l.
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

struct AttendParams {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* table;
  const int32_t* lens;
  void* out;
  float* lse;
  unsigned* flags;
  int64_t q_ld, out_ld, num_blocks;
  float scale;
  int32_t heads, kv_heads, max_blocks, sink, window;
};

template <class T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <>
__device__ __forceinline__ float to_float(__half x) {
  return __half2float(x);
}
template <class T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_float(float x) {
  return __float2half_rn(x);
}

// One block per (head, request): four warps take every fourth token, a lane
// holds HD / 32 channels, and the warps' partial results are joined.
template <class T, int HD>
__global__ void __launch_bounds__(128)
    attend_kernel(const __grid_constant__ AttendParams p) {
  constexpr int C = HD / 32;
  __shared__ float part[4][HD + 2];
  const int h = blockIdx.x, r = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t D = (int64_t)p.kv_heads * HD;
  const int64_t col = (int64_t)(h / (p.heads / p.kv_heads)) * HD + lane * C;
  const T* q = static_cast<const T*>(p.q) + r * p.q_ld + (int64_t)h * HD;
  float qf[C], o[C] = {}, m = -INFINITY, l = 0.f;
  for (int i = 0; i < C; ++i) qf[i] = to_float(q[lane * C + i]) * p.scale;
  int64_t len = max(p.lens[r], 0);
  if (len > (int64_t)p.max_blocks * kBlock) {
    len = (int64_t)p.max_blocks * kBlock;
    if (threadIdx.x == 0 && p.flags) atomicOr(p.flags, KVTC_FLAG_SPACE);
  }
  const int64_t recent = p.window ? len - p.window : 0;
  for (int64_t t = warp; t < len; t += 4) {
    if (p.window && t >= p.sink && t < recent) {
      // on to the first token of this warp inside the window
      t += (recent - t + 3) / 4 * 4 - 4;
      continue;
    }
    const int64_t id = p.table[(int64_t)r * p.max_blocks + t / kBlock];
    if (id < 0 || id >= p.num_blocks) {
      if (lane == 0 && p.flags) atomicOr(p.flags, KVTC_FLAG_BLOCK);
      continue;
    }
    const int64_t at = (id * kBlock + t % kBlock) * D + col;
    const T* k = static_cast<const T*>(p.k) + at;
    const T* v = static_cast<const T*>(p.v) + at;
    float s = 0.f;
    for (int i = 0; i < C; ++i) s += qf[i] * to_float(k[i]);
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    const float mn = fmaxf(m, s);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float a = expf(m - base), w = expf(s - base);
    m = mn;
    l = l * a + w;
    for (int i = 0; i < C; ++i) o[i] = o[i] * a + w * to_float(v[i]);
  }
  for (int i = 0; i < C; ++i) part[warp][lane * C + i] = o[i];
  if (lane == 0) {
    part[warp][HD] = m;
    part[warp][HD + 1] = l;
  }
  __syncthreads();
  float mx = -INFINITY;
  for (int w = 0; w < 4; ++w) mx = fmaxf(mx, part[w][HD]);
  const float base = mx == -INFINITY ? 0.f : mx;
  float a[4], total = 0.f;
  for (int w = 0; w < 4; ++w) {
    a[w] = expf(part[w][HD] - base);
    total += part[w][HD + 1] * a[w];
  }
  const bool none = total == 0.f;
  T* out = static_cast<T*>(p.out) + r * p.out_ld + (int64_t)h * HD;
  for (int d = threadIdx.x; d < HD; d += 128) {
    float x = 0.f;
    for (int w = 0; w < 4; ++w) x += part[w][d] * a[w];
    out[d] = from_float<T>(none ? 0.f : x / total);
  }
  if (threadIdx.x == 0 && p.lse)
    p.lse[(int64_t)r * p.heads + h] = none ? -INFINITY : base + logf(total);
}

template <class T>
cudaError_t launch(const AttendParams& p, int R, int head_dim,
                   cudaStream_t st) {
  const dim3 grid(p.heads, R);
  const auto kernel = head_dim == 64    ? attend_kernel<T, 64>
                      : head_dim == 128 ? attend_kernel<T, 128>
                                        : attend_kernel<T, 256>;
  const cudaError_t e = launch_kernel(kernel, grid, 128, 0, st, false, p);
  if (e == cudaSuccess) count_launch();
  return e;
}

inline bool misaligned4(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 3u) != 0;
}

// Shape errors shared by the call and its workspace query.
int check_shape(int cuda_device, int R, int heads, int kv_heads,
                int head_dim) {
  if (cuda_device < 0 || R < 0 || R > kMaxReq || heads <= 0 ||
      kv_heads <= 0 || heads % kv_heads || head_dim <= 0)
    return KVTC_EINVAL;
  if ((head_dim != 64 && head_dim != 128 && head_dim != 256) ||
      (int64_t)kv_heads * head_dim > kMaxD || heads / kv_heads > kMaxGroup)
    return KVTC_ENOTSUP;
  return KVTC_OK;
}

}  // namespace
}  // namespace kvtc

using namespace kvtc;

extern "C" {

int64_t kvtc_paged_attend_workspace_bytes(int cuda_device, int R, int heads,
                                          int kv_heads, int head_dim) {
  const int st = check_shape(cuda_device, R, heads, kv_heads, head_dim);
  return st != KVTC_OK ? st : 256;
}

int kvtc_paged_attend(int cuda_device, int R, int heads, int kv_heads,
                      int head_dim, int dtype, const void* q, int64_t q_ld,
                      const void* k_cache, const void* v_cache,
                      int64_t num_blocks, int block_size,
                      const int32_t* block_table, int max_blocks,
                      const int32_t* lens, int sink, int window, float scale,
                      void* out, int64_t out_ld, float* lse, void* workspace,
                      int64_t workspace_bytes, uint32_t* flags,
                      void* cuda_stream) {
  int ret = check_shape(cuda_device, R, heads, kv_heads, head_dim);
  if (ret != KVTC_OK) return ret;
  if ((dtype != KVTC_DTYPE_BF16 && dtype != KVTC_DTYPE_FP16) || !k_cache ||
      !v_cache || num_blocks <= 0 || num_blocks > INT32_MAX ||
      max_blocks <= 0 || sink < 0 || window < 0 || !std::isfinite(scale) ||
      !workspace || (R && (!q || !block_table || !lens || !out)))
    return KVTC_EINVAL;
  if (block_size != kBlock) return KVTC_ENOTSUP;
  const int64_t width = (int64_t)heads * head_dim;
  const int64_t need = kvtc_paged_attend_workspace_bytes(
      cuda_device, R, heads, kv_heads, head_dim);
  if (need < 0) return (int)need;
  if (q_ld < width || out_ld < width || workspace_bytes < need)
    return KVTC_ESIZE;
  if (q_ld % 8 || out_ld % 8 || !aligned16(q) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned16(out) || !aligned16(workspace) ||
      misaligned4(block_table) || misaligned4(lens) || misaligned4(lse) ||
      misaligned4(flags))
    return KVTC_EALIGN;
  if (R == 0) return KVTC_OK;
  DeviceGuard guard(cuda_device);
  if (!guard.ok) return KVTC_ECUDA;
  AttendParams p;
  p.q = q;
  p.k = k_cache;
  p.v = v_cache;
  p.table = block_table;
  p.lens = lens;
  p.out = out;
  p.lse = lse;
  p.flags = flags;
  p.q_ld = q_ld;
  p.out_ld = out_ld;
  p.num_blocks = num_blocks;
  p.scale = scale;
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.max_blocks = max_blocks;
  p.sink = sink;
  p.window = window;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e =
      dtype == KVTC_DTYPE_BF16
          ? launch<__nv_bfloat16>(p, R, head_dim, st)
          : launch<__half>(p, R, head_dim, st);
  return e == cudaSuccess ? KVTC_OK : KVTC_ECUDA;
}

}  // extern "C"
