// Norms and position rotation of the queries and keys of new tokens, and the
// way of their K and V rows into paged pools, in one pass.
//
// Per head x of a token at position p (head_dim elements):
//     y = x / sqrt(mean x^2 + eps) * w                (where there are weights)
//     (a, b) -> c (a cos t_i - b sin t_i, b cos t_i + a sin t_i),
// for the pairs i < rotary_dim / 2 of y, t_i = p f_i; the rest of y stays.
//
// The angle is needed modulo one turn only: f_i / 2 pi modulo 1 as a 64-bit
// fraction times p, in wrapping integers, is exact up to p 2^-65 of a turn,
// however far the position is; no 64-bit floating point per token.
//
// Work.  A block takes tiles of 1 to 8 tokens: a thread forms one angle of
// the tile (shared memory), then head_dim / 8 lanes take a head, 16 bytes a
// lane, which hold both elements of four pairs; a norm is a few shuffles.
//
// What bounds it: HBM.  Every element is read and written once.
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
constexpr int kThreads = 256;
constexpr int kMaxTile = 8;          // tokens per tile
constexpr int kAhead = 4;            // heads that a lane has under way

struct RotateParams {
  const char* src[3];                // q, k, v rows
  char* q_out;
  char* pool[2];                     // of K and V
  const int32_t* positions;
  const double* inv_freq;
  const int64_t* slots;
  const void* norm[2];               // weights of q and k, or null
  unsigned* flags;
  int64_t N, ld, q_out_ld, pool_rows;
  float scale, eps;
  int32_t heads, kv_heads;
  uint32_t inv[2];                   // 2^32 / heads (and kv_heads), up; 0: one
  int32_t pairs;                     // rotary_dim / 2
  int32_t tile;                      // tokens per tile
};

template <class T>
__device__ __forceinline__ float2 unpack2(uint32_t x);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t x) {
  return make_float2(__uint_as_float(x << 16),
                     __uint_as_float(x & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t x) {
  return __half22float2(*reinterpret_cast<const __half2*>(&x));
}
template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Bytes from a head's start to the two pieces (of 8 bytes) that lane c of the
// head holds.  Neighbours paired: 16 bytes in a row, elements 2i and 2i + 1 a
// pair.  Halves paired: elements i and i + pairs, four of each; of the part
// that is not rotated, four of either half.
template <int HD, bool kNeighbours>
struct Place {
  uint32_t a, b;
  __device__ __forceinline__ Place(int c, int pairs) {
    if (kNeighbours) {
      a = 16 * c;
      b = a + 8;
    } else if (4 * c < pairs) {
      a = 8 * c;
      b = a + 2 * pairs;
    } else {
      a = 4 * pairs + 2 * (4 * c - pairs);
      b = a + HD - 2 * pairs;
    }
  }
  __device__ __forceinline__ uint4 load(const char* p) const {
    if (kNeighbours) return *reinterpret_cast<const uint4*>(p + a);
    const uint2 x = *reinterpret_cast<const uint2*>(p + a);
    const uint2 y = *reinterpret_cast<const uint2*>(p + b);
    return make_uint4(x.x, x.y, y.x, y.y);
  }
  __device__ __forceinline__ void store(char* p, uint4 v) const {
    if (kNeighbours) {
      *reinterpret_cast<uint4*>(p + a) = v;
    } else {
      *reinterpret_cast<uint2*>(p + a) = make_uint2(v.x, v.y);
      *reinterpret_cast<uint2*>(p + b) = make_uint2(v.z, v.w);
    }
  }
};

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d, x = *reinterpret_cast<uint64_t*>(&a),
              y = *reinterpret_cast<uint64_t*>(&b);
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d, x = *reinterpret_cast<uint64_t*>(&a),
              y = *reinterpret_cast<uint64_t*>(&b),
              z = *reinterpret_cast<uint64_t*>(&c);
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
  return *reinterpret_cast<float2*>(&d);
}

template <class T, int HD, bool kNeighbours>
__global__ void __launch_bounds__(kThreads, 4)
    rotate_kernel(const __grid_constant__ RotateParams p) {
  constexpr int kLanes = HD / 8;                  // per head
  constexpr int kHeads = kThreads / kLanes;       // heads at once
  __shared__ __align__(16) float cosines[kMaxTile * HD / 2];
  __shared__ __align__(16) float sines[kMaxTile * HD / 2];
  __shared__ int64_t slot[kMaxTile];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, c = tid % kLanes;
  const Place<HD, kNeighbours> place(c, p.pairs);
  const bool turned = 4 * c < p.pairs;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // this thread's angle: pair and token of a tile
  const int pair = tid % (HD / 2);
  uint64_t step = 0;
  if (pair < p.pairs) {
    const double f = p.inv_freq[pair] * 0.15915494309189533577;   // 1 / 2 pi
    step = __double2ull_rn((f - floor(f)) * 18446744073709551616.0);
  }
  float2 w[2][4];                    // weights of the norms
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 x = p.norm[i] ? place.load(static_cast<const char*>(p.norm[i]))
                              : make_uint4(0, 0, 0, 0);
    w[i][0] = unpack2<T>(x.x);
    w[i][1] = unpack2<T>(x.y);
    w[i][2] = unpack2<T>(x.z);
    w[i][3] = unpack2<T>(x.w);
  }
  const int64_t tiles = (p.N + p.tile - 1) / p.tile;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t n0 = t * p.tile;
    const int tokens = (int)min((int64_t)p.tile, p.N - n0);
    __syncthreads();
    for (int i = tid / (HD / 2); pair < p.pairs && i < tokens;
         i += kThreads / (HD / 2)) {
      const uint64_t at = (uint64_t)(int64_t)p.positions[n0 + i] * step;
      float s, co;
      sincospif((float)(int32_t)(at >> 32) * 0x1p-31f, &s, &co);
      cosines[i * (HD / 2) + pair] = co * p.scale;
      sines[i * (HD / 2) + pair] = s * p.scale;
    }
    if (tid < tokens) {
      int64_t to = p.slots[n0 + tid];
      if (to >= p.pool_rows) {
        if (p.flags) atomicOr(p.flags, KVTC_FLAG_BLOCK);
        to = -1;
      }
      slot[tid] = to;
    }
    // Rounds of kHeads heads of the tile, of one kind each: q, then k, then v.
    const int of_q = (tokens * p.heads + kHeads - 1) / kHeads;
    const int of_k = (tokens * p.kv_heads + kHeads - 1) / kHeads;
    const int rounds = of_q + (p.src[2] ? 2 : 1) * of_k;
    bool first = true;
#pragma unroll 1
    for (int r0 = 0; r0 < rounds; r0 += kAhead) {
      uint4 x[kAhead];
      int ti[kAhead], hi[kAhead];     // token, or -1; head
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int r = r0 + k;
        const int what = r < of_q ? 0 : r < of_q + of_k ? 1 : 2;
        const int head0 = what == 0 ? r : what == 1 ? r - of_q
                                                    : r - of_q - of_k;
        const int n = what ? p.kv_heads : p.heads;
        const uint32_t at = head0 * kHeads + tid / kLanes;
        const uint32_t inv = p.inv[what ? 1 : 0];
        ti[k] = inv ? __umulhi(at, inv) : at;
        hi[k] = at - ti[k] * n;
        if (r >= rounds || ti[k] >= tokens) {
          ti[k] = -1;
          x[k] = make_uint4(0, 0, 0, 0);
        } else {
          x[k] = place.load(p.src[what] + (n0 + ti[k]) * p.ld * 2 +
                            hi[k] * (HD * 2));
        }
      }
      if (first) {
        __syncthreads();        // the angles, under the first loads
        first = false;
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int r = r0 + k;
        if (r >= rounds) break;
        if (r >= of_q + of_k) {
          if (ti[k] >= 0 && slot[ti[k]] >= 0)
            place.store(p.pool[1] + (slot[ti[k]] * p.kv_heads + hi[k]) *
                                        (HD * 2),
                        x[k]);
          continue;
        }
        const bool is_k = r >= of_q;
        // halves: a0 a1, a2 a3, b0 b1, b2 b3; neighbours: a0 b0, a1 b1, ...
        float2 v[4] = {unpack2<T>(x[k].x), unpack2<T>(x[k].y),
                       unpack2<T>(x[k].z), unpack2<T>(x[k].w)};
        if (p.norm[is_k]) {
          float2 sum2 = mul2(v[0], v[0]);
#pragma unroll
          for (int e = 1; e < 4; ++e) sum2 = fma2(v[e], v[e], sum2);
          float sum = sum2.x + sum2.y;
#pragma unroll
          for (int d = 1; d < kLanes; d <<= 1)
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
          // (to 2^-22, far below the output's step)
          const float inv = rsqrtf(fmaf(sum, 1.f / HD, p.eps));
          const float2 inv2 = make_float2(inv, inv);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = mul2(mul2(v[e], inv2), is_k ? w[1][e] : w[0][e]);
        }
        if (ti[k] < 0) continue;
        if (turned) {
          const int at = ti[k] * (HD / 2) + c * 4;
          const float4 co = *reinterpret_cast<const float4*>(cosines + at);
          const float4 si = *reinterpret_cast<const float4*>(sines + at);
          if (kNeighbours) {
            const float cc[4] = {co.x, co.y, co.z, co.w};
            const float ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = fma2(v[e], make_float2(cc[e], cc[e]),
                          mul2(make_float2(v[e].y, v[e].x),
                               make_float2(-ss[e], ss[e])));
          } else {
            const float2 c01 = make_float2(co.x, co.y);
            const float2 c23 = make_float2(co.z, co.w);
            const float2 s01 = make_float2(si.x, si.y);
            const float2 s23 = make_float2(si.z, si.w);
            const float2 m01 = make_float2(-si.x, -si.y);
            const float2 m23 = make_float2(-si.z, -si.w);
            const float2 a01 = fma2(v[0], c01, mul2(v[2], m01));
            const float2 a23 = fma2(v[1], c23, mul2(v[3], m23));
            v[2] = fma2(v[2], c01, mul2(v[0], s01));
            v[3] = fma2(v[3], c23, mul2(v[1], s23));
            v[0] = a01;
            v[1] = a23;
          }
        }
        const uint4 out =
            make_uint4(pack2<T>(v[0].x, v[0].y), pack2<T>(v[1].x, v[1].y),
                       pack2<T>(v[2].x, v[2].y), pack2<T>(v[3].x, v[3].y));
        if (!is_k) {
          place.store(p.q_out + (n0 + ti[k]) * p.q_out_ld * 2 +
                          hi[k] * (HD * 2),
                      out);
        } else if (slot[ti[k]] >= 0) {
          place.store(p.pool[0] + (slot[ti[k]] * p.kv_heads + hi[k]) *
                                      (HD * 2),
                      out);
        }
      }
    }
  }
}

inline bool misaligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

template <class T, int HD>
cudaError_t launch(const RotateParams& p, bool neighbours, cudaStream_t st) {
  const int64_t tiles = (p.N + p.tile - 1) / p.tile;
  const unsigned grid = (unsigned)std::min<int64_t>(tiles, 8 * 152);
  return neighbours ? launch_kernel(rotate_kernel<T, HD, true>, grid, kThreads,
                                    0, st, true, 0, p)
                    : launch_kernel(rotate_kernel<T, HD, false>, grid,
                                    kThreads, 0, st, true, 0, p);
}

}  // namespace
}  // namespace kvtc

using namespace kvtc;

extern "C" {

int kvtc_rotary_frequencies(int rotary_dim, double base, int scaling,
                            double factor, double context, double low,
                            double high, double* inv_freq) {
  if (rotary_dim <= 0 || rotary_dim % 2 || !inv_freq || !(base > 0) ||
      !std::isfinite(base))
    return KVTC_EINVAL;
  if (scaling != KVTC_ROTARY_PLAIN && scaling != KVTC_ROTARY_LINEAR &&
      scaling != KVTC_ROTARY_BASE && scaling != KVTC_ROTARY_BANDS)
    return KVTC_EINVAL;
  if (scaling != KVTC_ROTARY_PLAIN && !(factor > 0 && std::isfinite(factor)))
    return KVTC_EINVAL;
  if (scaling == KVTC_ROTARY_BANDS &&
      !(context > 0 && std::isfinite(context) && low >= 0 && high > low &&
        std::isfinite(high)))
    return KVTC_EINVAL;
  if (scaling == KVTC_ROTARY_BASE && rotary_dim == 2)
    return KVTC_EINVAL;                         // its one frequency is 1
  const auto frequency = [&](int i) {
    double f = std::pow(base, -2.0 * i / rotary_dim);
    if (scaling == KVTC_ROTARY_LINEAR) f /= factor;
    // (a factor of its own: the stretched base may lie out of range)
    if (scaling == KVTC_ROTARY_BASE)
      f *= std::pow(factor, -2.0 * i / (rotary_dim - 2.0));
    if (scaling == KVTC_ROTARY_BANDS) {
      const double turns = context * f / 6.283185307179586477;
      const double keep =
          std::min(1.0, std::max(0.0, (turns - low) / (high - low)));
      f *= keep + (1.0 - keep) / factor;
    }
    return f;
  };
  for (int i = 0; i < rotary_dim / 2; ++i)
    if (!std::isfinite(frequency(i))) return KVTC_EINVAL;
  for (int i = 0; i < rotary_dim / 2; ++i) inv_freq[i] = frequency(i);
  return KVTC_OK;
}

int kvtc_paged_rotate(int cuda_device, int64_t N, int heads, int kv_heads,
                      int head_dim, int dtype, const void* q, const void* k,
                      const void* v, int64_t ld, const int32_t* positions,
                      const double* inv_freq, int rotary_dim, int interleaved,
                      float rotary_scale, const void* q_norm,
                      const void* k_norm, float eps, void* q_out,
                      int64_t q_out_ld, const int64_t* slots, int block_size,
                      void* k_cache, void* v_cache, int64_t num_blocks,
                      uint32_t* flags, void* cuda_stream) {
  if (cuda_device < 0 || N < 0 || N > INT32_MAX || heads <= 0 ||
      kv_heads <= 0 || head_dim <= 0 ||
      (dtype != KVTC_DTYPE_BF16 && dtype != KVTC_DTYPE_FP16) ||
      rotary_dim < 0 || rotary_dim > head_dim || num_blocks <= 0 ||
      num_blocks > INT32_MAX || !k_cache || !std::isfinite(rotary_scale) ||
      !(eps >= 0.f) || !std::isfinite(eps) || (v && !v_cache) ||
      (!v && v_cache && N) || (rotary_dim && !inv_freq) ||
      (N && (!q || !k || !q_out || !slots || (rotary_dim && !positions))))
    return KVTC_EINVAL;
  if (block_size != kBlock || rotary_dim % 8 ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
      (int64_t)kv_heads * head_dim > kMaxD ||
      (int64_t)heads * head_dim > kMaxD * 16)
    return KVTC_ENOTSUP;
  if (ld < (int64_t)heads * head_dim || ld < (int64_t)kv_heads * head_dim ||
      q_out_ld < (int64_t)heads * head_dim)
    return KVTC_ESIZE;
  if (ld % 8 || q_out_ld % 8 || !aligned16(q) || !aligned16(k) ||
      !aligned16(v) || !aligned16(q_out) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned16(q_norm) || !aligned16(k_norm) ||
      misaligned(positions, 4) || misaligned(inv_freq, 8) ||
      misaligned(slots, 8) || misaligned(flags, 4))
    return KVTC_EALIGN;
  if (N == 0) return KVTC_OK;
  DeviceGuard guard(cuda_device);
  if (!guard.ok) return KVTC_ECUDA;
  RotateParams p;
  p.src[0] = static_cast<const char*>(q);
  p.src[1] = static_cast<const char*>(k);
  p.src[2] = static_cast<const char*>(v);
  p.q_out = static_cast<char*>(q_out);
  p.pool[0] = static_cast<char*>(k_cache);
  p.pool[1] = static_cast<char*>(v_cache);
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.slots = slots;
  p.norm[0] = q_norm;
  p.norm[1] = k_norm;
  p.flags = flags;
  p.N = N;
  p.ld = ld;
  p.q_out_ld = q_out_ld;
  p.pool_rows = num_blocks * kBlock;
  p.scale = rotary_scale;
  p.eps = eps;
  p.heads = heads;
  p.kv_heads = kv_heads;
  // (exact for the up to 8 x 2048 heads of a tile)
  p.inv[0] = heads > 1 ? (uint32_t)((1ull << 32) / heads + 1) : 0;
  p.inv[1] = kv_heads > 1 ? (uint32_t)((1ull << 32) / kv_heads + 1) : 0;
  p.pairs = rotary_dim / 2;
  // as many tokens as a block has angles to form, or one where that leaves
  // blocks without any
  const int most = kThreads / (head_dim / 2);
  p.tile = N >= (int64_t)most * 8 * 152 ? most : 1;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const bool near = interleaved != 0;
  cudaError_t e;
  if (dtype == KVTC_DTYPE_BF16)
    e = head_dim == 64    ? launch<__nv_bfloat16, 64>(p, near, st)
        : head_dim == 128 ? launch<__nv_bfloat16, 128>(p, near, st)
                          : launch<__nv_bfloat16, 256>(p, near, st);
  else
    e = head_dim == 64    ? launch<__half, 64>(p, near, st)
        : head_dim == 128 ? launch<__half, 128>(p, near, st)
                          : launch<__half, 256>(p, near, st);
  if (e != cudaSuccess) return KVTC_ECUDA;
  count_launch();
  return KVTC_OK;
}

}  // extern "C"
