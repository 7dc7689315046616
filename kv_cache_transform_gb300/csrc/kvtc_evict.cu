// Eviction from paged pools by weights per token: of a request longer than
// `keep`, the first `sink`, the last `window` and, of the others, those of the
// greatest weight stay, in their order.
//   select_kernel  a block per request finds the smallest weight that stays
//     by its bits, eight at a time (histograms), then lists the tokens in
//     order by sums over the block, and moves their weights.
//   move_kernel    rows of all pools by that list.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "../../include/kvtc.h"
#include "kvtc_hostutil.cuh"
#include "kvtc_internal.cuh"

namespace kvtc {
namespace {

constexpr int kBlock = 16;           // tokens per pool block
constexpr int kMaxReq = 4096;        // requests per call
constexpr int kMaxTable = INT32_MAX / kBlock - 1;

constexpr int kSelThreads = 1024;
constexpr int kMaxStreams = 64;      // pools per launch

struct EvictParams {
  const float* acc;
  const int32_t* lens;
  const int32_t* table;
  const int32_t* out_table;
  int32_t* kept;
  float* acc_out;
  int32_t* lens_out;
  int32_t* ids;        // [R][max_blocks * 16]: the block of a kept token
  unsigned* flags;
  int64_t acc_ld, num_blocks;
  int32_t R, keep, sink, window, max_blocks, in_place;
  int32_t pieces;      // 16-byte pieces per row
  int32_t slice;       // of which a block of move_kernel takes so many
  uint4* cache[kMaxStreams];
};

// The order of weights as that of unsigned numbers; both zeros are equal, a
// NaN comes before everything.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0;
  const uint32_t b = __float_as_uint(x + 0.f);   // -0 + 0 = 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Exclusive sums of a and b over the block's threads; totals in ta and tb.
__device__ __forceinline__ void block_sums2(int& a, int& b, int* ta, int* tb,
                                            int2* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int a0 = a, b0 = b;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(~0u, a, d), y = __shfl_up_sync(~0u, b, d);
    if (lane >= d) {
      a += x;
      b += y;
    }
  }
  __syncthreads();
  if (lane == 31) sums[warp] = make_int2(a, b);
  __syncthreads();
  const int2 w = sums[lane];          // (32 warps)
  int xa = lane < warp ? w.x : 0, xb = lane < warp ? w.y : 0;
  int sa = w.x, sb = w.y;
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    xa += __shfl_xor_sync(~0u, xa, d);
    xb += __shfl_xor_sync(~0u, xb, d);
    sa += __shfl_xor_sync(~0u, sa, d);
    sb += __shfl_xor_sync(~0u, sb, d);
  }
  a += xa - a0;
  b += xb - b0;
  *ta = sa;
  *tb = sb;
}

__global__ void __launch_bounds__(kSelThreads)
    select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int hist[256];
  __shared__ int2 sums[32];
  __shared__ int pick[2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x;
  const int32_t most = p.max_blocks * kBlock;
  const int32_t asked = p.lens[r];
  const int32_t len = min(max(asked, 0), most);
  const int32_t after = min(len, p.keep);
  const float* acc = p.acc + r * p.acc_ld;
  const int32_t* row = p.table + r * p.max_blocks;
  if (tid == 0 && asked > most && p.flags)
    atomicOr(p.flags, KVTC_FLAG_SPACE);
  // of tokens lo .. hi - 1, `want` stay
  const int32_t lo = len > p.keep ? p.sink : len;
  const int32_t hi = len > p.keep ? len - p.window : len;
  const int32_t want = len > p.keep ? p.keep - p.sink - p.window : 0;
  // the smallest key that stays, and how many of those equal to it
  uint32_t least = 0;
  int equal = want;
  if (len > p.keep) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t above = shift == 24 ? 0u : ~0u << (shift + 8);
      for (int32_t t = lo + tid; t < hi; t += kSelThreads) {
        const uint32_t key = key_of(acc[t]);
        if ((key & above) == least) atomicAdd(&hist[(key >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int left = equal, b = 255;
        while (b > 0 && hist[b] < left) left -= hist[b--];
        pick[0] = b;
        pick[1] = left;
      }
      __syncthreads();
      least |= (uint32_t)pick[0] << shift;
      equal = pick[1];
      __syncthreads();
    }
  }
  // the list, a stretch of tokens at a time
  int above = 0, same = 0;      // before this stretch
  int32_t* kept = p.kept + r * (int64_t)p.keep;
  int32_t* ids = p.ids + r * (int64_t)most;
  float* acc_out = p.acc_out + r * p.acc_ld;
  bool bad = false;
  for (int32_t t0 = 0; t0 < len; t0 += kSelThreads) {
    const int32_t t = t0 + tid;
    float w = 0.f;
    int is_above = 0, is_same = 0, stays = 0;
    if (t < len) {
      w = acc[t];
      if (t >= lo && t < hi) {
        const uint32_t key = key_of(w);
        is_above = key > least;
        is_same = key == least;
      } else {
        stays = 1;
      }
    }
    int a = is_above, s = is_same, ta, ts;
    block_sums2(a, s, &ta, &ts, sums);
    int32_t to = -1;
    if (stays) {
      to = t < lo ? t : t - (hi - lo) + want;
    } else if (is_above || (is_same && same + s < equal)) {
      to = lo + above + a + min(same + s, equal);
    }
    above += ta;
    same += ts;
    if (to >= 0) {
      const int32_t id = row[t / kBlock];
      const bool ok = id >= 0 && id < p.num_blocks;
      bad |= !ok;
      kept[to] = t;
      ids[to] = ok ? id : -1;
      acc_out[to] = w;
    }
  }
  __syncthreads();
  for (int32_t t = after + tid; t < len; t += kSelThreads) acc_out[t] = 0.f;
  for (int64_t j = after + tid; j < p.keep; j += kSelThreads) kept[j] = -1;
  if (tid == 0) p.lens_out[r] = after;
  if (bad && p.flags) atomicOr(p.flags, KVTC_FLAG_BLOCK);
}

// A block takes `slice` pieces of the rows of one request in one pool.  Where
// kept rows go into the blocks that they come from, it goes through them in
// order: row j's place is at or before the one it comes from, so that what is
// still to be read is never written, once all reads of a step are done.
// Otherwise several blocks share the rows of a slice.
constexpr int kMoveThreads = 256;
__global__ void __launch_bounds__(kMoveThreads)
    move_kernel(const __grid_constant__ EvictParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int slices = (p.pieces + p.slice - 1) / p.slice;
  const int64_t r = blockIdx.z;
  const int part = blockIdx.x / slices, parts = gridDim.x / slices;
  const int c = (blockIdx.x % slices) * p.slice + threadIdx.x % p.slice;
  const int step = kMoveThreads / p.slice;
  const int32_t most = p.max_blocks * kBlock;
  const int32_t n = p.lens_out[r];
  const int32_t* kept = p.kept + r * (int64_t)p.keep;
  const int32_t* ids = p.ids + r * (int64_t)most;
  const int32_t* to_row = p.out_table + r * p.max_blocks;
  uint4* pool = p.cache[blockIdx.y];
  bool bad = false;
  for (int32_t j0 = part * step; j0 < n; j0 += parts * step) {
    const int32_t j = j0 + (int32_t)threadIdx.x / p.slice;
    uint4 v;
    int64_t to = -1;
    if (j < n && threadIdx.x / p.slice < step && c < p.pieces) {
      const int32_t t = kept[j], id = ids[j], oid = to_row[j / kBlock];
      const bool ok = oid >= 0 && oid < p.num_blocks;
      bad |= !ok;
      if (ok && id >= 0 && !(p.in_place && t == j)) {
        to = (int64_t)oid * kBlock + j % kBlock;
        v = pool[((int64_t)id * kBlock + t % kBlock) * p.pieces + c];
      }
    }
    if (p.in_place) __syncthreads();
    if (to >= 0) pool[to * p.pieces + c] = v;
  }
  if (bad && p.flags) atomicOr(p.flags, KVTC_FLAG_BLOCK);
}

inline bool misaligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

}  // namespace
}  // namespace kvtc

using namespace kvtc;

extern "C" {

int64_t kvtc_paged_evict_workspace_bytes(int R, int max_blocks) {
  if (R < 0 || R > kMaxReq || max_blocks <= 0) return KVTC_EINVAL;
  if (max_blocks > kMaxTable) return KVTC_ENOTSUP;
  return std::max<int64_t>(256, (int64_t)R * max_blocks * kBlock * 4);
}

int kvtc_paged_evict(int cuda_device, int R, const float* acc, int64_t acc_ld,
                     const int32_t* lens, int keep, int sink, int window,
                     const int32_t* block_table, const int32_t* out_table,
                     int max_blocks, int block_size, int nstreams,
                     void* const* cache, int D, int64_t num_blocks,
                     int32_t* kept, float* acc_out, int32_t* lens_out,
                     void* workspace, int64_t workspace_bytes,
                     uint32_t* flags, void* cuda_stream) {
  const int64_t need = kvtc_paged_evict_workspace_bytes(R, max_blocks);
  if (need < 0) return (int)need;
  if (cuda_device < 0 || keep < 0 || sink < 0 || window < 0 ||
      (int64_t)sink + window > keep || nstreams < 0 || (nstreams && !cache) ||
      D <= 0 || num_blocks <= 0 || num_blocks > INT32_MAX || !workspace ||
      (R && (!acc || !lens || !block_table || !out_table || !acc_out ||
             !lens_out || (keep && !kept))))
    return KVTC_EINVAL;
  if (block_size != kBlock || D % 8 || D > kMaxD) return KVTC_ENOTSUP;
  if (acc_ld < (int64_t)max_blocks * kBlock || workspace_bytes < need)
    return KVTC_ESIZE;
  if (acc_ld % 4 || !aligned16(acc) || !aligned16(acc_out) ||
      !aligned16(workspace) || misaligned(lens, 4) ||
      misaligned(block_table, 4) || misaligned(out_table, 4) ||
      misaligned(kept, 4) || misaligned(lens_out, 4) || misaligned(flags, 4))
    return KVTC_EALIGN;
  for (int j = 0; j < nstreams; ++j) {
    if (!cache[j]) return KVTC_EINVAL;
    if (!aligned16(cache[j])) return KVTC_EALIGN;
  }
  if (R == 0) return KVTC_OK;
  DeviceGuard guard(cuda_device);
  if (!guard.ok) return KVTC_ECUDA;
  EvictParams p;
  p.acc = acc;
  p.lens = lens;
  p.table = block_table;
  p.out_table = out_table;
  p.kept = kept;
  p.acc_out = acc_out;
  p.lens_out = lens_out;
  p.ids = static_cast<int32_t*>(workspace);
  p.flags = flags;
  p.acc_ld = acc_ld;
  p.num_blocks = num_blocks;
  p.R = R;
  p.keep = keep;
  p.sink = sink;
  p.window = window;
  p.max_blocks = max_blocks;
  p.in_place = out_table == block_table;
  p.pieces = D / 8;
  p.slice = std::min(8, p.pieces);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (launch_kernel(select_kernel, R, kSelThreads, 0, st, true, 0, p) !=
      cudaSuccess)
    return KVTC_ECUDA;
  count_launch();
  const int slices = (p.pieces + p.slice - 1) / p.slice;
  for (int j0 = 0; j0 < nstreams; j0 += kMaxStreams) {
    const int n = std::min(kMaxStreams, nstreams - j0);
    for (int j = 0; j < n; ++j) p.cache[j] = static_cast<uint4*>(cache[j0 + j]);
    const int parts = p.in_place ? 1 : 4;
    if (launch_kernel(move_kernel, dim3(slices * parts, n, R), kMoveThreads,
                      0, st, true, 0, p) != cudaSuccess)
      return KVTC_ECUDA;
    count_launch();
  }
  return KVTC_OK;
}

}  // extern "C"
