// Blocks, slots and row writes of paged KV pools.
//
// kvtc_paged_assign: with n_r = max(0, lens_r - held_r) new tokens and b_r
// new blocks per request, cu is the exclusive sum of n, C the inclusive sum
// of b, and request r takes free[head + C_r - b_r ...] if it fits.  Both are
// integer sums, so the result is exact and does not depend on the launch.
//   assign_scan_kernel  one block of 1024 threads, four consecutive requests
//                       each: the two sums, who is served, head and held.
//   assign_fill_kernel  the block-table columns and the slot map.
// kvtc_paged_append: append_kernel copies 16-byte pieces of rows.
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
constexpr int kScanThreads = 1024;
constexpr int kScanPer = kMaxReq / kScanThreads;

__host__ __device__ __forceinline__ int64_t blocks_of(int64_t tokens) {
  return (tokens + kBlock - 1) / kBlock;
}

// What the fill pass needs of a request, in the workspace.
struct AssignRow {
  int64_t first;      // free-list index of its first new block
  int32_t held;       // tokens that had blocks
  int32_t blocks;     // new blocks; -1 where it is not served
};

struct AssignParams {
  const int32_t* held;
  const int32_t* lens;
  const int32_t* free_blocks;
  int64_t n_free;
  const int64_t* head;
  int32_t* table;
  int64_t* slots;
  int64_t slot_capacity;
  int64_t* cu;
  int32_t* held_out;
  int64_t* head_out;
  AssignRow* rows;
  unsigned* flags;
  int32_t R;
  int32_t max_blocks;
};

__device__ __forceinline__ int64_t warp_inclusive(int64_t v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

__global__ void __launch_bounds__(kScanThreads)
    assign_scan_kernel(const AssignParams p) {
  __shared__ int64_t warp_new[32], warp_need[32];
  __shared__ unsigned long long given;   // blocks given out
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) given = 0;
  const int64_t head = *p.head;
  const bool head_ok = head >= 0 && head <= p.n_free;
  const int64_t avail = head_ok ? p.n_free - head : 0;
  int64_t fresh[kScanPer], need[kScanPer];
  int32_t held[kScanPer], lens[kScanPer];
  int64_t sum_new = 0, sum_need = 0;
#pragma unroll
  for (int i = 0; i < kScanPer; ++i) {
    const int r = tid * kScanPer + i;
    held[i] = r < p.R ? max(p.held[r], 0) : 0;
    lens[i] = r < p.R ? max(p.lens[r], 0) : 0;
    fresh[i] = max((int64_t)lens[i] - held[i], (int64_t)0);
    const bool fits = lens[i] <= (int64_t)p.max_blocks * kBlock;
    need[i] = fresh[i] && fits ? blocks_of(lens[i]) - blocks_of(held[i]) : 0;
    sum_new += fresh[i];
    sum_need += need[i];
  }
  int64_t in_new = warp_inclusive(sum_new, lane);
  int64_t in_need = warp_inclusive(sum_need, lane);
  if (lane == 31) {
    warp_new[warp] = in_new;
    warp_need[warp] = in_need;
  }
  __syncthreads();
  if (warp == 0) {
    warp_new[lane] = warp_inclusive(warp_new[lane], lane);
    warp_need[lane] = warp_inclusive(warp_need[lane], lane);
  }
  __syncthreads();
  if (warp) {
    in_new += warp_new[warp - 1];
    in_need += warp_need[warp - 1];
  }
  int64_t at_new = in_new - sum_new, at_need = in_need - sum_need;
  bool short_of = tid == 0 && !head_ok;
#pragma unroll
  for (int i = 0; i < kScanPer; ++i) {
    const int r = tid * kScanPer + i;
    if (r >= p.R) break;
    p.cu[r] = at_new;
    at_new += fresh[i];
    at_need += need[i];
    const bool served = lens[i] <= (int64_t)p.max_blocks * kBlock &&
                        (need[i] == 0 || at_need <= avail);
    AssignRow row;
    row.first = head + at_need - need[i];
    row.held = held[i];
    row.blocks = served ? (int32_t)need[i] : -1;
    p.rows[r] = row;
    p.held_out[r] = served ? max(held[i], lens[i]) : held[i];
    if (served && need[i]) atomicMax(&given, (unsigned long long)at_need);
    short_of |= !served && fresh[i];
    if (r == p.R - 1) {
      p.cu[p.R] = at_new;
      short_of |= at_new > p.slot_capacity;
    }
  }
  if (short_of && p.flags) atomicOr(p.flags, KVTC_FLAG_SPACE);
  __syncthreads();
  if (tid == 0) {
    *p.head_out = head + (int64_t)given;
    if (p.R == 0) p.cu[0] = 0;
  }
}

__global__ void __launch_bounds__(256)
    assign_fill_kernel(const AssignParams p) {
  const int64_t tid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t threads = (int64_t)gridDim.x * blockDim.x;
  const int lane = threadIdx.x & 31;
  for (int64_t r = tid >> 5; r < p.R; r += threads >> 5) {
    const AssignRow row = p.rows[r];
    int32_t* to = p.table + r * p.max_blocks + blocks_of(row.held);
    for (int i = lane; i < row.blocks; i += 32)
      to[i] = p.free_blocks[row.first + i];
  }
  const int64_t total = p.R ? p.cu[p.R] : 0;
  for (int64_t j = tid; j < p.slot_capacity; j += threads) {
    int64_t slot = -1;
    if (j < total) {
      // the last request whose first new token is at or before j; of
      // several (requests with no new token) the one that holds j
      int lo = 0, hi = p.R - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu[mid] <= j) lo = mid; else hi = mid - 1;
      }
      const AssignRow row = p.rows[lo];
      if (row.blocks >= 0) {
        const int64_t t = row.held + (j - p.cu[lo]);
        const int64_t had = blocks_of(row.held), b = t / kBlock;
        const int64_t id = b < had
            ? p.table[(int64_t)lo * p.max_blocks + b]
            : p.free_blocks[row.first + (b - had)];
        if (id >= 0) slot = id * kBlock + t % kBlock;
      }
    }
    p.slots[j] = slot;
  }
}

constexpr int kAppendStreams = 64;   // streams per launch
struct AppendParams {
  const uint4* src[kAppendStreams];
  uint4* cache[kAppendStreams];
  const int64_t* slots;
  int64_t N;
  int64_t ld;            // 16-byte pieces per source row
  int64_t pool_rows;     // num_blocks * 16
  unsigned* flags;
  int32_t pieces;        // 16-byte pieces per row
  int32_t nstreams;
};

__global__ void __launch_bounds__(256)
    append_kernel(const __grid_constant__ AppendParams p) {
  const int64_t total = p.N * p.nstreams * p.pieces;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += step) {
    const int64_t row = i / p.pieces;
    const int c = (int)(i - row * p.pieces);
    const int j = (int)(row / p.N);
    const int64_t n = row - j * p.N;
    const int64_t slot = p.slots[n];
    if (slot < 0) continue;
    if (slot >= p.pool_rows) {
      if (p.flags) atomicOr(p.flags, KVTC_FLAG_BLOCK);
      continue;
    }
    p.cache[j][slot * p.pieces + c] = p.src[j][n * p.ld + c];
  }
}

inline bool misaligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

}  // namespace
}  // namespace kvtc

using namespace kvtc;

extern "C" {

int64_t kvtc_paged_assign_workspace_bytes(int R) {
  if (R < 0 || R > kMaxReq) return KVTC_EINVAL;
  return std::max<int64_t>(256, (int64_t)sizeof(AssignRow) * R);
}

int kvtc_paged_assign(int cuda_device, int R, const int32_t* held,
                      const int32_t* lens, const int32_t* free_blocks,
                      int64_t n_free, const int64_t* head,
                      int32_t* block_table, int max_blocks, int block_size,
                      int64_t* slots, int64_t slot_capacity, int64_t* cu,
                      int32_t* held_out, int64_t* head_out, void* workspace,
                      int64_t workspace_bytes, uint32_t* flags,
                      void* cuda_stream) {
  if (cuda_device < 0 || R < 0 || R > kMaxReq || n_free < 0 ||
      max_blocks <= 0 || slot_capacity < 0 || !head || !cu || !head_out ||
      !workspace || (R && (!held || !lens || !block_table || !held_out)) ||
      (n_free && !free_blocks) || (slot_capacity && !slots))
    return KVTC_EINVAL;
  if (block_size != kBlock) return KVTC_ENOTSUP;
  if (workspace_bytes < kvtc_paged_assign_workspace_bytes(R))
    return KVTC_ESIZE;
  if (misaligned(head, 8) || misaligned(cu, 8) || misaligned(head_out, 8) ||
      misaligned(slots, 8) || misaligned(workspace, 8) ||
      misaligned(held, 4) || misaligned(lens, 4) ||
      misaligned(free_blocks, 4) || misaligned(block_table, 4) ||
      misaligned(held_out, 4) || misaligned(flags, 4))
    return KVTC_EALIGN;
  DeviceGuard guard(cuda_device);
  if (!guard.ok) return KVTC_ECUDA;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  AssignParams p;
  p.held = held;
  p.lens = lens;
  p.free_blocks = free_blocks;
  p.n_free = n_free;
  p.head = head;
  p.table = block_table;
  p.slots = slots;
  p.slot_capacity = slot_capacity;
  p.cu = cu;
  p.held_out = held_out;
  p.head_out = head_out;
  p.rows = static_cast<AssignRow*>(workspace);
  p.flags = flags;
  p.R = R;
  p.max_blocks = max_blocks;
  if (launch_kernel(assign_scan_kernel, 1, kScanThreads, 0, st, false, 0, p) !=
      cudaSuccess)
    return KVTC_ECUDA;
  count_launch();
  const int64_t want = std::max((slot_capacity + 255) / 256,
                                ((int64_t)R * 32 + 255) / 256);
  if (want) {
    if (launch_kernel(assign_fill_kernel,
                      (unsigned)std::min<int64_t>(want, 8 * 152), 256, 0, st,
                      false, 0, p) != cudaSuccess)
      return KVTC_ECUDA;
    count_launch();
  }
  return KVTC_OK;
}

int kvtc_paged_append(int cuda_device, int nstreams, const void* const* src,
                      int64_t ld, int64_t N, const int64_t* slots, int D,
                      int block_size, void* const* cache, int64_t num_blocks,
                      uint32_t* flags, void* cuda_stream) {
  if (cuda_device < 0 || nstreams < 0 || N < 0 || N > INT32_MAX || D <= 0 ||
      num_blocks <= 0 || num_blocks > INT32_MAX ||
      (nstreams && (!src || !cache)) || (N && nstreams && !slots))
    return KVTC_EINVAL;
  if (block_size != kBlock || D % 8 || D > kMaxD) return KVTC_ENOTSUP;
  if (ld < D) return KVTC_ESIZE;
  if (ld % 8 || misaligned(slots, 8) || misaligned(flags, 4))
    return KVTC_EALIGN;
  for (int j = 0; j < nstreams; ++j) {
    if (!cache[j] || (N && !src[j])) return KVTC_EINVAL;
    if (!aligned16(cache[j]) || !aligned16(src[j])) return KVTC_EALIGN;
  }
  if (N == 0 || nstreams == 0) return KVTC_OK;
  DeviceGuard guard(cuda_device);
  if (!guard.ok) return KVTC_ECUDA;
  AppendParams p;
  p.slots = slots;
  p.N = N;
  p.ld = ld / 8;
  p.pool_rows = num_blocks * kBlock;
  p.flags = flags;
  p.pieces = D / 8;
  for (int j0 = 0; j0 < nstreams; j0 += kAppendStreams) {
    p.nstreams = std::min(kAppendStreams, nstreams - j0);
    for (int j = 0; j < p.nstreams; ++j) {
      p.src[j] = static_cast<const uint4*>(src[j0 + j]);
      p.cache[j] = static_cast<uint4*>(cache[j0 + j]);
    }
    const int64_t total = N * p.nstreams * p.pieces;
    if (launch_kernel(append_kernel,
                      (unsigned)std::min<int64_t>((total + 255) / 256,
                                                  8 * 152),
                      256, 0, static_cast<cudaStream_t>(cuda_stream), false,
                      0, p) != cudaSuccess)
      return KVTC_ECUDA;
    count_launch();
  }
  return KVTC_OK;
}

}  // extern "C"
