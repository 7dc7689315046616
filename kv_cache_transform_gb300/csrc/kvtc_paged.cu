// Blocks, slots and row writes of paged KV pools.
//
// kvtc_paged_assign: with n_r = max(0, lens_r - held_r) new tokens and b_r
// new blocks per request, cu is the exclusive sum of n, C the inclusive sum
// of b, and request r takes free[head + C_r - b_r ...] if it fits.  Both are
// integer sums, so the result is exact and does not depend on the launch.
//   few slots (decode steps): assign_small_kernel, one block, a thread per
//     request: a chain of three loads, 1.8 us;
//   more, or no slot map: assign_fill_kernel on the whole GPU writes the
//     table entries and the slots; every block forms the sums itself, or
//     assign_scan_kernel does so before it, in one block (more than 1024
//     requests, or a state that is kept in place).
// kvtc_paged_append: append_kernel, a warp per row.
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

__host__ __device__ __forceinline__ int64_t blocks_of(int64_t tokens) {
  return (tokens + kBlock - 1) / kBlock;
}

// What the fill pass needs of a request, in the workspace.
struct __align__(16) AssignRow {
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

// A request's demand.
struct Demand {
  int32_t held, lens;
  int64_t fresh;      // new tokens
  int32_t need;       // new blocks, 0 where they cannot fit the table
  bool fits;
  __device__ __forceinline__ Demand(const AssignParams& p, int r) {
    held = r < p.R ? max(p.held[r], 0) : 0;
    lens = r < p.R ? max(p.lens[r], 0) : 0;
    fresh = max((int64_t)lens - held, (int64_t)0);
    fits = lens <= (int64_t)p.max_blocks * kBlock;
    need = fresh && fits ? (int32_t)(blocks_of(lens) - blocks_of(held)) : 0;
  }
};

// Inclusive sums over the block's threads of two values each; `total` of the
// first.  sums: shared, two per warp.
__device__ __forceinline__ void block_sums(int64_t& a, int64_t& b,
                                           int64_t* sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = blockDim.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xFFFFFFFFu, a, d);
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, b, d);
    if (lane >= d) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    sums[2 * warp] = a;
    sums[2 * warp + 1] = b;
  }
  __syncthreads();
  // each warp adds up the warps before it
  int64_t x = lane < warps ? sums[2 * lane] : 0;
  int64_t y = lane < warps ? sums[2 * lane + 1] : 0;
  int64_t all = x;
  if (lane >= warp) x = y = 0;
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
    y += __shfl_xor_sync(0xFFFFFFFFu, y, d);
    all += __shfl_xor_sync(0xFFFFFFFFu, all, d);
  }
  a += x;
  b += y;
  *total = all;
}

__device__ __forceinline__ int64_t free_left(const AssignParams& p,
                                             int64_t head, bool* ok) {
  *ok = head >= 0 && head <= p.n_free;
  return *ok ? p.n_free - head : 0;
}

__device__ __forceinline__ int64_t slot_of(int64_t id, int64_t t) {
  return id >= 0 ? id * kBlock + t % kBlock : -1;
}

// One block, a thread per request (R <= 1024).  Where a request has few new
// tokens its thread writes their slots, else the warps share them.
// (64 requests of 16 new tokens 4.6 us, where the warps share all above four
// tokens 13.2, by assign_fill_kernel 7.3; of 32, 13.4 and 5.8; 1024 of 8, 8.6
// and 10.9, of 16, 14.7 and 10.9.  Table entries alone, without a slot map: 64
// requests of 2 blocks 10.3 and 3.8, of 2048 blocks 315 and 13.4; of one
// block 3.2 and 3.8.)
constexpr int kSmallReq = 1024;
constexpr int64_t kSmallSlots = 8192;  // and kSmallOwn a request
constexpr int kSmallOwn = 16;          // tokens that a thread writes itself
__global__ void __launch_bounds__(kSmallReq)
    assign_small_kernel(const __grid_constant__ AssignParams p) {
  __shared__ int64_t sums[64];
  __shared__ unsigned long long given;   // blocks given out
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int r = threadIdx.x, lane = r & 31;
  if (r == 0) given = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Demand d(p, r);
  const int64_t head = *p.head;
  bool head_ok;
  const int64_t left = free_left(p, head, &head_ok);
  // the block that the first new token continues, asked for ahead
  const int32_t had = (int32_t)blocks_of(d.held);
  int32_t* row = p.table + (int64_t)r * p.max_blocks;
  int32_t open = -1;
  if (d.fresh && d.fits && d.held % kBlock) open = row[had - 1];
  int64_t upto = d.fresh, used = d.need, total;
  block_sums(upto, used, sums, &total);
  const bool served = d.fits && (d.need == 0 || used <= left);
  const int64_t first = head + used - d.need;
  const int64_t at = upto - d.fresh;
  bool short_of = r == 0 && (!head_ok || total > p.slot_capacity);
  if (r < p.R) {
    p.cu[r] = at;
    p.held_out[r] = served ? max(d.held, d.lens) : d.held;
    if (served && d.need) atomicMax(&given, (unsigned long long)used);
    short_of |= !served && d.fresh;
  }
  if (r == 0) p.cu[p.R] = total;
  if (short_of && p.flags) atomicOr(p.flags, KVTC_FLAG_SPACE);
  // A request's new table entries, and the slots of its tokens as far as the
  // map goes: entries or tokens k, k + step, ...
  auto write = [&](int32_t held, int32_t open, int64_t fresh, int32_t blocks,
                   int64_t first, int64_t at, int32_t* row, int k, int step) {
    const int64_t had = blocks_of(held);
    for (int i = k; i < blocks; i += step)
      row[had + i] = p.free_blocks[first + i];
    fresh = min(fresh, p.slot_capacity - at);
    for (int64_t i = k; i < fresh; i += step) {
      const int64_t t = held + i, b = t / kBlock;
      int64_t slot = -1;
      if (blocks >= 0)
        slot = slot_of(b < had ? open : p.free_blocks[first + (b - had)], t);
      p.slots[at + i] = slot;
    }
  };
  const int32_t blocks = served ? d.need : -1;
  const bool own = d.fresh <= kSmallOwn;
  if (own) write(d.held, open, d.fresh, blocks, first, at, row, 0, 1);
  // the others, of one lane after the other
  for (uint32_t m = __ballot_sync(0xFFFFFFFFu, !own); m; m &= m - 1) {
    const int l = __ffs(m) - 1;
    write(__shfl_sync(0xFFFFFFFFu, d.held, l),
          __shfl_sync(0xFFFFFFFFu, open, l),
          __shfl_sync(0xFFFFFFFFu, d.fresh, l),
          __shfl_sync(0xFFFFFFFFu, blocks, l),
          __shfl_sync(0xFFFFFFFFu, first, l),
          __shfl_sync(0xFFFFFFFFu, at, l),
          p.table + (int64_t)((r & ~31) + l) * p.max_blocks, lane, 32);
  }
  for (int64_t j = total + r; j < p.slot_capacity; j += blockDim.x)
    p.slots[j] = -1;
  __syncthreads();
  if (r == 0) *p.head_out = head + (int64_t)given;
}

// One block forms the sums, `per` consecutive requests per thread, into cu
// and rows; where `writes`, it also writes what the call returns of them.
__device__ __forceinline__ void scan_requests(const AssignParams& p, int per,
                                              bool writes, int64_t* sums,
                                              unsigned long long* given,
                                              int64_t* cu, AssignRow* rows) {
  const int tid = threadIdx.x;
  const int64_t head = *p.head;
  bool head_ok;
  const int64_t left = free_left(p, head, &head_ok);
  int64_t fresh = 0, need = 0, total;
  for (int i = 0; i < per; ++i) {
    const Demand d(p, tid * per + i);
    fresh += d.fresh;
    need += d.need;
  }
  int64_t upto = fresh, used = need;
  block_sums(upto, used, sums, &total);
  upto -= fresh;
  used -= need;
  bool short_of = tid == 0 && (!head_ok || total > p.slot_capacity);
  for (int i = 0; i < per; ++i) {
    const int r = tid * per + i;
    if (r >= p.R) break;
    const Demand d(p, r);
    cu[r] = upto;
    if (writes) p.cu[r] = upto;
    upto += d.fresh;
    used += d.need;
    const bool served = d.fits && (d.need == 0 || used <= left);
    AssignRow row;
    row.first = head + used - d.need;
    row.held = d.held;
    row.blocks = served ? d.need : -1;
    rows[r] = row;
    if (!writes) continue;
    // (a request's held is read for the last time above)
    p.held_out[r] = served ? max(d.held, d.lens) : d.held;
    if (served && d.need) atomicMax(given, (unsigned long long)used);
    short_of |= !served && d.fresh;
  }
  if (tid == 0) cu[p.R] = total;
  if (writes) {
    if (short_of && p.flags) atomicOr(p.flags, KVTC_FLAG_SPACE);
    __syncthreads();
    if (tid == 0) {
      p.cu[p.R] = total;
      *p.head_out = head + (int64_t)*given;
    }
  }
}
__global__ void __launch_bounds__(kScanThreads)
    assign_scan_kernel(const __grid_constant__ AssignParams p, int per) {
  __shared__ int64_t sums[64];
  __shared__ unsigned long long given;   // blocks given out
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) given = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  scan_requests(p, per, true, sums, &given, p.cu, p.rows);
}

// Last request r in [lo, hi] with cu[r] <= j (cu[lo] <= j); the whole warp
// looks, 32 places at a time.
__device__ __forceinline__ int request_at(const int64_t* cu, int lo, int hi,
                                          int64_t j) {
  const int lane = threadIdx.x & 31;
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + 1 + lane * step;
    const bool in = at <= hi && cu[at] <= j;
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, in));
    if (n == 0) return lo;
    lo += 1 + (n - 1) * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// Slots and new table entries.  A warp takes runs of 256 tokens and finds
// their first request once; each lane goes on from there (tokens mostly lie
// many to a request).  The lane that has a new block's first token writes its
// table entry; blocks whose first token lies behind the slot map come after.
// 131 thousand slots (1 MB) take 4.6 us, 2.1 million (17 MB) 8.0 (with twice
// the blocks 9.2, with half of them 8.4).
//
// kOwnSums: every block forms the sums itself, in shared memory, instead of a
// launch before that does (7.4 and 10.9 us); not for a state kept in place,
// which one block would change while another still reads it.
constexpr int kFillRun = 256;
constexpr int kFillThreads = 256;
template <bool kOwnSums>
__global__ void __launch_bounds__(kFillThreads)
    assign_fill_kernel(const __grid_constant__ AssignParams p) {
  __shared__ int64_t own_cu[kOwnSums ? kSmallReq + 1 : 1];
  __shared__ AssignRow own_rows[kOwnSums ? kSmallReq : 1];
  __shared__ int64_t sums[64];
  __shared__ unsigned long long given;
  const int64_t* cu = kOwnSums ? own_cu : p.cu;
  const AssignRow* rows = kOwnSums ? own_rows : p.rows;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (kOwnSums && threadIdx.x == 0) given = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (kOwnSums) {
    scan_requests(p, (p.R + kFillThreads - 1) / kFillThreads,
                  blockIdx.x == 0, sums, &given, own_cu, own_rows);
    __syncthreads();
  }
  const int lane = threadIdx.x & 31;
  const int64_t warp = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  const int64_t total = cu[p.R];
  for (int64_t j0 = warp * kFillRun; j0 < p.slot_capacity;
       j0 += warps * kFillRun) {
    // (looked up before `total` is here to say whether it is of use)
    int r = p.R ? request_at(cu, 0, p.R - 1, j0) : 0;
    const AssignRow row0 = p.R ? rows[r] : AssignRow{0, 0, -1};
    const int64_t from0 = cu[r], to0 = p.R ? cu[r + 1] : 0;
    const int64_t end = min(total, p.slot_capacity);
    if (j0 + kFillRun <= min(end, to0)) {
      // the whole run is one request's (in a third of the instructions)
      const AssignRow row = row0;
      int64_t* to = p.slots + j0 + lane;
      if (row.blocks < 0) {
#pragma unroll
        for (int k = 0; k < kFillRun / 32; ++k) to[k * 32] = -1;
        continue;
      }
      const int32_t had = (int32_t)blocks_of(row.held);
      const int32_t* fresh = p.free_blocks + row.first - had;
      int32_t* table = p.table + (int64_t)r * p.max_blocks;
      const int32_t t0 = row.held + (int32_t)(j0 - from0) + lane;
      int32_t id[kFillRun / 32];
#pragma unroll
      for (int k = 0; k < kFillRun / 32; ++k) {
        const int32_t b = (t0 + k * 32) / kBlock;
        id[k] = b < had ? table[b] : fresh[b];
      }
#pragma unroll
      for (int k = 0; k < kFillRun / 32; ++k) {
        const int32_t t = t0 + k * 32, b = t / kBlock;
        if (t % kBlock == 0 && b >= had) table[b] = id[k];
        to[k * 32] = slot_of(id[k], t);
      }
      continue;
    }
    // of request r: tokens from, ..., to - 1 of the map (none looked up yet)
    int64_t from = 0, to = 0;
    const int32_t* fresh = nullptr;  // ids of its blocks, by block index
    int32_t* table = nullptr;
    int32_t held = 0, had = 0;
    bool served = false;
#pragma unroll
    for (int k = 0; k < kFillRun / 32; ++k) {
      const int64_t j = j0 + k * 32 + lane;
      int64_t slot = -1;
      if (j < end) {
        if (j >= to) {
          if (cu[r + 1] <= j && cu[++r + 1] <= j) {
            int hi = p.R - 1;
            while (r < hi) {
              const int mid = (r + hi + 1) >> 1;
              if (cu[mid] <= j) r = mid; else hi = mid - 1;
            }
          }
          const AssignRow row = rows[r];
          from = cu[r];
          to = cu[r + 1];
          held = row.held;
          had = (int32_t)blocks_of(held);
          served = row.blocks >= 0;
          fresh = p.free_blocks + row.first - had;
          table = p.table + (int64_t)r * p.max_blocks;
        }
        if (served) {
          const int32_t t = held + (int32_t)(j - from), b = t / kBlock;
          const int32_t id = b < had ? table[b] : fresh[b];
          slot = slot_of(id, t);
          if (b >= had && t % kBlock == 0) table[b] = id;
        }
      }
      if (j < p.slot_capacity) p.slots[j] = slot;
    }
  }
  if (total <= p.slot_capacity) return;
  for (int64_t r = warp; r < p.R; r += warps) {
    const AssignRow row = rows[r];
    // the first block whose first token has no place in the map
    const int64_t mapped = max(p.slot_capacity - cu[r], (int64_t)0);
    const int64_t had = blocks_of(row.held);
    const int64_t i0 = max(blocks_of(row.held + mapped) - had, (int64_t)0);
    int32_t* to = p.table + r * p.max_blocks + had;
    for (int64_t i = i0 + lane; i < row.blocks; i += 32)
      to[i] = p.free_blocks[row.first + i];
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

// A warp per (stream, row): the row's slot once, its pieces 32 at a time with
// four loads in flight a lane.  Bound by HBM and, for decode steps, by two
// loads one after the other: 8192 rows of K and V of 2 KB (67 MB moved)
// 11.5 us, 5.8 TB/s; with two rows in flight a warp 12.2.
__global__ void __launch_bounds__(256)
    append_kernel(const __grid_constant__ AppendParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const uint32_t warp = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const uint32_t warps = gridDim.x * (blockDim.x >> 5);
  const uint4* src = p.src[blockIdx.y];
  uint4* cache = p.cache[blockIdx.y];
  for (int64_t n = warp; n < p.N; n += warps) {
    const int64_t slot = p.slots[n];
    const uint4* from = src + n * p.ld;
    if (slot < 0) continue;
    if (slot >= p.pool_rows) {
      if (lane == 0 && p.flags) atomicOr(p.flags, KVTC_FLAG_BLOCK);
      continue;
    }
    uint4* to = cache + slot * p.pieces;
    for (int c0 = lane; c0 < p.pieces; c0 += 128) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c0 + i * 32 < p.pieces) v[i] = from[c0 + i * 32];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c0 + i * 32 < p.pieces) to[c0 + i * 32] = v[i];
    }
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
      misaligned(slots, 8) || !aligned16(workspace) ||
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
  // (capacity is what the host knows of the tokens; a map of less than half a
  // slot a request says that the table alone is wanted, of any length)
  if (R <= kSmallReq && slot_capacity >= (R + 1) / 2 &&
      slot_capacity <= std::min(kSmallSlots, (int64_t)kSmallOwn * R)) {
    if (launch_kernel(assign_small_kernel, 1, std::max(32, (R + 31) / 32 * 32),
                      0, st, true, 0, p) != cudaSuccess)
      return KVTC_ECUDA;
    count_launch();
    return KVTC_OK;
  }
  const int64_t runs = std::max<int64_t>(
      (slot_capacity + kFillRun - 1) / kFillRun, 152 * 8);
  const unsigned grid = (unsigned)std::min<int64_t>((runs + 7) / 8, 4 * 152);
  if (R <= kSmallReq && held_out != held && head_out != head) {
    if (launch_kernel(assign_fill_kernel<true>, grid, kFillThreads, 0, st,
                      true, 0, p) != cudaSuccess)
      return KVTC_ECUDA;
    count_launch();
    return KVTC_OK;
  }
  const int per = std::max(1, (R + kScanThreads - 1) / kScanThreads);
  const int threads = std::max(1, (R + per - 1) / per);
  if (launch_kernel(assign_scan_kernel, 1, (threads + 31) / 32 * 32, 0, st,
                    true, 0, p, per) != cudaSuccess)
    return KVTC_ECUDA;
  count_launch();
  if (launch_kernel(assign_fill_kernel<false>, grid, kFillThreads, 0, st,
                    true, 0, p) != cudaSuccess)
    return KVTC_ECUDA;
  count_launch();
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
    const dim3 grid((unsigned)std::min<int64_t>((N + 7) / 8, 16 * 152),
                    p.nstreams);
    if (launch_kernel(append_kernel, grid, 256, 0,
                      static_cast<cudaStream_t>(cuda_stream), true, 0, p) !=
        cudaSuccess)
      return KVTC_ECUDA;
    count_launch();
  }
  return KVTC_OK;
}

}  // extern "C"
