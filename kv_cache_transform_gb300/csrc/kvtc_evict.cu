// Eviction from paged pools by weights per token: of a request longer than
// `keep`, the first `sink`, the last `window` and, of the others, those of the
// greatest weight stay, in their order.
//   select_kernel  one to eight blocks per request find the smallest weight
//     that stays by its bits, eleven at a time (histograms), then list the
//     tokens in order by sums over the blocks, and move their weights.
//   move_kernel    rows of all pools by that list.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "../../include/kvtc.h"
#include "kvtc_hostutil.cuh"
#include "kvtc_internal.cuh"
#include "ptx.cuh"

namespace kvtc {
namespace {

constexpr int kBlock = 16;           // tokens per pool block
constexpr int kMaxReq = 4096;        // requests per call
constexpr int kMaxTable = INT32_MAX / kBlock - 1;

constexpr int kSelThreads = 1024;
constexpr int kMaxStreams = 64;      // pools per launch
constexpr int kBins = 2048;          // weights are told apart 11 bits at a time

struct EvictParams {
  const float* acc;
  const int32_t* lens;
  const int32_t* table;
  const int32_t* out_table;
  int32_t* kept;
  float* acc_out;
  int32_t* lens_out;
  int32_t* ids;        // [R][max_blocks * 16]: the block of a kept token
  float* weights;      // [R][max_blocks * 16]: its weight
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

// Exclusive sums of a over the block's threads (a may hold two counts, of 32
// bits each); the total in *all.
__device__ __forceinline__ uint64_t block_sums(uint64_t a, uint64_t* all,
                                               uint64_t* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t upto = a;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t x = __shfl_up_sync(~0u, upto, d);
    if (lane >= d) upto += x;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  const uint64_t w = sums[lane];              // (32 warps)
  uint64_t before = lane < warp ? w : 0, total = w;
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    before += __shfl_xor_sync(~0u, before, d);
    total += __shfl_xor_sync(~0u, total, d);
  }
  __syncthreads();
  *all = total;
  return upto - a + before;
}

// A cluster of blocks per request, each with a stretch of its tokens.  The
// smallest key that stays is found from the top, 11 bits a round: histograms of
// those that agree so far, added up through distributed shared memory, and their
// sums from above.  Then the tokens that stay are listed in order, four tokens a
// thread at a time.  (One request of 32K cut to 4K: 34 us in one block, 70 with
// 8 bits a round, a thread that goes through the bins and one token a thread.)
struct __align__(16) SelectShared {
  int hist[kBins];
  uint64_t sums[32];
  uint64_t counts;          // of the block's tokens: above, equal
  int pick[2];
};
__device__ __forceinline__ uint32_t cluster_blocks() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}
// 64 bits at the same place in another block's shared memory.
constexpr int kMaxBlocks = 8;
__device__ __forceinline__ uint2 load2_from(const void* at, uint32_t rank) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "r"(mapa_shared(smem_u32(at), rank))
               : "memory");
  return v;
}
// kMany: more than one block per request.
template <bool kMany>
__global__ void __launch_bounds__(kSelThreads)
    select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ SelectShared sm;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  const uint32_t blocks = kMany ? cluster_blocks() : 1;
  const uint32_t rank = kMany ? cluster_ctarank() : 0;
  const auto sync = [] {
    if (kMany) cluster_sync(); else __syncthreads();
  };
  const int64_t r = blockIdx.y;
  const int32_t most = p.max_blocks * kBlock;
  const int32_t asked = p.lens[r];
  const int32_t len = min(max(asked, 0), most);
  const int32_t after = min(len, p.keep);
  const float* acc = p.acc + r * p.acc_ld;
  const int32_t* row = p.table + r * p.max_blocks;
  if (tid == 0 && rank == 0 && asked > most && p.flags)
    atomicOr(p.flags, KVTC_FLAG_SPACE);
  // of tokens lo .. hi - 1, `want` stay
  const int32_t lo = len > p.keep ? p.sink : len;
  const int32_t hi = len > p.keep ? len - p.window : len;
  const int32_t want = len > p.keep ? p.keep - p.sink - p.window : 0;
  // This block's tokens.  (Places of tokens are unsigned: a request may have up
  // to 2^31 - 32 of them, and a stretch or a step of the block's threads that
  // begins before that may end behind 2^31.)
  const uint32_t each = ((uint32_t)len / blocks / 16 + 1) * 16;
  const uint32_t from = min(rank * each, (uint32_t)len);
  const uint32_t upto = min(from + each, (uint32_t)len);
  const uint32_t from_mid = max(from, (uint32_t)lo);
  const uint32_t upto_mid = min(upto, (uint32_t)hi);
  // the smallest key that stays, and how many of those equal to it
  uint32_t least = want ? 0u : ~0u;
  int equal = want;
  if (want) {
    for (int round = 0; round < 3; ++round) {
      const int shift = round == 0 ? 21 : round == 1 ? 10 : 0;
      const int bits = round == 2 ? 10 : 11;
      const uint32_t known = round == 0 ? 0u : ~0u << (shift + bits);
      for (int i = tid; i < kBins; i += kSelThreads) sm.hist[i] = 0;
      __syncthreads();
      constexpr int kAhead = 4;
      for (uint32_t t0 = from_mid + tid; t0 < upto_mid;
           t0 += kAhead * kSelThreads) {
        float w[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          w[i] = t0 + i * kSelThreads < upto_mid ? acc[t0 + i * kSelThreads]
                                                 : 0.f;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const uint32_t key = key_of(w[i]);
          if (t0 + i * kSelThreads < upto_mid && (key & known) == least)
            atomicAdd(&sm.hist[(key >> shift) & ((1u << bits) - 1)], 1);
        }
      }
      sync();
      // thread t: bins 2047 - 2 t and 2046 - 2 t; sums from the largest
      const int b1 = kBins - 1 - 2 * tid, b0 = b1 - 1;
      int n1 = 0, n0 = 0;
      {
        // (all asked for at once)
        uint2 v[kMaxBlocks] = {};
        if (!kMany) v[0] = *reinterpret_cast<const uint2*>(&sm.hist[b0]);
#pragma unroll
        for (int k = 0; kMany && k < kMaxBlocks; ++k)
          v[k] = k < blocks ? load2_from(&sm.hist[b0], k) : make_uint2(0, 0);
#pragma unroll
        for (int k = 0; k < kMaxBlocks; ++k) {
          n0 += (int)v[k].x;
          n1 += (int)v[k].y;
        }
      }
      uint64_t all;
      const int above = (int)block_sums((uint64_t)(n0 + n1), &all, sm.sums);
      if (above < equal && above + n1 >= equal) {
        sm.pick[0] = b1;
        sm.pick[1] = equal - above;
      } else if (above + n1 < equal && above + n1 + n0 >= equal) {
        sm.pick[0] = b0;
        sm.pick[1] = equal - above - n1;
      }
      // (all blocks have read all histograms)
      sync();
      least |= (uint32_t)sm.pick[0] << shift;
      equal = sm.pick[1];
    }
  }
  // 2 bits a token: 1 above, 2 equal, 3 stays in any case; four from t on
  const auto classify = [&](uint32_t t, const float (&w)[4], uint64_t* count) {
    uint32_t what = 0;
    *count = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (t + i >= upto) continue;
      uint32_t x = 3;
      if (t + i >= (uint32_t)lo && t + i < (uint32_t)hi) {
        const uint32_t key = key_of(w[i]);
        x = key > least ? 1u : key == least && equal ? 2u : 0u;
      }
      what |= x << (2 * i);
      *count += x == 1 ? 1ull : x == 2 ? 1ull << 32 : 0ull;
    }
    return what;
  };
  // (rows of acc are as long as the table, a multiple of 16)
  const auto load = [&](uint32_t t, float (&w)[4]) {
    const float4 x = t < upto ? *reinterpret_cast<const float4*>(acc + t)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
    w[0] = x.x;
    w[1] = x.y;
    w[2] = x.z;
    w[3] = x.w;
  };
  // counts of the blocks before this one
  uint32_t gone_above = 0, gone_same = 0;
  if (kMany && want) {
    uint64_t mine = 0, all;
    for (uint32_t t0 = from; t0 < upto; t0 += 4 * kSelThreads) {
      float w[4];
      uint64_t count;
      load(t0 + 4 * tid, w);
      classify(t0 + 4 * tid, w, &count);
      mine += count;
    }
    block_sums(mine, &all, sm.sums);
    if (tid == 0) sm.counts = all;
    sync();
    uint2 v[kMaxBlocks];
#pragma unroll
    for (int k = 0; k < kMaxBlocks; ++k)
      v[k] = k < rank ? load2_from(&sm.counts, k) : make_uint2(0, 0);
#pragma unroll
    for (int k = 0; k < kMaxBlocks; ++k) {
      gone_above += v[k].x;
      gone_same += v[k].y;
    }
  }
  // the list: tokens above `least`, and of those equal to it the first ones
  int32_t* kept = p.kept + r * (int64_t)p.keep;
  int32_t* ids = p.ids + r * (int64_t)most;
  float* weights = p.weights + r * (int64_t)most;
  float* acc_out = p.acc_out + r * p.acc_ld;
  bool bad = false;
  for (uint32_t t0 = from; t0 < upto; t0 += 4 * kSelThreads) {
    const uint32_t t = t0 + 4 * tid;
    float w[4];
    uint64_t count, all;
    load(t, w);
    const uint32_t what = classify(t, w, &count);
    const int32_t id = what ? row[t / kBlock] : 0;
    const uint64_t before = block_sums(count, &all, sm.sums);
    uint32_t above = gone_above + (uint32_t)before;
    uint32_t same = gone_same + (uint32_t)(before >> 32);
    gone_above += (uint32_t)all;
    gone_same += (uint32_t)(all >> 32);
    const bool ok = id >= 0 && id < p.num_blocks;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = (what >> (2 * i)) & 3;
      int32_t to = -1;
      if (x == 3)
        to = (int32_t)(t + i < (uint32_t)lo ? t + i : t + i - (hi - lo) + want);
      else if (x == 1 || (x == 2 && same < (uint32_t)equal))
        to = lo + (int32_t)(above + min(same, (uint32_t)equal));
      above += x == 1;
      same += x == 2;
      if (to < 0) continue;
      bad |= !ok;
      kept[to] = (int32_t)(t + i);
      ids[to] = ok ? id : -1;
      if (kMany) weights[to] = w[i]; else acc_out[to] = w[i];
    }
  }
  // (acc_out may be acc: a stretch's places lie at or before what it reads, so
  // one block may write them as it goes; of several, one would overtake another
  // that still reads, so theirs wait in the workspace)
  if (kMany) __threadfence();
  sync();
  const int32_t step = (int32_t)blocks * kSelThreads;
  const int32_t first = (int32_t)rank * kSelThreads + tid;
  for (int64_t t = (int64_t)(kMany ? 0 : after) + first;
       t < len; t += step)
    acc_out[t] = t < after ? __ldcg(weights + t) : 0.f;
  for (int64_t j = (int64_t)after + first; j < p.keep; j += step)
    kept[j] = -1;
  if (tid == 0 && rank == 0) p.lens_out[r] = after;
  if (bad && p.flags) atomicOr(p.flags, KVTC_FLAG_BLOCK);
}

// Blocks per request: as many as the GPU holds at once, and as 4096 tokens each
// can feed.
int select_blocks(int R, int64_t max_blocks) {
  int blocks = R <= 19 ? 8 : R <= 38 ? 4 : R <= 76 ? 2 : 1;
  while (blocks > 1 && max_blocks * kBlock <= 4096ll * (blocks / 2))
    blocks /= 2;
  return blocks;
}

// A block takes `slice` pieces of the rows of one request in one pool, four
// rows a thread under way.  Where kept rows go into the blocks that they come
// from, it goes through them in order: row j's place is at or before the one it
// comes from, so that what is still to be read is never written, once all reads
// of a step are done.  Otherwise several blocks share the rows of a slice.
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 4;         // per thread and step
__global__ void __launch_bounds__(kMoveThreads)
    move_kernel(const __grid_constant__ EvictParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int slices = (p.pieces + p.slice - 1) / p.slice;
  const int64_t r = blockIdx.z;
  const int part = blockIdx.x / slices, parts = gridDim.x / slices;
  const int c = (blockIdx.x % slices) * p.slice + threadIdx.x % p.slice;
  const int rows = kMoveThreads / p.slice, mine = threadIdx.x / p.slice;
  const bool in = mine < rows && c < p.pieces;
  const int32_t most = p.max_blocks * kBlock;
  const int32_t n = p.lens_out[r];
  const int32_t* kept = p.kept + r * (int64_t)p.keep;
  const int32_t* ids = p.ids + r * (int64_t)most;
  const int32_t* to_row = p.out_table + r * p.max_blocks;
  uint4* pool = p.cache[blockIdx.y];
  bool bad = false;
  const int64_t step = (int64_t)rows * kMoveRows;
  for (int64_t j0 = part * step; j0 < n; j0 += parts * step) {
    uint4 v[kMoveRows];
    int64_t to[kMoveRows];
    int32_t t[kMoveRows], id[kMoveRows], oid[kMoveRows];
#pragma unroll
    for (int i = 0; i < kMoveRows; ++i) {
      const int64_t j = j0 + i * rows + mine;
      const bool has = in && j < n;
      t[i] = has ? kept[j] : 0;
      id[i] = has ? ids[j] : -1;
      oid[i] = has ? to_row[j / kBlock] : -1;
      const bool ok = oid[i] >= 0 && oid[i] < p.num_blocks;
      bad |= has && !ok;
      to[i] = ok && id[i] >= 0 && !(p.in_place && t[i] == j)
                  ? (int64_t)oid[i] * kBlock + j % kBlock
                  : -1;
    }
#pragma unroll
    for (int i = 0; i < kMoveRows; ++i)
      if (to[i] >= 0)
        v[i] = pool[((int64_t)id[i] * kBlock + t[i] % kBlock) * p.pieces + c];
    if (p.in_place) __syncthreads();
#pragma unroll
    for (int i = 0; i < kMoveRows; ++i)
      if (to[i] >= 0) pool[to[i] * p.pieces + c] = v[i];
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
  return std::max<int64_t>(256, (int64_t)R * max_blocks * kBlock * 8);
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
  p.weights = reinterpret_cast<float*>(p.ids + (int64_t)R * max_blocks *
                                                   kBlock);
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
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const int blocks = select_blocks(R, max_blocks);
  if ((blocks > 1
           ? launch_kernel(select_kernel<true>, dim3(blocks, R), kSelThreads,
                           0, st, true, blocks, p)
           : launch_kernel(select_kernel<false>, dim3(1, R), kSelThreads, 0,
                           st, true, 0, p)) != cudaSuccess)
    return KVTC_ECUDA;
  count_launch();
  for (int j0 = 0; j0 < nstreams; j0 += kMaxStreams) {
    const int n = std::min(kMaxStreams, nstreams - j0);
    for (int j = 0; j < n; ++j) p.cache[j] = static_cast<uint4*>(cache[j0 + j]);
    // 512 bytes of a row, or in place, where a slice is one block's, as little
    // as 64 while there are fewer blocks than the GPU holds
    const int64_t pools = (int64_t)R * n;
    p.slice = std::min(32, p.pieces);
    while (p.in_place && p.slice > 4 &&
           pools * ((p.pieces + p.slice - 1) / p.slice) < 8 * 152)
      p.slice = (p.slice + 1) / 2;
    const int64_t slices = (p.pieces + p.slice - 1) / p.slice;
    const int64_t step = kMoveThreads / p.slice * kMoveRows;
    const int64_t steps =
        (std::min<int64_t>(keep, (int64_t)max_blocks * kBlock) + step - 1) /
        step;
    const int64_t parts =
        p.in_place ? 1
                   : std::max<int64_t>(
                         1, std::min(steps, 16 * 152 / (pools * slices)));
    if (launch_kernel(move_kernel, dim3((unsigned)(slices * parts), n, R),
                      kMoveThreads, 0, st, true, 0, p) != cudaSuccess)
      return KVTC_ECUDA;
    count_launch();
  }
  return KVTC_OK;
}

}  // extern "C"
