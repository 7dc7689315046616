// Attention of one new token per request over paged K and V pools.
//
// For a query head, s_t = scale q.k_t over the attended tokens.  With a
// running maximum m, l = sum 2^(s_t - m) and o = sum 2^(s_t - m) v_t (s in
// units of log2) are multiplied by 2^(m_old - m_new) when m grows, so K and
// V are read once; partial results of disjoint tokens join the same way:
//     m = max m_i,  l = sum l_i 2^(m_i - m),  o = sum o_i 2^(m_i - m),
// and out = o / l, lse = (m + log2 l) ln 2.
//
// Work.  A request's tokens fall into pages of 16; an item is (request, KV
// head, tile of query heads), a unit one page of an item, and all units of
// the call, in order, are dealt out to the grid's warps in equal runs: the
// kernel reads HBM at the same rate on every SM whatever the lengths are.
// The lengths are on the device, so each block sums them itself.  A warp
// writes an item that lies inside its run; parts of items are joined in
// three steps, each in a fixed order (equal calls give equal bits): the
// warps of a block through shared memory, then attend_join_kernel, launched
// behind, over the blocks.
//
// Inside a warp.  Each warp feeds itself: lane j of a batch of 32 units
// looks up its page's id and issues the two TMA boxes (16 tokens x head_dim
// of K and of V) into the warp's own ring; nothing but the warp waits for
// them, so there is no barrier between warps until the end.  The products
// are formed transposed, S^T = K Q^T (16 tokens x 8 heads) and O^T = V^T P^T
// (head_dim x 8 heads), so that the page fills the 16 rows of mma.sync and
// the few query heads only its 8 columns, the accumulators of eight heads
// take head_dim / 4 registers, and the softmax statistics sit in the lanes
// that rescale by them.  P enters the second product as two 16-bit terms
// (p = hi + lo to 2^-15), so that only the output's own rounding is of 16
// bits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/kvtc.h"
#include "kvtc_hostutil.cuh"
#include "kvtc_internal.cuh"
#include "ptx.cuh"

namespace kvtc {
namespace {

constexpr int kBlock = 16;           // tokens per pool block (a page)
constexpr int kMaxReq = 4096;        // requests per call
constexpr int kMaxGroup = 128;       // query heads per KV head
constexpr int kCtas = 152;           // one block per SM
constexpr int kRingBytes = 196608;   // shared memory for pages in flight
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Warps per block: the ring holds three pages a warp of head_dim 256, three
// of 128 or six of 64.
__host__ __device__ constexpr int warps_of(int hd) { return hd == 256 ? 4 : 8; }
__host__ __device__ constexpr int stage_bytes(int hd) { return hd * 64; }
__host__ __device__ constexpr int stages_of(int hd) {
  return kRingBytes / (warps_of(hd) * stage_bytes(hd));
}
// Floats of a partial result of nt x 8 query heads: o in fragment order
// ([channel tile][head tile][lane][4]), then m and l per head.
__host__ __device__ constexpr int slot_floats(int hd, int nt) {
  return nt * 8 * (hd + 2);
}

// Where the join finds the parts of an item that began in a block and did
// not end there; r < 0: there is none.
struct JoinDesc {
  int32_t r, sub, last_cta, pad;
};

struct AttendParams {
  CUtensorMap tm_k, tm_v;   // a pool as {64, 16, D / 64, num_blocks},
                            // box {64, 16, head_dim / 64, 1}
  const void* q;
  const int32_t* table;
  const int32_t* lens;
  void* out;
  float* lse;
  unsigned* flags;
  JoinDesc* desc;           // [kCtas]
  float* cta_slots;         // [kCtas][2] parts that cross blocks
  float* warp_slots;        // [kCtas * warps] parts that end inside a run
  int64_t q_ld, out_ld, num_blocks;
  float scale_log2;
  int32_t R, heads, kv_heads, max_blocks, sink, window;
  int32_t group, tiles, tile_heads;  // heads per KV head; tiles of them
};

// ------------------------------------------------------------ PTX wrappers
__device__ __forceinline__ void tma_load_page(uint32_t smem_dst,
                                              const void* tmap, int32_t slab,
                                              int32_t block, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_"
      "tx::bytes [%0], [%1, {%2, %2, %3, %4}], [%5];" ::"r"(smem_dst),
      "l"(tmap), "r"(0), "r"(slab), "r"(block), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr)
      : "memory");
}
// Transpose of an 8 x 8 matrix of 16-bit elements spread over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;"
               : "=r"(r)
               : "r"(x));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The two element types: conversion, packing (a in the low half) and
// D (16 x 8, fp32) += A (16 x 16) B (16 x 8).
//
// A weight w > 0 enters the product with V as hi + lo, hi = w kBelow cut to
// 16 bits and lo = w - hi (exact) rounded to 16 bits: w to 2^-15, and both
// terms positive, so that an infinite v gives an infinity and not inf - inf
// or 0 inf.  fp16 holds numbers from 2^-24: there weights are formed 2^15
// times as large, and what is lost lies 2^-39 below the largest.
template <class T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr float kBelow = 1.f - 0x1p-9f;  // by half a step or more
  static constexpr float kShift = 0.f;
  static __device__ __forceinline__ uint32_t pack_down(float a, float b) {
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t x) {
    return make_float2(__uint_as_float(x << 16),
                       __uint_as_float(x & 0xFFFF0000u));
  }
  static __device__ __forceinline__ void mma(float (&d)[4],
                                             const uint32_t (&a)[4],
                                             uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Elem<__half> {
  static constexpr float kBelow = 1.f - 0x1p-12f;
  static constexpr float kShift = 15.f;   // weights up to 2^15
  static __device__ __forceinline__ uint32_t pack_down(float a, float b) {
    uint32_t r;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
  }
  static __device__ __forceinline__ void mma(float (&d)[4],
                                             const uint32_t (&a)[4],
                                             uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

// ------------------------------------------------------------------- units
// The pages of a request that hold attended tokens: `units` of them, the
// first `front` at their own index, the others `gap` further on.  A request
// with none still has one unit, which writes its empty result.
struct Span {
  int32_t len, units, front, gap;
};
__device__ __forceinline__ Span span_of(const AttendParams& p, int r) {
  Span s;
  const int64_t room = (int64_t)p.max_blocks * kBlock;
  const int32_t len = max(__ldg(p.lens + r), 0);
  s.len = (int32_t)min((int64_t)len, room);
  const int32_t all = (int32_t)(((int64_t)s.len + kBlock - 1) / kBlock);
  s.front = all;
  s.gap = 0;
  if (p.window && (int64_t)p.sink + p.window < s.len) {
    s.front = (p.sink + kBlock - 1) / kBlock;     // sink < len: no overflow
    s.gap = max((s.len - p.window) / kBlock - s.front, 0);
  }
  s.units = max(all - s.gap, 1);
  return s;
}

// What a warp knows of a page in its ring.
struct __align__(16) UnitMeta {
  int32_t r;
  uint32_t sub;     // item within the request, and the bits below
  int32_t page;     // index in the request's table row
  int32_t len;
};
constexpr uint32_t kFirst = 1u << 31;   // first unit of its item
constexpr uint32_t kLast = 1u << 30;    // last unit of its item
constexpr uint32_t kSkip = 1u << 29;    // no page (bad id, empty request)
constexpr uint32_t kSubMask = kSkip - 1;

// A part of an item left by a warp: entry 0 of a warp holds the part of an
// item that ended in its run but began before it, entry 1 of one that goes
// on behind it.
struct __align__(8) PartRec {
  int64_t begin;    // first unit of the item, where kFirst is set
  int32_t r;
  uint32_t sub;     // kFirst: begun here; kLast: ended here
  int32_t present;  // 0, 1: in the warp's ring, 2: in its workspace slot
  int32_t pad;
};

template <int HD>
struct Smem {
  static constexpr int W = warps_of(HD), S = stages_of(HD);
  static constexpr int kBars = kRingBytes;
  static constexpr int kMeta = kBars + W * S * 8;
  static constexpr int kPrefix = kMeta + W * S * 16;
  static constexpr int kRecs = kPrefix + W * 32 * 8;
  static constexpr int kMisc = kRecs + W * 2 * (int)sizeof(PartRec);
  static constexpr int kBytes = kMisc + 128 + 1024;  // + alignment slack
};

// Heads of a column pair of a fragment: lane's columns 2 (lane & 3), + 1.
// Writes the rows of a tile pair's transposed accumulators: dims
// mt * 16 + {0, 8}, eight heads, scaled by inv (per column).
template <class T, int HD>
__device__ __forceinline__ void store_out_frag(const AttendParams& p, int r,
                                               int head0, int rows, int nt,
                                               int mt, const float (&c)[4],
                                               float inv0, float inv1) {
  const int lane = (int)lane_id(), gid = lane >> 2, tig = lane & 3;
  // the transpose puts head gid, channels 2 tig and 2 tig + 1 in a lane
  const uint32_t lo = transpose8(Elem<T>::pack(c[0] * inv0, c[1] * inv1));
  const uint32_t hi = transpose8(Elem<T>::pack(c[2] * inv0, c[3] * inv1));
  if (nt * 8 + gid < rows) {
    T* o = static_cast<T*>(p.out) + (int64_t)r * p.out_ld +
           (int64_t)(head0 + nt * 8 + gid) * HD + mt * 16 + tig * 2;
    *reinterpret_cast<uint32_t*>(o) = lo;
    *reinterpret_cast<uint32_t*>(o + 8) = hi;
  }
}

__device__ __forceinline__ float inverse(float l) {
  return l == 0.f ? 0.f : 1.f / l;
}
__device__ __forceinline__ float lse_of(float m, float l, float shift) {
  return l == 0.f ? -INFINITY : (m + (log2f(l) - shift)) * kLn2;
}
// What exponents are taken relative to: m, or 0 where no score is finite
// (so that 2^(-inf - base) is 0 and not NaN).
__device__ __forceinline__ float base_of(float m) {
  return m == -INFINITY ? 0.f : m;
}

__device__ __forceinline__ void head_range(const AttendParams& p,
                                           uint32_t sub, int* head0,
                                           int* rows) {
  const int j = (int)sub / p.tiles, t = (int)sub - j * p.tiles;
  *head0 = j * p.group + t * p.tile_heads;
  *rows = min(p.tile_heads, p.group - t * p.tile_heads);
}

// Sum of `n` parts (part(i): its slot) at one fragment position: o, and the
// joined m and l of its two columns.
template <int HD, int NT, class F>
__device__ __forceinline__ void join_parts(int n, int tile, F part,
                                           float (&o)[4], float (&m)[2],
                                           float (&l)[2]) {
  const int lane = (int)lane_id();
  const int col = (tile % NT) * 8 + (lane & 3) * 2;
  m[0] = m[1] = -INFINITY;
  for (int i = 0; i < n; ++i) {
    const float2 mi = *reinterpret_cast<const float2*>(
        part(i) + NT * 8 * HD + col);
    m[0] = fmaxf(m[0], mi.x);
    m[1] = fmaxf(m[1], mi.y);
  }
  const float b0 = base_of(m[0]), b1 = base_of(m[1]);
  l[0] = l[1] = 0.f;
  o[0] = o[1] = o[2] = o[3] = 0.f;
  for (int i = 0; i < n; ++i) {
    const float* s = part(i);
    const float2 mi = *reinterpret_cast<const float2*>(s + NT * 8 * HD + col);
    const float2 li =
        *reinterpret_cast<const float2*>(s + NT * 8 * (HD + 1) + col);
    const float4 x = *reinterpret_cast<const float4*>(s + (tile * 32 + lane) *
                                                              4);
    const float f0 = exp2_fast(mi.x - b0), f1 = exp2_fast(mi.y - b1);
    l[0] += li.x * f0;
    l[1] += li.y * f1;
    o[0] += x.x * f0;
    o[1] += x.y * f1;
    o[2] += x.z * f0;
    o[3] += x.w * f1;
  }
}

// Final values of an item from joined fragments: out and lse.
template <class T, int HD, int NT>
__device__ __forceinline__ void finish_item(const AttendParams& p, int r,
                                            uint32_t sub, int tile,
                                            const float (&o)[4],
                                            const float (&m)[2],
                                            const float (&l)[2]) {
  const int lane = (int)lane_id(), gid = lane >> 2, tig = lane & 3;
  const int mt = tile / NT, nt = tile % NT;
  int head0, rows;
  head_range(p, sub, &head0, &rows);
  store_out_frag<T, HD>(p, r, head0, rows, nt, mt, o, inverse(l[0]),
                        inverse(l[1]));
  if (p.lse && mt == 0 && gid == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int h = nt * 8 + tig * 2 + i;
      if (h < rows)
        p.lse[(int64_t)r * p.heads + head0 + h] = lse_of(m[i], l[i], Elem<T>::kShift);
    }
  }
}

// A joined part as a slot.
template <int HD, int NT>
__device__ __forceinline__ void store_part(float* slot, int tile,
                                           const float (&o)[4],
                                           const float (&m)[2],
                                           const float (&l)[2]) {
  const int lane = (int)lane_id();
  *reinterpret_cast<float4*>(slot + (tile * 32 + lane) * 4) =
      make_float4(o[0], o[1], o[2], o[3]);
  if (tile < NT && lane < 4) {
    const int col = tile * 8 + lane * 2;
    *reinterpret_cast<float2*>(slot + NT * 8 * HD + col) =
        make_float2(m[0], m[1]);
    *reinterpret_cast<float2*>(slot + NT * 8 * (HD + 1) + col) =
        make_float2(l[0], l[1]);
  }
}

// ------------------------------------------------------------------ kernel
// NT: tiles of eight query heads that a warp keeps.
template <class T, int HD, int NT>
__global__ void __launch_bounds__(warps_of(HD) * 32, 1)
    attend_kernel(const __grid_constant__ AttendParams p) {
  using L = Smem<HD>;
  constexpr int W = L::W, S = L::S, kThreads = W * 32;
  constexpr int MT = HD / 16;               // channel tiles of 16
  constexpr int kPage = HD * 32;            // bytes of one page of K or V
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars) + warp * S;
  UnitMeta* metas = reinterpret_cast<UnitMeta*>(smem + L::kMeta) + warp * S;
  int64_t* prefix = reinterpret_cast<int64_t*>(smem + L::kPrefix);
  PartRec* recs = reinterpret_cast<PartRec*>(smem + L::kRecs);
  int64_t* warp_sums = reinterpret_cast<int64_t*>(smem + L::kMisc);
  volatile int* abort_flag =
      reinterpret_cast<volatile int*>(smem + L::kMisc + 64);
  const int items = p.kv_heads * p.tiles;   // per request

  if (lane < S) mbar_init(bars + lane, 1);
  if (lane == 0) {
    recs[warp * 2].present = recs[warp * 2 + 1].present = 0;
    prefetch_tmap(&p.tm_k);
    prefetch_tmap(&p.tm_v);
  }
  if (tid == 0) *abort_flag = 0;
  fence_mbar_init();

  // Units of the requests before each thread's run of requests.
  const int per = (p.R + kThreads - 1) / kThreads;
  int64_t sum = 0;
  for (int i = 0; i < per; ++i) {
    const int r = tid * per + i;
    if (r >= p.R) break;
    sum += span_of(p, r).units;
    if (p.flags && blockIdx.x == 0 &&
        __ldg(p.lens + r) > (int64_t)p.max_blocks * kBlock)
      atomicOr(p.flags, KVTC_FLAG_SPACE);
  }
  int64_t upto = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) warp_sums[warp] = upto;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) upto += warp_sums[w];
    total += warp_sums[w];
  }
  prefix[tid] = (upto - sum) * items;
  total *= items;
  __syncthreads();

  // This warp's run of units, and the request that holds its first one.
  // Fewer units than warps leave blocks or warps out, so that every worker
  // has a unit and the parts of an item lie in consecutive blocks.
  const int64_t ctas = min(total, (int64_t)kCtas);
  const int64_t active = min(total / ctas, (int64_t)W);
  const int64_t workers = ctas * active;
  const int64_t worker = blockIdx.x * active + warp;
  const bool works = blockIdx.x < ctas && warp < active;
  const int64_t u0 = works ? worker * total / workers : 0;
  const int64_t u1 = works ? (worker + 1) * total / workers : 0;
  const int n = (int)(u1 - u0);
  int cur_r = 0;
  int64_t cur_s = 0;        // first unit of request cur_r
  if (n) {
    int lo = 0, hi = (p.R - 1) / per;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= u0) lo = mid; else hi = mid - 1;
    }
    cur_r = lo * per;
    cur_s = prefix[lo];
  }

  const uint32_t ring = smem_u32(smem) + warp * S * stage_bytes(HD);
  // Lane j's unit of the batch of 32 being issued.
  int b_r = 0, b_page = 0, b_len = 0, b_id = -1;
  uint32_t b_sub = 0;
  auto fill = [&](int i) {
    const int64_t u = u0 + i + lane;
    int r = cur_r;
    int64_t s = cur_s;
    if (u < u1) {
      Span sp = span_of(p, r);
      while (u >= s + (int64_t)sp.units * items) {
        s += (int64_t)sp.units * items;
        sp = span_of(p, ++r);
      }
      const int64_t o = u - s;
      const uint32_t sub = (o >> 32) ? (uint32_t)(o / sp.units)
                                     : (uint32_t)o / (uint32_t)sp.units;
      const int v = (int)(o - (int64_t)sub * sp.units);
      b_r = r;
      b_page = v < sp.front ? v : v + sp.gap;
      b_len = sp.len;
      b_sub = sub | (v == 0 ? kFirst : 0u) |
              (v == sp.units - 1 ? kLast : 0u);
      b_id = -1;
      if (sp.len) {
        b_id = __ldg(p.table + (int64_t)r * p.max_blocks + b_page);
        if (b_id < 0 || b_id >= p.num_blocks) {
          b_id = -1;
          if (p.flags) atomicOr(p.flags, KVTC_FLAG_BLOCK);
        }
      }
      if (b_id < 0) b_sub |= kSkip;
    }
    const int last = min(31, n - 1 - i);
    cur_r = __shfl_sync(0xFFFFFFFFu, r, last);
    cur_s = __shfl_sync(0xFFFFFFFFu, s, last);
  };
  auto issue = [&](int i) {
    if ((i & 31) == 0) fill(i);
    if (lane == (i & 31)) {
      const int st = i % S;
      UnitMeta m;
      m.r = b_r;
      m.sub = b_sub;
      m.page = b_page;
      m.len = b_len;
      metas[st] = m;
      if (b_sub & kSkip) {
        mbar_arrive(bars + st);
      } else {
        const int slab = (int)((b_sub & kSubMask) / p.tiles) * (HD / 64);
        const uint32_t dst = ring + st * stage_bytes(HD);
        mbar_arrive_expect_tx(bars + st, 2 * kPage);
        tma_load_page(dst, &p.tm_k, slab, b_id, bars + st);
        tma_load_page(dst + kPage, &p.tm_v, slab, b_id, bars + st);
      }
    }
    __syncwarp();
  };
  for (int i = 0; i < min(n, S); ++i) issue(i);

  // ldmatrix addresses inside a page: the row of this lane and its 128-byte
  // swizzle.  K: matrices (token half, chunk); V, transposed: (chunk, half).
  const uint32_t k_row = (lane & 7) + ((lane >> 3) & 1) * 8;
  const uint32_t v_row = (lane & 7) + (lane >> 4) * 8;
  const uint32_t swz = lane & 7;
  const uint32_t k_base = k_row * 128, v_base = v_row * 128;
  const uint32_t k_chunk = lane >> 4, v_chunk = (lane >> 3) & 1;

  uint32_t qf[MT][NT][2];
  float acc[MT][NT][4];
  float m_run[NT][2], l_run[NT][2];
  bool begun = false;          // the current item began in this run
  int64_t item_begin = 0;
  int pending = 0;             // kept across the loop for the drain below

  for (int c = 0; c < n; ++c) {
    const int st = c % S;
    if (!__all_sync(0xFFFFFFFFu,
                    mbar_wait(bars + st, (c / S) & 1, abort_flag))) {
      *abort_flag = 1;
      break;
    }
    pending = c + 1;
    const UnitMeta meta = metas[st];
    const uint32_t sub = meta.sub & kSubMask;
    if (c == 0 || (meta.sub & kFirst)) {
      begun = meta.sub & kFirst;
      item_begin = u0 + c;
      int head0, rows;
      head_range(p, sub, &head0, &rows);
      const T* q = static_cast<const T*>(p.q) + (int64_t)meta.r * p.q_ld +
                   (int64_t)head0 * HD;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const bool in = nt * 8 + gid < rows;
        const uint32_t* row = reinterpret_cast<const uint32_t*>(
            q + (int64_t)(nt * 8 + gid) * HD + tig * 2);
#pragma unroll
        for (int ks = 0; ks < MT; ++ks) {
          qf[ks][nt][0] = in ? __ldg(row + ks * 8) : 0u;
          qf[ks][nt][1] = in ? __ldg(row + ks * 8 + 4) : 0u;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[mt][nt][i] = 0.f;
        m_run[nt][0] = m_run[nt][1] = -INFINITY;
        l_run[nt][0] = l_run[nt][1] = 0.f;
      }
    }

    if (!(meta.sub & kSkip)) {
      const uint32_t kp = ring + st * stage_bytes(HD), vp = kp + kPage;
      float sc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < MT; ++ks) {
        uint32_t a[4];
        const uint32_t chunk = (ks & 3) * 2 + k_chunk;
        ldsm4(a, kp + (ks >> 2) * 2048 + k_base + ((chunk ^ swz) << 4));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          Elem<T>::mma(sc[nt], a, qf[ks][nt][0], qf[ks][nt][1]);
      }
      // tokens gid and gid + 8 of the page; columns are heads
      const int t0 = meta.page * kBlock;
      const int recent = p.window ? meta.len - p.window : 0;
      const bool whole =
          t0 + kBlock <= meta.len &&
          (t0 >= recent || (int64_t)t0 + kBlock <= p.sink);
      auto seen = [&](int t) {
        return t < meta.len && (t < p.sink || t >= recent);
      };
      const bool in0 = whole || seen(t0 + gid);
      const bool in1 = whole || seen(t0 + gid + 8);
      uint32_t ph[NT][2], pl[NT][2];
      bool grew = false;
      float alpha[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s[i] = (i < 2 ? in0 : in1) ? sc[nt][i] * p.scale_log2 : -INFINITY;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float mx = fmaxf(s[i], s[i + 2]);
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
          const float mn = fmaxf(m_run[nt][i], mx), base = base_of(mn);
          alpha[nt][i] = exp2_fast(m_run[nt][i] - base);
          grew |= mn != m_run[nt][i];
          m_run[nt][i] = mn;
          s[i] = exp2_fast(s[i] - (base - Elem<T>::kShift));
          s[i + 2] = exp2_fast(s[i + 2] - (base - Elem<T>::kShift));
          l_run[nt][i] = l_run[nt][i] * alpha[nt][i] + (s[i] + s[i + 2]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t hi = Elem<T>::pack_down(
              s[2 * h] * Elem<T>::kBelow, s[2 * h + 1] * Elem<T>::kBelow);
          const float2 f = Elem<T>::unpack(hi);
          const uint32_t lo =
              Elem<T>::pack(s[2 * h] - f.x, s[2 * h + 1] - f.y);
          ph[nt][h] = transpose8(hi);
          pl[nt][h] = transpose8(lo);
        }
      }
      if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[mt][nt][i] *= alpha[nt][i & 1];
      }
      auto pv = [&](auto masked) {
        // rows of V that are not attended may hold NaN: as zeros, 0 * 0
        uint32_t keep0 = 0xFFFFFFFFu, keep1 = 0xFFFFFFFFu;
        if (masked.value) {
          const int t = t0 + tig * 2;
          keep0 = (seen(t) ? 0xFFFFu : 0u) | (seen(t + 1) ? ~0xFFFFu : 0u);
          keep1 = (seen(t + 8) ? 0xFFFFu : 0u) | (seen(t + 9) ? ~0xFFFFu : 0u);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t a[4];
          const uint32_t chunk = (mt & 3) * 2 + v_chunk;
          ldsm4_trans(a, vp + (mt >> 2) * 2048 + v_base +
                             ((chunk ^ swz) << 4));
          if (masked.value) {
            a[0] &= keep0;
            a[1] &= keep0;
            a[2] &= keep1;
            a[3] &= keep1;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            Elem<T>::mma(acc[mt][nt], a, ph[nt][0], ph[nt][1]);
            Elem<T>::mma(acc[mt][nt], a, pl[nt][0], pl[nt][1]);
          }
        }
      };
      if (whole) pv(std::false_type{}); else pv(std::true_type{});
    }
    __syncwarp();
    if (c + S < n) issue(c + S);

    const bool ended = meta.sub & kLast;
    if (!ended && c + 1 < n) continue;
    // the sums over a head's tokens are still spread over the lanes
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1)
          l_run[nt][i] += __shfl_xor_sync(0xFFFFFFFFu, l_run[nt][i], d);
    if (begun && ended) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          finish_item<T, HD, NT>(p, meta.r, sub, mt * NT + nt, acc[mt][nt],
                                 m_run[nt], l_run[nt]);
      continue;
    }
    // a part: in the ring when the run ends with it (every page has been
    // read), else in the workspace
    const bool at_end = c + 1 == n;
    float* slot =
        at_end ? reinterpret_cast<float*>(smem + warp * S * stage_bytes(HD))
               : p.warp_slots + ((int64_t)blockIdx.x * W + warp) *
                                    slot_floats(HD, NT);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        store_part<HD, NT>(slot, mt * NT + nt, acc[mt][nt], m_run[nt],
                           l_run[nt]);
    if (lane == 0) {
      PartRec& rec = recs[warp * 2 + (ended ? 0 : 1)];
      rec.begin = item_begin;
      rec.r = meta.r;
      rec.sub = sub | (begun ? kFirst : 0u) | (ended ? kLast : 0u);
      rec.present = at_end ? 1 : 2;
    }
  }
  if (pending < n) {
    // a wait ran out: report it, and let the loads in flight land
    if (lane == 0 && p.flags) atomicOr(p.flags, KVTC_FLAG_TIMEOUT);
    for (int c = pending; c < min(n, pending + S); ++c)
      mbar_drain(bars + c % S, (c / S) & 1);
  }
  __syncthreads();

  // Join the block's parts: entries in order, those of one item together.
  auto entry = [&](int e) -> const float* {
    const int w = e >> 1;
    return recs[e].present == 1
               ? reinterpret_cast<const float*>(smem + w * S *
                                                           stage_bytes(HD))
               : p.warp_slots + ((int64_t)blockIdx.x * W + w) *
                                    slot_floats(HD, NT);
  };
  JoinDesc desc;
  desc.r = -1;
  desc.sub = desc.last_cta = desc.pad = 0;
  int e = 0;
  while (e < 2 * W) {
    if (!recs[e].present) {
      ++e;
      continue;
    }
    const PartRec first = recs[e];
    const uint32_t sub = first.sub & kSubMask;
    int list[W + 1], k = 0;
    uint32_t bits = first.sub & kFirst;
    for (; e < 2 * W; ++e) {
      if (!recs[e].present) continue;
      if (recs[e].r != first.r || (recs[e].sub & kSubMask) != sub) break;
      bits |= recs[e].sub & kLast;
      list[k++] = e;
    }
    for (int tile = warp; tile < MT * NT; tile += W) {
      float o[4], m[2], l[2];
      join_parts<HD, NT>(k, tile, [&](int i) { return entry(list[i]); }, o, m,
                         l);
      if (bits == (kFirst | kLast))
        finish_item<T, HD, NT>(p, first.r, sub, tile, o, m, l);
      else
        store_part<HD, NT>(p.cta_slots + ((int64_t)blockIdx.x * 2 +
                                          (bits & kFirst ? 1 : 0)) *
                                             slot_floats(HD, NT),
                           tile, o, m, l);
    }
    if (bits == kFirst) {
      // it ends in the block that holds its last unit
      desc.r = first.r;
      desc.sub = (int32_t)sub;
      const int64_t end = first.begin + span_of(p, first.r).units;
      desc.last_cta =
          (int)min((end * workers - 1) / total / active, ctas - 1);
    }
  }
  if (tid == 0) p.desc[blockIdx.x] = desc;
}

// Items that lie over several blocks: block c joins the one that began in
// block c of the attention, its own part and those of the blocks after it.
template <class T, int HD, int NT>
__global__ void __launch_bounds__(HD / 16 * NT * 32)
    attend_join_kernel(const __grid_constant__ AttendParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const JoinDesc d = p.desc[blockIdx.x];
  if (d.r < 0) return;
  const int c = blockIdx.x, tile = threadIdx.x >> 5;
  float o[4], m[2], l[2];
  join_parts<HD, NT>(
      d.last_cta - c + 1, tile,
      [&](int i) {
        return p.cta_slots + ((int64_t)(c + i) * 2 + (i == 0 ? 1 : 0)) *
                                 slot_floats(HD, NT);
      },
      o, m, l);
  finish_item<T, HD, NT>(p, d.r, (uint32_t)d.sub, tile, o, m, l);
}

template <class T, int HD, int NT>
cudaError_t launch_as(const AttendParams& p, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(
      attend_kernel<T, HD, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
      Smem<HD>::kBytes);
  if (e != cudaSuccess) return e;
  e = launch_kernel(attend_kernel<T, HD, NT>, kCtas, warps_of(HD) * 32,
                    Smem<HD>::kBytes, st, false, p);
  if (e != cudaSuccess) return e;
  count_launch();
  e = launch_kernel(attend_join_kernel<T, HD, NT>, kCtas, HD / 16 * NT * 32,
                    0, st, true, p);
  if (e == cudaSuccess) count_launch();
  return e;
}

// Tiles of eight query heads per warp: as many as the group needs, up to 32
// heads (16 at head_dim 256, where the accumulators of 32 heads would not
// fit the registers); larger groups are cut into equal tiles of heads, each
// of which reads the pages again (from L2, mostly).
int head_tiles(int head_dim, int group) {
  return group <= 8 ? 1 : group <= 16 || head_dim == 256 ? 2 : 4;
}

template <class T>
cudaError_t launch(const AttendParams& p, int head_dim, int nt,
                   cudaStream_t st) {
  if (head_dim == 64)
    return nt == 1   ? launch_as<T, 64, 1>(p, st)
           : nt == 2 ? launch_as<T, 64, 2>(p, st)
                     : launch_as<T, 64, 4>(p, st);
  if (head_dim == 128)
    return nt == 1   ? launch_as<T, 128, 1>(p, st)
           : nt == 2 ? launch_as<T, 128, 2>(p, st)
                     : launch_as<T, 128, 4>(p, st);
  return nt == 1 ? launch_as<T, 256, 1>(p, st) : launch_as<T, 256, 2>(p, st);
}

// A pool [num_blocks][16][D] as {64 channels, 16 tokens, D / 64, num_blocks}:
// a box is one block's rows of one head, as head_dim / 64 tiles [16][64].
bool encode_pages(CUtensorMap* m, const void* base, uint64_t D,
                  uint64_t num_blocks, uint32_t head_dim) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[4] = {64, kBlock, D / 64, num_blocks};
  cuuint64_t strides[3] = {D * 2, 128, D * 2 * kBlock};
  cuuint32_t box[4] = {64u, (cuuint32_t)kBlock, head_dim / 64, 1u};
  cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int64_t kDescBytes = (kCtas * sizeof(JoinDesc) + 255) / 256 * 256;

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
  if (st != KVTC_OK) return st;
  const int64_t slot =
      4 * slot_floats(head_dim, head_tiles(head_dim, heads / kv_heads));
  return kDescBytes + kCtas * (2 + warps_of(head_dim)) * slot;
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
  const uint64_t D = (uint64_t)kv_heads * head_dim;
  if (!encode_pages(&p.tm_k, k_cache, D, num_blocks, head_dim) ||
      !encode_pages(&p.tm_v, v_cache, D, num_blocks, head_dim))
    return KVTC_ECUDA;
  const int group = heads / kv_heads, nt = head_tiles(head_dim, group);
  p.q = q;
  p.table = block_table;
  p.lens = lens;
  p.out = out;
  p.lse = lse;
  p.flags = flags;
  p.desc = static_cast<JoinDesc*>(workspace);
  p.cta_slots = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                         kDescBytes);
  p.warp_slots = p.cta_slots + kCtas * 2 * slot_floats(head_dim, nt);
  p.q_ld = q_ld;
  p.out_ld = out_ld;
  p.num_blocks = num_blocks;
  p.scale_log2 = scale * kLog2e;
  p.R = R;
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.max_blocks = max_blocks;
  p.sink = window ? sink : 0;
  p.window = window;
  p.group = group;
  p.tiles = (group + 8 * nt - 1) / (8 * nt);
  p.tile_heads = (group + p.tiles - 1) / p.tiles;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = dtype == KVTC_DTYPE_BF16
                            ? launch<__nv_bfloat16>(p, head_dim, nt, st)
                            : launch<__half>(p, head_dim, nt, st);
  return e == cudaSuccess ? KVTC_OK : KVTC_ECUDA;
}

}  // extern "C"
