// Attention of one new token per request over paged K and V pools.
//
// For a query head, s_t = scale q.k_t over the attended tokens.  With a
// running reference m near the maximum, l = sum 2^(s_t - m) and o = sum
// 2^(s_t - m) v_t (s in units of log2) are multiplied by 2^(m_old - m_new)
// when m grows, so K and V are read once; partial results of disjoint tokens
// join the same way:
//     m = max m_i,  l = sum l_i 2^(m_i - m),  o = sum o_i 2^(m_i - m),
// and out = o / l, lse = (m + log2 l) ln 2.
//
// Work.  A request's tokens fall into pages of 16; an item is (request, KV
// head, tile of query heads), a unit one page of an item.  A warp takes a run
// of consecutive units, and writes an item that lies inside its run; of
// others it leaves a part.  The parts are joined in a fixed order (equal
// calls give equal bits), in one of two ways:
//   many items   all units of the call are dealt out to the warps of one
//                block per SM in equal runs, so that every SM reads at the
//                same rate whatever the lengths are (they are on the device:
//                each block sums them itself).  Parts are joined by the next
//                warp, by the block, and across blocks by attend_join_kernel
//                behind.
//   few items    a cluster of blocks takes one item and joins its parts
//                through distributed shared memory: one launch, and no
//                second round through L2.
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
//
// What bounds it.  HBM: each attended row of K and V is read once, at 4 heads
// flops a row element (50 TFLOP/s at eight query heads a KV head, a small
// part of what mma.sync gives).  While all warps have pages to ask for, the
// SMs read 7.8 TB/s together (570 MB, 16 requests up to 16K: 91 us in all,
// 6.3 TB/s); the rest is latency: 3 us until the first page (lengths, block
// table, page, one after the other), and after the last ones 4 us, more or
// less, of warps that end apart, 2 us of the block's join, 2 to 3 us of the
// launch behind.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
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
constexpr int kMaxTable = INT32_MAX / kBlock - 1;  // table columns: token
                                     // indices and a page more in 32 bits
constexpr int kCtas = 152;           // one block per SM
constexpr int kFewReq = 128;         // requests that each warp sums itself
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMaxScale = 0x1p127f;  // times log2 e still finite
constexpr float kSlack = 6.f;        // log2; see the reference in the loop

// Floats of a partial result of nt x 8 query heads: o in fragment order
// ([channel tile][head tile][lane][4]), then m and l per head.
__host__ __device__ constexpr int slot_floats(int hd, int nt) {
  return nt * 8 * (hd + 2);
}
// Warps per block, for nt tiles of eight query heads per warp: as many as
// registers and shared memory hold (a cluster's blocks need less of it), with
// one page each in flight (two where 12 or fewer warps read the small pages
// of head_dim 64).  More warps with one page mostly beat fewer with two: 64
// requests up to 4K at head_dim 128, 12 x 1 against 9 x 2: 48.5 and 49.7 us;
// 64 of 2K to 4K at head_dim 64 (8 KV heads), 16 x 1 against 12 x 2: 73.0 and
// 74.4 (32 of 4K to 8K, 4 KV heads: 40.0 and 38.3).  At head_dim 256 two head
// tiles' accumulators and queries alone are 192 registers: that form spills
// (255 registers, 172 bytes stored and 156 loaded a thread; in a cluster 24
// and 12).
__host__ __device__ constexpr int warps_of(int hd, int nt, bool cluster) {
  return hd == 64    ? (nt == 1 ? 16 : nt == 2 ? 12 : 8)
         : hd == 128 ? (nt == 1 ? (cluster ? 14 : 12) : 8)
                     : (cluster ? 8 : nt == 1 ? 7 : 5);
}
__host__ __device__ constexpr int stages_of(int hd, int nt) {
  return hd == 64 && nt > 1 ? 2 : 1;
}
__host__ __device__ constexpr int page_bytes(int hd) { return hd * 2 * kBlock; }
__host__ __device__ constexpr int query_bytes(int hd, int nt) {
  return nt * 16 * hd;
}

// Where the join finds the parts of an item that began in a block and did
// not end there; r < 0: there is none.
struct __align__(16) JoinDesc {
  int32_t r, sub, last_cta, pad;
};

struct AttendParams {
  // a pool as {64, 16, D / 64, num_blocks}: a page of a head, box {64, 16,
  // head_dim / 64, 1}, and 64 channels of half a page, box {64, 8, 1, 1}
  CUtensorMap tm_k, tm_v, tm_k8, tm_v8;
  const void* q;
  const int32_t* table;
  const int32_t* lens;
  void* out;
  float* lse;
  unsigned* flags;
  JoinDesc* desc;           // [kCtas]
  float* cta_slots;         // [kCtas][2] parts that cross blocks: 0 of an
                            // item begun in an earlier block, 1 in this one
  int64_t q_ld, out_ld, num_blocks;
  float scale_log2;
  int32_t R, heads, kv_heads, max_blocks, sink, window;
  int32_t group, tiles, tile_heads;  // heads per KV head; tiles of them
  uint32_t tiles_inv;                // 2^16 / tiles, rounded up
};

// ------------------------------------------------------------ PTX wrappers
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}
__device__ __forceinline__ uint32_t cluster_id() {    // in x
  uint32_t n;
  asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(n));
  return n;
}
__device__ __forceinline__ void tma_load_box(uint32_t smem_dst,
                                             const void* tmap, int32_t row,
                                             int32_t slab, int32_t block,
                                             uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_"
      "tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_dst),
      "l"(tmap), "r"(0), "r"(row), "r"(slab), "r"(block), "r"(smem_u32(bar))
      : "memory");
}
// Bulk copy global -> shared (both 16-byte aligned, bytes % 16 == 0).
__device__ __forceinline__ void bulk_load(uint32_t smem_dst, const void* src,
                                          uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1], %2, [%3];" ::"r"(smem_dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
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

// Loads from this block's shared memory, or from that of the cluster's blocks
// (which takes several times as long, for an own address too).
template <bool across>
__device__ __forceinline__ float2 lds2(uint32_t addr) {
  float2 v;
  if (across)
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(addr)
                 : "memory");
  return v;
}
template <bool across>
__device__ __forceinline__ float4 lds4(uint32_t addr) {
  float4 v;
  if (across)
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
  return v;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The two element types: conversion, packing (a in the low half) and
// D (16 x 8, fp32) += A (16 x 16) B (16 x 8).
//
// A weight w > 0 enters the product with V as hi + lo, hi = w kBelow cut to
// 16 bits and lo = w - hi (exact) rounded to 16 bits: w to 2^-15, and both
// terms positive, so that an infinite v gives an infinity and not inf - inf
// or 0 inf.  fp16 holds numbers from 2^-24: there weights are formed 2^9
// times as large, and what is lost lies 2^-33 below the largest.
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
  static constexpr float kShift = 9.f;    // weights up to 2^15
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
  bool hole;      // tokens between the sink and the window are left out
};
__device__ __forceinline__ Span span_of_len(const AttendParams& p,
                                            int32_t len) {
  Span s;       // (kMaxTable keeps all of this inside 32 bits)
  s.len = min(max(len, 0), p.max_blocks * kBlock);
  const int32_t all = (s.len + kBlock - 1) / kBlock;
  s.front = all;
  s.gap = 0;
  s.hole = p.window && (uint32_t)p.sink + p.window < (uint32_t)s.len;
  if (s.hole) {
    s.front = (p.sink + kBlock - 1) / kBlock;
    s.gap = max((s.len - p.window) / kBlock - s.front, 0);
  }
  s.units = max(all - s.gap, 1);
  return s;
}
__device__ __forceinline__ Span span_of(const AttendParams& p, int r) {
  return span_of_len(p, p.lens[r]);
}

// a / b and the remainder, for a quotient below 2^20 (a float quotient is
// then off by less than one): a 64-bit division is a hundred instructions.
__device__ __forceinline__ int small_quotient(int64_t a, int32_t b,
                                              int32_t* rest) {
  int q = (int)((float)a / (float)b);
  int64_t left = a - (int64_t)q * b;
  if (left < 0) {
    --q;
    left += b;
  } else if (left >= b) {
    ++q;
    left -= b;
  }
  *rest = (int32_t)left;
  return q;
}
// `total` units in order over the warps of the first `ctas` of `most` blocks:
// the first `more` warps take least + 1 units, the others `least`.  With few
// units, blocks are left out until every warp has one.  (With two a warp or
// more, one request of 1K, 32 heads on 8 of 128, took 9.3 us, not 8.1.)
template <int W>
struct Deal {
  int64_t least;
  int32_t more, ctas;
  __device__ __forceinline__ Deal(int64_t total, int most) {
    if (most == kCtas && total >= kCtas * W) {
      ctas = kCtas;
      least = total / (kCtas * W);       // by a constant
    } else {
      // (a cluster's item has less than 2^28 units)
      ctas = max(1, min(most, (int32_t)total / W));
      least = (uint32_t)total / (uint32_t)(ctas * W);
    }
    more = (int32_t)(total - least * (ctas * W));
  }
  __device__ __forceinline__ int64_t begin(int worker) const {
    return worker * least + min(worker, more);
  }
  // The block that holds a unit (the whole warp asks).
  __device__ __forceinline__ int cta_of(int64_t unit) const {
    int upto = 0;
    for (int i = 0; i < ctas; i += 32) {
      const int c = i + (int)lane_id();
      upto += __popc(__ballot_sync(0xFFFFFFFFu,
                                   c < ctas && begin(c * W) <= unit));
    }
    return upto - 1;
  }
};

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
constexpr uint32_t kWhole = 1u << 28;   // all 16 tokens are attended
constexpr uint32_t kNoLow = 1u << 27;   // none of the first eight is
constexpr uint32_t kNoHigh = 1u << 26;  // none of the last eight is
constexpr uint32_t kSubMask = kNoHigh - 1;

// A part of an item left by a warp: entry 0 of a warp is of an item that
// ended in its run but began before it (in the slot beside the ring), entry
// 1 of one that goes on behind it (in the ring, when every page is read).
struct __align__(16) PartRec {
  int64_t begin;    // first unit of the item, where kFirst is set
  int32_t r;        // < 0: there is no such part
  uint32_t sub;     // kFirst: begun here; kLast: ended here
};

template <int HD, int NT, bool kCluster>
struct Smem {
  static constexpr int W = warps_of(HD, NT, kCluster);
  static constexpr int S = stages_of(HD, NT);
  static constexpr int kSlot = 4 * slot_floats(HD, NT);
  static constexpr int kStage = 2 * page_bytes(HD);   // a page of K, one of V
  // A warp's ring of pages; when the last has been read, a part lies there.
  static constexpr int kRing =
      S * kStage >= kSlot ? S * kStage : (kSlot + 1023) / 1024 * 1024;
  // Queries of the pages in the ring that begin an item (in a cluster each
  // warp loads its one item's itself).
  static constexpr int kQueries = kCluster ? 0 : S;
  static constexpr int kQuery = W * kRing;
  // Parts of items that end inside a run (in a cluster there are none).
  static constexpr int kParts = kQuery + W * kQueries * query_bytes(HD, NT);
  static constexpr int kBlockPart = kParts + (kCluster ? 0 : W * kSlot);
  static constexpr int kRecs = kBlockPart + kSlot;
  static_assert(2 * W <= 32, "a warp's lanes hold the block's part records");
  static constexpr int kMeta = kRecs + W * 2 * (int)sizeof(PartRec);
  static constexpr int kBars = kMeta + W * S * (int)sizeof(UnitMeta);
  static constexpr int kPrefix = kBars + W * S * 16;
  static constexpr int kMisc = kPrefix + W * 32 * 8;
  static constexpr int kBytes = kMisc + 320 + 1024;  // + alignment slack
  static_assert(kBytes <= 232448, "shared memory of a block");
};

// What exponents are taken relative to: m, or 0 where no score is finite
// (so that 2^(-inf - base) is 0 and not NaN).
__device__ __forceinline__ float base_of(float m) {
  return m == -INFINITY ? 0.f : m;
}
// An item's KV head: sub / tiles, by a reciprocal of 16 bits.  (Items per
// request are at most 128 KV heads x 8 tiles: its error of at most 7 in 2^16
// stays below 1 / tiles.  A division would be 20 instructions to fetch.)
__device__ __forceinline__ int kv_head_of(const AttendParams& p,
                                          uint32_t sub) {
  return (int)((sub * p.tiles_inv) >> 16);
}
// The query heads of an item.
struct Heads {
  int first, rows;
  __device__ __forceinline__ Heads(const AttendParams& p, uint32_t sub) {
    const int j = kv_head_of(p, sub);
    const int t = (int)sub - j * p.tiles;
    first = j * p.group + t * p.tile_heads;
    rows = min(p.tile_heads, p.group - t * p.tile_heads);
  }
};

// Where an item's result goes.
template <class T>
struct Target {
  T* out;           // its first head
  float* lse;       // or null
  int rows;         // heads
  __device__ __forceinline__ Target(const AttendParams& p, int r,
                                    uint32_t sub, int hd) {
    const Heads h(p, sub);
    rows = h.rows;
    out = static_cast<T*>(p.out) + (int64_t)r * p.out_ld +
          (int64_t)h.first * hd;
    lse = p.lse ? p.lse + (int64_t)r * p.heads + h.first : nullptr;
  }
  // Lane: columns (heads) 2 (lane & 3) and + 1 of head tile nt.  The
  // accumulators o of channel tile mt (rows lane / 4 and + 8) times inv.
  template <int HD>
  __device__ __forceinline__ void store(int nt, int mt, const float (&o)[4],
                                        const float (&inv)[2]) const {
    const int lane = (int)lane_id(), gid = lane >> 2, tig = lane & 3;
    // the transpose puts head gid, channels 2 tig and 2 tig + 1 in a lane
    const uint32_t lo =
        transpose8(Elem<T>::pack(o[0] * inv[0], o[1] * inv[1]));
    const uint32_t hi =
        transpose8(Elem<T>::pack(o[2] * inv[0], o[3] * inv[1]));
    if (nt * 8 + gid < rows) {
      T* to = out + (nt * 8 + gid) * HD + mt * 16 + tig * 2;
      *reinterpret_cast<uint32_t*>(to) = lo;
      *reinterpret_cast<uint32_t*>(to + 8) = hi;
    }
  }
  __device__ __forceinline__ void store_lse(int nt, const float (&m)[2],
                                            const float (&l)[2]) const {
    const int lane = (int)lane_id(), h = nt * 8 + lane * 2;
    if (!lse || lane >= 4) return;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (h + i < rows)
        lse[h + i] = l[i] == 0.f
                         ? -INFINITY
                         : (m[i] + (log2f(l[i]) - Elem<T>::kShift)) * kLn2;
  }
};
// 1 / l; 0 for the empty sum.  (l >= 1 otherwise: some token's weight was 1
// when the reference was its score, and a part's factor of 2^-126 or less
// leaves nothing of it beside the largest part.)
__device__ __forceinline__ float inverse(float l) {
  return l == 0.f ? 0.f : rcp_fast(l);
}

// A part as a slot.
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

// Join n parts in shared memory, part i at at(i) (of this block or `across`
// the cluster's), kTiles channel tiles at a time (place, place + step, ...):
// into the result, or where `to` is given into a slot.  kBatch parts are
// loaded at once; more would only lengthen code that runs once a call and has
// to be fetched.  The sums are spelled out so that the same two parts give
// the same bits here and where a warp joins them in its registers.
template <class T, int HD, int NT, int kTiles, int kBatch, bool across,
          class F>
__device__ __forceinline__ void join_parts(int n, F at,
                                           const Target<T>& target, float* to,
                                           int place, int step) {
  constexpr int kPlaces = HD / 16 / kTiles;     // of a head tile
  const int lane = (int)lane_id();
#pragma unroll 1
  for (; place < kPlaces * NT; place += step) {
    const int nt = place / kPlaces, mt = place % kPlaces * kTiles;
    const uint32_t stat = (NT * 8 * HD + nt * 8 + (lane & 3) * 2) * 4;
    const uint32_t frag = ((mt * NT + nt) * 32 + lane) * 16;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[kTiles][4] = {};
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kBatch) {
      float2 mi[kBatch], li[kBatch];
      float4 oi[kBatch][kTiles];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const uint32_t slot = at(min(i0 + b, n - 1));
        mi[b] = lds2<across>(slot + stat);
        li[b] = lds2<across>(slot + stat + NT * 32);
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
          oi[b][t] = lds4<across>(slot + frag + t * NT * 512);
      }
      float mn[2] = {m[0], m[1]};
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {    // (the last one may come twice)
        mn[0] = fmaxf(mn[0], mi[b].x);
        mn[1] = fmaxf(mn[1], mi[b].y);
      }
      const float base[2] = {base_of(mn[0]), base_of(mn[1])};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float f = exp2_fast(m[c] - base[c]);
        m[c] = mn[c];
        l[c] = __fmul_rn(l[c], f);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          o[t][c] = __fmul_rn(o[t][c], f);
          o[t][c + 2] = __fmul_rn(o[t][c + 2], f);
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (i0 + b < n) {
          const float f0 = exp2_fast(mi[b].x - base[0]);
          const float f1 = exp2_fast(mi[b].y - base[1]);
          l[0] = __fmaf_rn(li[b].x, f0, l[0]);
          l[1] = __fmaf_rn(li[b].y, f1, l[1]);
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            o[t][0] = __fmaf_rn(oi[b][t].x, f0, o[t][0]);
            o[t][1] = __fmaf_rn(oi[b][t].y, f1, o[t][1]);
            o[t][2] = __fmaf_rn(oi[b][t].z, f0, o[t][2]);
            o[t][3] = __fmaf_rn(oi[b][t].w, f1, o[t][3]);
          }
        }
      }
    }
    if (to) {
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
        store_part<HD, NT>(to, (mt + t) * NT + nt, o[t], m, l);
    } else {
      const float inv[2] = {inverse(l[0]), inverse(l[1])};
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
        target.template store<HD>(nt, mt + t, o[t], inv);
      if (mt == 0) target.store_lse(nt, m, l);
    }
  }
}

// ------------------------------------------------------------------ kernel
// NT: tiles of eight query heads that a warp keeps.  kCluster: a cluster of
// blocks takes one item, else all items are dealt out to kCtas blocks.
template <class T, int HD, int NT, bool kCluster>
__global__ void __launch_bounds__(warps_of(HD, NT, kCluster) * 32, 1)
    attend_kernel(const __grid_constant__ AttendParams p) {
  using L = Smem<HD, NT, kCluster>;
  constexpr int W = L::W, S = L::S, kThreads = W * 32;
  constexpr int MT = HD / 16;               // channel tiles of 16
  constexpr int kPage = page_bytes(HD);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  // a barrier for K and the queries of each page in the ring, one for V
  uint64_t* k_bars = reinterpret_cast<uint64_t*>(smem + L::kBars) +
                     warp * 2 * S;
  uint64_t* v_bars = k_bars + S;
  UnitMeta* metas = reinterpret_cast<UnitMeta*>(smem + L::kMeta) + warp * S;
  int64_t* prefix = reinterpret_cast<int64_t*>(smem + L::kPrefix);
  PartRec* recs = reinterpret_cast<PartRec*>(smem + L::kRecs);
  // where a warp leaves its part of an item: one that goes on behind its run
  // (1), or one that ended in it (0)
  auto slot_at = [&](int w, int goes_on) {
    return goes_on || kCluster ? w * L::kRing : L::kParts + w * L::kSlot;
  };
  int64_t* warp_sums = reinterpret_cast<int64_t*>(smem + L::kMisc);
  volatile int* abort_flag =
      reinterpret_cast<volatile int*>(smem + L::kMisc + 128);
  volatile int* heads_ready =      // [W] entry 0 of the warp is complete
      reinterpret_cast<volatile int*>(smem + L::kMisc + 192);
  const int items = p.kv_heads * p.tiles;   // per request

  // the next launch's blocks may take their places: they wait for this grid
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (lane < 2 * S) mbar_init(k_bars + lane, 1);
  if (lane == 0) {
    recs[warp * 2].r = recs[warp * 2 + 1].r = -1;
    heads_ready[warp] = 0;
    prefetch_tmap(&p.tm_k);
    prefetch_tmap(&p.tm_v);
  }
  if (tid == 0) *abort_flag = 0;
  fence_mbar_init();
  __syncthreads();
  // Everything this call reads may come from the launch before it, and is
  // read by plain loads: this grid may have started under that one, so the
  // read-only path could hold what it held before.
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // This warp's run of units, and the request that holds its first one.
  const bool few = p.R <= kFewReq;
  const int per = few ? (p.R + 31) / 32 : (p.R + kThreads - 1) / kThreads;
  int64_t total, ahead = 0;    // ahead: units before this lane's requests
  int most = kCtas, rank = blockIdx.x, cur_r = 0;
  uint32_t fixed_sub = 0;
  if (kCluster) {
    most = (int)cluster_size();
    rank = (int)cluster_ctarank();
    cur_r = blockIdx.y;
    fixed_sub = cluster_id();
    total = span_of(p, cur_r).units;
    if (tid == 0 && p.flags &&
        p.lens[cur_r] > p.max_blocks * kBlock)
      atomicOr(p.flags, KVTC_FLAG_SPACE);
  } else if (few) {
    // Every warp sums them itself, `per` requests a lane: no barrier, and the
    // loop is kept short, as the code has to be fetched (64 requests up to 4K
    // 48.1 us, by the block below 48.5; but 256 windows 34.9 and 34.3).
    int32_t len[kFewReq / 32];
#pragma unroll
    for (int i = 0; i < kFewReq / 32; ++i) {
      const int r = lane * per + i;
      len[i] = i < per && r < p.R ? p.lens[r] : -1;
    }
    int64_t sum = 0;
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
      if (lane * per + i < p.R) sum += span_of_len(p, len[0]).units;
      if (p.flags && blockIdx.x == 0 && warp == 0 &&
          len[0] > p.max_blocks * kBlock)
        atomicOr(p.flags, KVTC_FLAG_SPACE);
#pragma unroll
      for (int j = 1; j < kFewReq / 32; ++j) len[j - 1] = len[j];
    }
    total = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xFFFFFFFFu, total, d);
      if (lane >= d) total += o;
    }
    ahead = (total - sum) * items;
    total = __shfl_sync(0xFFFFFFFFu, total, 31) * items;
  } else {
    // Units of the requests before each thread's run of requests.
    int64_t sum = 0;
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
      const int r = tid * per + i;
      if (r >= p.R) break;
      sum += span_of(p, r).units;
      if (p.flags && blockIdx.x == 0 &&
          p.lens[r] > p.max_blocks * kBlock)
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
    total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < warp) upto += warp_sums[w];
      total += warp_sums[w];
    }
    prefix[tid] = (upto - sum) * items;
    total *= items;
    __syncthreads();
  }
  const Deal<W> deal(total, most);
  const int worker = rank * W + warp;
  const bool works = rank < deal.ctas;
  const int64_t u0 = works ? deal.begin(worker) : 0;
  const int64_t u1 = works ? deal.begin(worker + 1) : 0;
  const int n = (int)(u1 - u0);
  int64_t cur_s = 0;        // first unit of request cur_r
  if (!kCluster && few && n) {
    const int l = 31 - __clz(__ballot_sync(
                           0xFFFFFFFFu, lane * per < p.R && ahead <= u0));
    cur_r = l * per;
    cur_s = __shfl_sync(0xFFFFFFFFu, ahead, l);
  } else if (!kCluster && n) {
    int before = 0;         // runs of requests that begin at or before u0
#pragma unroll
    for (int i = 0; i < W; ++i)
      before += __popc(__ballot_sync(
          0xFFFFFFFFu, (i * 32 + lane) * per < p.R &&
                           prefix[i * 32 + lane] <= u0));
    cur_r = (before - 1) * per;
    cur_s = prefix[before - 1];
  }

  const uint32_t ring = smem_u32(smem) + warp * L::kRing;
  const uint32_t queries = smem_u32(smem) + L::kQuery +
                           warp * L::kQueries * query_bytes(HD, NT);
  // Lane j's unit of the batch of 32 being issued.
  int b_r = 0, b_page = 0, b_len = 0, b_id = -1, b_slab = 0;
  uint32_t b_sub = 0;
  auto fill = [&](int i) {
    const int64_t u = u0 + i + lane;
    int r = cur_r;
    int64_t s = cur_s;
    if (u < u1) {
      Span sp = span_of(p, r);
      int v = (int)u;
      uint32_t sub = fixed_sub;
      if (!kCluster) {
        while (u >= s + (int64_t)sp.units * items) {
          s += (int64_t)sp.units * items;
          sp = span_of(p, ++r);
        }
        sub = small_quotient(u - s, sp.units, &v);
      }
      b_r = r;
      b_page = v < sp.front ? v : v + sp.gap;
      b_len = sp.len;
      b_sub = sub | (v == 0 ? kFirst : 0u) |
              (v == sp.units - 1 ? kLast : 0u);
      b_id = -1;
      if (sp.len) {
        b_id = p.table[(int64_t)r * p.max_blocks + b_page];
        if ((uint32_t)b_id >= (uint32_t)p.num_blocks) {
          b_id = -1;
          if (p.flags) atomicOr(p.flags, KVTC_FLAG_BLOCK);
        }
      }
      if (b_id < 0) b_sub |= kSkip;
      const int t0 = b_page * kBlock, recent = sp.hole ? sp.len - p.window : 0;
      if (sp.len - t0 >= kBlock &&
          (t0 >= recent || t0 + kBlock <= p.sink))
        b_sub |= kWhole;
      // (a cluster's items are few: it is not worth their code there)
      if (!kCluster && t0 + 8 <= recent && t0 >= p.sink) b_sub |= kNoLow;
      if (!kCluster &&
          (t0 + 8 >= sp.len || (t0 + 16 <= recent && t0 + 8 >= p.sink)))
        b_sub |= kNoHigh;
    }
    const int last = min(31, n - 1 - i);
    cur_r = __shfl_sync(0xFFFFFFFFu, r, last);
    cur_s = __shfl_sync(0xFFFFFFFFu, s, last);
  };
  // What is attended of a page: it whole, or half of it.
  auto page_loads = [&]() {
    return b_sub & kSkip ? 0
           : !kCluster && (b_sub & (kNoLow | kNoHigh)) ? kPage / 2
                                                       : kPage;
  };
  auto load_page = [&](uint32_t dst, const CUtensorMap& whole,
                       const CUtensorMap& half, uint64_t* bar) {
    if (kCluster || !(b_sub & (kNoLow | kNoHigh))) {
      tma_load_box(dst, &whole, 0, b_slab, b_id, bar);
    } else {
      const int row = b_sub & kNoLow ? 8 : 0;
#pragma unroll
      for (int i = 0; i < HD / 64; ++i)
        tma_load_box(dst + i * 2048 + row * 128, &half, row, b_slab + i, b_id,
                     bar);
    }
  };
  auto issue_k = [&](int i, int st) {
    if ((i & 31) == 0) fill(i);
    if (lane == (i & 31)) {
      UnitMeta m;
      m.r = b_r;
      m.sub = b_sub;
      m.page = b_page;
      m.len = b_len;
      metas[st] = m;
      const uint32_t sub = b_sub & kSubMask;
      const uint32_t page = page_loads();
      const uint32_t dst = ring + st * L::kStage;
      b_slab = kv_head_of(p, sub) * (HD / 64);
      if (!kCluster && (i == 0 || (b_sub & kFirst))) {
        // the rows of an item's query heads are consecutive
        const Heads h(p, sub);
        const uint32_t bytes = (uint32_t)h.rows * HD * 2;
        mbar_arrive_expect_tx(k_bars + st, bytes + page);
        bulk_load(queries + st * query_bytes(HD, NT),
                  static_cast<const T*>(p.q) + (int64_t)b_r * p.q_ld +
                      (int64_t)h.first * HD,
                  bytes, k_bars + st);
      } else if (page) {
        mbar_arrive_expect_tx(k_bars + st, page);
      } else {
        mbar_arrive(k_bars + st);
      }
      if (page) load_page(dst, p.tm_k, p.tm_k8, k_bars + st);
    }
    __syncwarp();
  };
  auto issue_v = [&](int i, int st) {
    if (lane == (i & 31)) {
      const uint32_t page = page_loads();
      if (!page) {
        mbar_arrive(v_bars + st);
      } else {
        mbar_arrive_expect_tx(v_bars + st, page);
        load_page(ring + st * L::kStage + kPage, p.tm_v, p.tm_v8,
                  v_bars + st);
      }
    }
  };

  // ldmatrix addresses inside a page: the row of this lane and its 128-byte
  // swizzle.  K: matrices (token half, chunk); V, transposed: (chunk, half).
  const uint32_t k_row = (lane & 7) + ((lane >> 3) & 1) * 8;
  const uint32_t v_row = (lane & 7) + (lane >> 4) * 8;
  const uint32_t swz = lane & 7;
  const uint32_t k_base = k_row * 128, v_base = v_row * 128;
  const uint32_t k_chunk = lane >> 4, v_chunk = (lane >> 3) & 1;

  uint32_t qf[MT][NT][2];
  float acc[MT][NT][4];
  float m_run[NT][2], limit[NT][2], l_run[NT][2];
  bool begun = false;          // the current item began in this run
  int64_t item_begin = 0;
  int k_used = 0, v_used = 0;  // pages waited for

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok =
        __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag));
    if (!ok) *abort_flag = 1;
    return ok;
  };

  // Turn c uses unit c and asks for unit c + S in its place, for K as soon as
  // the scores are formed and for V at the end; the first S turns only ask.
  int st = S - 1;
  uint32_t phase = 0;
  UnitMeta meta = {0, 0u, 0, 0};
  float sc[NT][4];
  for (int c = n ? -S : 0; c < n; ++c) {
    if (++st == S) {
      st = 0;
      phase ^= 1;
    }
    const uint32_t kp = ring + st * L::kStage, vp = kp + kPage;
    if (c >= 0) {
      meta = metas[st];
      if (kCluster && c == 0) {
        // (these loads are under way while the page is waited for)
        const Heads h(p, fixed_sub);
        const T* q = static_cast<const T*>(p.q) + (int64_t)cur_r * p.q_ld +
                     (int64_t)h.first * HD;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const bool in = nt * 8 + gid < h.rows;
          const uint32_t* row = reinterpret_cast<const uint32_t*>(
              q + (int64_t)(nt * 8 + gid) * HD + tig * 2);
#pragma unroll
          for (int ks = 0; ks < MT; ++ks) {
            qf[ks][nt][0] = in ? row[ks * 8] : 0u;
            qf[ks][nt][1] = in ? row[ks * 8 + 4] : 0u;
          }
        }
      }
      if (!wait(k_bars + st, phase)) break;
      k_used = c + 1;
    }
    if (c >= 0 && (c == 0 || (meta.sub & kFirst))) {
      begun = meta.sub & kFirst;
      item_begin = u0 + c;
      const int rows = Heads(p, meta.sub & kSubMask).rows;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const bool in = nt * 8 + gid < rows;
#pragma unroll
        for (int ks = 0; !kCluster && ks < MT; ks += 2) {
          uint32_t b[4];
          ldsm4(b, queries + st * query_bytes(HD, NT) +
                       (nt * 8 + (lane & 7)) * (HD * 2) + ks * 32 +
                       (lane >> 3) * 16);
          qf[ks][nt][0] = in ? b[0] : 0u;
          qf[ks][nt][1] = in ? b[1] : 0u;
          qf[ks + 1][nt][0] = in ? b[2] : 0u;
          qf[ks + 1][nt][1] = in ? b[3] : 0u;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[mt][nt][i] = 0.f;
        m_run[nt][0] = m_run[nt][1] = -INFINITY;
        limit[nt][0] = limit[nt][1] = -INFINITY;
        l_run[nt][0] = l_run[nt][1] = 0.f;
      }
    }
    const bool use = c >= 0 && !(meta.sub & kSkip);
    if (use) {
      // S^T, in two chains where there is one head tile
      constexpr int kChains = NT == 1 ? 2 : 1;
      float sd[4] = {0.f, 0.f, 0.f, 0.f};
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
          Elem<T>::mma(kChains == 2 && (ks & 1) ? sd : sc[nt], a,
                       qf[ks][nt][0], qf[ks][nt][1]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sc[nt][i] = (kChains == 2 ? sc[nt][i] + sd[i] : sc[nt][i]) *
                      p.scale_log2;
    }
    __syncwarp();
    if (c + S < n) issue_k(c + S, st);
    if (use) {
      const bool whole = meta.sub & kWhole;
      const int t0 = meta.page * kBlock;
      const int recent = p.window ? meta.len - p.window : 0;
      auto seen = [&](int t) {
        return t < meta.len && (t < p.sink || t >= recent);
      };
      // tokens gid and gid + 8 of the page; columns are heads
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!whole && !seen(t0 + gid + (i >> 1) * 8))
            sc[nt][i] = -INFINITY;
      // The reference that exponents are taken from moves only when a score
      // lies kSlack above it: the maximum over the lanes (six shuffles in
      // chains of three) and the rescaling are seldom needed.
      bool above = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          above |= sc[nt][i] > limit[nt][i & 1];
      if (__any_sync(0xFFFFFFFFu, above)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float mx = fmaxf(sc[nt][i], sc[nt][i + 2]);
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
            const float mn = fmaxf(m_run[nt][i], mx);
            const float alpha = exp2_fast(m_run[nt][i] - base_of(mn));
            m_run[nt][i] = mn;
            limit[nt][i] = mn + kSlack;
            l_run[nt][i] *= alpha;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              acc[mt][nt][i] *= alpha;
              acc[mt][nt][i + 2] *= alpha;
            }
          }
      }
      uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = exp2_fast(sc[nt][i] -
                           (base_of(m_run[nt][i & 1]) - Elem<T>::kShift));
        l_run[nt][0] += w[0] + w[2];
        l_run[nt][1] += w[1] + w[3];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t hi = Elem<T>::pack_down(
              w[2 * h] * Elem<T>::kBelow, w[2 * h + 1] * Elem<T>::kBelow);
          const float2 f = Elem<T>::unpack(hi);
          const uint32_t lo =
              Elem<T>::pack(w[2 * h] - f.x, w[2 * h + 1] - f.y);
          ph[nt][h] = transpose8(hi);
          pl[nt][h] = transpose8(lo);
        }
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
      if (!wait(v_bars + st, phase)) break;
      if (whole) pv(std::false_type{}); else pv(std::true_type{});
    }
    __syncwarp();
    if (c + S < n) issue_v(c + S, st);
    if (c < 0) continue;
    v_used = c + 1;

    const uint32_t sub = meta.sub & kSubMask;
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
    // (In a cluster, whose blocks run this once, every part is left to the
    // block's join: less code to fetch took 8K tokens of one request from
    // 12.2 to 11.9 us.)
    bool done = !kCluster && begun && ended;
    if (!kCluster && begun && !ended && warp + 1 < W &&
        __all_sync(0xFFFFFFFFu, heads_ready[warp + 1])) {
      // The item ends in the next warp's run, which has left that part (it
      // came first there): join it here, where the accumulators are.
      __threadfence_block();
      const float* slot =
          reinterpret_cast<const float*>(smem + slot_at(warp + 1, 0));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float* stat = slot + NT * 8 * HD + nt * 8 + tig * 2;
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float mn = fmaxf(m_run[nt][i], stat[i]), base = base_of(mn);
          const float a = exp2_fast(m_run[nt][i] - base);
          f[i] = exp2_fast(stat[i] - base);
          m_run[nt][i] = mn;
          l_run[nt][i] =
              __fmaf_rn(stat[NT * 8 + i], f[i], __fmul_rn(l_run[nt][i], a));
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            acc[mt][nt][i] = __fmul_rn(acc[mt][nt][i], a);
            acc[mt][nt][i + 2] = __fmul_rn(acc[mt][nt][i + 2], a);
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const float4 x = *reinterpret_cast<const float4*>(
              slot + ((mt * NT + nt) * 32 + lane) * 4);
          acc[mt][nt][0] = __fmaf_rn(x.x, f[0], acc[mt][nt][0]);
          acc[mt][nt][1] = __fmaf_rn(x.y, f[1], acc[mt][nt][1]);
          acc[mt][nt][2] = __fmaf_rn(x.z, f[0], acc[mt][nt][2]);
          acc[mt][nt][3] = __fmaf_rn(x.w, f[1], acc[mt][nt][3]);
        }
      }
      if (lane == 0) recs[(warp + 1) * 2].r = -1;
      done = true;
    }
    if (done) {
      const Target<T> target(p, meta.r, sub, HD);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float inv[2] = {inverse(l_run[nt][0]), inverse(l_run[nt][1])};
        target.store_lse(nt, m_run[nt], l_run[nt]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          target.template store<HD>(nt, mt, acc[mt][nt], inv);
      }
      continue;
    }
    float* slot =
        reinterpret_cast<float*>(smem + slot_at(warp, ended ? 0 : 1));
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        store_part<HD, NT>(slot, mt * NT + nt, acc[mt][nt], m_run[nt],
                           l_run[nt]);
    if (lane == 0) {
      PartRec rec;
      rec.begin = item_begin;
      rec.r = meta.r;
      rec.sub = sub | (begun ? kFirst : 0u) | (ended ? kLast : 0u);
      recs[warp * 2 + (ended ? 0 : 1)] = rec;
    }
    if (ended) {
      __threadfence_block();
      __syncwarp();
      if (lane == 0) heads_ready[warp] = 1;
    }
  }
  if (v_used < n) {
    // a wait ran out: report it, and let the loads in flight land
    if (lane == 0 && p.flags) atomicOr(p.flags, KVTC_FLAG_TIMEOUT);
    for (int c = v_used; c < min(n, v_used + S); ++c)
      mbar_drain(v_bars + c % S, (c / S) & 1);
    for (int c = k_used; c < min(n, k_used + S); ++c)
      mbar_drain(k_bars + c % S, (c / S) & 1);
  }
  __syncthreads();

  // Join the block's parts: runs of records of one item, in order.  Lane e
  // of every warp holds record e.  A run goes to one warp, or where there
  // are few (long items) to several, which share its channel tiles.
  PartRec rec = {0, -1, 0u};
  if (lane < 2 * W) rec = recs[lane];
  const uint32_t item = rec.sub & kSubMask;
  const uint32_t there = __ballot_sync(0xFFFFFFFFu, rec.r >= 0);
  const uint32_t before = there & ((1u << lane) - 1);
  const int prev = before ? 31 - __clz(before) : lane;
  const int prev_r = __shfl_sync(0xFFFFFFFFu, rec.r, prev);
  const uint32_t prev_item = __shfl_sync(0xFFFFFFFFu, item, prev);
  const uint32_t heads = __ballot_sync(
      0xFFFFFFFFu, rec.r >= 0 && (!before || prev_r != rec.r ||
                                  prev_item != item));
  const int runs = __popc(heads);
  const int share = runs && runs < W ? W / runs : 1;   // warps per run
  const uint32_t smem_at = smem_u32(smem);
  uint32_t left = heads;
#pragma unroll 1
  for (int i = 0, w = 0; i < runs; ++i, w = w + share < W ? w + share : 0) {
    const int e0 = __ffs(left) - 1;
    left &= left - 1;
    if (warp < w || warp >= w + share) continue;
    const uint32_t in_run =
        there & ~((1u << e0) - 1) & (left ? (left & (0u - left)) - 1 : ~0u);
    const int e1 = 31 - __clz(in_run);
    const bool begun_here = __shfl_sync(0xFFFFFFFFu, rec.sub, e0) & kFirst;
    const bool ended_here = __shfl_sync(0xFFFFFFFFu, rec.sub, e1) & kLast;
    // its parts: entry 1 of consecutive warps, and last what it is
    auto slot_of = [&](int e) { return smem_at + slot_at(e >> 1, e & 1); };
    float* to = nullptr;
    if (!(begun_here && ended_here))
      to = kCluster ? reinterpret_cast<float*>(smem + L::kBlockPart)
                    : p.cta_slots + ((int64_t)blockIdx.x * 2 +
                                     (begun_here ? 1 : 0)) *
                                        slot_floats(HD, NT);
    const Target<T> target(p, __shfl_sync(0xFFFFFFFFu, rec.r, e0),
                           __shfl_sync(0xFFFFFFFFu, item, e0), HD);
    const uint32_t first = slot_of(e0), last = slot_of(e1);
    const uint32_t base = slot_of(e0 | 1);
    const int k = __popc(in_run);
    // (a cluster's block has one run, and a warp for each of its tiles)
    join_parts<T, HD, NT, kCluster ? 1 : 2, kCluster ? 4 : 3, false>(
        k,
        [=](int i) {
          return i == 0 ? first
                 : i == k - 1 ? last : base + i * L::kRing;
        },
        target, to, warp - w, share);
  }

  if (kCluster) {
    if (deal.ctas == 1) return;
    cluster_sync();
    // one part in each working block, in their order
    const uint32_t mine = smem_at + L::kBlockPart;
    join_parts<T, HD, NT, 1, 8, true>(
        deal.ctas, [=](int i) { return mapa_shared(mine, (uint32_t)i); },
        Target<T>(p, cur_r, fixed_sub, HD), nullptr, rank + warp * most,
        most * W);
    cluster_sync();       // (the others have read this block's part)
    return;
  }
  // An item that goes on in the next blocks is the last run's.
  if (warp == W - 1) {
    const int e0 = heads ? 31 - __clz(heads) : 0;
    const int e1 = there ? 31 - __clz(there) : 0;
    const uint32_t first_sub = __shfl_sync(0xFFFFFFFFu, rec.sub, e0);
    const uint32_t last_sub = __shfl_sync(0xFFFFFFFFu, rec.sub, e1);
    const int64_t begin = __shfl_sync(0xFFFFFFFFu, rec.begin, e0);
    const int r = __shfl_sync(0xFFFFFFFFu, rec.r, e0);
    JoinDesc d = {-1, 0, 0, 0};
    if (there && (first_sub & kFirst) && !(last_sub & kLast)) {
      d.r = r;
      d.sub = (int32_t)(first_sub & kSubMask);
      d.last_cta = deal.cta_of(begin + span_of(p, r).units - 1);
    }
    if (lane == 0)
      *reinterpret_cast<int4*>(p.desc + blockIdx.x) =
          make_int4(d.r, d.sub, d.last_cta, 0);
  }
}

// A running join at one fragment position (two columns), of parts that other
// blocks left in the workspace.
template <int HD, int NT>
struct FarJoin {
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float o[4] = {0.f, 0.f, 0.f, 0.f};
  // Parts i0, i0 + kStep .. (N of them) of the item that began in block c, as
  // far as there are n; all loads are in flight before n is asked for.
  template <int N, int kStep, class F>
  __device__ __forceinline__ void add(const float* slots, int c, int i0,
                                      int tile, F n) {
    const int lane = (int)lane_id();
    const int col = tile % NT * 8 + (lane & 3) * 2;
    float2 mi[N], li[N];
    float4 oi[N];
#pragma unroll
    for (int b = 0; b < N; ++b) {
      const int i = i0 + b * kStep;
      const float* s = slots + ((int64_t)min(c + i, kCtas - 1) * 2 +
                                (i ? 0 : 1)) * slot_floats(HD, NT);
      mi[b] = __ldcg(reinterpret_cast<const float2*>(s + NT * 8 * HD + col));
      li[b] = __ldcg(
          reinterpret_cast<const float2*>(s + NT * 8 * (HD + 1) + col));
      oi[b] = __ldcg(reinterpret_cast<const float4*>(s) + tile * 32 + lane);
    }
    const int end = n();
    float mn[2] = {m[0], m[1]};
#pragma unroll
    for (int b = 0; b < N; ++b)
      if (i0 + b * kStep < end) {
        mn[0] = fmaxf(mn[0], mi[b].x);
        mn[1] = fmaxf(mn[1], mi[b].y);
      }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float f = exp2_fast(m[k] - base_of(mn[k]));
      m[k] = mn[k];
      l[k] *= f;
      o[k] *= f;
      o[k + 2] *= f;
    }
#pragma unroll
    for (int b = 0; b < N; ++b)
      if (i0 + b * kStep < end) {
        const float f0 = exp2_fast(mi[b].x - base_of(m[0]));
        const float f1 = exp2_fast(mi[b].y - base_of(m[1]));
        l[0] += li[b].x * f0;
        l[1] += li[b].y * f1;
        o[0] += oi[b].x * f0;
        o[1] += oi[b].y * f1;
        o[2] += oi[b].z * f0;
        o[3] += oi[b].w * f1;
      }
  }
  // Another such join, with {m, m, l, l}.
  __device__ __forceinline__ void more(const float4& x, const float4& y) {
    const float m0 = fmaxf(m[0], y.x), m1 = fmaxf(m[1], y.y);
    const float f0 = exp2_fast(m[0] - base_of(m0));
    const float f1 = exp2_fast(m[1] - base_of(m1));
    const float g0 = exp2_fast(y.x - base_of(m0));
    const float g1 = exp2_fast(y.y - base_of(m1));
    m[0] = m0;
    m[1] = m1;
    l[0] = l[0] * f0 + y.z * g0;
    l[1] = l[1] * f1 + y.w * g1;
    o[0] = o[0] * f0 + x.x * g0;
    o[1] = o[1] * f1 + x.y * g1;
    o[2] = o[2] * f0 + x.z * g0;
    o[3] = o[3] * f1 + x.w * g1;
  }
};

// Items that lie over several blocks: block c joins the one that began in
// block c of the attention, its own part and those of the blocks after it, a
// warp per channel tile.  With many items there are two or three parts mostly.
// Where an item lies over kFewParts blocks or more on average, join_groups
// groups of warps take every so-many-th part and are joined through shared
// memory.  The launch waits for no host, but its blocks start only as the
// attention's leave their SMs: those hold 64,512 of an SM's 65,536 registers
// at head_dim 128 with one head tile, where a block here takes 22,528 (9,984
// are free at head_dim 256, and 45,056 taken), so that the start and the first
// loads lie behind the attention's end.  One group and join_groups: 64
// requests up to 4K (256 items) 48.5 and 49.8 us; two of 32K (16 items) 39.6
// and 39.0, one (8 items) 30.5 and 29.2.
constexpr int kFewParts = 8;
__host__ __device__ constexpr int join_groups(int tiles) {
  return tiles > 16 ? 1 : tiles > 8 ? 2 : 4;
}
template <class T, int HD, int NT, int kGroups>
__global__ void __launch_bounds__(HD / 16 * NT * 32 * kGroups)
    attend_join_kernel(const __grid_constant__ AttendParams p) {
  constexpr int kTiles = HD / 16 * NT;
  constexpr int kFirst = kGroups > 1 ? 5 : 3;
  constexpr int kNext = kTiles * kGroups > 16 ? 5 : 8;   // by registers
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int c = blockIdx.x, warp = threadIdx.x >> 5;
  const int tile = warp % kTiles, group = warp / kTiles;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int4 d;
  int n;
  FarJoin<HD, NT> join;
  join.template add<kFirst, kGroups>(p.cta_slots, c, group, tile, [&] {
    d = __ldcg(reinterpret_cast<const int4*>(p.desc + c));
    n = d.x < 0 ? 0 : d.z - c + 1;
    return n;
  });
  if (n == 0) return;
#pragma unroll 1
  for (int i = group + kFirst * kGroups; i < n; i += kNext * kGroups)
    join.template add<kNext, kGroups>(p.cta_slots, c, i, tile,
                                      [&] { return n; });
  if (kGroups > 1) {
    __shared__ float4 part_o[kGroups][kTiles * 32];
    __shared__ float4 part_ml[kGroups][kTiles * 32];
    const int at = tile * 32 + (int)lane_id();
    part_o[group][at] =
        make_float4(join.o[0], join.o[1], join.o[2], join.o[3]);
    part_ml[group][at] =
        make_float4(join.m[0], join.m[1], join.l[0], join.l[1]);
    __syncthreads();
    if (group) return;
#pragma unroll
    for (int g = 1; g < kGroups; ++g) join.more(part_o[g][at], part_ml[g][at]);
  }
  const Target<T> target(p, d.x, (uint32_t)d.y, HD);
  const float inv[2] = {inverse(join.l[0]), inverse(join.l[1])};
  target.template store<HD>(tile % NT, tile / NT, join.o, inv);
  if (tile < NT) target.store_lse(tile % NT, join.m, join.l);
}

template <class T, int HD, int NT>
cudaError_t launch_as(const AttendParams& p, int cluster, int device,
                      cudaStream_t st) {
  static std::atomic<uint64_t> ready[2];     // devices, as bits
  cudaError_t e;
  if (cluster) {
    const auto kernel = attend_kernel<T, HD, NT, true>;
    using L = Smem<HD, NT, true>;
    e = allow_smem(kernel, L::kBytes, device, ready[0], true);
    if (e == cudaSuccess)
      e = launch_kernel(kernel, dim3(p.kv_heads * p.tiles * cluster, p.R),
                        L::W * 32, L::kBytes, st, true, cluster, p);
    if (e == cudaSuccess) count_launch();
    return e;
  }
  const auto kernel = attend_kernel<T, HD, NT, false>;
  using L = Smem<HD, NT, false>;
  e = allow_smem(kernel, L::kBytes, device, ready[1]);
  if (e == cudaSuccess)
    e = launch_kernel(kernel, kCtas, L::W * 32, L::kBytes, st, true, 0, p);
  if (e != cudaSuccess) return e;
  count_launch();
  constexpr int kTiles = HD / 16 * NT, kGroups = join_groups(kTiles);
  const bool few = (int64_t)p.R * p.kv_heads * p.tiles * kFewParts <= kCtas;
  e = launch_kernel(few ? attend_join_kernel<T, HD, NT, kGroups>
                        : attend_join_kernel<T, HD, NT, 1>,
                    kCtas, kTiles * 32 * (few ? kGroups : 1), 0, st, true, 0,
                    p);
  if (e == cudaSuccess) count_launch();
  return e;
}

// Blocks per item, or 0 for equal runs over all items.  The GPU holds 7
// clusters of 16 such blocks at once, 15 of 8, 36 of 4, 76 of 2 (what
// cudaOccupancyMaxActiveClusters says of it).  A cluster of more blocks than
// the longest item can feed is of no use.  What clusters save is the join
// across blocks, about 3 us; what they lose is that items * cluster blocks,
// at about 90 GB/s a block, may read slower than all SMs at 7000 GB/s, which
// is taken at the longest length that the table allows, for the others half
// of that.  Clusters and runs, 32 heads on 8 of 128: one request of 2K 8.0
// and 10.0 us, 8K 11.7 and 13.7, 16K 18.6 and 19.5, 32K 29.5 and 28.5; two of
// 4K 11.5 and 11.5, of 8K 18.0 and 16.6; 16 of up to 1K 13.7 and 15.9.
// The lengths themselves are on the device: under a table of 2048 columns one
// request of 256 tokens takes the runs' 9.9 us, not 6.8, of 1K 9.9 and not
// 8.1, of 8K 13.5 and not 11.7.
int cluster_of(int R, int64_t items, int64_t max_blocks, int head_dim,
               int nt) {
  if (items > kCtas) return 0;
  int cluster = items <= 7 ? 16 : items <= 15 ? 8 : items <= 36 ? 4
                : items <= 76 ? 2 : 1;
  const int64_t feeds = warps_of(head_dim, nt, true);
  while (cluster > 1 && max_blocks <= feeds * (cluster / 2)) cluster /= 2;
  const double bytes = 2.0 * (double)max_blocks * page_bytes(head_dim);
  const double others = R == 1 ? 1.0 : 0.5 + 0.5 / R;
  return bytes / (90.0 * cluster) - others * bytes * items / 7000.0 <= 3000.0
             ? cluster
             : 0;
}

// Tiles of eight query heads per warp: one or two, by the group, and four for
// large groups of head_dim 64.  Larger groups are cut into equal tiles of
// heads, each of which reads the pages again (from L2, mostly).  At 32 heads
// a KV head, one pass with four tiles takes 59.8 us at head_dim 64, two with
// two 69.1 (32 requests of 4K to 8K, 4 KV heads); at 128 it was 217 and 175
// (32 up to 8K, 8 KV heads): the accumulators of 32 heads leave too few warps.
int head_tiles(int head_dim, int group) {
  return group <= 8 ? 1 : group <= 16 || head_dim > 64 ? 2 : 4;
}

template <class T>
cudaError_t launch(const AttendParams& p, int head_dim, int nt, int cluster,
                   int device, cudaStream_t st) {
  if (head_dim == 64)
    return nt == 1   ? launch_as<T, 64, 1>(p, cluster, device, st)
           : nt == 2 ? launch_as<T, 64, 2>(p, cluster, device, st)
                     : launch_as<T, 64, 4>(p, cluster, device, st);
  if (head_dim == 128)
    return nt == 1 ? launch_as<T, 128, 1>(p, cluster, device, st)
                   : launch_as<T, 128, 2>(p, cluster, device, st);
  return nt == 1 ? launch_as<T, 256, 1>(p, cluster, device, st)
                 : launch_as<T, 256, 2>(p, cluster, device, st);
}

// A pool [num_blocks][16][D] as {64 channels, 16 tokens, D / 64, num_blocks}:
// a box is `rows` rows of one block, `slabs` times 64 channels of each, as
// tiles [rows][64].
bool encode_pages(CUtensorMap* m, const void* base, uint64_t D,
                  uint64_t num_blocks, uint32_t rows, uint32_t slabs) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[4] = {64, kBlock, D / 64, num_blocks};
  cuuint64_t strides[3] = {D * 2, 128, D * 2 * kBlock};
  cuuint32_t box[4] = {64u, rows, slabs, 1u};
  cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int64_t kDescBytes =
    (kCtas * sizeof(JoinDesc) + 255) / 256 * 256;

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
  const int nt = head_tiles(head_dim, heads / kv_heads);
  const int64_t slot = 4 * slot_floats(head_dim, nt);
  return kDescBytes + kCtas * 2 * slot;
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
      max_blocks <= 0 || sink < 0 || window < 0 ||
      !(std::fabs(scale) <= kMaxScale) ||      // (nor NaN)
      !workspace || (R && (!q || !block_table || !lens || !out)))
    return KVTC_EINVAL;
  if (block_size != kBlock || max_blocks > kMaxTable) return KVTC_ENOTSUP;
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
  const uint32_t slabs = (uint32_t)head_dim / 64;
  if (!encode_pages(&p.tm_k, k_cache, D, num_blocks, kBlock, slabs) ||
      !encode_pages(&p.tm_v, v_cache, D, num_blocks, kBlock, slabs) ||
      !encode_pages(&p.tm_k8, k_cache, D, num_blocks, 8, 1) ||
      !encode_pages(&p.tm_v8, v_cache, D, num_blocks, 8, 1))
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
  p.tiles_inv = (65536u + p.tiles - 1) / p.tiles;
  const int cluster = cluster_of(R, (int64_t)R * kv_heads * p.tiles,
                                 max_blocks, head_dim, nt);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = dtype == KVTC_DTYPE_BF16
                            ? launch<__nv_bfloat16>(p, head_dim, nt, cluster,
                                                    cuda_device, st)
                            : launch<__half>(p, head_dim, nt, cluster,
                                             cuda_device, st);
  return e == cudaSuccess ? KVTC_OK : KVTC_ECUDA;
}

}  // extern "C"
