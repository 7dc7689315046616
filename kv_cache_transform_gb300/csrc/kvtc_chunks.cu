// Attention of chunks of new tokens over paged K and V pools.
//
// Rows of a matrix product are (token, query head) pairs that read one KV
// head: row i * group + g is token i of the chunk and head g of the group, so
// that few tokens fill a tile too.  For a row, with a running reference m near
// the maximum,
//     S = Q K^T,  P = 2^(scale log2(e) S - m),  l += sum P,  O += P V,
// where a tile's maximum lies more than 2^8 above m, m moves to it, and l and
// O are multiplied by 2^(m_old - m_new); out = O / l, lse = (m + log2 l) ln 2.
//
// Work.  An item is (request, KV head, up to two tiles of 128 rows), a unit
// 128 tokens of K and V that an item's rows attend to.  All units of the call
// are dealt out to one block per SM in equal runs, whatever the lengths are
// (they are on the device: each block sums them itself).  A block whose run
// begins or ends inside an item leaves m, l and O of its part, and
// chunk_join_kernel joins the parts in a fixed order: equal calls give equal
// bits.
//
// Inside a block:
//   producer   goes through the run: item descriptors, Q, and the pages of K
//              and V by TMA into a ring of stages (128 tokens x up to 128
//              channels each);
//   MMA        issues S = Q K^T and O += P V (tcgen05, S, P and O in TMEM, P
//              over the S that it came from);
//   softmax    two warpgroups, a thread per row;
//   cleaner    rows of V in units that not every row attends to whole: those
//              that none attends to are zeroed, and infinities and NaN taken
//              out of the others (a weight of zero times them would be NaN);
//              the softmax threads add them to the rows that attend to them.
//
// P is rounded to 16 bits for the product with V; l is the sum of the
// unrounded weights.  Everything else is fp32.  (A second 16-bit term of P would
// be half as many products again.  One term leaves the error against 64 bits at
// that of the output's rounding where V's mean outweighs its spread, 1.4 times
// that where V has no mean: 1.19 times at 16 tokens, 1.39 at 4096.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/kvtc.h"
#include "kvtc_chunk.cuh"
#include "kvtc_hostutil.cuh"
#include "kvtc_internal.cuh"
#include "ptx.cuh"

namespace kvtc {
namespace {

constexpr float kSlack = 8.f;          // log2
// What an item's begin and end cost, in units: the first S, the last P V, O, and
// units that are attended in part.  (With 1, 2, 4 and 8 a prompt of 8192 tokens
// takes 505, 475, 424 and 439 us, 64 chunks up to 256 tokens 266, 238, 219 and
// 230.)
constexpr int kItemCost = 4;
constexpr int kWarps = 12;             // (the last one fills its warpgroup)
constexpr int kProducer = 8, kMma = 9, kCleaner = 10;
constexpr int kThreads = kWarps * 32;
constexpr int kItems = 4, kMetas = 8;  // entries of the rings

// Which blocks hold parts of an item that began in a block and did not end
// there; r < 0: there is none.
struct __align__(16) JoinDesc {
  int64_t row0;
  int32_t r, j, ntok, last;
};

struct ChunkParams {
  CUtensorMap tm_q;         // {64, HD / 64, heads, N}, box {64, 1, group, tq}
  CUtensorMap tm_k, tm_v;   // {64, 16, D / 64, num_blocks}, box {64, 16, x, 1}
  const int32_t* table;
  const int64_t* cu;
  const int32_t* lens;
  const void* v;
  void* out;
  float* lse;
  unsigned* flags;
  JoinDesc* desc;           // [kCtas]
  float* slots;             // [kCtas][2] parts: 0 of an item begun in an
                            // earlier block, 1 of one begun in this block
  int64_t N, out_ld, num_blocks;
  float scale;              // its magnitude, times log2 e; never 0
  int32_t negate;           // a negative scale: S is formed with -Q
  int32_t R, heads, kv_heads, max_blocks, sink, window;
  int32_t group, tq;        // query heads a KV head; tokens per row tile
  int32_t whole;            // a block per item: nothing to be joined
  int32_t split;            // items, where there are few; or 0
};

template <int HD_>
struct Cfg {
  static constexpr int HD = HD_;
  static constexpr int QT = HD == 256 ? 1 : 2;        // row tiles per item
  static constexpr int kChains = QT;
  static constexpr int U = HD == 256 ? 64 : 128;      // tokens of a unit
  static constexpr int kPages = U / kBlock;
  static constexpr int SC = HD < 128 ? HD : 128;      // channels per stage
  static constexpr int NS = HD / SC;                  // stages per K or V tile
  static constexpr int kSlabs = SC / 64;              // per stage
  static constexpr int kStage = U * SC * 2;
  static constexpr int S = HD == 64 ? 8 : HD == 128 ? 5 : 10;
  static constexpr int kQ = QT * kRows * HD * 2;
  static constexpr int kRing = kQ;
  static constexpr int kMisc = kRing + S * kStage;
  static constexpr int kBytes = kMisc + 2560;
  static_assert(kBytes <= 232448 && kMisc % 1024 == 0, "shared memory of a block");
  static_assert(S * kStage >= 8 * (kMaxReq + 1), "prefix of the requests");
  // TMEM columns
  static constexpr int kO = 256;                      // O of tile t: + 128 t
  static constexpr int kPart = kRows * (HD + 2);      // floats of a part tile
};

struct __align__(16) Item {
  int64_t row0;             // first row (token) of the call
  int32_t r, j;             // request, KV head
  int32_t ntok, pf;         // tokens, position of the first
  int32_t units;            // of this block; 0: the end
  int32_t flags;
};
constexpr int kStarts = 1, kEnds = 2, kDual = 4;

struct __align__(16) Meta {
  int32_t t0;               // first token
  uint32_t pages;           // which of its pages are there
  int32_t mixed;            // not every row attends to all of it
  int32_t pad;
  uint32_t odd[4];          // tokens whose V held infinities or NaN
};

// ------------------------------------------------------------------- spans
// Units of an item whose rows are at positions pf .. pl: `units` of them, the
// first `front` at their own place, the others `gap` further on.  An item
// whose rows attend to nothing still has one, which is empty.
template <int U>
struct Span {
  int32_t units, front, gap;
  __device__ __forceinline__ Span(const ChunkParams& p, int32_t pf,
                                  int32_t pl) {
    const int32_t all = pl >= 0 ? pl / U + 1 : 0;
    front = all;
    gap = 0;
    if (p.window) {
      const int64_t lo = (int64_t)pf - p.window + 1;
      const int32_t back = lo > 0 ? (int32_t)(lo / U) : 0;
      front = (int32_t)min(((int64_t)p.sink + U - 1) / U,
                           (int64_t)all);
      gap = max(back - front, 0);
    }
    units = max(all - gap, 1);
  }
};
__device__ __forceinline__ Request request(const ChunkParams& p, int r) {
  return Request(p.cu, p.lens, p.N, p.R, p.max_blocks, r);
}
// Cost of item i of a request (per KV head), in units.
template <int U>
__device__ __noinline__ int64_t item_cost(const ChunkParams& p,
                                             int32_t n, int32_t len, int32_t i,
                                             int32_t per) {
  if (p.whole) return 1;
  const int32_t first = i * per, last = first + min(per, n - first) - 1;
  return Span<U>(p, len - n + first, len - n + last).units + kItemCost;
}
// Which of the tokens t0 + 32 w .. + 31 the row at `pos` attends to.
__device__ __forceinline__ uint32_t seen_bits(const ChunkParams& p,
                                              const Meta& m, int64_t pos,
                                              int w) {
  const int64_t t = (int64_t)m.t0 + 32 * w;
  uint32_t bits = low_bits(pos - t + 1);
  if (p.window)
    bits &= low_bits(p.sink - t) | ~low_bits(pos - p.window + 1 - t);
  const uint32_t pages = m.pages >> (2 * w);
  return bits & ((pages & 1 ? 0xFFFFu : 0u) | (pages & 2 ? 0xFFFF0000u : 0u));
}

struct Bars {
  // A stage holds K and V in turn, and K's loads have another reader than V's:
  // what tells that loads have landed goes by units, so that each barrier has
  // one reader, which sees all of its phases.  (By stages, a reader of V would
  // take the phase before K's for its own while K's loads are under way.)
  uint64_t full[kMetas][2][2];     // K, V; stages of one
  uint64_t empty[10];              // stages
  uint64_t q_full, q_empty;
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t meta[kMetas], clean[kMetas];       // units
  uint64_t s_full[2], p_full[2];              // buffers of S
  uint64_t pv_done[2], fin;                   // chains
  uint64_t ready, taken;                      // chain 1's part of a lone tile
};

struct Smem {
  Bars bars;
  Item items[kItems];
  Meta metas[kMetas];
  int64_t sums[kWarps];
  float2 lone[kRows];       // m and l of chain 1's part of a lone tile
  uint32_t tmem;
  int abort_flag;
};
static_assert(sizeof(Smem) <= 2560, "the kernels' shared variables");

// --------------------------------------------------------------- producer
template <class T, class C>
__device__ __forceinline__ bool produce(const ChunkParams& p, Smem& sm,
                                        uint32_t smem, const int64_t* pre) {
  constexpr int HD = C::HD, NS = C::NS, S = C::S, U = C::U;
  constexpr int kPages = C::kPages;
  const int lane = (int)lane_id();
  Bars& b = sm.bars;
  volatile int* stop = &sm.abort_flag;
  Turn<S> st;
  Turn<kItems> it;
  Turn<kMetas> mt;
  uint32_t q_phase = 0;
  uint32_t fills = 0;                  // stages filled
  const int64_t total = pre[p.R];
  const Deal deal(total, p.whole ? 1 : kItemCost + 2);
  int64_t x = deal.begin(blockIdx.x);
  const int64_t end = deal.begin(blockIdx.x + 1);
  const int32_t per = C::QT * p.tq;
  int r = 0, j = 0, i = 0;
  int64_t y = 0;                       // x within its item
  if (x < end) {
    // the request (the last one that begins at or before x and is not empty)
    int lo = 0, hi = p.R;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= x) lo = mid; else hi = mid;
    }
    r = lo;
    const Request q = request(p, r);
    const int64_t head = (pre[r + 1] - pre[r]) / p.kv_heads;
    y = x - pre[r];
    j = (int)(y / head);
    y -= j * head;
    // the item, 32 at a time
    const int items = parts_of(q.n, per);
    for (;;) {
      const int64_t cost =
          i + lane < items ? item_cost<C::U>(p, q.n, q.len, i + lane, per) : 0;
      int64_t upto = cost;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(~0u, upto, d);
        if (lane >= d) upto += o;
      }
      const uint32_t past = __ballot_sync(~0u, upto > y);
      if (past) {
        const int at = __ffs(past) - 1;
        y -= __shfl_sync(~0u, upto - cost, at);
        i += at;
        break;
      }
      y -= __shfl_sync(~0u, upto, 31);
      i += 32;
    }
  }
  __syncwarp();
  // the prefix sums lay where the TMA is going to write
  asm volatile("fence.proxy.async;" ::: "memory");
  bool ok = true, left_desc = false;
  int base = r;                        // requests base .. base + 31
  Request batch = request(p, base + lane);
  while (x < end && ok) {
    if (r >= base + 32) {
      base = r;
      batch = request(p, base + lane);
    }
    const Request q(__shfl_sync(~0u, batch.c0, r - base),
                    __shfl_sync(~0u, batch.n, r - base),
                    __shfl_sync(~0u, batch.len, r - base));
    const int items = parts_of(q.n, per);
    if (items == 0) {
      ++r;
      continue;
    }
    const int32_t first = i * per, ntok = min(per, q.n - first);
    const int32_t pf = q.len - q.n + first, pl = pf + ntok - 1;
    const Span<U> span(p, pf, pl);
    const int64_t k0 = p.whole ? 0 : max(y - kItemCost, (int64_t)0);
    const int64_t k1 =
        p.whole ? span.units
                : min((int64_t)span.units, y + (end - x) - kItemCost);
    const bool dual = ntok > p.tq;
    if (k1 > k0) {
      if (!warp_wait(&b.item_empty[it.at], it.phase ^ 1, stop)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        Item d;
        d.row0 = q.c0 + first;
        d.r = r;
        d.j = j;
        d.ntok = ntok;
        d.pf = pf;
        d.units = (int32_t)(k1 - k0);
        d.flags = (k0 == 0 ? kStarts : 0) | (k1 == span.units ? kEnds : 0) |
                  (dual ? kDual : 0);
        sm.items[it.at] = d;
        mbar_arrive(&b.item_full[it.at]);
        if (k0 == 0 && k1 < span.units) {
          JoinDesc jd;
          jd.row0 = d.row0;
          jd.r = r;
          jd.j = j;
          jd.ntok = ntok;
          jd.last = deal.cta_of(x - y + kItemCost + span.units - 1);
          p.desc[blockIdx.x] = jd;
          left_desc = true;
        }
      }
      it.next();
      const int32_t* row = p.table + (int64_t)r * p.max_blocks;
      // a lane has a page and a slab of K
      const int page = lane % kPages, slab = lane / kPages;
      const int slab_all = j * (HD / 64) + slab;
      auto id_at = [&](int64_t k) -> int32_t {
        const int32_t t0 =
            (int32_t)(k < span.front ? k : k + span.gap) * U;
        const int32_t tp = t0 + page * kBlock;
        const bool need =
            pl >= 0 && tp <= pl &&
            (!p.window || tp < p.sink ||
             (int64_t)tp + kBlock - 1 > (int64_t)pf - p.window);
        return need ? row[tp / kBlock] : -1 - INT_MAX;
      };
      int32_t id = id_at(k0);
      for (int64_t k = k0; k < k1 && ok; ++k) {
        const int32_t next_id = k + 1 < k1 ? id_at(k + 1) : 0;
        const int32_t t0 =
            (int32_t)(k < span.front ? k : k + span.gap) * U;
        const bool fine = id >= 0 && id < p.num_blocks;
        const int32_t tp = t0 + page * kBlock;
        // (ids that are not asked for are -2^31; one in the table is bad too)
        if (!fine && slab == 0 && p.flags && pl >= 0 && tp <= pl &&
            (!p.window || tp < p.sink ||
             (int64_t)tp + kBlock - 1 > (int64_t)pf - p.window))
          atomicOr(p.flags, KVTC_FLAG_BLOCK);
        const uint32_t pages =
            __ballot_sync(~0u, fine) & ((1u << kPages) - 1);
        if (lane == 0) {
          Meta m;
          m.t0 = t0;
          m.pages = pages;
          const int64_t tl = (int64_t)t0 + U - 1;
          m.mixed = !(pages == (1u << kPages) - 1 && tl <= pf &&
                      (!p.window || tl < p.sink ||
                       (int64_t)t0 > (int64_t)pl - p.window));
          sm.metas[mt.at].t0 = m.t0;
          sm.metas[mt.at].pages = m.pages;
          sm.metas[mt.at].mixed = m.mixed;
          mbar_arrive(&b.meta[mt.at]);
        }
        const int unit = mt.at;
        mt.next();
        const uint32_t bytes = __popc(pages) * C::kSlabs * 2048;
#pragma unroll
        for (int kv = 0; kv < 2 && ok; ++kv) {
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            if (!warp_wait(&b.empty[st.at], st.phase ^ 1, stop)) {
              ok = false;
              break;
            }
            uint64_t* full = &b.full[unit][kv][s];
            if (lane == 0) mbar_arrive_expect_tx(full, bytes);
            __syncwarp();
            const uint32_t to = smem + C::kRing + st.at * C::kStage;
            if (kv == 0 && fine && slab / C::kSlabs == s && slab < HD / 64)
              tma_load_4d(to + slab % C::kSlabs * (U * 128) + page * 2048,
                          &p.tm_k, 0, 0, slab_all, id, full);
            if (kv == 1 && fine && slab == 0)
              tma_load_4d(to + page * (C::kSlabs * 2048), &p.tm_v, 0, 0,
                          slab_all + s * C::kSlabs, id, full);
            st.next();
            ++fills;
          }
        }
        id = next_id;
        if (k == k0 && ok) {
          // Q, behind the first unit: the item before has to be done with it
          if (!warp_wait(&b.q_empty, q_phase ^ 1, stop)) {
            ok = false;
            break;
          }
          const int tiles = dual ? 2 : 1;
          if (lane == 0)
            mbar_arrive_expect_tx(
                &b.q_full, tiles * (HD / 64) * p.tq * p.group * 128);
          __syncwarp();
          if (lane < tiles * (HD / 64)) {
            const int t = lane / (HD / 64), sl = lane % (HD / 64);
            tma_load_4d(smem + t * (kRows * HD * 2) + sl * (kRows * 128),
                        &p.tm_q, 0, sl, j * p.group,
                        (int32_t)(q.c0 + first) + t * p.tq, &b.q_full);
          }
          q_phase ^= 1;
        }
      }
    }
    const int64_t step = min(
        p.whole ? 1 : (int64_t)span.units + kItemCost - y, end - x);
    x += step;
    y = 0;
    if (++i == items) {
      i = 0;
      if (++j == p.kv_heads) {
        j = 0;
        ++r;
      }
    }
  }
  if (ok && warp_wait(&b.item_empty[it.at], it.phase ^ 1, stop)) {
    if (lane == 0) {
      sm.items[it.at].units = 0;
      mbar_arrive(&b.item_full[it.at]);
    }
  } else {
    ok = false;
  }
  if (lane == 0 && !left_desc) p.desc[blockIdx.x].r = -1;
  // loads under way land before the block's memory is given up
  __syncwarp();
  if (lane == 0) {
    mbar_drain(&b.q_full, q_phase ^ 1);
    for (uint32_t k = 1; k <= min(fills, (uint32_t)S); ++k) {
      const uint32_t f = fills - k, unit = f / (2 * NS);
      mbar_drain(&b.full[unit % kMetas][f / NS % 2][f % NS],
                 unit / kMetas & 1);
    }
  }
  return ok;
}

// -------------------------------------------------------------------- MMA
template <class T, class C>
__device__ __forceinline__ bool multiply(const ChunkParams& p, Smem& sm,
                                         uint32_t smem, uint32_t tmem) {
  constexpr int HD = C::HD, NS = C::NS, S = C::S, SC = C::SC, U = C::U;
  // (bit 13: A is negated)
  const uint32_t id_s =
      make_idesc(kRows, U, Elem<T>::kFormat) | (p.negate ? 1u << 13 : 0u);
  // (bit 16: B's rows are contiguous)
  constexpr uint32_t kIdO =
      make_idesc(kRows, SC, Elem<T>::kFormat) | (1u << 16);
  Bars& b = sm.bars;
  volatile int* stop = &sm.abort_flag;
  Turn<S> kt, vt;                // the next tile's first stage
  Turn<kItems> it;
  Turn<kMetas> km, mt;           // K's unit, V's
  uint32_t q_phase = 0;
  uint32_t p_phase = 0;          // a bit per barrier
  const uint32_t ring = smem + C::kRing;
  for (int s = 0; s < NS; ++s) vt.next();

  for (;;) {
    if (!warp_wait(&b.item_full[it.at], it.phase, stop)) return false;
    const int units = uniform(sm.items[it.at].units);
    const bool dual = uniform(sm.items[it.at].flags) & kDual;
    if (units == 0) return true;
    if (!warp_wait(&b.q_full, q_phase, stop)) return false;
    q_phase ^= 1;
    // Steps: a unit for each row tile in turn, or one unit after the other for
    // a lone tile; S, P (and with two chains O) of step n in buffer n & 1.  The
    // S of a step is formed as soon as the product with the P that lay in its
    // buffer has been issued.  (One place for each product, and loops that are
    // not unrolled: the code has to stay in the instruction cache.)
    const int steps = dual ? 2 * units : units;
#pragma unroll 1
    for (int n = 0; n < steps + 2; ++n) {
      const int buf = n & 1;
      const bool begins = !dual || buf == 0, ends = !dual || buf == 1;
      if (n >= 2) {
        // O += P V of step n - 2
        if (begins) {
          if (!warp_wait(&b.clean[mt.at], mt.phase, stop)) return false;
          mt.next();
        }
        if (!warp_wait(&b.p_full[buf], p_phase >> buf & 1, stop)) return false;
        p_phase ^= 1u << buf;
        tc_fence_after();
        const int chain = C::kChains == 2 ? buf : 0;
        Turn<S> v = vt;
#pragma unroll 1
        for (int s = 0; s < NS; ++s) {
          // (the next 64 channels lie a slab further on)
          const uint32_t bd =
              desc_base(ring + v.at * C::kStage, (uint32_t)(2048 >> 4));
          const uint32_t d = tmem + C::kO + chain * 128 + s * SC;
          const uint32_t a = tmem + buf * 128;
#pragma unroll
          for (int e = 0; e < U / 16; ++e)
            mma_ts_one(d, a + e * 8, bd + e * (C::kSlabs * 2048 >> 4), kIdO,
                       n - 2 >= C::kChains || e > 0);
          v.next();
        }
        tc_commit_one(&b.pv_done[chain]);
        if (ends) {
          for (int s = 0; s < NS; ++s) {
            tc_commit_one(&b.empty[vt.at]);
            vt.next();
          }
          for (int s = 0; s < NS; ++s) vt.next();     // (K's stages)
        }
      }
      if (n < steps) {
        // S of step n
        Turn<S> k = kt;
#pragma unroll 1
        for (int s = 0; s < NS; ++s) {
          if (begins && !warp_wait(&b.full[km.at][0][s], km.phase, stop))
            return false;
          tc_fence_after();
          const uint32_t bd = desc_base(ring + k.at * C::kStage);
          const uint32_t ad = desc_base(smem + (dual ? buf : 0) *
                                                   (kRows * HD * 2) +
                                        s * C::kSlabs * (kRows * 128));
          const uint32_t d = tmem + buf * 128;
#pragma unroll
          for (int e = 0; e < SC / 16; ++e)
            mma_ss_one(d, ad + (e / 4) * (kRows * 128 >> 4) + (e % 4) * 2,
                       bd + (e / 4) * (U * 128 >> 4) + (e % 4) * 2, id_s,
                       (s | e) > 0);
          k.next();
        }
        tc_commit_one(&b.s_full[buf]);
        if (ends) {
          km.next();
          for (int s = 0; s < NS; ++s) {
            tc_commit_one(&b.empty[kt.at]);
            kt.next();
          }
          for (int s = 0; s < NS; ++s) kt.next();     // (V's stages)
        }
        if (n + 1 == steps) tc_commit_one(&b.q_empty);
      }
    }
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(&b.item_empty[it.at]);
    it.next();
  }
}

// ---------------------------------------------------------------- cleaner
template <class T, class C>
__device__ __forceinline__ bool clean(const ChunkParams& p, Smem& sm,
                                      uint8_t* smem) {
  constexpr int NS = C::NS, S = C::S, U = C::U;
  const int lane = (int)lane_id();
  Bars& b = sm.bars;
  volatile int* stop = &sm.abort_flag;
  Turn<S> st;
  Turn<kItems> it;
  Turn<kMetas> mt;
  for (;;) {
    if (!warp_wait(&b.item_full[it.at], it.phase, stop)) return false;
    const Item item = sm.items[it.at];
    __syncwarp();
    if (lane == 0) mbar_arrive(&b.item_empty[it.at]);
    it.next();
    if (item.units == 0) return true;
    const int64_t pf = item.pf, pl = pf + item.ntok - 1;
    for (int k = 0; k < item.units; ++k) {
      if (!warp_wait(&b.meta[mt.at], mt.phase, stop)) return false;
      Meta& m = sm.metas[mt.at];
      const int32_t t0 = m.t0;
      const uint32_t pages = m.pages;
      const bool mixed = m.mixed;
      for (int s = 0; s < NS; ++s) st.next();     // K's
      uint32_t found[4] = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        if (!warp_wait(&b.full[mt.at][1][s], mt.phase, stop)) return false;
        if (mixed) {
          uint8_t* tile = smem + C::kRing + st.at * C::kStage;
          // four tokens at a time, eight lanes each
#pragma unroll 1
          for (int g = 0; g < U / 4; ++g) {
            const int row = g * 4 + lane / 8;
            const int64_t t = (int64_t)t0 + row;
            const bool none =
                !((pages >> (row / kBlock)) & 1) || t > pl ||
                (p.window && t >= p.sink && t <= pf - p.window);
            const bool every = t <= pf && (!p.window || t < p.sink ||
                                           t > pl - p.window);
            if (!__any_sync(~0u, none || !every)) continue;
            bool odd = false;
#pragma unroll
            for (int sl = 0; sl < C::kSlabs; ++sl) {
              uint4* at = reinterpret_cast<uint4*>(
                  tile + (row / kBlock * C::kSlabs + sl) * 2048 +
                  row % kBlock * 128 + (lane % 8) * 16);
              if (none) {
                *at = make_uint4(0, 0, 0, 0);
              } else if (!every) {
                const uint4 w = *at;
                const uint32_t o[4] = {odd_of<T>(w.x), odd_of<T>(w.y),
                                       odd_of<T>(w.z), odd_of<T>(w.w)};
                if (o[0] | o[1] | o[2] | o[3]) {
                  odd = true;
                  // (bit 15 of a half: all of its 16 bits)
                  auto keep = [](uint32_t x, uint32_t bits) {
                    return x & ~((bits >> 15) * 0xFFFFu);
                  };
                  *at = make_uint4(keep(w.x, o[0]), keep(w.y, o[1]),
                                   keep(w.z, o[2]), keep(w.w, o[3]));
                }
              }
            }
            const uint32_t who = __ballot_sync(~0u, odd);
            if (who) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if ((who >> (8 * e)) & 0xFF) {
                  const int at = g * 4 + e;
#pragma unroll
                  for (int w = 0; w < 4; ++w)
                    if (at / 32 == w) found[w] |= 1u << (at % 32);
                }
            }
          }
          if (s == NS - 1 && lane == 0) {
#pragma unroll
            for (int w = 0; w < 4; ++w) m.odd[w] = found[w];
          }
          fence_proxy_async_smem();
        }
        st.next();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&b.clean[mt.at]);
      mt.next();
    }
  }
}

// ---------------------------------------------------------------- softmax
// Of a unit's tokens whose V held infinities or NaN, those that this row
// attends to with a weight above 0 and with one of 0.
__device__ __noinline__ void find_odd(const ChunkParams& p, const Meta& meta,
                                      int64_t pos, uint32_t s_at,
                                      uint32_t (&has)[4],
                                      uint32_t (&none)[4]) {
#pragma unroll 1
  for (int w = 0; w < 4; ++w) {
    const uint32_t seen = seen_bits(p, meta, pos, w);
    has[w] = none[w] = 0;
#pragma unroll 1
    for (uint32_t x = meta.odd[w]; x; x &= x - 1) {
      const int bit = __ffs(x) - 1;
      const uint32_t word = tmem_ld1(s_at + w * 16 + bit / 2);
      tmem_wait_ld();
      const uint32_t half = bit & 1 ? word >> 16 : word & 0xFFFFu;
      if ((seen >> bit) & 1) {
        if (half) has[w] |= 1u << bit; else none[w] |= 1u << bit;
      }
    }
  }
}
// Infinities and NaN that the cleaner took out of V, for the rows that attend
// to them: v times the row's weight, added to O behind the unit's product.
// `has`: tokens of the unit that this row attends to with a weight above 0,
// `none`: with one of 0.
template <class T, int HD>
__device__ __noinline__ void add_odd(const ChunkParams& p, const Item& item,
                                     int32_t t0, const uint32_t (&odd)[4],
                                     const uint32_t (&has)[4],
                                     const uint32_t (&none)[4], uint32_t o) {
  for (int w = 0; w < 4; ++w) {
    for (uint32_t m = odd[w]; m; m &= m - 1) {
      const int bit = __ffs(m) - 1;
      const int64_t t = (int64_t)t0 + 32 * w + bit;
      const int64_t id =
          p.table[(int64_t)item.r * p.max_blocks + t / kBlock];
      const T* v = static_cast<const T*>(p.v) +
                   ((id * kBlock + t % kBlock) * p.kv_heads + item.j) * HD;
      const float weight = (has[w] >> bit) & 1    ? 1.f
                           : (none[w] >> bit) & 1 ? 0.f
                                                  : -1.f;
#pragma unroll 1
      for (int c = 0; c < HD; c += 16) {
        float acc[16];
        tmem_ld16(o + c, acc);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 x = Elem<T>::unpack(
              reinterpret_cast<const uint32_t*>(v + c)[e]);
          if (weight >= 0.f && !isfinite(x.x)) acc[2 * e] += x.x * weight;
          if (weight >= 0.f && !isfinite(x.y)) acc[2 * e + 1] += x.y * weight;
        }
        uint32_t r[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(acc[e]);
        tmem_st16(o + c, r);
        tmem_wait_st();
      }
    }
  }
}

template <int N>
__device__ __forceinline__ float row_max(const float (&s)[N]) {
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < N; c += 8) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      top[e] = fmaxf(fmaxf(top[e], s[c + 2 * e]), s[c + 2 * e + 1]);
  }
  return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
}
// Four rows' 64 bytes each, a row a lane, to four pieces of 16 bytes a lane:
// piece lane % 4 of the four rows, so that a store covers 64 bytes of a row.
__device__ __forceinline__ void transpose4(uint4 (&v)[4], int lane) {
#pragma unroll
  for (int d = 1; d <= 2; d <<= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint4& a = v[d == 1 ? 2 * k : k];
      uint4& z = v[d == 1 ? 2 * k + 1 : k + 2];
      const uint4 give = up ? a : z;
      uint4 get;
      get.x = __shfl_xor_sync(~0u, give.x, d);
      get.y = __shfl_xor_sync(~0u, give.y, d);
      get.z = __shfl_xor_sync(~0u, give.z, d);
      get.w = __shfl_xor_sync(~0u, give.w, d);
      if (up) a = get; else z = get;
    }
  }
}

template <class T, class C>
__device__ __forceinline__ bool soften(const ChunkParams& p, Smem& sm,
                                       uint32_t tmem, int warp) {
  constexpr int HD = C::HD, U = C::U;
  const int lane = (int)lane_id(), wg = warp >> 2;
  const int row = (warp & 3) * 32 + lane;
  const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
  const uint32_t o_at = lanes + C::kO + wg * 128;
  Bars& b = sm.bars;
  volatile int* stop = &sm.abort_flag;
  Turn<kItems> it;
  Turn<kMetas> mt;
  uint32_t s_phase = 0;          // a bit per barrier
  uint32_t pv_phase = 0;         // of the next product
  uint32_t lone_phase = 0;
  const float shift = Elem<T>::kShift;
  const int tok = row / p.group, head = row - tok * p.group;
  for (;;) {
    if (!warp_wait(&b.item_full[it.at], it.phase, stop)) return false;
    const Item item = sm.items[it.at];
    __syncwarp();
    if (lane == 0) mbar_arrive(&b.item_empty[it.at]);
    it.next();
    if (item.units == 0) return true;
    const bool dual = item.flags & kDual;
    // of a lone tile every second unit is this chain's
    const bool lone = C::kChains == 2 && !dual;
    const int32_t mine = (dual ? wg * p.tq : 0) + tok;    // the row's token
    const int64_t pos = (int64_t)item.pf + mine;
    const bool valid = tok < p.tq && mine < item.ntok;
    float m = -INFINITY;
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    bool first = true;
    for (int k = 0; k < item.units; ++k, mt.next()) {
      if (lone && (k & 1) != wg) continue;
      const int bar = C::kChains == 1 ? k & 1 : wg;
      const uint32_t s_at = lanes + bar * 128;
      if (!warp_wait(&b.meta[mt.at], mt.phase, stop)) return false;
      if (!warp_wait(&b.s_full[bar], (s_phase >> bar) & 1, stop)) return false;
      s_phase ^= 1u << bar;
      tc_fence_after();
      const Meta& meta = sm.metas[mt.at];
      const bool mixed = meta.mixed;
      float s[U];
#pragma unroll
      for (int c = 0; c < U; c += 32) tmem_ld32(s_at + c, s + c);
      tmem_wait_ld();
      if (mixed) {
#pragma unroll
        for (int w = 0; w < U / 32; ++w) {
          const uint32_t seen = seen_bits(p, meta, pos, w);
          if (__all_sync(~0u, seen == ~0u)) continue;
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!((seen >> c) & 1)) s[w * 32 + c] = -INFINITY;
        }
      }
      // A unit's weights are formed with the reference as it stands, beside
      // its maximum; the rare unit that moves the reference is gone through
      // again.  (The maximum first: 250 cycles more from S to P.)
      if (first) m = row_max(s) * p.scale;
      float2 part[2];
#pragma unroll 1
      for (;;) {
        // 0 where no score is finite; a score of +inf gives NaN
        const float base = m == -INFINITY  ? 0.f
                           : m == INFINITY ? __int_as_float(0x7FC00000)
                                           : m;
        const float2 scale2 = make_float2(p.scale, p.scale);
        const float2 base2 = make_float2(shift - base, shift - base);
        part[0] = part[1] = make_float2(0.f, 0.f);
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < U; c += 32) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float a = s[c + 2 * e], z = s[c + 2 * e + 1];
            const float2 x = fma2(make_float2(a, z), scale2, base2);
            const float2 y = make_float2(exp2_fast(x.x), exp2_fast(x.y));
            top[e & 1] = fmaxf(fmaxf(top[e & 1], a), z);
            part[e & 1] = add2(part[e & 1], y);
            w[e] = Elem<T>::pack(y.x, y.y);
          }
          tmem_st16(s_at + c / 2, w);
        }
        const float most = fmaxf(top[0], top[1]) * p.scale;
        const bool moves = most > m + kSlack;
        if (!__any_sync(~0u, moves)) break;
        const float factor = moves ? exp2_fast(m - most) : 1.f;
        if (moves) m = most;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sum[e].x *= factor;
          sum[e].y *= factor;
        }
        if (!first) {
          if (!warp_wait(&b.pv_done[wg], pv_phase ^ 1, stop)) return false;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < HD; c += 16) {
            float o[16];
            tmem_ld16(o_at + c, o);
            tmem_wait_ld();
            uint32_t r[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(o[e] * factor);
            tmem_st16(o_at + c, r);
          }
        }
      }
      sum[0] = add2(sum[0], part[0]);
      sum[1] = add2(sum[1], part[1]);
      tmem_wait_st();
      // infinities and NaN of V, rarely
      uint32_t odd[4] = {0, 0, 0, 0}, has[4], none[4];
      bool any_odd = false;
      int32_t t0 = 0;
      if (mixed) {
        if (!warp_wait(&b.clean[mt.at], mt.phase, stop)) return false;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          odd[w] = meta.odd[w];
          any_odd |= odd[w] != 0;
        }
        if (any_odd) {
          t0 = meta.t0;
          find_odd(p, meta, pos, s_at, has, none);
        }
      }
      // With one chain the last product may still be under way (with two it
      // ended before this S): a second one behind it would make its phase of
      // the barrier look like the one before.
      if (C::kChains == 1 && !first &&
          !warp_wait(&b.pv_done[0], pv_phase ^ 1, stop))
        return false;
      first = false;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b.p_full[bar]);
      pv_phase ^= 1;
      if (any_odd) {
        if (!warp_wait(&b.pv_done[wg], pv_phase ^ 1, stop)) return false;
        tc_fence_after();
        add_odd<T, HD>(p, item, t0, odd, has, none, o_at);
      }
    }
    // the item's result, or this block's part of it
    if (first) continue;         // (a lone tile's only unit was chain 0's)
    if (!warp_wait(&b.pv_done[wg], pv_phase ^ 1, stop)) return false;
    tc_fence_after();
    float l = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
    const bool joins = lone && item.units > 1;
    float mine_f = 1.f, their_f = 0.f;
    if (joins && wg) {
      sm.lone[row] = make_float2(m, l);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b.ready);
      // (O of this chain is read by the other)
      if (!warp_wait(&b.taken, lone_phase, stop)) return false;
      lone_phase ^= 1;
      tc_fence_after();
      continue;
    }
    if (joins) {
      if (!warp_wait(&b.ready, lone_phase, stop)) return false;
      lone_phase ^= 1;
      tc_fence_after();
      const float2 their = sm.lone[row];
      const float top = fmaxf(m, their.x);
      const float base = top == -INFINITY ? 0.f : top;
      mine_f = exp2_fast(m - base);
      their_f = exp2_fast(their.x - base);
      m = top;
      l = l * mine_f + their.y * their_f;
    }
    const bool whole =
        (item.flags & (kStarts | kEnds)) == (kStarts | kEnds);
    const float inv = l == 0.f ? 0.f : rcp_fast(l);
    const int64_t n = item.row0 + mine;
    const int h = item.j * p.group + head;
    T* out = static_cast<T*>(p.out) + lane % 4 * 8;
    // where the rows of this lane's four go
    const int64_t to = valid ? n * p.out_ld + (int64_t)h * HD : -1;
    int64_t at[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) at[e] = __shfl_sync(~0u, to, (lane & ~3) + e);
    float* part = p.slots + ((int64_t)(blockIdx.x * 2 +
                                       (item.flags & kStarts ? 1 : 0)) *
                                 C::QT + wg) * C::kPart;
#pragma unroll 1
    for (int c = 0; c < HD; c += 32) {
      float o[32];
      tmem_ld32(o_at + c, o);
      tmem_wait_ld();
      if (joins) {             // with the other chain's part
        float x[32];
        tmem_ld32(o_at + 128 + c, x);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = o[e] * mine_f + x[e] * their_f;
      }
      if (whole) {
        uint4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int f = 0; f < 4; ++f)
            w[f] = Elem<T>::pack(
                l == 0.f ? 0.f : o[8 * e + 2 * f] * inv,
                l == 0.f ? 0.f : o[8 * e + 2 * f + 1] * inv);
          v[e] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        transpose4(v, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (at[e] >= 0) *reinterpret_cast<uint4*>(out + at[e] + c) = v[e];
      } else if (valid) {
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          reinterpret_cast<float4*>(part)[(c + e) / 4 * kRows + row] =
              make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
      }
    }
    if (valid && whole && p.lse)
      p.lse[n * p.heads + h] =
          l == 0.f ? -INFINITY : (m + (log2f(l) - shift)) * kLn2;
    if (valid && !whole) {
      part[HD * kRows + row] = m;
      part[HD * kRows + kRows + row] = l;
    }
    // (the next product into O comes after the next arrival at p_full)
    tc_fence_before();
    if (joins) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&b.taken);
    }
  }
}

// ------------------------------------------------------------------ kernel
template <class T, int HD>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ ChunkParams p) {
  using C = Cfg<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Smem& sm = *reinterpret_cast<Smem*>(smem + C::kMisc);
  Bars& b = sm.bars;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < kMetas * 4; ++i)
      mbar_init(&b.full[i / 4][i / 2 % 2][i % 2], 1);
    for (int i = 0; i < C::S; ++i) mbar_init(&b.empty[i], 1);
    mbar_init(&b.q_full, 1);
    mbar_init(&b.q_empty, 1);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&b.item_full[i], 1);
      mbar_init(&b.item_empty[i], 4 * C::kChains + 2);  // (MMA, cleaner)
    }
    for (int i = 0; i < kMetas; ++i) {
      mbar_init(&b.meta[i], 1);
      mbar_init(&b.clean[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.s_full[i], 1);
      mbar_init(&b.p_full[i], 4);
      mbar_init(&b.pv_done[i], 1);
    }
    mbar_init(&b.fin, 1);
    mbar_init(&b.ready, 4);
    mbar_init(&b.taken, 4);
    sm.abort_flag = 0;
    prefetch_tmap(&p.tm_q);
    prefetch_tmap(&p.tm_k);
    prefetch_tmap(&p.tm_v);
  }
  fence_mbar_init();
  // Everything this call reads may come from the launch before it.  (TMEM is
  // taken behind this wait, too: a block of that launch may need it.)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == kMma) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  // costs of the requests, and their sums
  int64_t* pre = reinterpret_cast<int64_t*>(smem + C::kRing);
  const int32_t per = C::QT * p.tq;
  for (int r0 = warp * 32; r0 < p.R; r0 += kThreads) {
    const Request q = request(p, r0 + lane);
    const int items = parts_of(q.n, per);
    int64_t cost = 0;
    constexpr int kOwn = 4;             // items that a lane sums itself
    if (items <= kOwn)
      for (int i = 0; i < items; ++i)
        cost += item_cost<C::U>(p, q.n, q.len, i, per);
    for (uint32_t m = __ballot_sync(~0u, items > kOwn); m; m &= m - 1) {
      const int l = __ffs(m) - 1;
      const int32_t n = __shfl_sync(~0u, q.n, l);
      const int32_t len = __shfl_sync(~0u, q.len, l);
      int64_t part = 0;
      for (int i = lane; i < parts_of(n, per); i += 32)
        part += item_cost<C::U>(p, n, len, i, per);
#pragma unroll
      for (int d = 16; d; d >>= 1) part += __shfl_xor_sync(~0u, part, d);
      if (lane == l) cost = part;
    }
    if (r0 + lane < p.R) pre[r0 + lane] = cost * p.kv_heads;
    if (blockIdx.x == 0 && p.flags && r0 + lane < p.R &&
        (p.lens[r0 + lane] > p.max_blocks * kBlock ||
         p.cu[r0 + lane + 1] > p.N))
      atomicOr(p.flags, KVTC_FLAG_SPACE);
  }
  __syncthreads();
  {
    const int each = (p.R + kThreads - 1) / kThreads;
    int64_t sum = 0;
    for (int i = 0; i < each; ++i) {
      const int r = tid * each + i;
      if (r < p.R) sum += pre[r];
    }
    int64_t upto = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(~0u, upto, d);
      if (lane >= d) upto += o;
    }
    if (lane == 31) sm.sums[warp] = upto;
    __syncthreads();
    for (int w = 0; w < warp; ++w) upto += sm.sums[w];
    int64_t before = upto - sum;
    for (int i = 0; i < each; ++i) {
      const int r = tid * each + i;
      if (r < p.R) {
        const int64_t cost = pre[r];
        pre[r] = before;
        before += cost;
      }
    }
    if (tid == kThreads - 1) pre[p.R] = upto;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = sm.tmem, base = smem_u32(smem);
  bool ok = true;
  // The launch gives every thread 168 registers (384 x 168); a row of S takes
  // 128: 256 x 208 + 128 x 88 is the same number.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    if (warp < 4 * C::kChains) ok = soften<T, C>(p, sm, tmem, warp);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == kProducer) {
      ok = produce<T, C>(p, sm, base, pre);
    } else if (warp == kMma) {
      ok = multiply<T, C>(p, sm, base, uniform(tmem));
      // products under way end before the block's memory is given up
      __syncwarp();
      tc_commit_one(&b.fin);
      mbar_drain(&b.fin, 0);
      __syncwarp();
    } else if (warp == kCleaner) {
      ok = clean<T, C>(p, sm, smem);
    }
  }
  if (!ok) {
    *(volatile int*)&sm.abort_flag = 1;
    if (p.flags) atomicOr(p.flags, KVTC_FLAG_TIMEOUT);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(tmem, 512);
}

// Parts of items that cross blocks: block x joins the one begun in block x (or
// where there are few, the x-th of them), row tile y, 16 channels z.  A thread
// has a row and every kSplit-th part; the threads of a row then join theirs by
// halves.
constexpr int kJoinCh = 16;
struct Joined {
  float m, l, o[kJoinCh];
  __device__ __forceinline__ void add(float mi, float li,
                                      const float (&x)[kJoinCh]) {
    const float top = fmaxf(m, mi);
    const float base = top == -INFINITY ? 0.f : top;
    const float fo = exp2_fast(m - base), fi = exp2_fast(mi - base);
    m = top;
    l = l * fo + li * fi;
#pragma unroll
    for (int e = 0; e < kJoinCh; ++e) o[e] = o[e] * fo + x[e] * fi;
  }
};
template <class T, int HD, int kSplit>
__global__ void __launch_bounds__(kRows * kSplit)
    chunk_join_kernel(const __grid_constant__ ChunkParams p) {
  using C = Cfg<HD>;
  constexpr int kHalf = kSplit > 1 ? kSplit / 2 : 1;
  __shared__ float other[kHalf][kJoinCh + 2][kRows];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tile = blockIdx.y, ch = blockIdx.z * kJoinCh;
  int c = blockIdx.x;
  if (kSplit > 1) {
    // the c-th block that began an item that is to be joined
    constexpr int kEach = (kCtas + 31) / 32;
    uint32_t began[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int at = 32 * i + (int)lane_id();
      began[i] = __ballot_sync(~0u, at < kCtas && p.desc[at].r >= 0);
    }
    int left = c;
    c = -1;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int n = __popc(began[i]);
      if (left >= 0 && left < n) c = 32 * i + (int)__fns(began[i], 0, left + 1);
      left -= n;
    }
    if (c < 0) return;
  }
  const JoinDesc d = p.desc[c];
  if (d.r < 0) return;
  const int row = threadIdx.x % kRows, group = threadIdx.x / kRows;
  const int tok = row / p.group, head = row - tok * p.group;
  const int32_t mine = tile * p.tq + tok;
  const bool valid = tok < p.tq && mine < d.ntok;
  const int parts = valid ? d.last - c + 1 : 0;
  Joined a;
  a.m = -INFINITY;
  a.l = 0.f;
#pragma unroll
  for (int e = 0; e < kJoinCh; ++e) a.o[e] = 0.f;
#pragma unroll 2
  for (int i = group; i < parts; i += kSplit) {
    const float* part =
        p.slots +
        ((int64_t)((c + i) * 2 + (i == 0 ? 1 : 0)) * C::QT + tile) * C::kPart;
    const float mi = part[HD * kRows + row];
    const float li = part[HD * kRows + kRows + row];
    float x[kJoinCh];
#pragma unroll
    for (int e = 0; e < kJoinCh; e += 4) {
      const float4 w = reinterpret_cast<const float4*>(
          part)[(ch + e) / 4 * kRows + row];
      x[e] = w.x;
      x[e + 1] = w.y;
      x[e + 2] = w.z;
      x[e + 3] = w.w;
    }
    a.add(mi, li, x);
  }
#pragma unroll
  for (int half = kSplit / 2; half; half /= 2) {
    if (group >= half && group < 2 * half) {
      float(&to)[kJoinCh + 2][kRows] = other[group - half];
      to[kJoinCh][row] = a.m;
      to[kJoinCh + 1][row] = a.l;
#pragma unroll
      for (int e = 0; e < kJoinCh; ++e) to[e][row] = a.o[e];
    }
    __syncthreads();
    if (group < half) {
      const float(&from)[kJoinCh + 2][kRows] = other[group];
      float x[kJoinCh];
#pragma unroll
      for (int e = 0; e < kJoinCh; ++e) x[e] = from[e][row];
      a.add(from[kJoinCh][row], from[kJoinCh + 1][row], x);
    }
    __syncthreads();
  }
  if (!valid || group) return;
  const float inv = a.l == 0.f ? 0.f : rcp_fast(a.l);
  const int64_t n = d.row0 + mine;
  const int h = d.j * p.group + head;
  T* out = static_cast<T*>(p.out) + n * p.out_ld + (int64_t)h * HD + ch;
#pragma unroll
  for (int e = 0; e < kJoinCh; e += 8) {
    uint32_t w[4];
#pragma unroll
    for (int f = 0; f < 4; ++f)
      w[f] = Elem<T>::pack(a.l == 0.f ? 0.f : a.o[e + 2 * f] * inv,
                           a.l == 0.f ? 0.f : a.o[e + 2 * f + 1] * inv);
    *reinterpret_cast<uint4*>(out + e) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (p.lse && ch == 0)
    p.lse[n * p.heads + h] =
        a.l == 0.f ? -INFINITY
                   : (a.m + (log2f(a.l) - Elem<T>::kShift)) * kLn2;
}

template <class T, int HD>
cudaError_t launch_as(const ChunkParams& p, int device, cudaStream_t st) {
  using C = Cfg<HD>;
  static std::atomic<uint64_t> ready;          // devices, as bits
  const auto kernel = chunk_kernel<T, HD>;
  cudaError_t e = allow_smem(kernel, C::kBytes, device, ready);
  if (e == cudaSuccess)
    e = launch_kernel(kernel, kCtas, kThreads, C::kBytes, st, true, 0, p);
  if (e != cudaSuccess) return e;
  count_launch();
  if (p.whole) return e;
  const dim3 grid(p.split ? p.split : kCtas, C::QT, HD / kJoinCh);
  e = p.split ? launch_kernel(chunk_join_kernel<T, HD, 8>, grid, kRows * 8, 0,
                              st, true, 0, p)
              : launch_kernel(chunk_join_kernel<T, HD, 1>, grid, kRows, 0, st,
                              true, 0, p);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <class T>
cudaError_t launch(const ChunkParams& p, int head_dim, int device,
                   cudaStream_t st) {
  return head_dim == 64    ? launch_as<T, 64>(p, device, st)
         : head_dim == 128 ? launch_as<T, 128>(p, device, st)
                           : launch_as<T, 256>(p, device, st);
}

constexpr int64_t kDescBytes =
    (kCtas * sizeof(JoinDesc) + 255) / 256 * 256;
template <int HD>
constexpr int64_t part_bytes() {
  return 4ll * kCtas * 2 * Cfg<HD>::QT * Cfg<HD>::kPart;
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
  return kDescBytes + (head_dim == 64    ? part_bytes<64>()
                       : head_dim == 128 ? part_bytes<128>()
                                         : part_bytes<256>());
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
  p.group = heads / kv_heads;
  p.tq = kRows / p.group;
  const uint64_t D = (uint64_t)kv_heads * head_dim;
  if (!encode_pages(&p.tm_k, k_cache, D, num_blocks, 1) ||
      !encode_pages(&p.tm_v, v_cache, D, num_blocks,
                    head_dim == 64 ? 1 : 2) ||
      !encode_rows(&p.tm_q, q, head_dim, heads, N, q_ld, p.group, p.tq))
    return KVTC_ECUDA;
  p.table = block_table;
  p.cu = cu;
  p.lens = lens;
  p.v = v_cache;
  p.out = out;
  p.lse = lse;
  p.flags = flags;
  p.desc = static_cast<JoinDesc*>(workspace);
  p.slots = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                     kDescBytes);
  p.N = N;
  p.out_ld = out_ld;
  p.num_blocks = num_blocks;
  // (the maximum is taken of the products, before the scale; that of 0 is the
  // smallest number, so that -inf stays what it is for tokens left out)
  p.negate = scale < 0.f;
  p.scale = std::max(std::fabs(scale) * kLog2e, 0x1p-149f);
  p.R = R;
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.max_blocks = max_blocks;
  p.sink = window ? sink : 0;
  p.window = window;
  // Few items that are short whatever the lengths are (the table is narrow) go to
  // a block each, without the second launch, which is worth about eight units of
  // one block: 8 x 128 tokens (8 KV heads, 16 rows, lengths of 128, 512 and 1024:
  // 12.2, 16.7 and 22.0 us from a graph against 19.7, 21.7 and 24.7 in runs that
  // are joined; at head_dim 64 11.3, 14.7 and 19.2 against 17.0, 18.8 and 21.0),
  // at head_dim 256 8 x 64 (256, 512, 768 and 1024 tokens: 18.2, 24.3, 30.2 and
  // 36.3 against 23.1, 26.1, 25.9 and 26.7).  Where more than half of the blocks
  // have an item, longer ones too: runs cut few of them (136 items at head_dim
  // 256, 768 and 1024 tokens: 29.5 and 35.4 against 33.6 and 39.7; 60 items 27.7
  // and 33.8 against 23.5 and 24.3).
  const int per = p.tq * (head_dim == 256 ? 1 : 2);
  const int64_t items = (int64_t)kv_heads * ((N + per - 1) / per + R);
  const int unit = head_dim == 256 ? 64 : 128;
  p.whole = items <= kCtas && max_blocks <= 8 * 128 / kBlock &&
            (max_blocks <= 8 * unit / kBlock || items > kCtas / 2);
  // Few items are cut into many parts each, which eight threads a row join (64
  // rows behind 128K tokens, one head: 95 us a call with one thread a row, 31 with
  // eight; 36 items 43 and 40).  More items have few parts, and so many threads
  // cost more than they save (68 items 60 and 66, 144 items 43 and 67).
  p.split = items <= kCtas / 4 ? (int32_t)items : 0;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = dtype == KVTC_DTYPE_BF16
                            ? launch<__nv_bfloat16>(p, head_dim, cuda_device, st)
                            : launch<__half>(p, head_dim, cuda_device, st);
  return e == cudaSuccess ? KVTC_OK : KVTC_ECUDA;
}

}  // extern "C"
