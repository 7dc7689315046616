// The attention weight that cached tokens receive:
//     acc_out[t] = decay acc[t] + sum over rows i and heads h of
//                  e^(scale q_ih . k_t - lse_ih),
// with the log-sum-exp that the attention of the same rows returned, so K is
// read once and nothing but the sums is written.
//
// The products are formed transposed, S^T = K Q^T: 128 tokens (eight of each of
// 16 pages) fill the 128 lanes of TMEM and the (row, head) pairs of a KV head
// the columns, so that a thread owns a token, adds up its columns in a
// register, and nothing is summed across threads.  Few pairs (a decode step: the heads of one row) make
// a narrow product, down to 16 columns.
//
// Rounding.  Scores are summed by the tensor cores in fp32, which cut a sum off
// where others round it, so that weights are too small by half a step of the
// score (one of 20 in natural units: 5e-7) rather than off to either side;
// scale s - lse is formed in one instruction, in log2, the sums in fp32.  (The
// difference formed before the factor log2 e, and half a step given back: 1.4
// times as far from 64 bits as fp32 throughout instead of 1.9 times, and 99 us
// instead of 93 for 16 requests of 32 rows.)
//
// Work.  An item is (request, 256 tokens), a unit one KV head of an item.  All
// units are dealt out to one block per SM in equal runs; a block whose run
// begins or ends inside an item leaves its part of the sums, which
// weigh_join_kernel adds in a fixed order.  Tokens that no row attends to (a
// gap between sink and window, a request without rows) are items of one unit
// and no products.
//
// Inside a block: a producer warp (K pages and rows of Q by TMA into two
// rings), an MMA warp, two warps that fetch the log-sum-exps, and two
// warpgroups, a thread per token, which take the products from two buffers in
// TMEM.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "../../include/kvtc.h"
#include "kvtc_chunk.cuh"
#include "kvtc_internal.cuh"

namespace kvtc {
namespace {

constexpr int kThreads = 384;
constexpr int kProducer = 8, kMma = 9, kFetch = 10;   // (and 11)
constexpr int kTile = 256;           // tokens of an item
constexpr int kPages = kTile / kBlock;
constexpr int kCols = 128;           // columns of a product
constexpr int kItems = 4;
constexpr int kBoxes = 8;            // tokens of Q at once: 1, 2, ... 128

struct __align__(16) JoinDesc {
  int32_t r, t0, last, pad;          // r < 0: nothing to join
};

struct WeighParams {
  CUtensorMap tm_q[kBoxes];  // {64, HD / 64, heads, N}, box {64, 1, group, x}
  CUtensorMap tm_k;
  const int32_t* table;
  const int64_t* cu;
  const int32_t* lens;
  const float* lse;
  const float* acc;
  float* acc_out;
  unsigned* flags;
  JoinDesc* desc;            // [kCtas]
  float* slots;              // [kCtas][2][kTile]: 0 of an item begun in an
                             // earlier block, 1 of one begun in this block
  int64_t N, num_blocks, acc_ld;
  float scale, decay;        // scale times log2 e
  int32_t R, heads, kv_heads, max_blocks, sink, window;
  int32_t group, tq;         // query heads a KV head; rows per product
};

template <int HD_>
struct Cfg {
  static constexpr int HD = HD_;
  static constexpr int SC = HD < 128 ? HD : 128;      // channels per stage
  static constexpr int NS = HD / SC;                  // stages per tile
  static constexpr int kSlabs = SC / 64;
  static constexpr int kPage = kSlabs * 2048;         // bytes of a page
  static constexpr int kStageK = kPages * kPage;      // both token tiles'
  static constexpr int kStage = kRows * SC * 2;       // of Q
  static constexpr int SK = HD == 64 ? 4 : 2;         // stages of K
  static constexpr int SQ = HD == 64 ? 4 : 3;         // stages of Q
  static constexpr int kQ = SK * kStageK;
  static constexpr int kMisc = kQ + SQ * kStage;
  static constexpr int kBytes = kMisc + 2048 + 1024;  // + alignment slack
  static_assert(kBytes <= 232448, "shared memory of a block");
  static_assert(SK * kStageK >= 8 * (kMaxReq + 1), "prefix of the requests");
};

struct __align__(16) Item {
  int64_t row0;              // first row of the request
  int32_t r, t0, n, pf;      // rows, position of the first
  int32_t j0, j1;            // KV heads of this block
  int32_t steps;             // products per KV head; 0: none to be formed
  int32_t len;
  uint32_t pages;            // pages that are there
  int32_t flags;
};
constexpr int kStarts = 1, kEnds = 2, kStop = 4;

struct Bars {
  uint64_t k_full[4], k_empty[4], q_full[4], q_empty[4];
  uint64_t item_full[kItems], item_empty[kItems];
  // buffer, token tile: products and log-sum-exps are there; products have
  // been read; log-sum-exps too
  uint64_t s_full[2][2], s_empty[2][2], l_empty[2];
  uint64_t fin;
};
struct Smem {
  Bars bars;
  Item items[kItems];
  int64_t sums[kThreads / 32];
  uint32_t tmem;
  int abort_flag;
  uint32_t dead[2];     // columns without weight, a bit per 32
  __align__(16) float lse[2][kCols];   // minus log-sum-exp, in log2
};
static_assert(sizeof(Smem) <= 2048, "the kernel's shared variables");

// A request's token tiles: those that rows attend to come first (`front` at
// their own place, the others `gap` further on), then those of the gap.
struct Tiles {
  int32_t all, live, front, gap, steps;
  __device__ __forceinline__ Tiles(const WeighParams& p, const Request& q) {
    all = parts_of(q.len, kTile);
    front = live = q.n ? all : 0;
    gap = 0;
    steps = parts_of(q.n, p.tq);
    if (p.window && q.n) {
      const int64_t lo = (int64_t)q.len - q.n - p.window + 1;
      const int32_t back = lo > 0 ? (int32_t)min(lo / kTile, (int64_t)all) : 0;
      front = (int32_t)min(((int64_t)p.sink + kTile - 1) / kTile,
                           (int64_t)all);
      gap = max(back - front, 0);
      live = all - gap;
    }
  }
  // (of what the host sees as i: the tile, and whether it is a live one)
  __device__ __forceinline__ int32_t tile(int32_t i) const {
    return i < front ? i : i < live ? i + gap : i - live + front;
  }
  __device__ __forceinline__ int64_t cost(const WeighParams& p) const {
    return (int64_t)live * p.kv_heads * steps + (all - live);
  }
};

__device__ __forceinline__ Request request(const WeighParams& p, int r) {
  return Request(p.cu, p.lens, p.N, p.R, p.max_blocks, r);
}

// --------------------------------------------------------------- producer
template <class T, class C>
__device__ __forceinline__ bool produce(const WeighParams& p, Smem& sm,
                                        uint32_t smem, const int64_t* pre) {
  constexpr int HD = C::HD, NS = C::NS;
  const int lane = (int)lane_id();
  Bars& b = sm.bars;
  volatile int* stop = &sm.abort_flag;
  Turn<C::SK> kt;
  Turn<C::SQ> qt;
  Turn<kItems> it;
  int k_fills = 0, q_fills = 0;
  const Deal deal(pre[p.R], 1);
  int64_t x = deal.begin(blockIdx.x);
  const int64_t end = deal.begin(blockIdx.x + 1);
  int r = 0;
  if (x < end) {
    int lo = 0, hi = p.R;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= x) lo = mid; else hi = mid;
    }
    r = lo;
  }
  int64_t y = x - pre[r];              // x within the request
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
    const Tiles tiles(p, q);
    const int64_t cost = tiles.cost(p);
    if (y >= cost) {                   // (an empty request, or the next one)
      ++r;
      y = 0;
      continue;
    }
    const int64_t each = (int64_t)p.kv_heads * tiles.steps;
    const bool live = y < tiles.live * each;
    // the item, where y lies in it, and the KV heads that begin in this run
    const int32_t i = (int32_t)(live ? y / each : y - tiles.live * each +
                                                      tiles.live);
    const int64_t in = live ? y - i * each : 0;
    const int64_t all = live ? each : 1;
    const int64_t upto = min(all, in + (end - x));
    const int32_t steps = live ? tiles.steps : 0;
    const int j0 = live ? (int)((in + steps - 1) / steps) : 0;
    const int j1 = live ? (int)((upto + steps - 1) / steps) : 1;
    // (a run inside one KV head of an item: nothing for the join to add)
    for (int k = lane; j1 == j0 && k < kTile; k += 32)
      p.slots[blockIdx.x * 2 * kTile + k] = 0.f;
    if (j1 > j0) {
      const int32_t t0 = tiles.tile(i) * kTile;
      const int64_t pf = (int64_t)q.len - q.n, pl = (int64_t)q.len - 1;
      const int page = lane % kPages;
      const int64_t tp = (int64_t)t0 + page * kBlock;
      const bool need = live && tp <= pl &&
                        (!p.window || tp < p.sink ||
                         tp + kBlock - 1 > pf - p.window);
      const int32_t id =
          need ? p.table[(int64_t)r * p.max_blocks + tp / kBlock] : -1;
      const bool fine = id >= 0 && id < p.num_blocks;
      if (need && !fine && lane < kPages && p.flags)
        atomicOr(p.flags, KVTC_FLAG_BLOCK);
      const uint32_t pages = __ballot_sync(~0u, fine) & 0xFFFFu;
      if (!warp_wait(&b.item_empty[it.at], it.phase ^ 1, stop)) {
        ok = false;
        break;
      }
      const bool starts = j0 == 0, ends = !live || j1 == p.kv_heads;
      if (lane == 0) {
        Item d;
        d.row0 = q.c0;
        d.r = r;
        d.t0 = t0;
        d.n = q.n;
        d.pf = (int32_t)pf;
        d.j0 = j0;
        d.j1 = j1;
        d.steps = steps;
        d.len = q.len;
        d.pages = pages;
        d.flags = (starts ? kStarts : 0) | (ends ? kEnds : 0);
        sm.items[it.at] = d;
        mbar_arrive(&b.item_full[it.at]);
        if (starts && !ends) {
          JoinDesc jd;
          jd.r = r;
          jd.t0 = t0;
          // the block in which the last KV head begins
          jd.last = deal.cta_of(x - in + all - steps);
          jd.pad = q.len;
          p.desc[blockIdx.x] = jd;
          left_desc = true;
        }
      }
      it.next();
      for (int j = j0; j < j1 && ok && steps; ++j) {
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          if (!warp_wait(&b.k_empty[kt.at], kt.phase ^ 1, stop)) {
            ok = false;
            break;
          }
          if (lane == 0)
            mbar_arrive_expect_tx(&b.k_full[kt.at], __popc(pages) * C::kPage);
          __syncwarp();
          if (fine && lane < kPages)
            tma_load_4d(smem + kt.at * C::kStageK + page * C::kPage, &p.tm_k,
                        0, 0, j * (HD / 64) + s * C::kSlabs, id,
                        &b.k_full[kt.at]);
          kt.next();
          ++k_fills;
        }
        for (int st = 0; st < steps && ok; ++st) {
          // Q: the box of the fewest tokens that hold the rows
          const int rows = min(p.tq, q.n - st * p.tq);
          const int pow = 32 - __clz(rows - 1);
          const int box = min(1 << pow, p.tq);
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            if (!warp_wait(&b.q_empty[qt.at], qt.phase ^ 1, stop)) {
              ok = false;
              break;
            }
            if (lane == 0)
              mbar_arrive_expect_tx(&b.q_full[qt.at],
                                    C::kSlabs * box * p.group * 128);
            __syncwarp();
            if (lane < C::kSlabs)
              tma_load_4d(smem + C::kQ + qt.at * C::kStage +
                              lane * (kRows * 128),
                          &p.tm_q[pow], 0, s * C::kSlabs + lane, j * p.group,
                          (int32_t)q.c0 + st * p.tq, &b.q_full[qt.at]);
            qt.next();
            ++q_fills;
          }
        }
      }
    }
    const int64_t step = min(all - in, end - x);
    x += step;
    y += step;
  }
  if (ok && warp_wait(&b.item_empty[it.at], it.phase ^ 1, stop)) {
    if (lane == 0) {
      sm.items[it.at].flags = kStop;
      mbar_arrive(&b.item_full[it.at]);
    }
  } else {
    ok = false;
  }
  if (lane == 0 && !left_desc) p.desc[blockIdx.x].r = -1;
  // loads under way land before the block's memory is given up
  __syncwarp();
  if (lane == 0) {
    for (int k = min(k_fills, C::SK); k > 0; --k) {
      if (kt.at-- == 0) {
        kt.at = C::SK - 1;
        kt.phase ^= 1;
      }
      mbar_drain(&b.k_full[kt.at], kt.phase);
    }
    for (int k = min(q_fills, C::SQ); k > 0; --k) {
      if (qt.at-- == 0) {
        qt.at = C::SQ - 1;
        qt.phase ^= 1;
      }
      mbar_drain(&b.q_full[qt.at], qt.phase);
    }
  }
  return ok;
}

// Columns of a product: the (row, head) pairs of up to tq rows, up to a
// multiple of 16.
__device__ __forceinline__ int columns(const WeighParams& p, int n, int st) {
  return (min(p.tq, n - st * p.tq) * p.group + 15) & ~15;
}

// -------------------------------------------------------------------- MMA
template <class T, class C>
__device__ __forceinline__ bool multiply(const WeighParams& p, Smem& sm,
                                         uint32_t smem, uint32_t tmem) {
  constexpr int NS = C::NS, SC = C::SC;
  Bars& b = sm.bars;
  volatile int* stop = &sm.abort_flag;
  Turn<C::SK> kt;
  Turn<C::SQ> qt;
  Turn<kItems> it;
  uint32_t step = 0;                  // over all items
  for (;;) {
    if (!warp_wait(&b.item_full[it.at], it.phase, stop)) return false;
    const Item& item = sm.items[it.at];
    const int flags = uniform(item.flags), steps = uniform(item.steps);
    const int heads = uniform(item.j1 - item.j0), n = uniform(item.n);
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(&b.item_empty[it.at]);
    it.next();
    if (flags & kStop) return true;
    if (steps == 0) continue;
#pragma unroll 1
    for (int j = 0; j < heads; ++j) {
#pragma unroll 1
      for (int st = 0; st < steps; ++st, ++step) {
        const uint32_t buf = step & 1, phase = (step >> 1) & 1;
        const uint32_t idesc =
            make_idesc(kRows, columns(p, n, st), Elem<T>::kFormat);
        Turn<C::SQ> q0 = qt;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          if (!warp_wait(&b.q_full[qt.at], qt.phase, stop)) return false;
          qt.next();
        }
        Turn<C::SK> k = kt;
        Turn<C::SQ> q = q0;
#pragma unroll 1
        for (int s = 0; s < NS; ++s) {
          if (st == 0 && !warp_wait(&b.k_full[k.at], k.phase, stop))
            return false;
          const uint32_t bd = desc_base(smem + C::kQ + q.at * C::kStage);
#pragma unroll 1
          for (int tile = 0; tile < 2; ++tile) {
            if (s == 0 && !warp_wait(&b.s_empty[buf][tile], phase ^ 1, stop))
              return false;
            // (rows 0 .. 7 of the 16 pages, or 8 .. 15)
            tc_fence_after();
            const uint32_t ad =
                desc_base(smem + k.at * C::kStageK + tile * 1024);
            const uint32_t d = tmem + (buf * 2 + tile) * kCols;
#pragma unroll
            for (int e = 0; e < SC / 16; ++e)
              mma_ss_one<desc_high(C::kPage)>(
                  d, ad + (e / 4) * (2048 >> 4) + (e % 4) * 2,
                  bd + (e / 4) * (kRows * 128 >> 4) + (e % 4) * 2, idesc,
                  (s | e) > 0);
            if (s == NS - 1) tc_commit_one(&b.s_full[buf][tile]);
          }
          if (st + 1 == steps) tc_commit_one(&b.k_empty[k.at]);
          k.next();
          q.next();
        }
        for (int s = 0; s < NS; ++s) {
          tc_commit_one(&b.q_empty[q0.at]);
          q0.next();
        }
        if (st + 1 == steps) kt = k;
      }
    }
  }
}

// ------------------------------------------------------- log-sum-exps
// Minus lse log2(e) of a product's columns; -inf where a head has no weight
// to give (no attended token), and behind the last column.
__device__ __forceinline__ bool fetch(const WeighParams& p, Smem& sm,
                                      int which) {
  const int lane = (int)lane_id();
  Bars& b = sm.bars;
  volatile int* stop = &sm.abort_flag;
  Turn<kItems> it;
  uint32_t step = 0;
  int64_t at[kCols / 32];            // this lane's columns, from the first row
#pragma unroll
  for (int i = 0; i < kCols / 32; ++i) {
    const int c = lane + 32 * i;
    at[i] = c < p.tq * p.group
                ? (int64_t)(c / p.group) * p.heads + c % p.group
                : -1;
  }
  for (;;) {
    if (!warp_wait(&b.item_full[it.at], it.phase, stop)) return false;
    const Item item = sm.items[it.at];
    __syncwarp();
    if (lane == 0) mbar_arrive(&b.item_empty[it.at]);
    it.next();
    if (item.flags & kStop) return true;
    if (item.steps == 0) continue;
    for (int j = item.j0; j < item.j1; ++j) {
      for (int st = 0; st < item.steps; ++st, ++step) {
        if ((int)(step & 1) != which) continue;
        const int slot = step & 1;
        const int cols = min(p.tq, item.n - st * p.tq) * p.group;
        const float* lse = p.lse + (item.row0 + st * p.tq) * p.heads +
                           (int64_t)j * p.group;
        float v[kCols / 32];
#pragma unroll
        for (int i = 0; i < kCols / 32; ++i)
          v[i] = lane + 32 * i < cols ? lse[at[i]] : -INFINITY;
        const uint32_t phase = (step >> 1) & 1;
        if (!warp_wait(&b.l_empty[slot], phase ^ 1, stop)) return false;
        uint32_t dead = 0;
#pragma unroll
        for (int i = 0; i < kCols / 32; ++i) {
          const float x = v[i] == -INFINITY ? -INFINITY : -v[i] * kLog2e;
          sm.lse[slot][lane + 32 * i] = x;
          if (__any_sync(~0u, x == -INFINITY)) dead |= 1u << i;
        }
        if (lane == 0) sm.dead[slot] = dead;
        __syncwarp();
        if (lane < 2) mbar_arrive(&b.s_full[slot][lane]);
      }
    }
  }
}

// ---------------------------------------------------------------- weights
// The sum of `kN` columns' weights; `whole`: this token is attended to by all
// of them, and none is without weight.
template <int kN>
__device__ __forceinline__ float add_columns(const float (&s)[kN],
                                             const float* lse, float scale,
                                             bool whole, int lo, int hi) {
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  const float2 scale2 = make_float2(scale, scale);
  if (whole) {
#pragma unroll
    for (int c = 0; c < kN; c += 4) {
      const float4 l = *reinterpret_cast<const float4*>(lse + c);
      const float2 x = fma2(make_float2(s[c], s[c + 1]), scale2,
                            make_float2(l.x, l.y));
      const float2 y = fma2(make_float2(s[c + 2], s[c + 3]), scale2,
                            make_float2(l.z, l.w));
      sum[0] = add2(sum[0], make_float2(exp2_fast(x.x), exp2_fast(x.y)));
      sum[1] = add2(sum[1], make_float2(exp2_fast(y.x), exp2_fast(y.y)));
    }
  } else {
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      const float l = lse[c];
      const bool in = c >= lo && c < hi && l != -INFINITY;
      const float x = exp2_fast(in ? fmaf(s[c], scale, l) : -INFINITY);
      if (c & 1) sum[(c >> 1) & 1].y += x; else sum[(c >> 1) & 1].x += x;
    }
  }
  return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

template <class T, class C>
__device__ __forceinline__ bool weigh(const WeighParams& p, Smem& sm,
                                      uint32_t tmem, int warp) {
  const int lane = (int)lane_id(), tile = warp >> 2;
  const int row = (warp & 3) * 32 + lane;
  const uint32_t lanes =
      tmem + ((uint32_t)(warp & 3) << 21) + (uint32_t)tile * kCols;
  Bars& b = sm.bars;
  volatile int* stop = &sm.abort_flag;
  Turn<kItems> it;
  uint32_t step = 0;
  for (;;) {
    if (!warp_wait(&b.item_full[it.at], it.phase, stop)) return false;
    const Item item = sm.items[it.at];
    __syncwarp();
    if (lane == 0) mbar_arrive(&b.item_empty[it.at]);
    it.next();
    if (item.flags & kStop) return true;
    // (eight rows of each page to a tile: the pages lie one behind the other)
    const int in_item = row / 8 * kBlock + tile * 8 + row % 8;
    const int64_t t = (int64_t)item.t0 + in_item;
    const bool here = (item.pages >> (row / 8)) & 1;
    // rows that attend to this token: from, ..., upto - 1
    const int64_t from = max(t - item.pf, (int64_t)0);
    int64_t upto = item.n;
    if (p.window && t >= p.sink)
      upto = min(upto, t + p.window - item.pf);
    if (!here) upto = 0;
    float sum = 0.f;
    for (int j = item.j0; item.steps && j < item.j1; ++j) {
      for (int st = 0; st < item.steps; ++st, ++step) {
        const uint32_t buf = step & 1, phase = (step >> 1) & 1;
        const int64_t first = (int64_t)st * p.tq;
        const int lo = (int)min(max(from - first, (int64_t)0),
                                (int64_t)kCols) * p.group;
        const int hi = (int)min(max(upto - first, (int64_t)0),
                                (int64_t)p.tq) * p.group;
        const int n = columns(p, item.n, st);
        if (!warp_wait(&b.s_full[buf][tile], phase, stop)) return false;
        tc_fence_after();
        const uint32_t dead = sm.dead[buf];
        const uint32_t at = lanes + buf * 2 * kCols;
        float part = 0.f;
        if (n == kCols && dead == 0 && __all_sync(~0u, lo <= 0 && hi >= n)) {
          // (read at once: the next product may go into the buffer)
          float s[kCols];
#pragma unroll
          for (int c = 0; c < kCols; c += 32) tmem_ld32(at + c, s + c);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b.s_empty[buf][tile]);
          part = add_columns(s, sm.lse[buf], p.scale, true, 0, 0);
        } else {
          int c = 0;
#pragma unroll 1
          for (; c + 32 <= n; c += 32) {
            float s[32];
            tmem_ld32(at + c, s);
            tmem_wait_ld();
            const bool whole = __all_sync(~0u, lo <= c && hi >= c + 32) &&
                               !((dead >> (c / 32)) & 1);
            part += add_columns(s, &sm.lse[buf][c], p.scale, whole, lo - c,
                                hi - c);
          }
          if (c < n) {
            float s[16];
            tmem_ld16(at + c, s);
            tmem_wait_ld();
            part += add_columns(s, &sm.lse[buf][c], p.scale, false, lo - c,
                                hi - c);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b.s_empty[buf][tile]);
        }
        sum += part;
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.l_empty[buf]);
      }
    }
    if ((item.flags & (kStarts | kEnds)) == (kStarts | kEnds)) {
      if (t < item.len) {
        const int64_t to = item.r * p.acc_ld + t;
        p.acc_out[to] =
            p.decay == 0.f ? sum : fmaf(p.decay, p.acc[to], sum);
      }
    } else {
      p.slots[(blockIdx.x * 2 + (item.flags & kStarts ? 1 : 0)) * kTile +
              in_item] = sum;
    }
  }
}

// ------------------------------------------------------------------ kernel
template <class T, int HD>
__global__ void __launch_bounds__(kThreads, 1)
    weigh_kernel(const __grid_constant__ WeighParams p) {
  using C = Cfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  Smem& sm = *reinterpret_cast<Smem*>(smem + C::kMisc);
  Bars& b = sm.bars;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < C::SK; ++i) {
      mbar_init(&b.k_full[i], 1);
      mbar_init(&b.k_empty[i], 1);
    }
    for (int i = 0; i < C::SQ; ++i) {
      mbar_init(&b.q_full[i], 1);
      mbar_init(&b.q_empty[i], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&b.item_full[i], 1);
      mbar_init(&b.item_empty[i], 11);    // eight warps, MMA, two fetchers
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&b.s_full[i / 2][i % 2], 2);    // MMA, fetcher
      mbar_init(&b.s_empty[i / 2][i % 2], 4);
      if (i < 2) mbar_init(&b.l_empty[i], 8);
    }
    mbar_init(&b.fin, 1);
    sm.abort_flag = 0;
    if (p.N) prefetch_tmap(&p.tm_q[0]);
    prefetch_tmap(&p.tm_k);
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
  int64_t* pre = reinterpret_cast<int64_t*>(smem);
  const int each = (p.R + kThreads - 1) / kThreads;
  int64_t sum = 0;
  for (int i = 0; i < each; ++i) {
    const int r = tid * each + i;
    if (r >= p.R) break;
    const int64_t cost = Tiles(p, request(p, r)).cost(p);
    pre[r] = cost;
    sum += cost;
    if (blockIdx.x == 0 && p.flags &&
        (p.lens[r] > p.max_blocks * kBlock || p.cu[r + 1] > p.N))
      atomicOr(p.flags, KVTC_FLAG_SPACE);
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
    if (r >= p.R) break;
    const int64_t cost = pre[r];
    pre[r] = before;
    before += cost;
  }
  if (tid == kThreads - 1) pre[p.R] = upto;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = sm.tmem, base = smem_u32(smem);
  bool ok = true;
  if (warp < 8) {
    ok = weigh<T, C>(p, sm, tmem, warp);
  } else if (warp == kProducer) {
    ok = produce<T, C>(p, sm, base, pre);
  } else if (warp == kMma) {
    ok = multiply<T, C>(p, sm, base, uniform(tmem));
    // products under way end before the block's memory is given up
    __syncwarp();
    tc_commit_one(&b.fin);
    mbar_drain(&b.fin, 0);
  } else {
    ok = fetch(p, sm, warp - kFetch);
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

// Block x adds up the parts of the item that began in block x; a thread per
// token.
__global__ void __launch_bounds__(kTile)
    weigh_join_kernel(const __grid_constant__ WeighParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, i = threadIdx.x;
  const JoinDesc d = p.desc[c];
  if (d.r < 0) return;
  const int64_t t = (int64_t)d.t0 + i;
  if (t >= d.pad) return;
  float sum = p.slots[(c * 2 + 1) * kTile + i];
#pragma unroll 4
  for (int k = c + 1; k <= d.last; ++k) sum += p.slots[k * 2 * kTile + i];
  const int64_t to = d.r * p.acc_ld + t;
  p.acc_out[to] = p.decay == 0.f ? sum : fmaf(p.decay, p.acc[to], sum);
}

template <class T, int HD>
cudaError_t launch_as(const WeighParams& p, int device, cudaStream_t st) {
  using C = Cfg<HD>;
  static std::atomic<uint64_t> ready;          // devices, as bits
  const auto kernel = weigh_kernel<T, HD>;
  cudaError_t e = allow_smem(kernel, C::kBytes, device, ready);
  if (e == cudaSuccess)
    e = launch_kernel(kernel, kCtas, kThreads, C::kBytes, st, true, 0, p);
  if (e != cudaSuccess) return e;
  count_launch();
  e = launch_kernel(weigh_join_kernel, kCtas, kTile, 0, st, true, 0, p);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <class T>
cudaError_t launch(const WeighParams& p, int head_dim, int device,
                   cudaStream_t st) {
  return head_dim == 64    ? launch_as<T, 64>(p, device, st)
         : head_dim == 128 ? launch_as<T, 128>(p, device, st)
                           : launch_as<T, 256>(p, device, st);
}

constexpr int64_t kDescBytes = (kCtas * sizeof(JoinDesc) + 255) / 256 * 256;

}  // namespace
}  // namespace kvtc

using namespace kvtc;

extern "C" {

int64_t kvtc_paged_weigh_workspace_bytes(int cuda_device, int R, int64_t N,
                                         int heads, int kv_heads,
                                         int head_dim) {
  if (cuda_device < 0 || R < 0 || R > kMaxReq || N < 0 || N > INT32_MAX ||
      heads <= 0 || kv_heads <= 0 || heads % kv_heads || head_dim <= 0)
    return KVTC_EINVAL;
  if ((head_dim != 64 && head_dim != 128 && head_dim != 256) ||
      (int64_t)kv_heads * head_dim > kMaxD || heads / kv_heads > kMaxGroup)
    return KVTC_ENOTSUP;
  return kDescBytes + kCtas * 2 * kTile * 4;
}

int kvtc_paged_weigh(int cuda_device, int R, int64_t N, int heads,
                     int kv_heads, int head_dim, int dtype, const void* q,
                     int64_t q_ld, const void* k_cache, int64_t num_blocks,
                     int block_size, const int32_t* block_table,
                     int max_blocks, const int64_t* cu, const int32_t* lens,
                     int sink, int window, float scale, const float* lse,
                     float decay, const float* acc, float* acc_out,
                     int64_t acc_ld, void* workspace, int64_t workspace_bytes,
                     uint32_t* flags, void* cuda_stream) {
  const int64_t need = kvtc_paged_weigh_workspace_bytes(
      cuda_device, R, N, heads, kv_heads, head_dim);
  if (need < 0) return (int)need;
  if ((dtype != KVTC_DTYPE_BF16 && dtype != KVTC_DTYPE_FP16) || !k_cache ||
      num_blocks <= 0 || num_blocks > INT32_MAX || max_blocks <= 0 ||
      sink < 0 || window < 0 || !(std::fabs(scale) <= kMaxScale) ||
      !std::isfinite(decay) || !workspace ||
      (R && (!block_table || !cu || !lens || !acc_out ||
             (decay != 0.f && !acc))) ||
      (R && N && (!q || !lse)))
    return KVTC_EINVAL;
  if (block_size != kBlock || max_blocks > kMaxTable) return KVTC_ENOTSUP;
  if (q_ld < (int64_t)heads * head_dim ||
      acc_ld < (int64_t)max_blocks * kBlock || workspace_bytes < need)
    return KVTC_ESIZE;
  if (q_ld % 8 || acc_ld % 4 || !aligned16(q) || !aligned16(k_cache) ||
      !aligned16(acc) || !aligned16(acc_out) || !aligned16(workspace) ||
      misaligned(block_table, 4) || misaligned(cu, 8) ||
      misaligned(lens, 4) || misaligned(lse, 4) || misaligned(flags, 4))
    return KVTC_EALIGN;
  if (R == 0) return KVTC_OK;
  DeviceGuard guard(cuda_device);
  if (!guard.ok) return KVTC_ECUDA;
  WeighParams p;
  p.group = heads / kv_heads;
  p.tq = kCols / p.group;
  if (!encode_pages(&p.tm_k, k_cache, (uint64_t)kv_heads * head_dim,
                    num_blocks, head_dim == 64 ? 1 : 2))
    return KVTC_ECUDA;
  // (without rows no box is read: their maps are never made)
  for (int i = 0; N && i < kBoxes; ++i) {
    if (i && (1 << (i - 1)) >= p.tq) break;
    if (!encode_rows(&p.tm_q[i], q, head_dim, heads, N, q_ld, p.group,
                     std::min(1 << i, p.tq)))
      return KVTC_ECUDA;
  }
  p.table = block_table;
  p.cu = cu;
  p.lens = lens;
  p.lse = lse;
  p.acc = acc;
  p.acc_out = acc_out;
  p.flags = flags;
  p.desc = static_cast<JoinDesc*>(workspace);
  p.slots = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                     kDescBytes);
  p.N = N;
  p.num_blocks = num_blocks;
  p.acc_ld = acc_ld;
  p.scale = scale * kLog2e;
  p.decay = decay;
  p.R = R;
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.max_blocks = max_blocks;
  p.sink = window ? sink : 0;
  p.window = window;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = dtype == KVTC_DTYPE_BF16
                            ? launch<__nv_bfloat16>(p, head_dim, cuda_device,
                                                    st)
                            : launch<__half>(p, head_dim, cuda_device, st);
  return e == cudaSuccess ? KVTC_OK : KVTC_ECUDA;
}

}  // extern "C"
