// What the tensor-core kernels over chunks of rows and paged pools share.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "kvtc_hostutil.cuh"
#include "ptx.cuh"

namespace kvtc {
namespace {

constexpr int kBlock = 16;           // tokens per pool block (a page)
constexpr int kMaxReq = 4096;        // requests per call
constexpr int kMaxGroup = 128;       // query heads per KV head
constexpr int kMaxTable = INT32_MAX / kBlock - 1;
constexpr int kCtas = 152;           // one block per SM
constexpr int kRows = 128;           // rows of a tile (TMEM lanes)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMaxScale = 0x1p127f;  // times log2 e still finite

// ------------------------------------------------------------ PTX wrappers
__device__ __forceinline__ void tma_load_4d(uint32_t smem_dst,
                                            const void* tmap, int32_t x,
                                            int32_t y, int32_t z, int32_t w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_"
      "tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
      "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];"
               : "=r"(r)
               : "r"(taddr));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d, x = *reinterpret_cast<uint64_t*>(&a),
              y = *reinterpret_cast<uint64_t*>(&b),
              z = *reinterpret_cast<uint64_t*>(&c);
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d, x = *reinterpret_cast<uint64_t*>(&a),
              y = *reinterpret_cast<uint64_t*>(&b);
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return *reinterpret_cast<float2*>(&d);
}
template <class T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr uint32_t kFormat = 1;
  static constexpr float kShift = 0.f;
  static constexpr uint32_t kExp = 0x7F807F80u, kOne = 0x00800080u;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t x) {
    return make_float2(__uint_as_float(x << 16),
                       __uint_as_float(x & 0xFFFF0000u));
  }
};
// fp16 holds numbers from 2^-24 to 2^16: weights are formed 2^7 times as
// large, up to 2^15, and what is lost lies 2^-32 below the largest.
template <>
struct Elem<__half> {
  static constexpr uint32_t kFormat = 0;
  static constexpr float kShift = 7.f;
  static constexpr uint32_t kExp = 0x7C007C00u, kOne = 0x04000400u;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
  }
};
// Halves of a word that are infinite or NaN, as bits 15 and 31.
template <class T>
__device__ __forceinline__ uint32_t odd_of(uint32_t w) {
  return ((w & Elem<T>::kExp) + Elem<T>::kOne) & 0x80008000u;
}

// Parts of up to `of` that n >= 0 falls into.  (n + of - 1 may lie behind
// 2^31.)
__device__ __forceinline__ int32_t parts_of(int32_t n, int32_t of) {
  return n / of + (n % of != 0);
}
// A request's rows and length.
struct Request {
  int64_t c0;
  int32_t n, len;
  __device__ __forceinline__ Request(const int64_t* cu,
                                     const int32_t* lens, int64_t N,
                                     int32_t R, int32_t max_blocks, int r) {
    c0 = 0;
    n = len = 0;
    if (r < R) {
      c0 = min(max(cu[r], (int64_t)0), N);
      n = (int32_t)max(min(max(cu[r + 1], (int64_t)0), N) - c0,
                       (int64_t)0);
      len = min(max(lens[r], 0), max_blocks * kBlock);
    }
  }
  __device__ __forceinline__ Request(int64_t c0, int32_t n, int32_t len)
      : c0(c0), n(n), len(len) {}
};
// `total` costs in equal runs over the first `ctas` blocks, of `each` or more.
struct Deal {
  int64_t least;
  int32_t more, ctas;
  __device__ __forceinline__ Deal(int64_t total, int64_t each) {
    ctas = (int32_t)min((int64_t)kCtas, max(total / each, (int64_t)1));
    least = total / ctas;
    more = (int32_t)(total - least * ctas);
  }
  __device__ __forceinline__ int64_t begin(int c) const {
    return c >= ctas ? least * ctas + more : c * least + min(c, more);
  }
  __device__ __forceinline__ int cta_of(int64_t x) const {
    const int64_t wide = more * (least + 1);
    return (int)(x < wide ? x / (least + 1) : more + (x - wide) / least);
  }
};

__device__ __forceinline__ uint32_t low_bits(int64_t n) {
  return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << (int)n) - 1u;
}
// A phase of a ring of N barriers.
template <int N>
struct Turn {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      phase ^= 1;
    }
  }
};

// The MMA warp runs as one: all lanes compute the same, one of them, the same
// each time, issues.  Where the operands lie in uniform registers a product of
// 64 cycles is issued in fewer; out of others each takes 90 to 100.
template <class I>
__device__ __forceinline__ I uniform(I x) {
  return (I)__reduce_max_sync(~0u, (unsigned)x);
}
// Shared-memory matrix descriptors as in sw128_desc: the low word of one, with
// a leading byte offset (of operands whose rows are contiguous), and the high
// word, with the bytes from one group of eight rows to the next.
__device__ __forceinline__ uint32_t desc_base(uint32_t smem_addr,
                                              uint32_t lead = 1) {
  return uniform(((smem_addr & 0x3FFFFu) >> 4) | lead << 16);
}
__host__ __device__ constexpr uint32_t desc_high(uint32_t stride) {
  return (stride >> 4) | 1u << 14 | 2u << 29;
}
template <uint32_t kHighA = desc_high(1024)>
__device__ __forceinline__ void mma_ss_one(uint32_t d_tmem, uint32_t a_desc,
                                           uint32_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "elect.sync _|q, 0xFFFFFFFF;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\t"
      "mov.b64 b, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(
          d_tmem),
      "r"(a_desc), "r"(b_desc), "r"(idesc), "r"(accumulate), "n"(kHighA),
      "n"(desc_high(1024))
      : "memory");
}
__device__ __forceinline__ void mma_ts_one(uint32_t d_tmem, uint32_t a_tmem,
                                           uint32_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
      "elect.sync _|q, 0xFFFFFFFF;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(
          d_tmem),
      "r"(a_tmem), "r"(b_desc), "r"(idesc), "r"(accumulate),
      "n"(desc_high(1024))
      : "memory");
}
__device__ __forceinline__ void tc_commit_one(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xFFFFFFFF;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 "
      "[%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

// A bounded wait (mbar_wait's limit) that the warp goes through as one: every
// branch is on a vote, so that no lane falls behind the others.  (Lanes that
// leave a loop one by one stay apart after it, and each product that the MMA
// warp issues then gathers them again: 330 cycles.)  The lanes may ask for
// barriers of their own.
// (Kept short: the kernels' code competes for the instruction cache.)
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity,
                                          const volatile int* stop) {
  const uint32_t t0 = (uint32_t)globaltimer_ns();
#pragma unroll 1
  while (!__all_sync(~0u, mbar_try_wait_sleep(bar, parity, 20000u)))
    if (__any_sync(~0u, *stop ||
                            (uint32_t)globaltimer_ns() - t0 > kWaitNs))
      return false;
  return true;
}

// ---------------------------------------------------------------- host
// A pool [num_blocks][16][D] as {64 channels, 16 tokens, D / 64, num_blocks}:
// a box is `slabs` times 64 channels of a block.
bool encode_pages(CUtensorMap* m, const void* base, uint64_t D,
                  uint64_t num_blocks, uint32_t slabs) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[4] = {64, kBlock, D / 64, num_blocks};
  cuuint64_t strides[3] = {D * 2, 128, D * 2 * kBlock};
  cuuint32_t box[4] = {64u, (cuuint32_t)kBlock, slabs, 1u};
  cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Rows [N][ld] of `heads` heads as {64 channels, head_dim / 64, heads, N}: a
// box is 64 channels of the `group` heads of `tokens` rows.
bool encode_rows(CUtensorMap* m, const void* base, uint64_t head_dim,
                 uint64_t heads, uint64_t N, uint64_t ld, uint32_t group,
                 uint32_t tokens) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[4] = {64, head_dim / 64, heads, N};
  cuuint64_t strides[3] = {128, head_dim * 2, ld * 2};
  cuuint32_t box[4] = {64u, 1u, group, tokens};
  cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool misaligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

}  // namespace
}  // namespace kvtc
