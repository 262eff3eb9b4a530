// umma.cuh -- 5th-generation tensor-core products on tiles in shared memory:
// operand images, descriptors, the instruction, and FP32 products made of
// BF16 terms.
//
// Images.  An operand image is a matrix of bf16 rows of kRowBytes (128 or 64)
// bytes, row after row, whose 16-byte chunks are permuted inside each row the
// way the matrix unit's swizzle of that width expects: chunk c of row r lies
// at c ^ (r % 8) for 128-byte rows and at c ^ (r / 2 % 4) for 64-byte rows.
// Every image starts on a 1024-byte boundary.  The same image serves as an
// operand whose contraction runs along its rows (K-major: one row per M / N
// index) and as one whose contraction runs down its rows (MN-major: one row
// per contraction index), so no operand is ever transposed by hand.
//
// Terms.  An FP32 value is carried as the sum of NT bf16 values, each the
// rounding of what the earlier ones leave: two terms hold 16 bits of the
// significand (relative error at most 2^-16), three hold all 24.  A product of
// two such sums keeps the pairs (i, j) with i + j < NT; the dropped ones are
// below the last kept term.  Accumulation is FP32 in tensor memory.
#pragma once

#include "common.cuh"

namespace vssm {

__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

// ------------------------------------------------------------------ images
template <int kRowBytes>
__device__ __forceinline__ uint32_t image_chunk(int row, int chunk) {
  static_assert(kRowBytes == 128 || kRowBytes == 64, "rows of 64 or 128 bytes");
  if (kRowBytes == 128) return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4));
  return (uint32_t)(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
}

// Two FP32 values as NT bf16 pairs (first value in the low half).
template <int NT>
__device__ __forceinline__ void split_pair(float2 v, uint32_t (&t)[NT]) {
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    t[i] = *reinterpret_cast<const uint32_t*>(&h);
    if (i + 1 < NT)  // what this term leaves (exact)
      v = fma2(make_float2(__uint_as_float(t[i] << 16), __uint_as_float(t[i] & 0xffff0000u)), splat2(-1.0f), v);
  }
}

__device__ __forceinline__ float bf16_lo(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

// ------------------------------------------------------------------ descriptors
// Shared-memory matrix descriptor: address and strides in 16-byte units, the
// version field 1 of this generation, the swizzle width.
// K-major:  sbo = bytes between groups of 8 rows (lbo unused).
// MN-major: sbo = bytes between groups of 8 contraction rows, lbo = bytes
//           between blocks of one row width along M / N.
template <int kRowBytes>
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo = 16, uint32_t sbo = 8 * kRowBytes) {
  constexpr uint64_t kSwizzle = kRowBytes == 128 ? 2 : 4;
  return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)((lbo >> 4) & 0x3fff) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3fff) << 32) | (1ull << 46) | (kSwizzle << 61);
}

enum : uint32_t { kKMajor = 0, kMnMajor = 1 };

// bf16 x bf16 -> FP32, M = 128.
__host__ __device__ constexpr uint32_t umma_idesc(uint32_t a_major, uint32_t b_major, uint32_t n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_major << 15) | (b_major << 16) | ((n >> 3) << 17) |
         ((128u >> 4) << 24);
}

// One M = 128, K = 16 instruction; issued by one thread.  accumulate = 0
// overwrites D.
__device__ __forceinline__ void umma(uint32_t tmem_d, uint64_t desc_a, uint64_t desc_b, uint32_t idesc,
                                     uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(desc_a), "l"(desc_b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrives on `bar` once every product issued so far by this thread is done.
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// Makes this thread's shared-memory writes visible to the matrix unit and the
// bulk copies (the async proxy).
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Bulk copy shared -> global (both 16-byte aligned, bytes % 16 == 0), in this
// thread's bulk group.
__device__ __forceinline__ void bulk_store_1d(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Waits until this thread's bulk stores have read their shared memory.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
// Waits until this thread's bulk stores are complete.
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// An operand at a shared-memory address: kTerms images kTermBytes apart, rows
// of kRowBytes, read K-major or MN-major.  Contraction step s (16 indices) of
// a K-major operand lies 32 bytes further along the row, kPanelBytes further
// for each full row width; of an MN-major operand, 16 rows further.
// kLbo (MN-major): distance between row-wide blocks along M / N.
template <int kRowBytes_, uint32_t kMajor_, int kTerms_, int kTermBytes_, int kPanelBytes_ = 0, int kLbo_ = 16>
struct Operand {
  static constexpr int kRowBytes = kRowBytes_, kTerms = kTerms_;
  static constexpr uint32_t kMajor = kMajor_;
  uint64_t desc;
  __device__ __forceinline__ explicit Operand(uint32_t addr) : desc(smem_desc<kRowBytes_>(addr, kLbo_)) {}
  __device__ __forceinline__ uint64_t at(int term, int step) const {
    constexpr int kStepsPerRow = kRowBytes_ / 32;
    const int off = kMajor_ == kKMajor
                        ? (step / kStepsPerRow) * kPanelBytes_ + (step % kStepsPerRow) * 32
                        : step * 16 * kRowBytes_;
    return desc + (uint64_t)((term * kTermBytes_ + off) >> 4);  // addresses stay below 2^18: no carry out
  }
};

// D (128 x N at tmem_d) = or += the sum over the term pairs (i, j), i + j <
// kKeep, of A_i B_j over kSteps contraction steps, the small pairs first.
// Issued by one thread.
template <int N, int kSteps, int kKeep, typename A, typename B>
__device__ __forceinline__ void umma_terms(uint32_t tmem_d, const A& a, const B& b, bool accumulate) {
  constexpr uint32_t idesc = umma_idesc(A::kMajor, B::kMajor, N);
  uint32_t acc = accumulate ? 1u : 0u;
#pragma unroll
  for (int sum = kKeep - 1; sum >= 0; --sum) {
#pragma unroll
    for (int i = 0; i < A::kTerms; ++i) {
      const int j = sum - i;
      if (j < 0 || j >= B::kTerms) continue;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        umma(tmem_d, a.at(i, s), b.at(j, s), idesc, acc);
        acc = 1u;
      }
    }
  }
}

// The same product with the terms of B side by side along N: B's image is
// [term][column block][rows], MN-major, so that one instruction multiplies a
// term of A with several terms of B and reads A from shared memory once (at
// N = 64 reading A takes longer than the products).  Order s = i + j of the
// pairs has its own kCols columns of D, and the sum of D's kKeep blocks,
// smallest first, is the product:
//   D[block i ..] += A_i [B_0 .. B_{kKeep - 1 - i}]
// kFresh: overwrite D.  A B of one term leaves the blocks from A's other terms.
template <int kCols, int kSteps, int kKeep, bool kFresh, typename A, typename B>
__device__ __forceinline__ void umma_blocks(uint32_t tmem_d, const A& a, const B& b) {
  static_assert(B::kMajor == kMnMajor, "terms along N need an MN-major B");
  static_assert(B::kTerms >= kKeep || B::kTerms == 1, "");
#pragma unroll
  for (int i = 0; i < kKeep && i < A::kTerms; ++i) {
    const int terms = B::kTerms < kKeep - i ? B::kTerms : kKeep - i;
    const uint32_t idesc = umma_idesc(A::kMajor, kMnMajor, (uint32_t)(terms * kCols));
    const bool fresh = kFresh && (i == 0 || B::kTerms == 1);
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      umma(tmem_d + i * kCols, a.at(i, s), b.at(0, s), idesc, fresh && s == 0 ? 0u : 1u);
  }
}

// ------------------------------------------------------------------ tensor memory of `kCols` columns
template <int kCols>
__device__ __forceinline__ void tmem_alloc(uint32_t* dst) {  // warp-collective
  __syncwarp();
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "n"(kCols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <int kCols>
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr) {  // warp-collective
  __syncwarp();
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(kCols) : "memory");
}

// 16 consecutive columns of this thread's lane as pairs, summed over kBlocks
// blocks `stride` columns apart, last block first.  All loads are in flight
// together.
template <int kBlocks>
__device__ __forceinline__ void tmem_sum(uint32_t taddr, int stride, float2 (&v)[8]) {
  __syncwarp();  // the load is warp-collective; a thread may come from a wait or from issuing products
  uint32_t r[kBlocks][16];
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) tmem_ld16(taddr + b * stride, r[b]);
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) tmem_wait_ld16(r[b]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = make_float2(__uint_as_float(r[kBlocks - 1][2 * i]), __uint_as_float(r[kBlocks - 1][2 * i + 1]));
#pragma unroll
    for (int b = kBlocks - 2; b >= 0; --b)
      v[i] = add2(v[i], make_float2(__uint_as_float(r[b][2 * i]), __uint_as_float(r[b][2 * i + 1])));
  }
}

// 16 consecutive columns of this thread's lane, as floats.
__device__ __forceinline__ void tmem_row(uint32_t taddr, float (&v)[16]) {
  float2 p[8];
  tmem_sum<1>(taddr, 0, p);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = p[i].x;
    v[2 * i + 1] = p[i].y;
  }
}

}  // namespace vssm
