// linear_bf16.cu -- linear attention's walks in bf16: the forward and each of
// its three gradients (lin_walk), and what a segment adds to the state (lin_state).
#include "linear.cuh"

namespace vssm {
namespace {

// ------------------------------------------------------------------ the walk
// One CTA per (segment, value head, role).  A chunk of 128 tokens is four
// products on the matrix unit:
//   A  = X Y^T             read back, weighted and masked: P, bf16 terms in tensor memory
//   D1 = X S
//   S  = exp(G_end) S + Y^T (up * W)   as bf16 terms in shared memory for D1
//   D2 = P W               out = in * D1 + D2
// with in and up the weights of a row for the state and in it.  The two paths,
// of the state (up * W, S) and of the results (P, out), need each other only
// through the products, so each has warps of its own, and one thread issues the
// products, one the copies and one warp makes the gates; every hand-over is an
// mbarrier, and each phase of one is a chunk.  Chunks of 128 rows fill the
// lanes of tensor memory and halve the steps of the chain A, P, D2 (and U, S,
// D1), which is what a CTA alone on its SM waits for; all columns in one CTA
// spare a second A, P and copy of X and Y.  What bounds it is that chain: a chunk
// takes 9500 cycles, with dots 16000, of which the matrix unit is busy for a
// quarter, and each of its 56 (80) products takes 60 to 80 to issue.  32768 tokens,
// 32 heads of 128: 266 us forward (807 MB, 3.0 TB/s), the gradients 477 (dq), 466
// (dk) and 276 us (dv); a key head shared by 8 value heads writes its dq and dk as
// f32 parts of each, 512 MB more (16384 tokens, 64 heads of 64: 524 and 511 us).
//
// Terms: inputs are exact in one.  Without dots up * W, P and S have two, 16
// bits, so that results lose no more than their own rounding to bf16 (with one
// term of P and S out was 2.3e-3 of its norm off, 1.7e-3 with two), and S is left
// in tensor memory, where the products add to it.  Rows with dots, whose sums
// give dg, have three, all 24 bits, and S, whose terms are a float's digits, takes
// up U = Y^T (up * W) with one rounding a chunk (the matrix unit cuts off what it
// adds to a running sum).  They have room because up * W comes in stretches of
// rows, issued by a thread of their own, P reaches over A, and D1 comes after D2,
// where P was.  dg is 6e-7 to 8e-7 of its norm off, where two terms left 3e-6 to
// 7e-6, at 470 us a walk instead of 310 to 350 (32768 tokens, 32 heads of 128).  D1
// before D2, which then adds to it in its place, takes 432 us, but all 24 additions of
// D2 are cut off at D1's size: 1.1e-6.  Walks of 64 columns, with room for all of
// that, issue twice the products: 600 us.
constexpr int kC = 128, kStateWarps = 8;
template <bool has_dot>
struct WalkWarps {
  static constexpr int kParts = 2, kOut = 4 * kParts;  // for the results: threads to a row
  static constexpr int kProducts = kStateWarps + kOut, kCopies = kProducts + 1, kGates = kProducts + 2, kStateMma = kProducts + 3;
  static constexpr int kThreads = 32 * (kProducts + 4);
};
constexpr int kPanel = kC * 128;  // bytes of 64 columns of a chunk's rows
constexpr int kStep = 16 * 128;   // bytes of 16 rows, a step of a product over the rows

enum Bar : int {
  kFullX, kFullY, kFullW, kFullW2, kGatesFull, kGatesFree, kStateReady, kPReady, kOutDone, kDoneA, kDoneX, kDoneU, kDoneO, kDrained,
  kUpReady, kUpReadyLast = kUpReady + 3, kUpFree, kUpFreeLast = kUpFree + 3,  // rows with dots: of each stretch; otherwise the first
  kWClean, kWClean2, kDrained2, kBars
};

template <int KP, int NP, bool has_dot>  // panels of 64 columns of X and Y, and of W
struct WalkSmem {
  static constexpr int kTerms = has_dot ? 3 : 2;  // of up * W and S
  static constexpr bool kRoom = KP == 1 || NP == 1;  // for a second buffer of W, and for four stretches of up * W
  static constexpr int kX = KP * kPanel, kW = NP * kPanel, kSBlock = KP * 8192, kSTerm = NP * kSBlock;
  // up * W: all rows, or with dots stretches of them in two places or four
  static constexpr int kUpRows = has_dot ? 32 / NP : kC, kUpPanel = kUpRows * 128, kUpTerm = NP * kUpPanel, kUp = kTerms * kUpTerm;
  static constexpr int kUps = !has_dot ? 1 : kRoom ? 4 : 2;
  static constexpr int oX = 0, oY = kX, oW = 2 * kX, oUp = oW + kW, oS = oUp + kUps * kUp, oGates = oS + kTerms * kSTerm;
  static constexpr int oW2 = kRoom ? oGates : oW, oTokens = kRoom ? oGates + kW : oGates;
  static constexpr int oMisc = oTokens + 5 * 4 * kC, oBar = oMisc + 64, kBytes = oBar + kBars * 8;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};
// Columns of tensor memory.  P of two terms takes A's place.  P of three reaches from before A into it, and D1 comes
// after D2, where P was.
template <bool has_dot>
struct WalkTmem {
  static constexpr int kStep = has_dot ? 24 : 16;  // of 16 columns of P
  static constexpr int tP = 0, tA = has_dot ? 128 : 0, tD1 = has_dot ? 0 : 128, tU = 256, tO = 384;
};

// S in tensor memory is left undecayed, in a unit that shrinks with the sum of
// g, until that is down to 2^-kFar, which leaves the rest of a float's range to
// the values; it is read and written for its decay no more often than that.
constexpr float kFar = 48.0f;

struct Segment {
  int64_t start, inner_before;
  int seq, len, n;
  bool is_first, is_last;
  __device__ __forceinline__ explicit Segment(int4 e)
      : start(e.y), inner_before((unsigned)e.w >> kLinPlaceShift), seq(e.x), len(e.z), n((e.z + kC - 1) / kC),
        is_first(e.w & kLinFirst), is_last(e.w & kLinLast) {}
};

__device__ __forceinline__ void copy_panels(const CUtensorMap* map, uint8_t* to, int panels, int head, int64_t token, uint64_t* bar) {
#pragma unroll 1
  for (int p = 0; p < panels; ++p)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_u32(to + p * kPanel)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(p * 64), "r"(head), "r"((int)token), "r"(smem_u32(bar))
        : "memory");
}

// The warps of a path wait at a barrier for one that waits for the mbarrier:
// two dozen that ask for its phase keep the others from their work.

// A warp's arrival, behind what all its lanes wrote.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// 16 columns each from two places of this thread's lane, on their way together.
__device__ __forceinline__ void load_two(uint32_t from0, uint32_t from1, float2 (&v)[2][8]) {
  uint32_t w[2][16];
  __syncwarp();
  tmem_ld16(from0, w[0]);
  tmem_ld16(from1, w[1]);
  tmem_wait_ld16(w[0]);
  tmem_wait_ld16(w[1]);
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[u][i] = make_float2(__uint_as_float(w[u][2 * i]), __uint_as_float(w[u][2 * i + 1]));
}

// kCols columns of this thread's row of S, times `decay`.
template <int kCols>
__device__ __noinline__ void decay_state(uint32_t at, float decay) {
#pragma unroll 1
  for (int u = 0; u < kCols / 16; ++u) {
    uint32_t w[16];
    __syncwarp();
    tmem_ld16(at + 16 * u, w);
    tmem_wait_ld16(w);
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * decay);
    tmem_st16(at + 16 * u, w);
  }
  tmem_wait_st();
}

// Whether 16 values of every row of every head lie on 32-byte boundaries.
__device__ __forceinline__ bool whole_rows(const void* base, int64_t stride, int n) {
  return ((reinterpret_cast<uintptr_t>(base) | (uintptr_t)(2 * stride) | (uintptr_t)(2 * n)) & 31) == 0;
}

// 16 bf16 values of a row, of which `cols` exist (a multiple of 8): a sector, read and written at once where it is
// one, so that a warp's access of 32 rows touches each of its sectors once.
struct Row16 {
  uint32_t v[8];
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int cols, bool whole) {
    if (whole && cols >= 16) {
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                   : "l"(p));
      return;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 q = 8 * i < cols ? reinterpret_cast<const uint4*>(p)[i] : make_uint4(0, 0, 0, 0);
      v[4 * i] = q.x;
      v[4 * i + 1] = q.y;
      v[4 * i + 2] = q.z;
      v[4 * i + 3] = q.w;
    }
  }
  __device__ __forceinline__ void store_whole(__nv_bfloat16* p) const {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, int cols) const {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (8 * i < cols) reinterpret_cast<uint4*>(p)[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  }
  __device__ __forceinline__ float2 get(int i) const { return make_float2(bf16_lo(v[i]), bf16_hi(v[i])); }
  __device__ __forceinline__ void put(int i, float2 x) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
    v[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
};

// 0 in the place of what is not finite, in `count` chunks `step` bytes apart.
__device__ __noinline__ void clear_odd(uint8_t* at, int step, int count) {
  for (int u = 0; u < count; ++u)
    for (int k = 0; k < 4; ++k) {
      uint32_t* p = reinterpret_cast<uint32_t*>(at + u * step) + k;
      if ((*p & 0x7f80u) == 0x7f80u) *p &= 0xffff0000u;
      if ((*p & 0x7f800000u) == 0x7f800000u) *p &= 0xffffu;
    }
}

// A 16-byte chunk of W times its row's weight as bf16 terms.
template <int kTerms>
__device__ __forceinline__ void weigh(uint4 q, float up, uint4 (&terms)[kTerms]) {
  const uint32_t p[4] = {q.x, q.y, q.z, q.w};
  uint32_t t[4][kTerms];
#pragma unroll
  for (int k = 0; k < 4; ++k) split_pair<kTerms>(mul2(make_float2(bf16_lo(p[k]), bf16_hi(p[k])), splat2(up)), t[k]);
#pragma unroll
  for (int i = 0; i < kTerms; ++i) terms[i] = make_uint4(t[0][i], t[1][i], t[2][i], t[3][i]);
}
// x * 0 added up: not 0 once a value is not finite.
__device__ __forceinline__ void look_over(uint4 q, __nv_bfloat162& trace) {
  const uint32_t p[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    trace = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&p[k]), __floats2bfloat162_rn(0.0f, 0.0f), trace);
}
__device__ __forceinline__ bool is_odd(__nv_bfloat162 trace) { return *reinterpret_cast<const uint32_t*>(&trace) & 0x7fff7fffu; }

// Up * W as images of kTerms terms from W's image, by kThreads threads, each along
// a column of 16-byte chunks whose place in the swizzle is the same in all its
// rows.  A value of W that is not finite reaches the state, and so every later
// row, through up * W; in D2, where 0 times it would reach earlier rows, 0 takes
// its place in W, and *odd has the rows it should reach made NaN when they are
// written.
template <int NP, int kTerms, int kThreads>
__device__ __forceinline__ void weigh_all(uint8_t* w_image, uint8_t* up_image, const float* up, int t, volatile int* odd) {
  constexpr int kRowChunks = NP * 8, kRows = kThreads / kRowChunks;
  static_assert(kRows % 8 == 0, "the swizzle repeats every 8 rows");
  const int r0 = t / kRowChunks, ch = t % kRowChunks;
  const uint32_t at = (ch >> 3) * kPanel + image_chunk<128>(r0, ch & 7);
  __nv_bfloat162 trace = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll 2
  for (int u = 0; u < kC / kRows; ++u) {
    const uint4 q = *reinterpret_cast<const uint4*>(w_image + at + u * kRows * 128);
    uint4 terms[kTerms];
    if (odd) look_over(q, trace);
    weigh<kTerms>(q, up[r0 + u * kRows], terms);
    uint8_t* to = up_image + at + u * kRows * 128;
#pragma unroll
    for (int i = 0; i < kTerms; ++i) *reinterpret_cast<uint4*>(to + i * NP * kPanel) = terms[i];
  }
  if (odd && is_odd(trace)) {
    clear_odd(w_image + at, kRows * 128, kC / kRows);
    *odd = 1;
  }
}

// Rows past the segment, which the copies fill with another's: 0 times them could be NaN.
template <int KP>
__device__ __forceinline__ void clear_rows(uint8_t* image, int rows, int t, int threads) {
  for (int i = rows * KP * 8 + t; i < kC * KP * 8; i += threads) {
    const int r = i / (KP * 8), ch = i % (KP * 8);
    *reinterpret_cast<uint4*>(image + (ch >> 3) * kPanel + image_chunk<128>(r, ch & 7)) = make_uint4(0, 0, 0, 0);
  }
}

// NaN in those of a row's results (`cols` of them, from `at` on) in whose column
// a value of W at the row or an earlier one (back: a later one) is not finite.
// Whether one is at another row: then the row's dot product has it, too.
__device__ __noinline__ bool spoil_row(const LinRole& role, const __nv_bfloat16* w, int64_t at, int row, int rows, int cols) {
  const int from = role.back ? row : 0, to = role.back ? rows : row + 1;
  const float nan = __int_as_float(0x7fffffff);
  bool others = false;
  for (int c = 0; c < cols; ++c) {
    bool odd = false;
    for (int r = from; r < to; ++r) {
      const bool here = !isfinite(__bfloat162float(w[(int64_t)r * role.sw + c]));
      odd = odd || here;
      others = others || (here && r != row);
    }
    if (!odd) continue;
    if (role.part) static_cast<float*>(role.out)[at + c] = nan;
    else static_cast<__nv_bfloat16*>(role.out)[at + c] = __float2bfloat16_rn(nan);
  }
  return others;
}

// `role`'s walk of the segment a.order[item], head h.  Its direction, and whether rows have a dot product, are known
// where it is compiled.
template <int KP, int NP, bool back, bool has_dot>
__device__ __forceinline__ void walk(const LinArgs& a, const LinMaps& maps, const LinRole& role, int h, int64_t item) {
  using T = __nv_bfloat16;
  using L = WalkSmem<KP, NP, has_dot>;
  using M = WalkTmem<has_dot>;
  using Warps = WalkWarps<has_dot>;
  constexpr int kParts = Warps::kParts, kOutWarps = Warps::kOut, kProducts = Warps::kProducts, kCopies = Warps::kCopies;
  constexpr int kTerms = L::kTerms;  // of P, of up * W and of S
  constexpr int tP = M::tP, tA = M::tA, tD1 = M::tD1, tU = M::tU, tO = M::tO;
  constexpr int kN = NP * 64, kCols = NP * 32;  // columns of W, and to a thread of the state's path
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::oBar);
  const float* s_up = reinterpret_cast<const float*>(sm + L::oTokens);  // up, G / ln 2 in two floats, P's columns' factors
  const float *s_hi = s_up + kC, *s_lo = s_up + 2 * kC, *s_col = s_up + 3 * kC;
  float* s_self = reinterpret_cast<float*>(sm + L::oTokens) + 4 * kC;  // rows with dots: the weight of the token's own pair
  float* s_sums = reinterpret_cast<float*>(sm + L::oMisc);  // 8
  float *s_decay = s_sums + 8, *s_unit = s_sums + 9;
  volatile int *odd = reinterpret_cast<int*>(s_sums + 10), *stop = odd + 1, *s_steep = odd + 2;
  Pair* s_last = reinterpret_cast<Pair*>(s_sums + 14);  // the chunk's sum
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(s_sums + 13);

  constexpr bool two_w = L::kRoom;
  auto w_image = [&](int k) { return sm + (two_w && (k & 1) ? L::oW2 : L::oW); };
  const int seg_at = a.order[item];
  const Segment seg(a.table[seg_at]);
  const int n1 = role.n1, n2 = role.n2, n = seg.n;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, quad = warp & 3, row = quad * 32 + lane;
  if (t == 0) {
    for (int i = 0; i < kBars; ++i)
      mbar_init(bars + i, i == kStateReady || i == kWClean || i == kWClean2 ? kStateWarps
                          : i >= kUpReady && i <= kUpReadyLast              ? (has_dot ? kStateWarps / 2 : kStateWarps)
                          : i == kPReady || i == kOutDone                   ? kOutWarps
                          : i == kGatesFree                                 ? kStateWarps + kOutWarps
                                                                            : 1);
    *stop = *odd = 0;
    fence_mbar_init();
  }
  if (warp == kProducts) tmem_alloc<512>(tmem_at);
  // the state the segment starts from, if any
  const int64_t state_size = (int64_t)n1 * n2;
  const float* carry = nullptr;
  if (back ? seg.is_last : seg.is_first) {
    if (role.first) carry = role.first + ((int64_t)seg.seq * a.Hv + h) * state_size;
  } else {
    carry = role.slots + ((back ? seg.inner_before : seg.inner_before - 1) * a.Hv + h) * state_size;
  }
  const bool has_carry = carry != nullptr;
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tm = *tmem_at, lane_at = (uint32_t)(quad * 32) << 16;
  LinWaiter wait{a, stop};
  auto chunk_of = [&](int k) { return back ? n - 1 - k : k; };

  if (warp < kStateWarps) {  // the state's path
    const int c0 = (warp >> 2) * kCols;
    float unit = 1.0f, decay = 1.0f;  // without dots S is `unit` times what tensor memory has
    const bool has_row = row < KP * 64;
    auto state_at = [&](int col) { return (int64_t)row * role.srow + (int64_t)col * role.scol; };
    auto put_state = [&](int col, const float2 (&d)[8]) {
      uint8_t* image = sm + L::oS + col / 64 * L::kSBlock;
      put_row<kTerms, 128>(image, L::kSTerm, row, col % 64 / 8, d);
    };
    auto next_state = [&](int col, float2 (&d)[8]) {  // with dots: of S, whose three terms are its digits, and U
      tmem_sum<1>(tm + tU + lane_at + col, 0, d);
      const uint8_t* image = sm + L::oS + col / 64 * L::kSBlock;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t place = image_chunk<128>(row, col % 64 / 8 + q);
        float2 sum[4];
#pragma unroll
        for (int term = kTerms - 1; term >= 0; --term) {
          float2 v[4];
          unpack(*reinterpret_cast<const uint4*>(image + term * L::kSTerm + place), v);
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[i] = term == kTerms - 1 ? v[i] : add2(sum[i], v[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) d[4 * q + i] = fma2(splat2(decay), sum[i], d[4 * q + i]);
      }
    };
    auto load_state = [&](const float* from, int col, float2 (&d)[8]) {  // 16 columns of this thread's row
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (row < n1 && col + 2 * i < n2) {
          const float* p = from + state_at(col + 2 * i);
          f = role.scol == 1 ? *reinterpret_cast<const float4*>(p)
                             : make_float4(p[0], p[role.scol], p[2 * role.scol], p[3 * role.scol]);
        }
        d[i] = make_float2(f.x, f.y);
        d[i + 1] = make_float2(f.z, f.w);
      }
    };
    if (has_row && n > 0 || has_carry && has_row) {  // without one, zeros: D1 is added in any case
#pragma unroll 1
      for (int u = 0; u < kCols / 16; ++u) {
        float2 d[8];
        if (has_carry) {
          load_state(carry, c0 + 16 * u, d);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = splat2(0.0f);
        }
        if constexpr (!has_dot) {
          uint32_t words[16];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            words[2 * i] = __float_as_uint(d[i].x);
            words[2 * i + 1] = __float_as_uint(d[i].y);
          }
          __syncwarp();
          tmem_st16(tm + tU + lane_at + c0 + 16 * u, words);
        }
        put_state(c0 + 16 * u, d);
      }
      if constexpr (!has_dot) tmem_wait_st();
      tmem_fence_before_sync();
    }
    fence_async_smem();
    warp_arrive(bars + kStateReady, lane);
    const bool wanted = has_dot && role.cross && (!back || seg.is_first);
    // with dots: the first four warps weigh every other stretch of rows, the others those between.  A thread's chunks of W
    // have the same place in the swizzle.
    constexpr int kHalf = L::kUpRows / 2;
    const int half = warp >> 2, r = (t & 127) / (NP * 8), ch = (t & 127) % (NP * 8);
    int put = ~0;  // the phases of the places
    for (int k = 0; k < n; ++k) {
      const uint32_t p = k & 1;
      const bool more = k + 1 < n;
      const int rows = min(kC, seg.len - chunk_of(k) * kC);
      if (warp == 0) {
        wait(bars + kGatesFull, p);
        if (two_w) wait(bars + kFullW + p, (k >> 1) & 1);
        else wait(bars + kFullW, p);
        if (rows < kC) wait(bars + kFullY, p);
      }
      named_barrier(1, 32 * kStateWarps);
      decay = *s_decay;
      unit = *s_unit;
      if (rows < kC) {
        clear_rows<KP>(sm + L::oY, rows, t, 32 * kStateWarps);
        clear_rows<NP>(w_image(k), rows, t, 32 * kStateWarps);
        named_barrier(1, 32 * kStateWarps);
      }
      if constexpr (has_dot) {
        uint8_t* w = w_image(k) + (ch >> 3) * kPanel + half * L::kUpPanel + image_chunk<128>(r, ch & 7);
        __nv_bfloat162 trace = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < kC / L::kUpRows; ++i)
          look_over(*reinterpret_cast<const uint4*>(w + (i / 2 * 2 * L::kUpRows + i % 2 * kHalf) * 128), trace);
        const bool any_odd = __any_sync(0xffffffffu, is_odd(trace));
        tmem_fence_before_sync();  // what was read of U
        fence_async_smem();        // rows cleared
        if (!any_odd) warp_arrive(bars + kWClean + p, lane);
#pragma unroll 1
        for (int row0 = 0; row0 + half * L::kUpRows < rows; row0 += 2 * L::kUpRows) {
          uint4 terms[2][kTerms];
#pragma unroll
          for (int j = 0; j < 2; ++j)
            weigh<kTerms>(*reinterpret_cast<const uint4*>(w + (row0 + j * kHalf) * 128), s_up[row0 + half * L::kUpRows + j * kHalf + r], terms[j]);
          const int place = half + (L::kUps > 2 ? row0 / L::kUpRows & 2 : 0);
          if (lane == 0) wait(bars + kUpFree + place, put >> place & 1);
          __syncwarp();
          put ^= 1 << place;
          uint8_t* to = sm + L::oUp + place * L::kUp + (ch >> 3) * L::kUpPanel + image_chunk<128>(r, ch & 7);
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < kTerms; ++i) *reinterpret_cast<uint4*>(to + i * L::kUpTerm + j * kHalf * 128) = terms[j][i];
          fence_async_smem();
          warp_arrive(bars + kUpReady + place, lane);
        }
        if (any_odd) {
          if (is_odd(trace)) {
            for (int i = 0; i < 2; ++i) clear_odd(w + i * kHalf * 128, 2 * L::kUpRows * 128, kC / (2 * L::kUpRows));
            *odd = 1;
          }
          fence_async_smem();
          warp_arrive(bars + kWClean + p, lane);
        }
        warp_arrive(bars + kGatesFree, lane);
      } else {
        weigh_all<NP, kTerms, 32 * kStateWarps>(w_image(k), sm + L::oUp, s_up, t, odd);
        warp_arrive(bars + kGatesFree, lane);
        if (decay != 1.0f && has_row) decay_state<kCols>(tm + tU + lane_at + c0, decay);
        tmem_fence_before_sync();
        fence_async_smem();
        warp_arrive(bars + kUpReady, lane);
      }
      if (more || wanted) {
        if (warp == 0) {
          wait(bars + kDoneX, p);
          wait(bars + kDoneU, p);
        }
        named_barrier(1, 32 * kStateWarps);
        tmem_fence_after_sync();
      }
      if (more) {
        if (has_row) {
#pragma unroll 1
          for (int u = 0; u < kCols / 16; ++u) {
            float2 d[8];
            if constexpr (has_dot) {
              next_state(c0 + 16 * u, d);
            } else {
              tmem_sum<1>(tm + tU + lane_at + c0 + 16 * u, 0, d);
              scale_row(d, unit);
            }
            put_state(c0 + 16 * u, d);
          }
        }
        fence_async_smem();
        tmem_fence_before_sync();
        warp_arrive(bars + kStateReady, lane);
      }
    }
    if (has_dot && wanted) {
      const float *e = nullptr, *at_end = nullptr;  // between segments: the state as it was made for the next one
      if (!back && !seg.is_last) {
        at_end = role.slots + (seg.inner_before * a.Hv + h) * state_size;
        e = role.against + (seg.inner_before * a.Hv + h) * state_size;
      } else if (role.against_last) {
        e = role.against_last + ((int64_t)seg.seq * a.Hv + h) * state_size;
      }
      float2 sum = splat2(0.0f);
      if (has_row && e) {
#pragma unroll 1
        for (int u = 0; u < kCols / 16; ++u) {
          float2 d[8], x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = splat2(0.0f);
          if (at_end) load_state(at_end, c0 + 16 * u, d);
          else if (n > 0) next_state(c0 + 16 * u, d);
          else if (has_carry) load_state(carry, c0 + 16 * u, d);
          load_state(e, c0 + 16 * u, x);
#pragma unroll
          for (int i = 0; i < 8; ++i)  // past the state d may be what the matrix unit made of other rows
            if (row < n1 && c0 + 16 * u + 2 * i < n2) sum = fma2(d[i], x[i], sum);
        }
      }
      float v = sum.x + sum.y;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) s_sums[warp] = v;
      named_barrier(1, 32 * kStateWarps);
      if (t == 0) {
        for (int i = 1; i < kStateWarps; ++i) v += s_sums[i];
        role.cross[(int64_t)seg_at * a.Hv + h] = v;
      }
    }
  } else if (warp < kStateWarps + kOutWarps) {  // the results' path
    const int part = (warp - kStateWarps) >> 2;
    const int64_t dot_at = has_dot ? (int64_t)(h / role.rdot) * n2 : 0, w_at = (int64_t)(h / role.rw) * n2;
    const bool whole_out = whole_rows(role.out, (int64_t)a.Hv * n2, n2), whole_dot = whole_rows(role.dot, role.sdot, n2);
    for (int k = 0; k < n; ++k) {
      const uint32_t p = k & 1;
      const int c = chunk_of(k), rows = min(kC, seg.len - c * kC);
      if (warp == kStateWarps) {
        wait(bars + kGatesFull, p);
        wait(bars + kDoneA, p);
      }
      named_barrier(2, 32 * kOutWarps);
      const float hi = s_hi[row], lo = s_lo[row];
      const Pair G{hi, lo};
      const float in = back ? exp2_of(add(*s_last, minus(G))) : a.scale * exp2_of(G);
      const bool steep = *s_steep;
      tmem_fence_after_sync();
#pragma unroll 1
      for (int u = 0; u < 8 / kParts; ++u) {
        // a thread's blocks of 16 columns of P, spread over its columns: P is triangular
        const int j0 = 16 * (kParts * u + (u & 1 ? kParts - 1 - part : part));
        uint32_t words[kTerms][8];
        if (back ? j0 + 15 < quad * 32 || j0 >= rows : j0 > quad * 32 + 31) {  // no row of the warp sees these columns
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int q = 0; q < kTerms; ++q) words[q][i] = 0;
        } else {
          float2 d[8];
          tmem_sum<1>(tm + tA + lane_at + j0, 0, d);
          const bool all = back ? j0 > quad * 32 + 31 && j0 + 15 < rows : j0 + 15 < quad * 32;
          const int at = row - j0;  // the diagonal's column
          if (has_dot && !all) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (at == i) s_self[row] = a.scale * (i % 2 ? d[i / 2].y : d[i / 2].x);
          }
          // exp(G_i - G_j) in two factors, by way of the block's end: neither is above 1 where every row sees every
          // column, and on the diagonal the row's has no more than 32 tokens to grow over
          const int ref = back ? j0 : j0 + 15;
          const float e = (hi - s_hi[ref]) + (lo - s_lo[ref]);
          if (all || !steep) {
            const float f = a.scale * ex2(back ? -e : e);
            const float4* col = reinterpret_cast<const float4*>(s_col + j0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 q = col[i];
              d[2 * i] = mul2(d[2 * i], mul2(make_float2(q.x, q.y), splat2(f)));
              d[2 * i + 1] = mul2(d[2 * i + 1], mul2(make_float2(q.z, q.w), splat2(f)));
            }
          } else {
            #pragma unroll 1
            for (int i = 0; i < 16; ++i) {  // little code: see LinWaiter
              const float w = a.scale * ex2((back ? -1.0f : 1.0f) * ((hi - s_hi[j0 + i]) + (lo - s_lo[j0 + i])));
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                d[q].x *= i == 2 * q ? w : 1.0f;
                d[q].y *= i == 2 * q + 1 ? w : 1.0f;
              }
            }
          }
          if (!all) {
            constexpr int own = has_dot ? 0 : 1;
            const int from = back ? at + 1 - own : 0, count = max((back ? rows - j0 : at + own) - from, 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if ((unsigned)(2 * i - from) >= (unsigned)count) d[i].x = 0.0f;
              if ((unsigned)(2 * i + 1 - from) >= (unsigned)count) d[i].y = 0.0f;
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t term[kTerms];
            split_pair<kTerms>(d[i], term);
#pragma unroll
            for (int q = 0; q < kTerms; ++q) words[q][i] = term[q];
          }
        }
        __syncwarp();
        if (has_dot && u == 2) named_barrier(3 + quad, 32 * kParts);  // the last blocks of P lie on the first ones of A
#pragma unroll
        for (int q = 0; q < kTerms; ++q) tmem_st8(tm + tP + lane_at + j0 / 16 * M::kStep + 8 * q, words[q]);
      }
      tmem_wait_st();
      warp_arrive(bars + kGatesFree, lane);
      tmem_fence_before_sync();
      warp_arrive(bars + kPReady, lane);

      const int64_t token = seg.start + (int64_t)c * kC + row;
      const bool mine = row < rows;
      const int64_t out_row = (token * a.Hv + h) * n2;
      constexpr int kRuns = kN / 16 / kParts;
      const int first = part * (kN / kParts), cols = mine ? n2 - first : 0;
      Row16 r[kRuns];  // the partner's rows, then the results
      if (has_dot) {
        const T* from = static_cast<const T*>(role.dot) + token * role.sdot + dot_at + first;
#pragma unroll
        for (int s = 0; s < kRuns; ++s) r[s].load(from + 16 * s, cols - 16 * s, whole_dot);
      }
      if (warp == kStateWarps) {
        if (has_dot) wait(bars + kFullW + (two_w ? p : 0), two_w ? (k >> 1) & 1 : p);
        wait(bars + (has_dot ? kDoneX : kDoneO), p);  // the later of D1 and D2; behind the weighing of this chunk, too
      }
      named_barrier(2, 32 * kOutWarps);
      tmem_fence_after_sync();
      const bool spoilt = *odd;
      Pair dot{0.0f, 0.0f};  // short sums, put together without a rounding: over a segment dg adds thousands of them
#pragma unroll
      for (int s = 0; s < kRuns; ++s) {
        const int c0 = first + 16 * s;
        float2 e[2][8];
        float2 sum = splat2(0.0f);
        load_two(tm + tO + lane_at + c0, tm + tD1 + lane_at + c0, e);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          e[0][i] = fma2(splat2(in), e[1][i], e[0][i]);
          if (has_dot) sum = fma2(r[s].get(i), e[0][i], sum);
        }
        if (has_dot) {
          dot = add(dot, Pair{sum.x + sum.y, 0.0f});
          const float2 self = splat2(s_self[row]);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float2 w[4];
            unpack(*reinterpret_cast<const uint4*>(w_image(k) + (c0 >> 6) * kPanel + image_chunk<128>(row, (c0 & 63) / 8 + q)), w);
#pragma unroll
            for (int i = 0; i < 4; ++i) e[0][4 * q + i] = fma2(self, w[i], e[0][4 * q + i]);
          }
        }
        if (role.part) {
          float* to = static_cast<float*>(role.out) + out_row + c0;
#pragma unroll
          for (int i = 0; i < 8; i += 4)
            if (16 * s + 2 * i < cols) st_io8(to + 2 * i, &e[0][i].x);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) r[s].put(i, e[0][i]);
        }
      }
      // the next products may have D1's and D2's places
      tmem_fence_before_sync();
      warp_arrive(bars + kOutDone, lane);
      if (!role.part) {
        T* to = static_cast<T*>(role.out) + out_row + first;
        if (whole_out) {
#pragma unroll
          for (int s = 0; s < kRuns; ++s)
            if (16 * s < cols) r[s].store_whole(to + 16 * s);
        } else {
#pragma unroll
          for (int s = 0; s < kRuns; ++s) r[s].store(to + 16 * s, cols - 16 * s);
        }
      }
      float rest = dot.hi + dot.lo;
      if (spoilt && mine &&
          spoil_row(role, static_cast<const T*>(role.w) + (token - row) * role.sw + w_at + first, out_row + first, row, rows, cols))
        rest = __int_as_float(0x7fffffff);
      if (has_dot && mine) role.dots[((int64_t)part * a.Hv + h) * a.T + token] = rest;
    }
  } else {
    // W's copies are asked for by whoever knows that its place is free: whoever waits for a phase has to have done so
    // before it can come around again
    int ws[2] = {0, 0};
    constexpr int ahead = two_w ? 1 : 0;
    auto load_w = [&](int k) {
      const int b = two_w ? k & 1 : 0;
      mbar_arrive_expect_tx(bars + kFullW + b, (uint32_t)L::kW);
      copy_panels(maps.m + role.mw, w_image(k), NP, h / role.rw, seg.start + (int64_t)chunk_of(k) * kC, bars + kFullW + b);
      ++ws[b];
    };
    auto drain_w = [&]() {  // what is on its way comes in before the memory is given back
      drain_copies(bars + kFullW, ws[0]);
      drain_copies(bars + kFullW2, ws[1]);
    };
    if (warp == kProducts) {  // all lanes go through it together, so that addresses are uniform; one issues
      {
        const bool lead = elect_one();
        const uint64_t x = smem_desc<128>(smem_u32(sm + L::oX)), y = smem_desc<128>(smem_u32(sm + L::oY));
        const uint64_t yt = smem_desc<128>(smem_u32(sm + L::oY), kPanel);
        const uint64_t up = smem_desc<128>(smem_u32(sm + L::oUp), kPanel), st = smem_desc<128>(smem_u32(sm + L::oS), L::kSBlock);
        if (!has_dot && lead && n > 0) load_w(0);
        if (!has_dot && lead && two_w && n > 1) load_w(1);
        auto add_state = [&](uint32_t p) {  // D1
          wait(bars + kStateReady, p);
          if (__all_sync(0xffffffffu, wait.ok)) {
            tmem_fence_after_sync();
            constexpr uint32_t idesc = umma_idesc(kKMajor, kMnMajor, kN);
#pragma unroll 1
            for (int i = 0; i < kTerms * KP; ++i) {  // the smallest term first
              const int term = kTerms - 1 - i / KP, panel = i % KP;
#pragma unroll
              for (int s = 0; s < 4; ++s)
                umma_one(tm + tD1, x + (panel * kPanel + s * 32) / 16, st + (term * L::kSTerm + (4 * panel + s) * kStep) / 16, idesc,
                        i + s > 0 ? 1u : 0u);
            }
            if (lead) umma_commit(bars + kDoneX);
          }
        };
        for (int k = 0; k < n; ++k) {
          const uint32_t p = k & 1;
          wait(bars + kFullX, p, k == 0 && forced_here(a));
          wait(bars + kFullY, p);
          if (!has_dot && k > 0) {
            wait(bars + kDoneO, p ^ 1);  // P's place, and W's
            if (lead && wait.ok && k + ahead < n) load_w(k + ahead);
          }
          if (__all_sync(0xffffffffu, wait.ok)) {
            tmem_fence_after_sync();
            constexpr uint32_t idesc = umma_idesc(kKMajor, kKMajor, kC);
#pragma unroll 1
            for (int i = 0; i < KP; ++i)
#pragma unroll
              for (int s = 0; s < 4; ++s)
                umma_one(tm + tA, x + (i * kPanel + s * 32) / 16, y + (i * kPanel + s * 32) / 16, idesc, i + s > 0 ? 1u : 0u);
            if (lead) umma_commit(bars + kDoneA);
          }
          if (k > 0) wait(bars + kOutDone, p ^ 1);
          if constexpr (!has_dot) add_state(p);
          if (has_dot) wait(bars + kWClean + p, (k >> 1) & 1);
          else wait(bars + kUpReady, p);
          if (!has_dot && __all_sync(0xffffffffu, wait.ok)) {
            tmem_fence_after_sync();
            constexpr uint32_t idesc = umma_idesc(kMnMajor, kMnMajor, kN);
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              const int term = 1 - i / 2;
#pragma unroll
              for (int s = 0; s < 4; ++s)
                umma_one(tm + tU, yt + ((i & 1) * 4 + s) * (kStep / 16), up + (term * L::kW + ((i & 1) * 4 + s) * kStep) / 16, idesc, 1u);
            }
            if (lead) umma_commit(bars + kDoneU);
          }
          wait(bars + kPReady, p);
          if (__all_sync(0xffffffffu, wait.ok)) {
            tmem_fence_after_sync();
            const uint64_t w = smem_desc<128>(smem_u32(w_image(k)), kPanel);
            constexpr uint32_t idesc = umma_idesc(kKMajor, kMnMajor, kN);
#pragma unroll 1
            for (int i = 0; i < 2 * kTerms; ++i) {
              const int term = kTerms - 1 - i / 2;
#pragma unroll
              for (int s = 0; s < 4; ++s)
                umma_ta_one(tm + tO, tm + tP + M::kStep * ((i & 1) * 4 + s) + 8 * term, w + ((i & 1) * 4 + s) * (kStep / 16), idesc,
                            i + s > 0 ? 1u : 0u);
            }
            if (lead) umma_commit(bars + kDoneO);
          }
          if constexpr (has_dot) {
            wait(bars + kDoneO, p);  // D1 takes P's place
            add_state(p);
          }
        }
        if (lead) drain_w();
        if (lead && *stop) {  // products that were not waited for
          umma_commit(bars + kDrained);
          mbar_wait(bars + kDrained, 0, kCopyDrainNs);
        }
      }
      __syncwarp();
    } else if (warp == kCopies) {
      if (lane == 0 && n > 0) {
        int asked = 0;
        if (has_dot) load_w(0);
        if (has_dot && two_w && n > 1) load_w(1);
        // X and Y in turn, each once the products are through with what is in its place; then, with dots, W
#pragma unroll 1
        for (int i = 0; i < 2 * n; ++i) {
          const int k = i / 2;
          const bool is_x = i % 2 == 0;
          if (k > 0) {
            wait(bars + (is_x ? kDoneX : kDoneU), (k - 1) & 1);
            if (!is_x && has_dot) wait(bars + kDoneA, (k - 1) & 1);  // otherwise issued before U
          }
          if (!wait.ok) break;
          uint64_t* bar = bars + (is_x ? kFullX : kFullY);
          mbar_arrive_expect_tx(bar, (uint32_t)L::kX);
          copy_panels(maps.m + (is_x ? role.mx : role.my), sm + (is_x ? L::oX : L::oY), KP, is_x ? h / role.rx : h / role.ry,
                      seg.start + (int64_t)chunk_of(k) * kC, bar);
          ++asked;
          if (has_dot && !is_x && k > 0 && k + ahead < n) {
            wait(bars + kOutDone, (k - 1) & 1);  // rows' own pairs are read from W
            if (wait.ok) load_w(k + ahead);
          }
        }
        drain_copies(bars + kFullX, (asked + 1) / 2);
        drain_copies(bars + kFullY, asked / 2);
        if (has_dot) drain_w();
      }
      __syncwarp();
    } else if (warp == Warps::kGates) {
      const float* g_base = a.g + seg.start * a.g_token + h;
      auto load_g = [&](int c, float (&g)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = c * kC + lane * 4 + i;
          g[i] = r < seg.len ? g_base[(int64_t)r * a.g_token] : 0.0f;
        }
      };
      float g[4];
      Pair unit{0.0f, 0.0f};  // what S in tensor memory counts in, over ln 2
      if (n > 0) load_g(chunk_of(0), g);
      for (int k = 0; k < n; ++k) {
        Pair last, run = running_sums(g, lane, last);
        const Pair next = has_dot ? last : add(unit, last);  // with dots S is decayed in every chunk
        const bool keep = !has_dot && fabsf(next.hi) < kFar;
        float up[4] = {}, hi[4] = {}, lo[4] = {}, col[4];
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          run = add(run, Pair{clamp_g(i == 0 ? g[0] : i == 1 ? g[1] : i == 2 ? g[2] : g[3]), 0.0f});
          const Pair G = over_ln2(run), w = back ? G : add(last, minus(G));
          const float f = (back ? a.scale : 1.0f) * exp2_of(keep ? add(w, minus(next)) : w);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            up[q] = q == i ? f : up[q];
            hi[q] = q == i ? G.hi : hi[q];
            lo[q] = q == i ? G.lo : lo[q];
          }
        }
        if (k + 1 < n) load_g(chunk_of(k + 1), g);
        // a column's factor of P's weights, up to the end (back: from the start) of its block of 16
        const int ref = back ? lane & ~3 : lane | 3;
        const float rh = __shfl_sync(0xffffffffu, back ? hi[0] : hi[3], ref), rl = __shfl_sync(0xffffffffu, back ? lo[0] : lo[3], ref);
        // whether G changes more over 32 tokens than a factor can span
        const float from = __shfl_sync(0xffffffffu, hi[0], lane & ~7);
        bool flat = true;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float d = (rh - hi[i]) + (rl - lo[i]);
          col[i] = ex2(back ? -d : d);
          flat = flat && fabsf(hi[i] - from) < 60.0f;
        }
        const bool steep = !__all_sync(0xffffffffu, flat);
        const float decay = keep ? 1.0f : exp2_of(next), in_unit = keep ? exp2_of(next) : 1.0f;
        unit = keep ? next : Pair{0.0f, 0.0f};
        if (k > 0) wait(bars + kGatesFree, (k - 1) & 1);
        __syncwarp();
        float4* to = reinterpret_cast<float4*>(sm + L::oTokens) + lane;
        to[0] = make_float4(up[0], up[1], up[2], up[3]);
        to[kC / 4] = make_float4(hi[0], hi[1], hi[2], hi[3]);
        to[kC / 2] = make_float4(lo[0], lo[1], lo[2], lo[3]);
        to[3 * kC / 4] = make_float4(col[0], col[1], col[2], col[3]);
        if (lane == 0) {
          *s_steep = steep;
          *s_decay = decay;
          *s_unit = in_unit;
          *s_last = last;
        }
        warp_arrive(bars + kGatesFull, lane);
      }
    } else if (has_dot && warp == Warps::kStateMma) {  // U, stretch by stretch; all lanes together, as for the other products
      const bool lead = elect_one();
      const uint64_t yt = smem_desc<128>(smem_u32(sm + L::oY), kPanel);
      const uint64_t up = smem_desc<128>(smem_u32(sm + L::oUp), L::kUpPanel);
      constexpr uint32_t idesc = umma_idesc(kMnMajor, kMnMajor, kN);
      int got = 0;  // the phases of the places
      for (int k = 0; k < n; ++k) {
        const int rows = min(kC, seg.len - chunk_of(k) * kC);
        wait(bars + kFullY, k & 1);
#pragma unroll 1
        for (int row0 = 0; row0 < rows; row0 += L::kUpRows) {
          const int j = row0 / L::kUpRows & (L::kUps - 1);
          wait(bars + kUpReady + j, got >> j & 1);
          got ^= 1 << j;
          if (!__all_sync(0xffffffffu, wait.ok)) continue;
          tmem_fence_after_sync();
#pragma unroll
          for (int q = 0; q < L::kUpRows / 16; ++q)
#pragma unroll
            for (int term = kTerms - 1; term >= 0; --term)  // the smallest first
              umma_one(tm + tU, yt + (row0 * 128 + q * kStep) / 16, up + (j * L::kUp + term * L::kUpTerm + q * kStep) / 16,
                       idesc, row0 + q > 0 || term < kTerms - 1 ? 1u : 0u);
          if (lead) umma_commit(bars + kUpFree + j);
        }
        if (lead && wait.ok) umma_commit(bars + kDoneU);
        __syncwarp();
      }
      if (lead && n > 0) wait(bars + kDoneU, (n - 1) & 1);  // nobody else may
      if (lead && *stop) {
        umma_commit(bars + kDrained2);
        mbar_wait(bars + kDrained2, 0, kCopyDrainNs);
      }
      __syncwarp();
    }
  }
  tmem_fence_before_sync();
  __syncthreads();
  if (warp == kProducts) tmem_dealloc<512>(tm);
}

template <int KP, int NP, bool back, bool has_dot>
__global__ void __launch_bounds__(WalkWarps<has_dot>::kThreads, 1)
    lin_walk_bf16_kernel(const __grid_constant__ LinArgs a, const __grid_constant__ LinMaps maps, int which) {
  const int64_t item = blockIdx.x / a.Hv;
  if (item < a.info[0]) walk<KP, NP, back, has_dot>(a, maps, a.role[which], blockIdx.x % a.Hv, item);
}

// ------------------------------------------------------------------ what a segment adds to the state
// One CTA per (segment, value head, role): the sum of Y^T (up * W) with up the
// weights up to the segment's end, in which the chunks just add up: the one next
// to that end comes first, and each earlier one's weights carry the decay over
// the ones behind it.  up * W has three terms, all 24 bits, and a chunk's sum is
// added in registers while the next one's is made: the matrix unit cuts off what
// it adds to a running sum, which left the state of 4096 tokens of slow decays
// 6.6e-6 too small.  First the segments that others follow, for the scan; once
// the states before all segments are known, those that a sequence ends with (back:
// starts with), where its last state is asked for.
// One sequence of 32768 tokens, 32 heads of 128: 139 us (537 MB, 3.9 TB/s) and, for
// its last segment, 25.
constexpr int kStateTerms = 3;
template <int KP, int NP>
struct StateSmem {
  static constexpr int kY = KP * kPanel, kW = NP * kPanel, kUp = kStateTerms * kW;
  static constexpr int oY = 0, oW = 2 * kY, oUp = oW + 2 * kW, oGates = oUp + kUp, oMisc = oGates + 2 * 4 * kC;
  static constexpr int oBar = oMisc + 64, kBytes = oBar + 16 * 8;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};
constexpr int kWeighWarps = 16, kProducts = kWeighWarps, kCopies = kProducts + 1, kGatesWarp = kProducts + 2, kWarps = kProducts + 3;

template <int KP, int NP>
__global__ void __launch_bounds__(kWarps * 32, 1)
    lin_state_bf16_kernel(const __grid_constant__ LinArgs a, const __grid_constant__ LinMaps maps, int roles, bool ends) {
  using L = StateSmem<KP, NP>;
  constexpr int kN = NP * 64, kCols = NP * 16;  // columns of W, and to a thread of the sum
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::oBar);
  uint64_t *full = bars, *gates_full = bars + 2, *used = bars + 4, *up_ready = bars + 6, *done = bars + 7, *drained = bars + 9;
  float* s_total = reinterpret_cast<float*>(sm + L::oMisc);
  volatile int* stop = reinterpret_cast<int*>(s_total + 1);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(s_total + 2);
  const int which = blockIdx.x % roles, h = blockIdx.x / roles % a.Hv;
  const int64_t item = blockIdx.x / roles / a.Hv;
  if (item >= a.info[ends ? 0 : 1]) return;
  const LinRole& role = a.role[which];
  const bool back = role.back != 0;
  const Segment seg(a.table[ends ? a.order[item] : a.inner[item] + (back ? 1 : 0)]);
  if (ends && !(back ? seg.is_first : seg.is_last)) return;
  const int n1 = role.n1, n2 = role.n2, n = seg.n;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, quad = warp & 3, row = quad * 32 + lane;
  if (t == 0) {
    for (int i = 0; i < 10; ++i) mbar_init(bars + i, i == 6 || (i == 4 || i == 5) ? kWeighWarps : 1);
    *stop = 0;
    fence_mbar_init();
  }
  if (warp == kProducts) tmem_alloc<256>(tmem_at);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tm = *tmem_at, lane_at = (uint32_t)(quad * 32) << 16;
  LinWaiter wait{a, stop};
  auto chunk_of = [&](int k) { return back ? k : n - 1 - k; };

  if (warp == kProducts) {
    const bool lead = elect_one();
    const uint64_t up = smem_desc<128>(smem_u32(sm + L::oUp), kPanel);
    constexpr uint32_t idesc = umma_idesc(kMnMajor, kMnMajor, kN);
    for (int k = 0; k < n; ++k) {
      wait(up_ready, k & 1, k == 0 && forced_here(a));
      if (__all_sync(0xffffffffu, wait.ok)) {
        tmem_fence_after_sync();
        const uint64_t yt = smem_desc<128>(smem_u32(sm + L::oY + (k & 1) * L::kY), kPanel);
#pragma unroll 1
        for (int i = 0; i < 2 * kStateTerms; ++i) {  // the smallest term first
          const int term = kStateTerms - 1 - i / 2;
#pragma unroll
          for (int s = 0; s < 4; ++s)
            umma_one(tm + (k & 1) * 128, yt + ((i & 1) * 4 + s) * (kStep / 16), up + (term * L::kW + ((i & 1) * 4 + s) * kStep) / 16,
                    idesc, i + s > 0 ? 1u : 0u);
        }
        if (lead) umma_commit(done + (k & 1));
      }
      __syncwarp();
    }
    if (lead && *stop) {
      umma_commit(drained);
      mbar_wait(drained, 0, kCopyDrainNs);
    }
    __syncwarp();
  } else if (warp == kCopies) {
    if (lane == 0) {
      int asked[2] = {0, 0};
      auto load = [&](int k) {
        const int b = k & 1;
        const int64_t token = seg.start + (int64_t)chunk_of(k) * kC;
        mbar_arrive_expect_tx(full + b, L::kY + L::kW);
        copy_panels(maps.m + role.my, sm + L::oY + b * L::kY, KP, h / role.ry, token, full + b);
        copy_panels(maps.m + role.mw, sm + L::oW + b * L::kW, NP, h / role.rw, token, full + b);
        ++asked[b];
      };
      for (int k = 0; k < 2 && k < n; ++k) load(k);
      for (int k = 0; k + 2 < n; ++k) {
        wait(done + (k & 1), (k >> 1) & 1);  // Y's buffer; W's was read before
        if (wait.ok) load(k + 2);
      }
      for (int b = 0; b < 2; ++b) drain_copies(full + b, asked[b]);
    }
    __syncwarp();
  } else if (warp == kGatesWarp) {
    const float* g_base = a.g + seg.start * a.g_token + h;
    auto load_g = [&](int c, float (&g)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = c * kC + lane * 4 + i;
        g[i] = r < seg.len ? g_base[(int64_t)r * a.g_token] : 0.0f;
      }
    };
    float g[4];
    if (n > 0) load_g(chunk_of(0), g);
    Pair behind{0.0f, 0.0f};
    for (int k = 0; k < n; ++k) {
      Pair last, run = running_sums(g, lane, last);
      float up[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        run = add(run, Pair{clamp_g(g[i]), 0.0f});
        const Pair G = over_ln2(run);
        up[i] = back ? a.scale * exp2_of(add(behind, G)) : exp2_of(add(behind, add(last, minus(G))));
      }
      if (k + 1 < n) load_g(chunk_of(k + 1), g);
      behind = add(behind, last);
      if (k >= 2) wait(used + (k & 1), ((k - 2) >> 1) & 1);
      __syncwarp();
      reinterpret_cast<float4*>(sm + L::oGates + (k & 1) * 4 * kC)[lane] = make_float4(up[0], up[1], up[2], up[3]);
      if (k + 1 == n && lane == 0) {
        *s_total = exp2_of(behind);
        if (!ends) role.decay[item * a.Hv + h] = *s_total;
      }
      warp_arrive(gates_full + (k & 1), lane);
    }
  } else if (warp < kWeighWarps) {
    constexpr int kThreads = 32 * kWeighWarps;
    const int c0 = (warp >> 2) * kCols;
    float2 sum[kCols / 16][8];
#pragma unroll
    for (int u = 0; u < kCols / 16; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[u][i] = splat2(0.0f);
    auto take = [&](int k) {
      if (row >= KP * 64) return;
#pragma unroll
      for (int u = 0; u < kCols / 16; ++u) {
        float2 d[8];
        tmem_sum<1>(tm + (k & 1) * 128 + lane_at + c0 + 16 * u, 0, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[u][i] = add2(sum[u][i], d[i]);
      }
    };
    for (int k = 0; k < n; ++k) {
      const int b = k & 1, rows = min(kC, seg.len - chunk_of(k) * kC);
      if (warp == 0) {
        wait(gates_full + b, (k >> 1) & 1);
        wait(full + b, (k >> 1) & 1);
        if (k > 0) wait(done + ((k - 1) & 1), ((k - 1) >> 1) & 1);  // up * W's place is free, and there is a sum
      }
      named_barrier(1, kThreads);
      if (rows < kC) {
        clear_rows<KP>(sm + L::oY + b * L::kY, rows, t, kThreads);
        clear_rows<NP>(sm + L::oW + b * L::kW, rows, t, kThreads);
        named_barrier(1, kThreads);
      }
      weigh_all<NP, kStateTerms, kThreads>(sm + L::oW + b * L::kW, sm + L::oUp, reinterpret_cast<const float*>(sm + L::oGates + b * 4 * kC), t,
                                       nullptr);
      tmem_fence_before_sync();
      fence_async_smem();
      warp_arrive(used + b, lane);
      if (lane == 0) mbar_arrive(up_ready);
      if (k > 0) {
        tmem_fence_after_sync();
        take(k - 1);
      }
    }
    if (n > 0) {
      if (warp == 0) wait(done + ((n - 1) & 1), ((n - 1) >> 1) & 1);
      named_barrier(1, kThreads);
      tmem_fence_after_sync();
      take(n - 1);
    }
    const int64_t size = (int64_t)n1 * n2;
    const float total = n > 0 ? *s_total : 1.0f;
    const float* carry = nullptr;
    if (back ? seg.is_last : seg.is_first) {
      if (role.first) carry = role.first + ((int64_t)seg.seq * a.Hv + h) * size;
    } else if (ends) {
      carry = role.slots + ((back ? seg.inner_before : seg.inner_before - 1) * a.Hv + h) * size;
    }
    float* to = ends ? role.last + ((int64_t)seg.seq * a.Hv + h) * size : role.slots + (item * a.Hv + h) * size;
#pragma unroll
    for (int u = 0; u < kCols / 16; ++u)
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const int col = c0 + 16 * u + 2 * i;
        if (row >= n1 || col >= n2) continue;
        const int64_t at = (int64_t)row * n2 + col;
        float2 x = sum[u][i], y = sum[u][i + 1];
        if (carry) {
          const float4 f = *reinterpret_cast<const float4*>(carry + at);
          x = fma2(splat2(total), make_float2(f.x, f.y), x);
          y = fma2(splat2(total), make_float2(f.z, f.w), y);
        }
        *reinterpret_cast<float4*>(to + at) = make_float4(x.x, x.y, y.x, y.y);
      }
  }
  tmem_fence_before_sync();
  __syncthreads();
  if (warp == kProducts) tmem_dealloc<256>(tm);
}

template <int KP, int NP, bool back, bool has_dot>
cudaError_t run_walk(const LinArgs& a, const LinMaps& maps, int which, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const auto kernel = lin_walk_bf16_kernel<KP, NP, back, has_dot>;
  constexpr size_t bytes = WalkSmem<KP, NP, has_dot>::kBytes;
  const cudaError_t e = set_smem(reinterpret_cast<const void*>(kernel), bytes, done);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)(a.max_segs * a.Hv), WalkWarps<has_dot>::kThreads, bytes, st>>>(a, maps, which);
  return cudaGetLastError();
}

template <int KP, int NP>
cudaError_t run_state(const LinArgs& a, const LinMaps& maps, int roles, bool ends, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const auto kernel = lin_state_bf16_kernel<KP, NP>;
  constexpr size_t bytes = StateSmem<KP, NP>::kBytes;
  const cudaError_t e = set_smem(reinterpret_cast<const void*>(kernel), bytes, done);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)((ends ? a.max_segs : a.max_inner) * a.Hv * roles), kWarps * 32, bytes, st>>>(a, maps, roles, ends);
  return cudaGetLastError();
}

// A kernel for each direction, with dot products or without: in one for all,
// whatever each needs would take registers and code from the others.
template <int KP, int NP>
cudaError_t run_role(const LinArgs& a, const LinMaps& maps, int i, cudaStream_t st) {
  const LinRole& r = a.role[i];
  if (r.back) return r.dot ? run_walk<KP, NP, true, true>(a, maps, i, st) : run_walk<KP, NP, true, false>(a, maps, i, st);
  return r.dot ? run_walk<KP, NP, false, true>(a, maps, i, st) : run_walk<KP, NP, false, false>(a, maps, i, st);
}

}  // namespace

cudaError_t launch_lin_state_bf16(const LinArgs& a, const LinMaps& maps, int roles, bool ends, cudaStream_t st) {
  if ((ends ? a.max_segs : a.max_inner) == 0) return cudaSuccess;
  const bool k2 = a.role[0].n1 > 64, v2 = a.role[0].n2 > 64;  // of all roles: K x V
  if (k2) return v2 ? run_state<2, 2>(a, maps, roles, ends, st) : run_state<2, 1>(a, maps, roles, ends, st);
  return v2 ? run_state<1, 2>(a, maps, roles, ends, st) : run_state<1, 1>(a, maps, roles, ends, st);
}

cudaError_t launch_lin_walk_bf16(const LinArgs& a, const LinMaps& maps, int roles, cudaStream_t st) {
  if (a.max_segs == 0) return cudaSuccess;
  for (int i = 0; i < roles; ++i) {
    const bool k2 = a.role[i].n1 > 64, v2 = a.role[i].n2 > 64;
    const cudaError_t e = k2 ? (v2 ? run_role<2, 2>(a, maps, i, st) : run_role<2, 1>(a, maps, i, st))
                             : (v2 ? run_role<1, 2>(a, maps, i, st) : run_role<1, 1>(a, maps, i, st));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace vssm
