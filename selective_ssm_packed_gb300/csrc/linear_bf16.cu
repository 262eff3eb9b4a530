// linear_bf16.cu -- linear attention's walks in bf16: the forward and each of
// its three gradients (lin_walk), and what a segment adds to the state (lin_state).
#include "linear.cuh"

namespace vssm {
namespace {

// ------------------------------------------------------------------ the walk
// One CTA per (segment, value head, role).  A chunk of 128 tokens is four
// products on the matrix unit:
//   A  = X Y^T             read back, weighted and masked: P, bf16 terms in A's place in tensor memory
//   D1 = X S
//   S  = S + Y^T (up * W)  in tensor memory, decayed by exp(G_end) before; as bf16 terms in shared memory for D1
//   D2 = P W               out = in * D1 + D2
// with in and up the weights of a row for the state and in it.  The two paths,
// of the state (up * W, S) and of the results (P, out), need each other only
// through the products, so each has warps of its own, and one thread issues the
// products, one the copies and one warp makes the gates; every hand-over is an
// mbarrier, and each phase of one is a chunk.
constexpr int kC = 128, kPathWarps = 8, kProducts = 16, kCopies = 17, kGatesWarp = 18, kWarps = 20;
constexpr int kPanel = kC * 128;  // bytes of 64 columns of a chunk's rows

enum Bar : int { kFullX, kFullY, kFullW, kGatesFull, kGatesFree, kUpReady, kStateReady, kPReady, kOutDone, kDoneA, kDoneX, kDoneU, kDoneO, kDrained, kBars };

template <int KP, int NP>  // panels of 64 columns of X and Y, and of W
struct WalkSmem {
  static constexpr int kX = KP * kPanel, kW = NP * kPanel, kUp = 2 * kW, kSBlock = KP * 8192, kSTerm = NP * kSBlock;
  static constexpr int oX = 0, oY = kX, oW = 2 * kX, oUp = oW + kW, oS = oUp + kUp, oGates = oS + 2 * kSTerm;
  static constexpr int oDiag = oGates + 4 * 4 * kC, oMisc = oDiag + 4 * kC, oBar = oMisc + 64, kBytes = oBar + kBars * 8;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};
constexpr int tA = 0, tD1 = 128, tU = 256, tO = 384;  // columns of tensor memory

struct Segment {
  int64_t start, inner_before;
  int seq, len, n;
  bool is_first, is_last;
  __device__ __forceinline__ explicit Segment(int4 e)
      : start(e.y), inner_before((unsigned)e.w >> kLinPlaceShift), seq(e.x), len(e.z), n((e.z + kC - 1) / kC),
        is_first(e.w & kLinFirst), is_last(e.w & kLinLast) {}
};

__device__ __forceinline__ void copy_panels(const CUtensorMap* map, uint8_t* to, int panels, int head, int64_t token, uint64_t* bar) {
  for (int p = 0; p < panels; ++p)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_u32(to + p * kPanel)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(p * 64), "r"(head), "r"((int)token), "r"(smem_u32(bar))
        : "memory");
}

// A warp's arrival, behind what all its lanes wrote.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Up * W as images of two terms from W's image, by kThreads threads.  Rows past
// the segment, which the copies fill with another's, become zero in W too.  A
// value of W that is not finite reaches the state, and so every later row,
// through up * W; in D2, where 0 times it would reach earlier rows, 0 takes its
// place in W, and *odd has the rows it should reach made NaN when they are written.
template <int NP, int kThreads>
__device__ __forceinline__ void weigh(uint8_t* w_image, uint8_t* up_image, const float* up, int rows, int t, volatile int* odd) {
#pragma unroll 2
  for (int u = 0; u < kC * NP * 8 / kThreads; ++u) {
    const int i = t + u * kThreads, r = i / (NP * 8), ch = i % (NP * 8);
    uint4* at = reinterpret_cast<uint4*>(w_image + (ch >> 3) * kPanel + image_chunk<128>(r, ch & 7));
    uint4 q = *at;
    if (r >= rows) {
      q = make_uint4(0, 0, 0, 0);
      if (odd) *at = q;
    }
    float2 v[4];
    unpack(q, v);
    float2 trace = splat2(0.0f);
    const float f = up[r];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      trace = fma2(v[k], splat2(0.0f), trace);
      v[k] = mul2(v[k], splat2(r < rows ? f : 0.0f));
    }
    put_chunk<2, 128>(up_image + (ch >> 3) * kPanel, NP * kPanel, r, ch & 7, v);
    if (odd && trace.x + trace.y != 0.0f) {
      uint32_t p[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if ((p[k] & 0x7f80u) == 0x7f80u) p[k] &= 0xffff0000u;
        if ((p[k] & 0x7f800000u) == 0x7f800000u) p[k] &= 0xffffu;
      }
      *at = make_uint4(p[0], p[1], p[2], p[3]);
      *odd = 1;
    }
  }
}

// Rows of Y past the segment: 0 times what the copies brought could be NaN.
template <int KP>
__device__ __forceinline__ void clear_rows(uint8_t* image, int rows, int t, int threads) {
  for (int i = rows * KP * 8 + t; i < kC * KP * 8; i += threads) {
    const int r = i / (KP * 8), ch = i % (KP * 8);
    *reinterpret_cast<uint4*>(image + (ch >> 3) * kPanel + image_chunk<128>(r, ch & 7)) = make_uint4(0, 0, 0, 0);
  }
}

// The columns (of 16 from w on) in which a value of W at the row or an earlier
// one (back: a later one) is not finite.
__device__ __noinline__ uint32_t odd_columns(const LinRole& role, const __nv_bfloat16* w, int row, int rows, int cols) {
  uint32_t mask = 0;
  if (row >= rows) return mask;
  const int from = role.back ? row : 0, to = role.back ? rows : row + 1;
  for (int c = 0; c < 16 && c < cols; ++c)
    for (int r = from; r < to; ++r)
      if (!isfinite(__bfloat162float(w[(int64_t)r * role.sw + c]))) mask |= 1u << c;
  return mask;
}

template <int KP, int NP>
__global__ void __launch_bounds__(kWarps * 32, 1)
    lin_walk_bf16_kernel(const __grid_constant__ LinArgs a, const __grid_constant__ LinMaps maps, int roles) {
  using T = __nv_bfloat16;
  using L = WalkSmem<KP, NP>;
  using R = WalkRow<T, 2>;  // 16 columns of a thread's at a time
  using RF = WalkRow<float, 2>;
  constexpr int kN = NP * 64, kCols = NP * 32;  // columns of W, and to a thread
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::oBar);
  const float* s_in = reinterpret_cast<const float*>(sm + L::oGates);  // in, up, and two of P's factors or of G
  const float *s_up = s_in + kC, *s_f = s_in + 2 * kC, *s_h = s_in + 3 * kC;
  float* s_diag = reinterpret_cast<float*>(sm + L::oDiag);
  float* s_sums = reinterpret_cast<float*>(sm + L::oMisc);  // 8
  float* s_end = s_sums + 8;
  volatile int* s_near = reinterpret_cast<int*>(s_end + 1);
  volatile int *odd = s_near + 1, *stop = s_near + 2;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(s_end + 4);

  const int which = blockIdx.x % roles, h = blockIdx.x / roles % a.Hv;
  const int64_t item = blockIdx.x / roles / a.Hv;
  if (item >= a.info[0]) return;
  const LinRole& role = a.role[which];
  const bool back = role.back != 0, has_dot = role.dot != nullptr;
  const int seg_at = a.order[item];
  const Segment seg(a.table[seg_at]);
  const int n1 = role.n1, n2 = role.n2, n = seg.n;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, quad = warp & 3, part = (warp >> 2) & 1, row = quad * 32 + lane;
  if (t == 0) {
    for (int i = 0; i < kBars; ++i)
      mbar_init(bars + i, i == kUpReady || i == kStateReady || i == kPReady || i == kOutDone ? kPathWarps
                          : i == kGatesFree                                                  ? 2 * kPathWarps
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

  if (warp == kProducts) {
    if (lane == 0) {
      const Operand<128, kKMajor, 1, L::kX, kPanel> X(smem_u32(sm + L::oX)), Y(smem_u32(sm + L::oY));
      const Operand<128, kMnMajor, 1, L::kX, 0, kPanel> Yt(smem_u32(sm + L::oY));
      const Operand<128, kMnMajor, 2, L::kSTerm, 0, L::kSBlock> S(smem_u32(sm + L::oS));
      const Operand<128, kMnMajor, 2, L::kW, 0, kPanel> Up(smem_u32(sm + L::oUp));
      const Operand<128, kMnMajor, 1, L::kW, 0, kPanel> W(smem_u32(sm + L::oW));
      for (int k = 0; k < n; ++k) {
        const uint32_t p = k & 1;
        const bool has_state = k > 0 || has_carry;
        wait(bars + kFullX, p, k == 0 && forced_here(a));
        wait(bars + kFullY, p);
        if (k > 0) wait(bars + kDoneO, p ^ 1);  // P's place
        if (wait.ok) {
          tmem_fence_after_sync();
          umma_terms<kC, KP * 4, 1>(tm + tA, X, Y, false);
          umma_commit(bars + kDoneA);
        }
        wait(bars + kStateReady, p);
        if (k > 0) wait(bars + kOutDone, p ^ 1);
        if (wait.ok) {
          tmem_fence_after_sync();
          if (has_state) umma_terms<kN, KP * 4, 2>(tm + tD1, X, S, false);
          umma_commit(bars + kDoneX);
        }
        wait(bars + kUpReady, p);
        if (wait.ok) {
          tmem_fence_after_sync();
          umma_terms<kN, kC / 16, 2>(tm + tU, Yt, Up, has_state);
          umma_commit(bars + kDoneU);
        }
        wait(bars + kPReady, p);
        if (wait.ok) {
          tmem_fence_after_sync();
          constexpr uint32_t idesc = umma_idesc(kKMajor, kMnMajor, kN);
#pragma unroll
          for (int term = 1; term >= 0; --term)
#pragma unroll
            for (int s = 0; s < kC / 16; ++s)
              umma_ta(tm + tO, tm + tA + 16 * s + 8 * term, W.at(0, s), idesc, term == 1 && s == 0 ? 0u : 1u);
          umma_commit(bars + kDoneO);
        }
      }
      if (*stop) {  // products that were not waited for
        umma_commit(bars + kDrained);
        mbar_wait(bars + kDrained, 0, kCopyDrainNs);
      }
    }
    __syncwarp();
  } else if (warp == kCopies) {
    if (lane == 0 && n > 0) {
      int xs = 0, ys = 0, ws = 0;  // copies asked for
      auto load = [&](int map, int head, int at, int panels, int bar, int& asked, int c) {
        mbar_arrive_expect_tx(bars + bar, (uint32_t)(panels * kPanel));
        copy_panels(maps.m + map, sm + at, panels, head, seg.start + (int64_t)c * kC, bars + bar);
        ++asked;
      };
      auto load_x = [&](int c) { load(role.mx, h / role.rx, L::oX, KP, kFullX, xs, c); };
      auto load_y = [&](int c) { load(role.my, h / role.ry, L::oY, KP, kFullY, ys, c); };
      auto load_w = [&](int c) { load(role.mw, h / role.rw, L::oW, NP, kFullW, ws, c); };
      load_x(chunk_of(0));
      load_y(chunk_of(0));
      load_w(chunk_of(0));
      for (int k = 0; k + 1 < n; ++k) {
        const uint32_t p = k & 1;
        wait(bars + kDoneX, p);
        if (wait.ok) load_x(chunk_of(k + 1));
        wait(bars + kDoneU, p);
        if (wait.ok) load_y(chunk_of(k + 1));
        wait(bars + kDoneO, p);
        if (wait.ok) load_w(chunk_of(k + 1));
      }
      // what is on its way comes in before the memory is given back
      drain_copies(bars + kFullX, xs);
      drain_copies(bars + kFullY, ys);
      drain_copies(bars + kFullW, ws);
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
    for (int k = 0; k < n; ++k) {
      const GateSums<4> sums(g, lane);
      if (k + 1 < n) load_g(chunk_of(k + 1), g);
      const float mid = 0.5f * sums.last.hi;
      bool near = true;  // both factors of every weight are normal numbers
      float in[4], up[4], f[4], q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Pair G = sums.G[i], d = add(G, Pair{-mid, 0.0f});
        const float from = a.scale * exp2_of(G), to = exp2_of(add(sums.last, minus(G)));
        in[i] = back ? to : from;
        up[i] = back ? from : to;
        f[i] = a.scale * exp2_of(back ? minus(d) : d);
        q[i] = exp2_of(back ? d : minus(d));
        near = near && fabsf(d.hi) < 120.0f;
      }
      near = __all_sync(0xffffffffu, near);
      if (!near) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[i] = sums.G[i].hi;
          q[i] = sums.G[i].lo;
        }
      }
      const float end = exp2_of(sums.last);
      if (k > 0) wait(bars + kGatesFree, (k - 1) & 1);
      __syncwarp();
      float4* to = reinterpret_cast<float4*>(sm + L::oGates) + lane;
      to[0] = make_float4(in[0], in[1], in[2], in[3]);
      to[kC / 4] = make_float4(up[0], up[1], up[2], up[3]);
      to[kC / 2] = make_float4(f[0], f[1], f[2], f[3]);
      to[3 * kC / 4] = make_float4(q[0], q[1], q[2], q[3]);
      if (lane == 0) {
        *s_end = end;
        *s_near = near;
      }
      warp_arrive(bars + kGatesFull, lane);
    }
  } else if (warp < kPathWarps) {  // the state's path
    const int c0 = part * kCols;
    const bool has_row = row < KP * 64;
    auto state_at = [&](int col) { return (int64_t)row * role.srow + (int64_t)col * role.scol; };
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
    if (has_carry && has_row) {
#pragma unroll 1
      for (int u = 0; u < kCols / 16; ++u) {
        float2 d[8];
        uint32_t words[16];
        load_state(carry, c0 + 16 * u, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          words[2 * i] = __float_as_uint(d[i].x);
          words[2 * i + 1] = __float_as_uint(d[i].y);
        }
        __syncwarp();
        tmem_st16(tm + tU + lane_at + c0 + 16 * u, words);
        put_row<2, 128>(sm + L::oS + (c0 + 16 * u) / 64 * L::kSBlock, L::kSTerm, row, (c0 + 16 * u) % 64 / 8, d);
      }
      tmem_wait_st();
      tmem_fence_before_sync();
    }
    fence_async_smem();
    warp_arrive(bars + kStateReady, lane);
    const bool wanted = role.cross || (role.last && (back ? seg.is_first : seg.is_last));
    for (int k = 0; k < n; ++k) {
      const uint32_t p = k & 1;
      const bool more = k + 1 < n;
      const int rows = min(kC, seg.len - chunk_of(k) * kC);
      wait(bars + kGatesFull, p);
      wait(bars + kFullW, p);
      const float end = *s_end;
      weigh<NP, 256>(sm + L::oW, sm + L::oUp, s_up, rows, t, odd);
      warp_arrive(bars + kGatesFree, lane);
      if (rows < kC) {
        wait(bars + kFullY, p);
        clear_rows<KP>(sm + L::oY, rows, t, 256);
      }
      if ((k > 0 || has_carry) && has_row) {
#pragma unroll
        for (int u = 0; u < kCols / 32; ++u) {
          uint32_t w[32];
          __syncwarp();
          tmem_ld32(tm + tU + lane_at + c0 + 32 * u, w);
          tmem_wait_ld32(w);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 d = mul2(make_float2(__uint_as_float(w[i]), __uint_as_float(w[i + 1])), splat2(end));
            w[i] = __float_as_uint(d.x);
            w[i + 1] = __float_as_uint(d.y);
          }
          tmem_st32(tm + tU + lane_at + c0 + 32 * u, w);
        }
        tmem_wait_st();
      }
      tmem_fence_before_sync();
      fence_async_smem();
      warp_arrive(bars + kUpReady, lane);
      if (more || wanted) wait(bars + kDoneU, p);
      if (more) {
        wait(bars + kDoneX, p);
        tmem_fence_after_sync();
        if (has_row) {
#pragma unroll
          for (int u = 0; u < kCols / 16; ++u) {
            float2 d[8];
            tmem_sum<1>(tm + tU + lane_at + c0 + 16 * u, 0, d);
            put_row<2, 128>(sm + L::oS + (c0 + 16 * u) / 64 * L::kSBlock, L::kSTerm, row, (c0 + 16 * u) % 64 / 8, d);
          }
        }
        fence_async_smem();
        tmem_fence_before_sync();
        warp_arrive(bars + kStateReady, lane);
      }
    }
    if (wanted) {
      tmem_fence_after_sync();
      float* to = role.last && (back ? seg.is_first : seg.is_last) ? role.last + ((int64_t)seg.seq * a.Hv + h) * state_size : nullptr;
      const float* e = nullptr;
      if (role.cross) {
        if (!seg.is_last) e = role.against + (seg.inner_before * a.Hv + h) * state_size;
        else if (role.against_last) e = role.against_last + ((int64_t)seg.seq * a.Hv + h) * state_size;
      }
      float2 sum = splat2(0.0f);
      if (has_row && (to || e)) {
#pragma unroll 1
        for (int u = 0; u < kCols / 16; ++u) {
          float2 d[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = splat2(0.0f);
          if (n > 0 || has_carry) tmem_sum<1>(tm + tU + lane_at + c0 + 16 * u, 0, d);
          if (e) {
            float2 x[8];
            load_state(e, c0 + 16 * u, x);
#pragma unroll
            for (int i = 0; i < 8; ++i)  // past the state d may be what the matrix unit made of other rows
              if (row < n1 && c0 + 16 * u + 2 * i < n2) sum = fma2(d[i], x[i], sum);
          }
          if (to)
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const int col = c0 + 16 * u + 2 * i;
              if (row >= n1 || col >= n2) continue;
              float* q = to + state_at(col);  // these are never the transposed ones
              *reinterpret_cast<float4*>(q) = make_float4(d[i].x, d[i].y, d[i + 1].x, d[i + 1].y);
            }
        }
      }
      if (role.cross) {
        float v = sum.x + sum.y;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) s_sums[warp] = v;
        named_barrier(1, 32 * kPathWarps);
        if (t == 0) {
          for (int i = 1; i < kPathWarps; ++i) v += s_sums[i];
          role.cross[(int64_t)seg_at * a.Hv + h] = v;
        }
      }
    }
  } else if (warp < 2 * kPathWarps) {  // the results' path
    for (int k = 0; k < n; ++k) {
      const uint32_t p = k & 1;
      const int c = chunk_of(k), rows = min(kC, seg.len - c * kC);
      const bool has_state = k > 0 || has_carry;
      wait(bars + kGatesFull, p);
      const float in = s_in[row], mine = s_f[row], rest = s_h[row];
      const bool near = *s_near;
      const int see = back ? row + (has_dot ? 1 : 0) : row + (has_dot ? 0 : 1);  // the columns a row sees: j < see, back: see <= j < rows
      wait(bars + kDoneA, p);
      tmem_fence_after_sync();
#pragma unroll 1
      for (int u = 0; u < 4; ++u) {
        // a thread's blocks of 16 columns, spread: P is triangular
        const int j0 = 16 * (u & 1 ? 2 * u + 1 - part : 2 * u + part);
        uint32_t words[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) words[i] = 0;
        if (back ? j0 + 15 >= quad * 32 && j0 < rows : j0 <= quad * 32 + 31) {  // the warp has rows that see these columns
          float2 d[8];
          tmem_sum<1>(tm + tA + lane_at + j0, 0, d);
          const bool all = back ? j0 > quad * 32 + 31 && j0 + 15 < rows : j0 + 15 < quad * 32;
          if (!all && has_dot) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (j0 + i == row) s_diag[row] = a.scale * (i % 2 ? d[i / 2].y : d[i / 2].x);
          }
          const float4* h4 = reinterpret_cast<const float4*>(s_h + j0);
          if (near) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 f = h4[i];
              d[2 * i] = mul2(d[2 * i], mul2(make_float2(f.x, f.y), splat2(mine)));
              d[2 * i + 1] = mul2(d[2 * i + 1], mul2(make_float2(f.z, f.w), splat2(mine)));
            }
          } else {
            const float sign = back ? -1.0f : 1.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              d[i].x *= a.scale * ex2(sign * ((mine - s_f[j0 + 2 * i]) + (rest - s_h[j0 + 2 * i])));
              d[i].y *= a.scale * ex2(sign * ((mine - s_f[j0 + 2 * i + 1]) + (rest - s_h[j0 + 2 * i + 1])));
            }
          }
          if (!all) {
            const int lo = back ? see - j0 : 0, count = (back ? rows : see) - j0 - lo;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if ((unsigned)(2 * i - lo) >= (unsigned)max(count, 0)) d[i].x = 0.0f;
              if ((unsigned)(2 * i + 1 - lo) >= (unsigned)max(count, 0)) d[i].y = 0.0f;
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t term[2];
            split_pair<2>(d[i], term);
            words[i] = term[0];
            words[8 + i] = term[1];
          }
        }
        __syncwarp();
        tmem_st16(tm + tA + lane_at + j0, words);
      }
      tmem_wait_st();
      warp_arrive(bars + kGatesFree, lane);
      float self = 0.0f;
      if (has_dot) {
        named_barrier(2, 32 * kPathWarps);
        self = s_diag[row];
      }
      tmem_fence_before_sync();
      warp_arrive(bars + kPReady, lane);

      const int64_t at = (int64_t)c * kC + quad * 32;  // the warp's first token
      float2 dot = splat2(0.0f);
#pragma unroll 1
      for (int s = 0; s < kCols / 16; ++s) {
        const int c0 = part * kCols + 16 * s;
        typename R::Raw raw_y, raw_w;
        if (has_dot) {  // the partner's rows, and the values of the token's own pair
          R::load(static_cast<const T*>(role.dot) + (seg.start + at) * role.sdot + (int64_t)(h / role.rdot) * n2 + c0, role.sdot,
                  seg.len - at, n2 - c0, lane, raw_y);
          R::load(static_cast<const T*>(role.w) + (seg.start + at) * role.sw + (int64_t)(h / role.rw) * n2 + c0, role.sw,
                  seg.len - at, n2 - c0, lane, raw_w);
        }
        if (s == 0) {
          wait(bars + kUpReady, p);  // what weigh() found
          wait(bars + kDoneO, p);
          tmem_fence_after_sync();
        }
        float2 o[8];
        tmem_sum<1>(tm + tO + lane_at + c0, 0, o);
        if (has_state) {
          float2 e[8];
          tmem_sum<1>(tm + tD1 + lane_at + c0, 0, e);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = fma2(splat2(in), e[i], o[i]);
        }
        if (has_dot) {
          transpose(raw_y[0], lane);
          transpose(raw_w[0], lane);
          R::each(raw_y, 0, [&](int i, float2 y) { dot = fma2(y, o[i], dot); });
          R::each(raw_w, 0, [&](int i, float2 w) { o[i] = fma2(splat2(self), w, o[i]); });
        }
        if (*odd) {
          const uint32_t mask = odd_columns(
              role, static_cast<const T*>(role.w) + (seg.start + (int64_t)c * kC) * role.sw + (int64_t)(h / role.rw) * n2 + c0, row,
              rows, n2 - c0);
          const float nan = __int_as_float(0x7fffffff);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (mask >> (2 * i) & 1) o[i].x = nan;
            if (mask >> (2 * i + 1) & 1) o[i].y = nan;
          }
        }
        const int64_t out_at = ((seg.start + at) * a.Hv + h) * n2 + c0;
        auto store = [&](auto rows_of, auto* base) {
          using Q = decltype(rows_of);
          typename Q::Raw raw;
          Q::put(raw, 0, o);
          Q::store(base + out_at, (int64_t)a.Hv * n2, seg.len - at, n2 - c0, lane, raw);
        };
        if (role.part) store(RF(), static_cast<float*>(role.out));
        else store(R(), static_cast<T*>(role.out));
      }
      if (has_dot && row < rows) role.dots[((int64_t)part * a.T + seg.start + at + lane) * a.Hv + h] = dot.x + dot.y;
      tmem_fence_before_sync();
      warp_arrive(bars + kOutDone, lane);
    }
  }
  tmem_fence_before_sync();
  __syncthreads();
  if (warp == kProducts) tmem_dealloc<512>(tm);
}

// ------------------------------------------------------------------ what a segment adds to the state
// One CTA per (inner segment, value head, role): the sum of Y^T (up * W) with up
// the weights up to the segment's end, so that the chunks add up in tensor
// memory with nothing read back in between: the chunk next to that end comes
// first, and each earlier one's weights carry the decay over the ones behind it.
template <int KP, int NP>
struct StateSmem {
  static constexpr int kY = KP * kPanel, kW = NP * kPanel, kUp = 2 * kW;
  static constexpr int oY = 0, oW = 2 * kY, oUp = oW + 2 * kW, oGates = oUp + kUp, oMisc = oGates + 2 * 4 * kC;
  static constexpr int oBar = oMisc + 64, kBytes = oBar + 16 * 8;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};
constexpr int kWeighWarps = 16;

template <int KP, int NP>
__global__ void __launch_bounds__(kWarps * 32, 1)
    lin_state_bf16_kernel(const __grid_constant__ LinArgs a, const __grid_constant__ LinMaps maps, int roles) {
  using L = StateSmem<KP, NP>;
  constexpr int kN = NP * 64, kCols = NP * 32;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::oBar);
  uint64_t *full = bars, *gates_full = bars + 2, *used = bars + 4, *up_ready = bars + 6, *done = bars + 7, *drained = bars + 8;
  float* s_total = reinterpret_cast<float*>(sm + L::oMisc);
  volatile int* stop = reinterpret_cast<int*>(s_total + 1);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(s_total + 2);
  const int which = blockIdx.x % roles, h = blockIdx.x / roles % a.Hv;
  const int64_t item = blockIdx.x / roles / a.Hv;
  if (item >= a.info[1]) return;
  const LinRole& role = a.role[which];
  const bool back = role.back != 0;
  const Segment seg(a.table[a.inner[item] + (back ? 1 : 0)]);
  const int n1 = role.n1, n2 = role.n2, n = seg.n;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, quad = warp & 3, row = quad * 32 + lane;
  if (t == 0) {
    for (int i = 0; i < 9; ++i) mbar_init(bars + i, i == 6 || (i == 4 || i == 5) ? kWeighWarps : 1);
    *stop = 0;
    fence_mbar_init();
  }
  if (warp == kProducts) tmem_alloc<128>(tmem_at);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tm = *tmem_at, lane_at = (uint32_t)(quad * 32) << 16;
  LinWaiter wait{a, stop};
  auto chunk_of = [&](int k) { return back ? k : n - 1 - k; };

  if (warp == kProducts) {
    if (lane == 0) {
      const Operand<128, kMnMajor, 2, L::kW, 0, kPanel> Up(smem_u32(sm + L::oUp));
      for (int k = 0; k < n; ++k) {
        wait(up_ready, k & 1, k == 0 && forced_here(a));
        if (wait.ok) {
          tmem_fence_after_sync();
          const Operand<128, kMnMajor, 1, L::kY, 0, kPanel> Yt(smem_u32(sm + L::oY + (k & 1) * L::kY));
          umma_terms<kN, kC / 16, 2>(tm, Yt, Up, k > 0);
          umma_commit(done);
        }
      }
      if (*stop) {
        umma_commit(drained);
        mbar_wait(drained, 0, kCopyDrainNs);
      }
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
        wait(done, k & 1);  // Y's buffer; W's was read before
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
    load_g(chunk_of(0), g);
    Pair behind{0.0f, 0.0f};
    for (int k = 0; k < n; ++k) {
      const GateSums<4> sums(g, lane);
      if (k + 1 < n) load_g(chunk_of(k + 1), g);
      float up[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        up[i] = back ? a.scale * exp2_of(add(behind, sums.G[i])) : exp2_of(add(behind, add(sums.last, minus(sums.G[i]))));
      behind = add(behind, sums.last);
      if (k >= 2) wait(used + (k & 1), ((k - 2) >> 1) & 1);
      __syncwarp();
      reinterpret_cast<float4*>(sm + L::oGates + (k & 1) * 4 * kC)[lane] = make_float4(up[0], up[1], up[2], up[3]);
      if (k + 1 == n && lane == 0) {
        *s_total = exp2_of(behind);
        role.decay[item * a.Hv + h] = *s_total;
      }
      warp_arrive(gates_full + (k & 1), lane);
    }
  } else if (warp < kWeighWarps) {
    for (int k = 0; k < n; ++k) {
      const int b = k & 1, rows = min(kC, seg.len - chunk_of(k) * kC);
      wait(gates_full + b, (k >> 1) & 1);
      wait(full + b, (k >> 1) & 1);
      if (k > 0) wait(done, (k - 1) & 1);  // up * W's place is free
      weigh<NP, 32 * kWeighWarps>(sm + L::oW + b * L::kW, sm + L::oUp, reinterpret_cast<const float*>(sm + L::oGates + b * 4 * kC), rows, t,
                                  nullptr);
      if (rows < kC) clear_rows<KP>(sm + L::oY + b * L::kY, rows, t, 32 * kWeighWarps);
      fence_async_smem();
      warp_arrive(used + b, lane);
      if (lane == 0) mbar_arrive(up_ready);
    }
    wait(done, (n - 1) & 1);
    tmem_fence_after_sync();
    if (warp < kPathWarps) {
      const int c0 = (warp >> 2) * kCols;
      const float total = *s_total;
      const float* carry = role.first && (back ? seg.is_last : seg.is_first)
                               ? role.first + ((int64_t)seg.seq * a.Hv + h) * ((int64_t)n1 * n2) : nullptr;
      float* to = role.slots + (item * a.Hv + h) * ((int64_t)n1 * n2);
#pragma unroll 1
      for (int u = 0; u < kCols / 16; ++u) {
        float2 d[8];
        tmem_sum<1>(tm + lane_at + c0 + 16 * u, 0, d);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const int col = c0 + 16 * u + 2 * i;
          if (row >= n1 || col >= n2) continue;
          const int64_t at = (int64_t)row * n2 + col;
          if (carry) {
            const float4 f = *reinterpret_cast<const float4*>(carry + at);
            d[i] = fma2(splat2(total), make_float2(f.x, f.y), d[i]);
            d[i + 1] = fma2(splat2(total), make_float2(f.z, f.w), d[i + 1]);
          }
          *reinterpret_cast<float4*>(to + at) = make_float4(d[i].x, d[i].y, d[i + 1].x, d[i + 1].y);
        }
      }
    }
  }
  tmem_fence_before_sync();
  __syncthreads();
  if (warp == kProducts) tmem_dealloc<128>(tm);
}

template <int KP, int NP, bool kState>
cudaError_t run(const LinArgs& a, const LinMaps& maps, int roles, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const auto kernel = kState ? lin_state_bf16_kernel<KP, NP> : lin_walk_bf16_kernel<KP, NP>;
  constexpr size_t bytes = kState ? (size_t)StateSmem<KP, NP>::kBytes : (size_t)WalkSmem<KP, NP>::kBytes;
  const cudaError_t e = set_smem(reinterpret_cast<const void*>(kernel), bytes, done);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (kState ? a.max_inner : a.max_segs) * a.Hv * roles;
  kernel<<<(unsigned)blocks, kWarps * 32, bytes, st>>>(a, maps, roles);
  return cudaGetLastError();
}

template <bool kState>
cudaError_t pick(const LinArgs& a, const LinMaps& maps, int roles, cudaStream_t st) {
  int n1 = 0, n2 = 0;
  for (int i = 0; i < roles; ++i) {
    n1 = n1 > a.role[i].n1 ? n1 : a.role[i].n1;
    n2 = n2 > a.role[i].n2 ? n2 : a.role[i].n2;
  }
  if (n1 > 64) return n2 > 64 ? run<2, 2, kState>(a, maps, roles, st) : run<2, 1, kState>(a, maps, roles, st);
  return n2 > 64 ? run<1, 2, kState>(a, maps, roles, st) : run<1, 1, kState>(a, maps, roles, st);
}

}  // namespace

cudaError_t launch_lin_walk_bf16(const LinArgs& a, const LinMaps& maps, int roles, bool state_only, cudaStream_t st) {
  if ((state_only ? a.max_inner : a.max_segs) == 0) return cudaSuccess;
  return state_only ? pick<true>(a, maps, roles, st) : pick<false>(a, maps, roles, st);
}

}  // namespace vssm
