// linear.cu -- linear attention's walk over the chunks of a segment in f32: the
// forward, each of its three gradients, and the states between segments.  The
// bf16 walks are linear_bf16.cu's.
#include "linear.cuh"

namespace vssm {
namespace {

// One CTA per (segment, value head, role, 64 columns of the state; the columns
// never mix).  A chunk of 64 tokens is four products on the matrix unit, every
// operand in three bf16 terms (24 bits):
//   A  = X Y^T             read back, weighted and masked: P, bf16 terms in tensor memory
//   D1 = X S
//   U  = Y^T (up * W)      S = exp(G_end) S + U, in registers and as bf16 terms in shared memory
//   D2 = P W               out = in * D1 + D2
// with in and up the weights of a row for the state and in it.  Sixteen warps
// work on the operands and results, four threads to a row; another issues the
// products and makes the next chunk's gates meanwhile.  What one product
// leaves is worked on while the next one runs: up * W during A and D1, P
// during U, S during D2.  Chunks of 64 tokens and tiles of 64 columns are what
// shared memory holds of three terms; the chain of a chunk is what bounds it
// (3001 tokens, 6 heads of 96 x 80: 51 us forward, 130 the gradients; 11 us for
// 16 tokens).
constexpr int kLinWorkers = 128 * kLinParts, kLinThreads = kLinWorkers + 32, kLinCtrl = kLinWorkers / 32;

constexpr int kC = 64, kTerms = 3;  // tokens of a chunk, bf16 terms of a value
constexpr int kBlockWords = 32;     // columns of tensor memory that a block of 16 columns of P takes, its terms one after the other
constexpr int tA = 0, tP = 64, tD1 = 192, tU = 256, tO = 320;  // columns of tensor memory

template <int KP>
struct LinSmem {
  static constexpr int kPanel = kC * 128;  // bytes of 64 columns of a chunk's rows
  static constexpr int kX = kTerms * KP * kPanel, kW = kTerms * kPanel, kSTerm = KP * 64 * 128, kS = kTerms * kSTerm;
  // (the products take 128 rows of X's 64: what follows it counts as rows whose results nobody reads)
  static constexpr int oX = 0, oY = kX, oW = oY + kX, oUp = oW + kW, oS = oUp + kW, oGates = oS + kS;
  // of the tokens: G / ln 2 as two floats; in and up; the two factors of P's weights
  static constexpr int oInUp = 8 * kC, oRow = 16 * kC, oCol = 20 * kC, kGates = 24 * kC;
  static constexpr int oEnd = oGates + 2 * kGates;       // exp(G_end) of either buffer, and whether the factors serve
  static constexpr int oDiag = oEnd + 16, oBad = oDiag + 4 * kC, oAnyBad = oBad + 2 * 64 * 4;
  static constexpr int oBar = oAnyBad + 16, kBytes = oBar + 64 + 1024;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

// The six pairs of three terms whose product counts, smallest first.
__device__ __forceinline__ int first_term(int i) { return (0x124 >> (2 * i)) & 3; }
__device__ __forceinline__ int second_term(int i) { return (0x046 >> (2 * i)) & 3; }

template <int KP, bool kStateOnly>
__global__ void __launch_bounds__(kLinThreads, 1) lin_walk_kernel(const __grid_constant__ LinArgs a, int roles, int all_tiles) {
  using L = LinSmem<KP>;
  using R = WalkRow<float, 2>;  // 16 columns to a thread
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  uint64_t* bar_a = reinterpret_cast<uint64_t*>(sm + L::oBar);
  uint64_t *bar_u = bar_a + 1, *bar_o = bar_a + 2, *drained = bar_a + 3;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(bar_a + 4);
  volatile int* stop = reinterpret_cast<int*>(tmem_at + 1);
  volatile int* leave = stop + 1;
  float* s_end = reinterpret_cast<float*>(sm + L::oEnd);
  int* s_near = reinterpret_cast<int*>(s_end + 2);
  float* s_diag = reinterpret_cast<float*>(sm + L::oDiag);
  int* s_bad = reinterpret_cast<int*>(sm + L::oBad);
  volatile int* any_bad = reinterpret_cast<int*>(sm + L::oAnyBad);

  // what this CTA walks
  int tile = blockIdx.x % all_tiles, which = 0;
  const int h = blockIdx.x / all_tiles % a.Hv;
  const int64_t item = blockIdx.x / all_tiles / a.Hv;
  while (which + 1 < roles && tile >= lin_tiles(a.role[which].n2)) tile -= lin_tiles(a.role[which++].n2);
  const LinRole& role = a.role[which];
  const bool back = role.back != 0, has_dot = role.dot != nullptr;
  if (item >= a.info[kStateOnly ? 1 : 0]) return;
  const int seg = kStateOnly ? a.inner[item] + (back ? 1 : 0) : a.order[item];
  const int4 entry = a.table[seg];
  const int64_t start = entry.y;
  const int len = entry.z, n = (len + kC - 1) / kC;
  const bool is_first = entry.w & kLinFirst, is_last = entry.w & kLinLast;
  const int64_t inner_before = (unsigned)entry.w >> kLinPlaceShift;
  const int n1 = role.n1, n2 = role.n2, tiles = lin_tiles(n2);

  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  auto bad_none = [&]() { return back ? -1 : kC; };
  if (t == 0) {
    mbar_init(bar_a, 1);
    mbar_init(bar_u, 1);
    mbar_init(bar_o, 1);
    mbar_init(drained, 1);
    *stop = *leave = 0;
    any_bad[0] = any_bad[1] = 0;
    fence_mbar_init();
  }
  if (t < 128) s_bad[t] = bad_none();
  if (warp == kLinCtrl) tmem_alloc<512>(tmem_at);

  const float* g_base = a.g + start * a.g_token + h;
  // the gates of chunk c; returns the chunk's sum of g over ln 2
  auto make_gates = [&](int c, int buf) -> Pair {
    constexpr int kPer = kC / 32;
    const int rows = min(kC, len - c * kC);
    Pair own[kPer], incl{0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = lane * kPer + i;
      incl = add(incl, Pair{r < rows ? clamp_g(g_base[(int64_t)(c * kC + r) * a.g_token]) : 0.0f, 0.0f});
      own[i] = incl;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Pair v{__shfl_up_sync(0xffffffffu, incl.hi, o), __shfl_up_sync(0xffffffffu, incl.lo, o)};
      if (lane >= o) incl = add(v, incl);
    }
    const Pair last = over_ln2(Pair{__shfl_sync(0xffffffffu, incl.hi, 31), __shfl_sync(0xffffffffu, incl.lo, 31)});
    Pair before{__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
    if (lane == 0) before = Pair{0.0f, 0.0f};
    uint8_t* gates = sm + L::oGates + buf * L::kGates;
    const float mid = 0.5f * last.hi;
    bool near = true;  // both factors of every weight are normal numbers
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = lane * kPer + i;
      const Pair G = over_ln2(add(before, own[i]));
      const float from = a.scale * exp2_of(G), to = exp2_of(add(last, Pair{-G.hi, -G.lo}));
      const Pair d = add(G, Pair{-mid, 0.0f});
      const float up = exp2_of(d), down = exp2_of(Pair{-d.hi, -d.lo});
      near = near && fabsf(d.hi) < 120.0f;
      reinterpret_cast<float2*>(gates)[r] = make_float2(G.hi, G.lo);
      reinterpret_cast<float2*>(gates + L::oInUp)[r] = back ? make_float2(to, from) : make_float2(from, to);
      reinterpret_cast<float*>(gates + L::oRow)[r] = a.scale * (back ? down : up);
      reinterpret_cast<float*>(gates + L::oCol)[r] = back ? up : down;
    }
    near = __all_sync(0xffffffffu, near);
    if (lane == 0) s_near[buf] = near;
    if (lane == 0) s_end[buf] = exp2_of(last);
    return last;
  };

  const float* xb = static_cast<const float*>(role.x) + start * role.sx + (int64_t)(h / role.rx) * n1;
  const float* yb = static_cast<const float*>(role.y) + start * role.sy + (int64_t)(h / role.ry) * n1;
  const float* wb = static_cast<const float*>(role.w) + start * role.sw + (int64_t)(h / role.rw) * n2 + tile * kLinTile;
  const int wcols = n2 - tile * kLinTile;  // of W from this tile on

  auto note_bad = [&](int which_buf, int col, int r) {
    if (back) atomicMax(s_bad + which_buf * 64 + col, r); else atomicMin(s_bad + which_buf * 64 + col, r);
    any_bad[which_buf] = 1;
  };
  // The images of X, Y, W and up * W, through registers.  A value of W that is
  // not finite reaches the state, and so every later row, through up * W; in D2,
  // where 0 times it would reach earlier rows, 0 takes its place, and its
  // column's rows from it on are made NaN when they are written.
  constexpr int kLoadX = kC * KP * 8 / kLinWorkers, kLoadW = kC * 8 / kLinWorkers;
  auto load_images = [&](int c, int buf) {
    {
      const int rows = len - c * kC;
      float4 x[kLoadX][2], y[kLoadX][2], w[kLoadW][2];
      auto get = [&](float4 (&f)[2], const float* base, int64_t stride, int r, int ch, int cols) {
        f[0] = f[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < rows && ch * 8 < cols) {
          const float4* src = reinterpret_cast<const float4*>(base + (c * kC + r) * stride + ch * 8);
          f[0] = src[0];
          f[1] = src[1];
        }
      };
#pragma unroll
      for (int u = 0; u < kLoadX; ++u) {
        const int i = t + u * kLinWorkers, r = i / (KP * 8), ch = i % (KP * 8);
        get(y[u], yb, role.sy, r, ch, n1);
        if (!kStateOnly) get(x[u], xb, role.sx, r, ch, n1);
      }
#pragma unroll
      for (int u = 0; u < kLoadW; ++u) get(w[u], wb, role.sw, (t + u * kLinWorkers) / 8, t % 8, wcols);
#pragma unroll
      for (int u = 0; u < kLoadX; ++u) {
        const int i = t + u * kLinWorkers, r = i / (KP * 8), ch = i % (KP * 8);
        auto put = [&](int o, const float4 (&f)[2]) {
          const float2 v[4] = {make_float2(f[0].x, f[0].y), make_float2(f[0].z, f[0].w), make_float2(f[1].x, f[1].y),
                               make_float2(f[1].z, f[1].w)};
          put_chunk<kTerms, 128>(sm + o + (ch >> 3) * L::kPanel, KP * L::kPanel, r, ch & 7, v);
        };
        put(L::oY, y[u]);
        if (!kStateOnly) put(L::oX, x[u]);
      }
      const float2* in_up = reinterpret_cast<const float2*>(sm + L::oGates + buf * L::kGates + L::oInUp);
#pragma unroll
      for (int u = 0; u < kLoadW; ++u) {
        const int r = (t + u * kLinWorkers) / 8, ch = t % 8;
        float2 v[4] = {make_float2(w[u][0].x, w[u][0].y), make_float2(w[u][0].z, w[u][0].w),
                       make_float2(w[u][1].x, w[u][1].y), make_float2(w[u][1].z, w[u][1].w)};
        float2 up[4];
        float2 trace = splat2(0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          up[i] = mul2(v[i], splat2(in_up[r].y));
          trace = fma2(v[i], splat2(0.0f), trace);
        }
        put_chunk<kTerms, 128>(sm + L::oUp, L::kPanel, r, ch, up);
        if (trace.x + trace.y != 0.0f) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (v[i].x * 0.0f != 0.0f) { note_bad(buf, ch * 8 + 2 * i, r); v[i].x = 0.0f; }
            if (v[i].y * 0.0f != 0.0f) { note_bad(buf, ch * 8 + 2 * i + 1, r); v[i].y = 0.0f; }
          }
        }
        if (!kStateOnly) put_chunk<kTerms, 128>(sm + L::oW, L::kPanel, r, ch, v);
      }
    }
  };
  const int quad = warp & 3, part = (warp >> 2) & (kLinParts - 1), row = quad * 32 + lane;
  const int col0 = tile * kLinTile + part * 16;  // this thread's columns of the state and of the results
  const bool state_row = row < n1 && warp < kLinCtrl;
  // the state the segment starts from, if any
  const int64_t state_at = (int64_t)row * role.srow + (int64_t)col0 * role.scol;
  const int64_t state_size = (int64_t)n1 * n2;
  const float* carry = nullptr;
  if (back ? is_last : is_first) {
    if (role.first) carry = role.first + ((int64_t)entry.x * a.Hv + h) * state_size;
  } else if (!kStateOnly) {
    carry = role.slots + ((back ? inner_before : inner_before - 1) * a.Hv + h) * state_size;
  }
  float2 S[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) S[i] = splat2(0.0f);
  auto state_io = [&](auto f) {  // f(i, offset) for the pairs i of this thread's columns that exist
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (state_row && col0 + 2 * i < n2) f(i, state_at + 2 * i * role.scol);
  };
  if (carry) state_io([&](int i, int64_t at) { S[i] = make_float2(carry[at], carry[at + role.scol]); });
  const bool has_carry = carry != nullptr;

  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tm = *tmem_at;
  const uint32_t lane_at = (uint32_t)(quad * 32) << 16;
  LinWaiter wait{a, stop};
  auto chunk_of = [&](int k) { return back ? n - 1 - k : k; };

  if (warp == kLinCtrl) {  // all lanes go through it together, so that addresses are uniform; one issues
    const bool lead = elect_one();
    Pair total{0.0f, 0.0f};
    if (n > 0) total = make_gates(chunk_of(0), 0);
    if (n > 0) named_barrier(4, kLinThreads);
    for (int k = 0; k < n; ++k) {
      const int buf = k & 1;
      if (lane == 0) *leave = *stop;
      named_barrier(1, kLinThreads);
      if (*leave) break;
      const uint64_t x = smem_desc<128>(smem_u32(sm + L::oX)), y = smem_desc<128>(smem_u32(sm + L::oY));
      if (!kStateOnly && !*stop) {
        tmem_fence_after_sync();
        constexpr uint32_t idesc = umma_idesc(kKMajor, kKMajor, kC), idesc_s = umma_idesc(kKMajor, kMnMajor, 64);
#pragma unroll 1
        for (int i = 0; i < 6 * KP; ++i) {
          const int first = first_term(i / KP), second = second_term(i / KP), panel = i % KP;
#pragma unroll
          for (int s = 0; s < 4; ++s)
            umma_one(tm + tA, x + ((first * KP + panel) * L::kPanel + s * 32) / 16,
                    y + ((second * KP + panel) * L::kPanel + s * 32) / 16, idesc, i + s > 0 ? 1u : 0u);
        }
        if (lead) umma_commit(bar_a);
        if (k > 0 || has_carry) {
          const uint64_t st = smem_desc<128>(smem_u32(sm + L::oS), L::kSTerm);
#pragma unroll 1
          for (int i = 0; i < 6 * KP; ++i) {
            const int first = first_term(i / KP), second = second_term(i / KP), panel = i % KP;
#pragma unroll
            for (int s = 0; s < 4; ++s)
              umma_one(tm + tD1, x + ((first * KP + panel) * L::kPanel + s * 32) / 16,
                      st + (second * L::kSTerm + (4 * panel + s) * 2048) / 16, idesc_s, i + s > 0 ? 1u : 0u);
          }
        }
      }
      __syncwarp();
      named_barrier(2, kLinThreads);
      if (!*stop) {
        tmem_fence_after_sync();
        constexpr uint32_t idesc = umma_idesc(kMnMajor, kMnMajor, 64);
        const uint64_t yt = smem_desc<128>(smem_u32(sm + L::oY), L::kPanel), up = smem_desc<128>(smem_u32(sm + L::oUp), L::kPanel);
#pragma unroll 1
        for (int i = 0; i < 6; ++i)
#pragma unroll
          for (int s = 0; s < kC / 16; ++s)
            umma_one(tm + tU, yt + (first_term(i) * KP * L::kPanel + s * 2048) / 16, up + (second_term(i) * L::kPanel + s * 2048) / 16,
                    idesc, i + s > 0 ? 1u : 0u);
        if (lead) umma_commit(bar_u);
      }
      __syncwarp();
      if (k + 1 < n) total = add(total, make_gates(chunk_of(k + 1), buf ^ 1));
      if constexpr (!kStateOnly) {
        named_barrier(3, kLinThreads);
        if (!*stop) {
          tmem_fence_after_sync();
          constexpr uint32_t idesc = umma_idesc(kKMajor, kMnMajor, 64);
          const uint64_t w = smem_desc<128>(smem_u32(sm + L::oW));
#pragma unroll 1
          for (int i = 0; i < 6; ++i)
#pragma unroll
            for (int s = 0; s < kC / 16; ++s)
              umma_ta_one(tm + tO, tm + tP + kBlockWords * s + 8 * first_term(i), w + (second_term(i) * L::kPanel + s * 2048) / 16,
                         idesc, i + s > 0 ? 1u : 0u);
          if (lead) umma_commit(bar_o);
        }
        __syncwarp();
      }
      if (k + 1 < n) named_barrier(4, kLinThreads);
    }
    if (kStateOnly && lane == 0 && tile == 0) role.decay[item * a.Hv + h] = exp2_of(total);
  } else {
    uint32_t phase = 0;
    if (n > 0) {
      named_barrier(4, kLinThreads);  // the gates
      load_images(chunk_of(0), 0);
    }
    if (!kStateOnly && has_carry && row < KP * 64)
      put_row<kTerms, 128>(sm + L::oS, L::kSTerm, row, part * 2, S);
    for (int k = 0; k < n; ++k, phase ^= 1) {
      const int c = chunk_of(k), buf = k & 1;
      const int rows = min(kC, len - c * kC);
      const bool more = k + 1 < n, has_state = k > 0 || has_carry;
      fence_async_smem();
      tmem_fence_before_sync();
      named_barrier(1, kLinThreads);
      tmem_fence_after_sync();
      if (*leave) break;
      if (t < 64) s_bad[(buf ^ 1) * 64 + t] = bad_none();
      if (t == 0) any_bad[buf ^ 1] = 0;
      asm volatile("bar.arrive %0, %1;" ::"r"(2), "r"(kLinThreads) : "memory");

      if constexpr (!kStateOnly) {
        wait(bar_a, phase, k == 0 && t == 0 && forced_here(a));
        tmem_fence_after_sync();
        if (row < kC) {
          const uint8_t* gates = sm + L::oGates + buf * L::kGates;
          const float row_factor = reinterpret_cast<const float*>(gates + L::oRow)[row];
          // the columns a row sees: fwd j < see, back see <= j < rows
          const int see = back ? row + (has_dot ? 1 : 0) : row + (has_dot ? 0 : 1);
          const bool near = s_near[buf];
          {
            const int j0 = 16 * part;
            uint32_t words[kBlockWords];
#pragma unroll
            for (int i = 0; i < kBlockWords; ++i) words[i] = 0;
            if (back ? j0 + 15 >= quad * 32 && j0 < rows : j0 <= quad * 32 + 31) {  // the warp has rows that see these columns
              float2 d[8];
              tmem_sum<1>(tm + tA + lane_at + j0, 0, d);
              const bool all = back ? j0 > quad * 32 + 31 && j0 + 15 < rows : j0 + 15 < quad * 32;
              if (!all && has_dot) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (j0 + i == row) s_diag[row] = a.scale * (i % 2 ? d[i / 2].y : d[i / 2].x);
              }
              if (near) {
                const float4* col = reinterpret_cast<const float4*>(gates + L::oCol) + j0 / 4;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float4 f = col[i];
                  d[2 * i] = mul2(d[2 * i], mul2(make_float2(f.x, f.y), splat2(row_factor)));
                  d[2 * i + 1] = mul2(d[2 * i + 1], mul2(make_float2(f.z, f.w), splat2(row_factor)));
                }
              } else {
                const float2* sums = reinterpret_cast<const float2*>(gates);
                const float2 mine = sums[row];
                const float sign = back ? -1.0f : 1.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const float2 x = sums[j0 + 2 * i], y = sums[j0 + 2 * i + 1];
                  d[i].x *= a.scale * ex2(sign * ((mine.x - x.x) + (mine.y - x.y)));
                  d[i].y *= a.scale * ex2(sign * ((mine.x - y.x) + (mine.y - y.y)));
                }
              }
              if (!all) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const int j = j0 + 2 * i;
                  if (back ? j < see || j >= rows : j >= see) d[i].x = 0.0f;
                  if (back ? j + 1 < see || j + 1 >= rows : j + 1 >= see) d[i].y = 0.0f;
                }
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                uint32_t term[kTerms];
                split_pair<kTerms>(d[i], term);
#pragma unroll
                for (int q = 0; q < kTerms; ++q) words[8 * q + i] = term[q];
              }
            }
            __syncwarp();
            tmem_st32(tm + tP + lane_at + 2 * j0, words);
          }
          tmem_wait_st();
        }
        tmem_fence_before_sync();
        named_barrier(3, kLinThreads);
      }

      wait(bar_u, phase, kStateOnly && k == 0 && t == 0 && forced_here(a));
      tmem_fence_after_sync();
      if (row < KP * 64) {
        const float end = s_end[buf];
        float2 d[8];
        tmem_sum<1>(tm + tU + lane_at + part * 16, 64, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) S[i] = fma2(splat2(end), S[i], d[i]);
        if (!kStateOnly && more) put_row<kTerms, 128>(sm + L::oS, L::kSTerm, row, part * 2, S);
      }

      if constexpr (!kStateOnly) {
        wait(bar_o, phase);
        tmem_fence_after_sync();
        if (row < kC) {
          const int64_t at = (int64_t)c * kC + quad * 32;  // the warp's first token
          float2 o[8];
          tmem_sum<1>(tm + tO + lane_at + part * 16, 0, o);
          if (has_state) {
            const float in = reinterpret_cast<const float2*>(sm + L::oGates + buf * L::kGates + L::oInUp)[row].x;
            float2 e[8];
            tmem_sum<1>(tm + tD1 + lane_at + part * 16, 64, e);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = fma2(splat2(in), e[i], o[i]);
          }
          float dot = 0.0f;
          if (has_dot) {  // rho or sigma, then the token's own pair
            typename R::Raw raw;
            R::load(static_cast<const float*>(role.dot) + (start + at) * role.sdot + (int64_t)(h / role.rdot) * n2 + col0, role.sdot,
                    len - at, n2 - col0, lane, raw);
#pragma unroll
            for (int i = 0; i < R::kParts; ++i) transpose(raw[i], lane);
            float2 sum = splat2(0.0f);
            R::each(raw, 0, [&](int i, float2 y) { sum = fma2(y, o[i], sum); });
            dot = sum.x + sum.y;
            const float self = s_diag[row];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint32_t place = image_chunk<128>(row, part * 2 + q);
#pragma unroll
              for (int term = kTerms - 1; term >= 0; --term) {
                float2 w[4];
                unpack(*reinterpret_cast<const uint4*>(sm + L::oW + term * L::kPanel + place), w);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[4 * q + i] = fma2(splat2(self), w[i], o[4 * q + i]);
              }
            }
          }
          if (any_bad[buf]) {
            const float nan = __int_as_float(0x7fffffff);
            const int* bad = s_bad + buf * 64 + part * 16;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (back ? row <= bad[2 * i] : row >= bad[2 * i]) o[i].x = nan;
              if (back ? row <= bad[2 * i + 1] : row >= bad[2 * i + 1]) o[i].y = nan;
              if (back ? row < max(bad[2 * i], bad[2 * i + 1]) : row > min(bad[2 * i], bad[2 * i + 1])) dot = nan;  // another row's
            }
          }
          if (has_dot && row < rows) role.dots[((int64_t)(tile * kLinParts + part) * a.Hv + h) * a.T + start + at + lane] = dot;
          const int64_t out_at = ((start + at) * a.Hv + h) * n2 + col0;
          typename R::Raw raw;
          R::put(raw, 0, o);
          R::store(static_cast<float*>(role.out) + out_at, (int64_t)a.Hv * n2, len - at, n2 - col0, lane, raw);
        }
      }
      if (more) {
        named_barrier(4, kLinThreads);  // everyone is through with the images, and the next gates are there
        load_images(chunk_of(k + 1), buf ^ 1);
      }
    }
    // the state the segment leaves
    float* to = nullptr;
    if (kStateOnly) to = role.slots + (item * a.Hv + h) * state_size;
    else if (role.last && (back ? is_first : is_last)) to = role.last + ((int64_t)entry.x * a.Hv + h) * state_size;
    if (to) state_io([&](int i, int64_t at) {
      to[at] = S[i].x;
      to[at + role.scol] = S[i].y;
    });
    if (!kStateOnly && role.cross && (!back || is_first)) {
      const float* e = nullptr;
      if (!back && !is_last) e = role.against + (inner_before * a.Hv + h) * state_size;
      else if (role.against_last) e = role.against_last + ((int64_t)entry.x * a.Hv + h) * state_size;
      float2 sum = splat2(0.0f);
      if (e) state_io([&](int i, int64_t at) { sum = fma2(S[i], make_float2(e[at], e[at + role.scol]), sum); });
      float v = sum.x + sum.y;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      float* sums = reinterpret_cast<float*>(sm + L::oGates);  // the gates are not needed any more
      named_barrier(5, kLinWorkers);
      if (lane == 0) sums[warp] = v;
      named_barrier(5, kLinWorkers);
      if (t == 0) {
        for (int i = 1; i < kLinCtrl; ++i) v += sums[i];
        role.cross[((int64_t)seg * a.Hv + h) * tiles + tile] = v;
      }
    }
  }
  tmem_fence_before_sync();
  __syncthreads();
  if (warp == kLinCtrl) {
    if (elect_one() && *stop) {  // products that were not waited for
      umma_commit(drained);
      mbar_wait(drained, 0, kCopyDrainNs);
    }
    __syncwarp();
    tmem_dealloc<512>(tm);
  }
}

template <int KP, bool kStateOnly>
cudaError_t run_walk(const LinArgs& a, int roles, cudaStream_t st) {
  constexpr size_t bytes = LinSmem<KP>::kBytes;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = set_smem(reinterpret_cast<const void*>(lin_walk_kernel<KP, kStateOnly>), bytes, done);
  if (e != cudaSuccess) return e;
  int tiles = 0;
  for (int i = 0; i < roles; ++i) tiles += lin_tiles(a.role[i].n2);
  const int64_t blocks = (kStateOnly ? a.max_inner : a.max_segs) * a.Hv * tiles;
  lin_walk_kernel<KP, kStateOnly><<<(unsigned)blocks, kLinThreads, bytes, st>>>(a, roles, tiles);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lin_walk(const LinArgs& a, const LinMaps& maps, int roles, bool state_only, IO io, cudaStream_t st) {
  if (io == IO::BF16) return state_only ? launch_lin_state_bf16(a, maps, roles, false, st) : launch_lin_walk_bf16(a, maps, roles, st);
  if ((state_only ? a.max_inner : a.max_segs) == 0) return cudaSuccess;
  int width = 0;
  for (int i = 0; i < roles; ++i) width = width > a.role[i].n1 ? width : a.role[i].n1;
  if (width > 64) return state_only ? run_walk<2, true>(a, roles, st) : run_walk<2, false>(a, roles, st);
  return state_only ? run_walk<1, true>(a, roles, st) : run_walk<1, false>(a, roles, st);
}

}  // namespace vssm
