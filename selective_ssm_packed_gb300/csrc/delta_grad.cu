// delta_grad.cu -- the gated delta rule's gradients that need no walk: dq,
// dk, dg and dbeta of a chunk from the states and state gradients around it.
#include "delta.cuh"

namespace vssm {
namespace {

// An item is a chunk and a key head; the value heads that share the key head
// follow each other, and dq and dk are summed over them in registers, in that
// order.  Where that leaves SMs idle (delta_split_grads) an item is one value
// head, whose part of dq and dk goes to `partial` and is added to the others by
// a second kernel, in the same order and so with the same bits.  CTAs of 256 threads, one an SM, take every gridDim-th item, so that the
// next item's tiles and [K; Q] arrive while this one is worked on.  Products over the state's columns (tile by tile)
// and over the chunk's tokens, rows 0-63 for the keys' tokens and 64-127 for
// the queries':
//   [A, W] = [dV; dO] [S0; E]^T    B = E dS1^T (rows 0-63)    QK = [K; Q] K^T
//   C = [M2; M1] K       F = [M2; M1]^T [K; Q] (rows 0-63)
// A, B, C and F are as wide as a state has rows; C takes W's and QK's columns,
// so the four fill the SM's tensor memory.  Thread = one row, half the columns
// (warp w: lanes 32 (w % 4) .., half w / 4).
template <IO kIO, int KP>
struct GradSmem {
  using D = DeltaTerms<kIO>;
  static constexpr int NT = D::kMid;
  static constexpr int kStages = kIO == IO::BF16 ? 2 : 1;  // of tiles, and of [K; Q]
  static constexpr int kKq = D::kIn * KP * 16384;
  static constexpr int kSTerm = KP * 64 * 64, kS = NT * kSTerm, kE = NT * kRowTile, kW = NT * 2 * kRowTile;
  // a stage: term by term S0 and, below it, E, so that one instruction has both for columns; dS1; then
  // term by term 64 rows of dV and 64 of dO
  static constexpr int kSE = kSTerm + kRowTile, oS0 = 0, oE = kSTerm, oDs = NT * kSE, oW = oDs + kS, kStage = oW + kW;
  static constexpr int kM = NT * 16384;  // [M2; M1], 128 rows of 64
  // M of its own, or (FP32, one stage) over the stage
  static constexpr bool kOwnM = kIO == IO::BF16;
  static constexpr int oKq = 0, oStage = kStages * kKq, oM = kOwnM ? oStage + kStages * kStage : oStage;
  // F's instructions read 8 KB past M's last image for rows that are not read back
  static constexpr int kBehindM = oM + kM + 8192, kBehindStage = oStage + kStages * kStage;
  static constexpr int oF = kBehindM > kBehindStage ? kBehindM : kBehindStage;  // floats below
  static constexpr int kFloats = 320 + 256 + 256 + 256 + 256 + 64 + 64;
  static constexpr int oBar = oF + kFloats * 4;
  static constexpr int kBytes = oBar + 128 + 1024;
};

// Lane l gets the sum over the warp's lanes of v[l]: 31 exchanges, fixed order.
__device__ __forceinline__ float lane_column_sum(float (&v)[32], int lane) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float give = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  return v[0];
}

// 8 elements of row `row` of the [K; Q] images, from column col: the sums of
// their terms.
template <int NQ, int KP>
__device__ __forceinline__ void kq_at(const uint8_t* images, int row, int col, float2 (&v)[4]) {
  const uint8_t* p = images + (col >> 6) * 16384 + image_chunk<128>(row, (col >> 3) & 7);
  unpack(*reinterpret_cast<const uint4*>(p + (NQ - 1) * KP * 16384), v);
#pragma unroll
  for (int i = NQ - 2; i >= 0; --i) {
    float2 w[4];
    unpack(*reinterpret_cast<const uint4*>(p + i * KP * 16384), w);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = add2(v[j], w[j]);
  }
}

// A warp's 32 rows, kMine columns from half * kMine on: lane = row.
template <typename T, int kMine>
__device__ __forceinline__ void write_rows(T* out, int64_t stride, int rows, int width, int half, int lane,
                                           const float2 (&x)[kMine / 2]) {
  constexpr int kPer = 64 / (int)sizeof(T);  // values of a 64-byte piece of a row
#pragma unroll
  for (int p = 0; p < kMine / kPer; ++p) {
    uint4 q[4];
#pragma unroll
    for (int u = 0; u < kPer / 16; ++u) {
      float2 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = x[p * (kPer / 2) + 8 * u + i];
      pack(v, q + u * 2, T());
    }
    const int col = half * kMine + p * kPer;
    store_rows(out + col, stride, rows, width - col, lane, q);
  }
}

template <IO kIO, int KP>
__global__ void __launch_bounds__(256, 1) delta_grad_kernel(DeltaArgs a) {
  using T = typename IoType<kIO>::type;
  using L = GradSmem<kIO, KP>;
  constexpr int NQ = DeltaTerms<kIO>::kIn, NT = DeltaTerms<kIO>::kMid, ST = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  float* sgate = reinterpret_cast<float*>(sm + L::oF);
  float* scol = sgate + 320;   // [quad][64]: column sums of W / beta, no diagonal
  float* sdots = scol + 256;   // [half][128]: rows of A times rows of [K; Q]
  float* skap = sdots + 256;   // [half][64]: rows of B times rows of K
  float* srow = skap + 256;    // [half][128]: row sums of W, no diagonal
  float* sdot = srow + 256;    // [warp]: parts of <dS1, S0>
  float* sdiag = sdot + 64;    // diagonal of W / beta
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::oBar);
  uint64_t* empty = full + ST;  // the products and the 8 warps have read a stage
  uint64_t* kq_full = empty + ST;
  uint64_t* done = kq_full + ST;
  uint64_t* drained = done + 1;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(drained + 1);
  int* stop = reinterpret_cast<int*>(tmem_at + 1);

  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, quad = warp & 3, half = warp >> 2;
  const int rep = a.Hv / a.Hk;
  const int tiles = delta_tiles(a.V);
  const int heads = a.partial ? 1 : rep, shares = rep / heads;  // value heads of an item, items of a key head
  const int64_t all = a.info[1] != a.key || a.info[0] < 0 ? 0 : (int64_t)a.info[0] * a.Hk * shares;
  if (blockIdx.x >= all) return;
  const int items = (int)((all - 1 - blockIdx.x) / gridDim.x) + 1, per_item = heads * tiles;
  Waiter wait{a, stop};

  if (t == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 9);
      mbar_init(&kq_full[i], 1);
    }
    mbar_init(done, 1);
    mbar_init(drained, 1);
    *stop = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc<512>(tmem_at);
  // dO has fewer terms than dV: the rows beside dV's later terms are zero
  if constexpr (NQ < NT) {
    for (int i = t; i < ST * (NT - NQ) * (kRowTile / 16); i += 256) {
      const int st = i / ((NT - NQ) * (kRowTile / 16)), k = i % ((NT - NQ) * (kRowTile / 16));
      const int term = NQ + k / (kRowTile / 16);
      *reinterpret_cast<uint4*>(sm + L::oStage + st * L::kStage + L::oW + (2 * term + 1) * kRowTile +
                                k % (kRowTile / 16) * 16) = make_uint4(0, 0, 0, 0);
    }
  }
  fence_async_smem();
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tm = *tmem_at;

  auto item_of = [&](int k) { return (int64_t)blockIdx.x + (int64_t)k * gridDim.x; };  // (chunk * Hk + key head) * shares + share
  // tile i of this CTA's (item, head, tile) triples; an item's run on in every array
  auto load = [&](int64_t i) {
    const int st = (int)(i % ST);
    uint8_t* to = sm + L::oStage + st * L::kStage;
    const size_t at = item_of((int)(i / per_item)) * per_item + i % per_item;
    mbar_arrive_expect_tx(&full[st], 2 * L::kS + L::kE + (NT + NQ) * kRowTile);
    bulk_load_1d(to + L::oDs, a.ds + at * L::kS, L::kS, &full[st]);
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      bulk_load_1d(to + L::oS0 + k * L::kSE, a.s0 + (at * NT + k) * L::kSTerm, L::kSTerm, &full[st]);
      bulk_load_1d(to + L::oE + k * L::kSE, a.e + (at * NT + k) * kRowTile, kRowTile, &full[st]);
      bulk_load_1d(to + L::oW + 2 * k * kRowTile, a.dvi + (at * NT + k) * kRowTile, kRowTile, &full[st]);
      if (k < NQ)
        bulk_load_1d(to + L::oW + (2 * k + 1) * kRowTile, a.doi + (at * NQ + k) * kRowTile, kRowTile, &full[st]);
    }
  };
  int64_t asked = 0, kq_asked = 0;  // tiles and [K; Q] that the copier has asked for, from the first on
  // one thread: once tile i's stage has been read, fill it for tile i + ST
  auto refill = [&](int64_t i) {
    if (i + ST >= (int64_t)items * per_item) return;
    if (!wait(&empty[i % ST], (uint32_t)(i / ST) & 1)) return;
    load(i + ST);
    asked = i + ST + 1;
  };
  auto load_kq = [&](int k) {
    mbar_arrive_expect_tx(&kq_full[k % ST], L::kKq);
    bulk_load_1d(sm + L::oKq + k % ST * L::kKq, a.kq + item_of(k) / shares * (size_t)L::kKq, L::kKq, &kq_full[k % ST]);
  };
  const bool copier = t == 7 * 32;
  if (copier) {
    for (; kq_asked < ST && kq_asked < items; ++kq_asked) load_kq((int)kq_asked);
    for (; asked < ST && asked < items * per_item; ++asked) load(asked);
  }
  constexpr int kWide = KP * 64, kMine = kWide / 2, kSteps = kMine / 16;  // state rows, and a thread's share of them
  const int row = quad * 32 + lane, r = row & 63;
  const bool is_k = row < 64;
  const uint32_t tA = tm, tW = tm + kWide, tQK = tW + 64, tC = tW, tB = tm + 256, tF = tm + 384;
  const uint32_t lane_at = (uint32_t)(quad * 32) << 16;
  const uint32_t m_at = smem_u32(sm + L::oM);
  const bool leader = t == 3 * 32;  // issues the products; its warp takes no part in <dS1, S0>
  uint32_t done_phase = 0;

  bool fine = true;
  for (int k = 0; k < items; ++k) {
    const int kh = (int)(item_of(k) / shares % a.Hk), share = (int)(item_of(k) % shares);
    const int64_t c = item_of(k) / shares / a.Hk;
    const int4 chunk = a.table[c];
    const int64_t start = chunk.y;
    const int len = chunk.z;
    uint8_t* kq_image = sm + L::oKq + k % ST * L::kKq;
    const uint32_t kq = smem_u32(kq_image);
    wait(&kq_full[k % ST], (uint32_t)(k / ST) & 1, k == 0 && leader && forced_here(a));

    float2 sum[kMine / 2];  // of dk (rows 0-63) or dq
#pragma unroll
    for (int i = 0; i < kMine / 2; ++i) sum[i] = splat2(0.0f);

    for (int hh = 0; hh < heads; ++hh) {
      const int h = kh * rep + share + hh;
      float2 acc[kMine / 2];  // this head's part
      const float* gates = a.gates + (c * a.Hv + h) * kDeltaGates;
      const float gate0 = gates[t], gate1 = t < 64 ? gates[256 + t] : 0.0f;  // on their way through the tiles
      float dot = 0.0f;
      if (leader && wait.ok) {
        tmem_fence_after_sync();
        const Operand<128, kKMajor, NQ, KP * 16384, 16384> KQ(kq);
        umma_terms<64, KP * 4, NQ>(tQK, KQ, KQ, false);
      }
      for (int p = 0; p < tiles; ++p) {
        const int64_t i = (int64_t)k * per_item + hh * tiles + p;
        const int st = (int)(i % ST);
        uint8_t* stage = sm + L::oStage + st * L::kStage;
        wait(&full[st], (uint32_t)(i / ST) & 1);
        if (warp == 3) {
          if (leader && wait.ok) {
            const uint32_t at = smem_u32(stage);
            const Operand<64, kKMajor, NT, L::kSE> SE(at + L::oS0), E(at + L::oE);
            const Operand<64, kKMajor, NT, L::kSTerm> dS(at + L::oDs);
            const Operand<64, kKMajor, NT, 2 * kRowTile> dW(at + L::oW);
            umma_terms<kWide + 64, 2, NT>(tA, dW, SE, p > 0);
            umma_terms<kWide, 2, NT>(tB, E, dS, p > 0);
            umma_commit(&empty[st]);
            if (p + 1 == tiles) umma_commit(done);
          }
          __syncwarp();
        } else {
          // <dS1, S0> over the tile: both images are permuted alike
          for (int q = t - (warp > 3 ? 32 : 0); q < L::kSTerm / 16; q += 224) {
            float2 x[4], y[4], w[4];
            unpack(*reinterpret_cast<const uint4*>(stage + L::oS0 + (NT - 1) * L::kSE + q * 16), x);
            unpack(*reinterpret_cast<const uint4*>(stage + L::oDs + (NT - 1) * L::kSTerm + q * 16), y);
#pragma unroll
            for (int m = NT - 2; m >= 0; --m) {
              unpack(*reinterpret_cast<const uint4*>(stage + L::oS0 + m * L::kSE + q * 16), w);
#pragma unroll
              for (int j = 0; j < 4; ++j) x[j] = add2(x[j], w[j]);
              unpack(*reinterpret_cast<const uint4*>(stage + L::oDs + m * L::kSTerm + q * 16), w);
#pragma unroll
              for (int j = 0; j < 4; ++j) y[j] = add2(y[j], w[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) dot = fmaf(x[j].x, y[j].x, fmaf(x[j].y, y[j].y, dot));
          }
          __syncwarp();
        }
        if (lane == 0 && wait.ok) mbar_arrive(&empty[st]);
        if (copier && (L::kOwnM || p + 1 < tiles)) refill(i);
      }
      wait(done, done_phase);
      done_phase ^= 1;
      tmem_fence_after_sync();
      named_barrier(1, 256);  // every warp is through with the last tile, and with the last head's sums
      sgate[t] = gate0;
      if (t < 64) sgate[256 + t] = gate1;
      named_barrier(1, 256);

      // M1 and M2, and what their elements add to dg and dbeta
      {
        float rows = 0.0f, cols[32];
        if (half && (quad & 1) == 0) {  // rows 0-31 end before column 32
#pragma unroll
          for (int k = 0; k < 4 * NT; ++k)
            *reinterpret_cast<uint4*>(sm + L::oM + k / 4 * 16384 + image_chunk<128>(row, 4 + k % 4)) = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 32; ++i) cols[i] = 0.0f;
        } else {
          const float gi = sgate[192 + r], gl = sgate[256 + r], sign = is_k ? -1.0f : a.scale;
          const int end = is_k ? r : r + 1;  // columns j < end
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float m[16], qk[16];
            tmem_row(tW + lane_at + half * 32 + u * 16, m);
            tmem_row(tQK + lane_at + half * 32 + u * 16, qk);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int j0 = half * 32 + u * 16 + 4 * q;
              const float4 gh = *reinterpret_cast<const float4*>(sgate + 192 + j0);
              const float4 gw = *reinterpret_cast<const float4*>(sgate + 256 + j0);
              const float4 bt = *reinterpret_cast<const float4*>(sgate + 128 + j0);
              const float g4[4] = {gh.x, gh.y, gh.z, gh.w}, l4[4] = {gw.x, gw.y, gw.z, gw.w}, b4[4] = {bt.x, bt.y, bt.z, bt.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int k = 4 * q + i, j = j0 + i;
                const float d = ex2((gi - g4[i]) + (gl - l4[i])) * sign;
                const float w = j < end ? d * m[k] : 0.0f;
                const float x = j < end ? w * qk[k] : 0.0f;
                m[k] = w * b4[i];
                if (j == r && !is_k) sdiag[r] = x;
                cols[u * 16 + k] = j == r ? 0.0f : x;
                rows = fmaf(cols[u * 16 + k], b4[i], rows);
              }
            }
            float2 mp[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) mp[i] = make_float2(m[2 * i], m[2 * i + 1]);
            put_row<NT, 128>(sm + L::oM, 16384, row, half * 4 + 2 * u, mp);
          }
        }
        srow[half * 128 + row] = rows;
        scol[quad * 64 + half * 32 + lane] = lane_column_sum(cols, lane);
      }
      fence_async_smem();
      tmem_fence_before_sync();
      named_barrier(1, 256);
      if (leader && wait.ok) {
        tmem_fence_after_sync();
        const Operand<128, kMnMajor, NQ, KP * 16384, 0, 16384> KQ(kq);
        const Operand<128, kKMajor, NT, 16384> M(m_at);
        const Operand<128, kMnMajor, NT, 16384, 0, 8192> Mt(m_at);
        umma_terms<kWide, 4, NT>(tC, M, KQ, false);   // the rows of K
        umma_terms<kWide, 8, NT>(tF, Mt, KQ, false);
        umma_commit(done);
      }
      // while that runs: the parts of dq and dk from the states
      {
        const float f = is_k ? -sgate[r] : a.scale * sgate[r], db = sgate[64 + r];
        float2 da = splat2(0.0f), dk = splat2(0.0f);
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          const int col = half * kMine + 16 * u;
          float2 x[8], k0[4], k1[4];
          tmem_sum<1>(tA + lane_at + col, 0, x);
          kq_at<NQ, KP>(kq_image, row, col, k0);
          kq_at<NQ, KP>(kq_image, row, col + 8, k1);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            da = fma2(x[i], i < 4 ? k0[i & 3] : k1[i & 3], da);
            acc[8 * u + i] = mul2(splat2(f), x[i]);
          }
          if (is_k) {
            tmem_sum<1>(tB + lane_at + col, 0, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              dk = fma2(x[i], i < 4 ? k0[i & 3] : k1[i & 3], dk);
              acc[8 * u + i] = fma2(splat2(db), x[i], acc[8 * u + i]);
            }
          }
        }
        sdots[half * 128 + row] = f * (da.x + da.y);
        if (is_k) skap[half * 64 + row] = dk.x + dk.y;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0) sdot[warp] = dot;
      }
      wait(done, done_phase);
      done_phase ^= 1;
      tmem_fence_after_sync();
      if (copier && !L::kOwnM) refill((int64_t)k * per_item + (hh + 1) * tiles - 1);  // M lay in the stage
      __syncwarp();
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        const int col = half * kMine + 16 * u;
        float2 x[8];
        tmem_sum<1>(tC + lane_at + col, 0, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[8 * u + i] = add2(acc[8 * u + i], x[i]);
        if (is_k) {
          tmem_sum<1>(tF + lane_at + col, 0, x);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[8 * u + i] = add2(acc[8 * u + i], x[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[8 * u + i] = add2(sum[8 * u + i], acc[8 * u + i]);
      }
      tmem_fence_before_sync();
      fine = vote(1, 256, wait.ok);  // the sums are in; the next head's products may begin
      if (!fine) break;
      if (warp == 0) {
        // tokens 2 lane and 2 lane + 1
        float dg[2], end = 0.0f;
        const float g_last = sgate[192 + 63], l_last = sgate[256 + 63];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int j = 2 * lane + i;
          const float kap = skap[j] + skap[64 + j];
          const float tau = (sdots[j] + sdots[128 + j]) + (sdots[64 + j] + sdots[192 + j]);
          const float col = (scol[j] + scol[64 + j]) + (scol[128 + j] + scol[192 + j]);
          const float rows = (srow[j] + srow[128 + j]) + (srow[64 + j] + srow[192 + j]);
          const float dec = ex2((g_last - sgate[192 + j]) + (l_last - sgate[256 + j]));
          const float beta = sgate[128 + j];
          const float db = fmaf(dec, kap, col);
          end = fmaf(sgate[64 + j], kap, end);
          dg[i] = tau + (rows - beta * db);
          if (j < len) a.dbeta[(start + j) * a.Hv + h] = db + sdiag[j];
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) end += __shfl_xor_sync(0xffffffffu, end, o);
        float d = 0.0f;
        for (int w = 0; w < 8; ++w) d += sdot[w];
        end = fmaf(sgate[63], d, end);
        float suffix = dg[0] + dg[1];
        const float own = suffix;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float v = __shfl_down_sync(0xffffffffu, suffix, o);
          if (lane + o < 32) suffix += v;
        }
        float next = __shfl_down_sync(0xffffffffu, suffix, 1);
        if (lane == 31) next = 0.0f;
        const int j = 2 * lane;
        if (j < len) a.dg[(start + j) * a.Hv + h] = end + (next + own);
        if (j + 1 < len) a.dg[(start + j + 1) * a.Hv + h] = end + (next + dg[1]);
      }
    }

    if (!fine) break;
    const int first = (quad & 1) * 32;
    if (a.partial) {
      float* out = a.partial + ((item_of(k) * 2 + !is_k) * 64 + first) * a.K;
      write_rows<float, kMine>(out, a.K, len - first, a.K, half, lane, sum);
    } else {
      T* out = static_cast<T*>(is_k ? a.dk : a.dq) + ((start + first) * a.Hk + kh) * a.K;
      write_rows<T, kMine>(out, (int64_t)a.Hk * a.K, len - first, a.K, half, lane, sum);
    }
    if (copier && k + ST < items) {
      load_kq(k + ST);
      kq_asked = k + ST + 1;
    }  // behind the last barrier nothing reads this item's
  }
  tmem_fence_before_sync();
  if (!__syncthreads_and(wait.ok)) {
    // nobody asks for anything any more: what is on its way comes in before the memory is given back
    if (leader) umma_commit(drained);
    if (copier) {
      for (int i = 0; i < ST; ++i) {
        drain_copies(&full[i], (asked - i + ST - 1) / ST);
        drain_copies(&kq_full[i], (kq_asked - i + ST - 1) / ST);
      }
      mbar_wait(drained, 0, kCopyDrainNs);
    }
    __syncthreads();
  }
  if (warp == 0) tmem_dealloc<512>(tm);
}

// The value heads' parts of dk or dq of a chunk and key head, added in order:
// 16 rows a CTA.
template <typename T>
__global__ void __launch_bounds__(256) delta_grad_sum_kernel(DeltaArgs a) {
  if (a.info[1] != a.key || (int64_t)blockIdx.x >= (int64_t)a.info[0] * a.Hk) return;
  const int rep = a.Hv / a.Hk, kh = blockIdx.x % a.Hk, wide = a.K / 4;
  const int4 chunk = a.table[blockIdx.x / a.Hk];
  const float* part = a.partial + ((int64_t)blockIdx.x * rep * 2 + blockIdx.y / 4) * 64 * a.K;
  T* out = static_cast<T*>(blockIdx.y / 4 ? a.dq : a.dk) + ((int64_t)chunk.y * a.Hk + kh) * a.K;
  const int r0 = blockIdx.y % 4 * 16, rows = min(16, chunk.z - r0);
  for (int i = threadIdx.x; i < rows * wide; i += 256) {
    const int r = r0 + i / wide, c = i % wide * 4;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int h = 0; h < rep; ++h) {
      const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)h * 128 * a.K + r * a.K + c);
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    st_io2(out + (int64_t)r * a.Hk * a.K + c, make_float2(s.x, s.y));
    st_io2(out + (int64_t)r * a.Hk * a.K + c + 2, make_float2(s.z, s.w));
  }
}

template <IO kIO, int KP>
cudaError_t run_grads(const DeltaArgs& a, cudaStream_t st) {
  constexpr size_t bytes = GradSmem<kIO, KP>::kBytes;
  static_assert(bytes <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> done{0};
  cudaError_t e = set_smem(reinterpret_cast<const void*>(delta_grad_kernel<kIO, KP>), bytes, done);
  if (e != cudaSuccess) return e;
  const int64_t items = a.max_chunks * (a.partial ? a.Hv : a.Hk);
  delta_grad_kernel<kIO, KP><<<(unsigned)(items < 152 ? items : 152), 256, bytes, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.partial) return e;
  delta_grad_sum_kernel<typename IoType<kIO>::type><<<dim3((unsigned)(a.max_chunks * a.Hk), 8), 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_grads(const DeltaArgs& a, IO io, cudaStream_t st) {
  if (a.max_chunks == 0) return cudaSuccess;
  const bool two = delta_panels_k(a.K) == 2;
  if (io == IO::BF16) return two ? run_grads<IO::BF16, 2>(a, st) : run_grads<IO::BF16, 1>(a, st);
  return two ? run_grads<IO::F32, 2>(a, st) : run_grads<IO::F32, 1>(a, st);
}

}  // namespace vssm
