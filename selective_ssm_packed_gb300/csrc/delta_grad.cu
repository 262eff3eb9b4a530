// delta_grad.cu -- the gated delta rule's gradients that need no walk: dq,
// dk, dg and dbeta of a chunk from the states and state gradients around it.
#include "delta.cuh"

namespace vssm {
namespace {

// One CTA of 256 threads per chunk and key head; the value heads that share the key head follow each other, and dq and dk are summed
// over them in registers, in that order.  Products over the state's columns
// (tile by tile) and over the chunk's tokens; dq and dk appear transposed,
// state row by token, so that every product fills the matrix unit's 128 rows:
//   A1 = S0 dV^T   A2 = dS1 E^T   A3 = S0 dO^T   (rows: state rows)
//   W  = [dV; dO] E^T             QK = [K; Q] K^T
//   CK = K^T M2^T + K^T M2 + Q^T M1               CQ = K^T M1^T
// All are 64 columns wide: 448 of the SM's 512 columns of tensor memory.
// What the call reads (two states and three sets of rows per head) bounds it,
// so the next tiles are on their way through everything else.
template <IO kIO, int KP>
struct GradSmem {
  using D = DeltaTerms<kIO>;
  static constexpr int NT = D::kMid;
  static constexpr int kStages = kIO == IO::BF16 ? 2 : 1;
  static constexpr int kKq = D::kIn * KP * 16384;
  static constexpr int kSTerm = KP * 64 * 64, kS = NT * kSTerm, kE = NT * kRowTile, kW = NT * 2 * kRowTile;
  // a stage: S0, dS1, E, then term by term 64 rows of dV and 64 of dO
  static constexpr int oS0 = 0, oDs = kS, oE = 2 * kS, oW = oE + kE, kStage = oW + kW;
  static constexpr int kM = NT * 8192;
  // M2 and M1: of their own, or (FP32, one stage) over S0 and dS1
  static constexpr bool kOwnM = kIO == IO::BF16;
  static constexpr int oKq = 0, oStage = kKq, oM2 = kOwnM ? oStage + kStages * kStage : oStage, oM1 = oM2 + kM;
  static constexpr int kBehindM = oM1 + kM, kBehindStage = oStage + kStages * kStage;
  static constexpr int oF = kBehindM > kBehindStage ? kBehindM : kBehindStage;  // floats below
  static constexpr int kFloats = 320 + 256 + 256 + 256 + 256 + 64 + 64;
  static constexpr int oBar = oF + kFloats * 4;
  static constexpr int kBytes = oBar + 64 + 1024;
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

// Element (row, col) of the [K; Q] images: the sum of its terms.
template <int NQ, int KP>
__device__ __forceinline__ float kq_at(const uint8_t* images, int row, int col) {
  const uint8_t* p = images + (col >> 6) * 16384 + image_chunk<128>(row, (col >> 3) & 7) + (col & 7) * 2;
  float v = 0.0f;
#pragma unroll
  for (int i = NQ - 1; i >= 0; --i) v += __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p + i * KP * 16384));
  return v;
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
  float* skap = scol + 256;    // [quad][64]
  float* stau = skap + 256;    // [quad][64]
  float* srow = stau + 256;    // [half][128]: row sums of W, no diagonal
  float* sdot = srow + 256;    // [warp]: parts of <dS1, S0>
  float* sdiag = sdot + 64;    // diagonal of W / beta
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::oBar);
  uint64_t* empty = full + ST;  // the products and the 8 warps have read a stage
  uint64_t* kq_full = empty + ST;
  uint64_t* done = kq_full + 1;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(done + 1);

  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, quad = warp & 3, half = warp >> 2;
  const int kh = blockIdx.x % a.Hk;
  const int64_t c = blockIdx.x / a.Hk;
  if (c >= a.info[0]) return;
  const int4 chunk = a.table[c];
  const int64_t start = chunk.y;
  const int len = chunk.z;
  const int rep = a.Hv / a.Hk;
  const int tiles = delta_tiles(a.V);
  Waiter wait{a.wait_ns, a.status};

  if (t == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 9);
    }
    mbar_init(kq_full, 1);
    mbar_init(done, 1);
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

  // tile i of the (head, tile) pairs, which run on in every array
  auto load = [&](int i) {
    const int st = i % ST;
    uint8_t* to = sm + L::oStage + st * L::kStage;
    const size_t at = (c * a.Hv + kh * rep) * tiles + i;
    mbar_arrive_expect_tx(&full[st], 2 * L::kS + L::kE + (NT + NQ) * kRowTile);
    bulk_load_1d(to + L::oS0, a.s0 + at * L::kS, L::kS, &full[st]);
    bulk_load_1d(to + L::oDs, a.ds + at * L::kS, L::kS, &full[st]);
    bulk_load_1d(to + L::oE, a.e + at * L::kE, L::kE, &full[st]);
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      bulk_load_1d(to + L::oW + 2 * k * kRowTile, a.dvi + (at * NT + k) * kRowTile, kRowTile, &full[st]);
      if (k < NQ)
        bulk_load_1d(to + L::oW + (2 * k + 1) * kRowTile, a.doi + (at * NQ + k) * kRowTile, kRowTile, &full[st]);
    }
  };
  // one thread: once tile i's stage has been read, fill it for tile i + ST
  auto refill = [&](int i) {
    if (i + ST >= rep * tiles) return;
    wait(&empty[i % ST], (i / ST) & 1);
    load(i + ST);
  };
  const bool copier = t == 7 * 32;
  if (copier) {
    mbar_arrive_expect_tx(kq_full, L::kKq);
    bulk_load_1d(sm + L::oKq, a.kq + (size_t)(c * a.Hk + kh) * L::kKq, L::kKq, kq_full);
    for (int i = 0; i < ST && i < rep * tiles; ++i) load(i);
  }
  {
    const int row = quad * 32 + lane, r = row & 63;
    const bool is_k = row < 64;
    const uint32_t tA1 = tm, tA2 = tm + 64, tA3 = tm + 128, tW = tm + 192, tQK = tm + 256, tCK = tm + 320, tCQ = tm + 384;
    const uint32_t mine = ((uint32_t)(quad * 32) << 16) + half * 32;
    const uint32_t kq = smem_u32(sm + L::oKq);
    uint32_t done_phase = 0;

    float acc_k[32], acc_q[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) acc_k[i] = acc_q[i] = 0.0f;

    for (int hh = 0; hh < rep; ++hh) {
      const int h = kh * rep + hh;
      const int64_t ch = c * a.Hv + h;
      float dot = 0.0f;
      for (int i = t; i < 320; i += 256) sgate[i] = a.gates[ch * kDeltaGates + i];
      if (t == 0 && hh == 0) {
        wait(kq_full, 0);
        tmem_fence_after_sync();
        const Operand<128, kKMajor, NQ, KP * 16384, 16384> KQ(kq);
        umma_terms<64, KP * 4, NQ>(tQK, KQ, KQ, false);
      }
      for (int p = 0; p < tiles; ++p) {
        const int i = hh * tiles + p, st = i % ST;
        uint8_t* stage = sm + L::oStage + st * L::kStage;
        wait(&full[st], (i / ST) & 1);
        if (t == 0) {
          tmem_fence_after_sync();
          const uint32_t at = smem_u32(stage);
          const Operand<64, kKMajor, NT, L::kSTerm> S0(at + L::oS0), dS(at + L::oDs);
          const Operand<64, kKMajor, NT, kRowTile> E(at + L::oE);
          const Operand<64, kKMajor, NT, 2 * kRowTile> dW(at + L::oW);
          const Operand<64, kKMajor, NQ, 2 * kRowTile> dO(at + L::oW + kRowTile);
          umma_terms<64, 2, NT>(tW, dW, E, p > 0);
          umma_terms<64, 2, NT>(tA1, S0, dW, p > 0);
          umma_terms<64, 2, NT>(tA3, S0, dO, p > 0);
          umma_terms<64, 2, NT>(tA2, dS, E, p > 0);
          umma_commit(&empty[st]);
          if (p + 1 == tiles) umma_commit(done);
        }
        // <dS1, S0> over the tile: both images are permuted alike
        for (int k = t; k < L::kSTerm / 16; k += 256) {
          float x[8], y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = y[j] = 0.0f;
#pragma unroll
          for (int m = NT - 1; m >= 0; --m) {
            float w[8];
            ld_io8(reinterpret_cast<const __nv_bfloat16*>(stage + L::oS0 + m * L::kSTerm + k * 16), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] += w[j];
            ld_io8(reinterpret_cast<const __nv_bfloat16*>(stage + L::oDs + m * L::kSTerm + k * 16), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] += w[j];
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) dot = fmaf(x[j], y[j], dot);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        if (copier && (L::kOwnM || p + 1 < tiles)) refill(i);
      }
      wait(done, done_phase);
      done_phase ^= 1;
      tmem_fence_after_sync();
      named_barrier(1, 256);  // the gates are in; every warp is through with the last tile

      // M1 and M2, and what their elements add to dg and dbeta
      {
        float m[32], qk[32];
        tmem_row<32>(tW + mine, m);
        tmem_row<32>(tQK + mine, qk);
        const float gi = sgate[192 + r], gl = sgate[256 + r];
        float rows = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int j = half * 32 + i;
          const float d = ex2((gi - sgate[192 + j]) + (gl - sgate[256 + j]));
          const bool in = is_k ? j < r : j <= r;
          const float w = in ? (is_k ? -d : a.scale * d) * m[i] : 0.0f;
          const float b = sgate[128 + j];
          m[i] = w * b;
          qk[i] = in ? w * qk[i] : 0.0f;
          if (j == r) {
            if (!is_k) sdiag[r] = qk[i];
            qk[i] = 0.0f;
          }
          rows = fmaf(qk[i], b, rows);
        }
        float2 mp[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) mp[i] = make_float2(m[2 * i], m[2 * i + 1]);
        put_row<NT, 128>(sm + (is_k ? L::oM2 : L::oM1), 8192, r, half * 4, mp);
        srow[half * 128 + row] = rows;
        scol[quad * 64 + half * 32 + lane] = lane_column_sum(qk, lane);
      }
      fence_async_smem();
      tmem_fence_before_sync();
      named_barrier(1, 256);
      if (t == 0) {
        tmem_fence_after_sync();
        const Operand<128, kMnMajor, NQ, KP * 16384, 0, 16384> K(kq), Q(kq + 64 * 128);
        const Operand<128, kKMajor, NT, 8192> M2t(smem_u32(sm + L::oM2)), M1t(smem_u32(sm + L::oM1));
        const Operand<128, kMnMajor, NT, 8192> M2(smem_u32(sm + L::oM2)), M1(smem_u32(sm + L::oM1));
        umma_terms<64, 4, NT>(tCK, K, M2t, false);
        umma_terms<64, 4, NT>(tCK, K, M2, true);
        umma_terms<64, 4, NT>(tCK, Q, M1, true);
        umma_terms<64, 4, NT>(tCQ, K, M1t, false);
        umma_commit(done);
      }
      // while that runs: the parts of dq and dk from the states
      {
        float kap[32], tau[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) kap[i] = tau[i] = 0.0f;
        if (row < KP * 64) {
          float x[32];
          tmem_row<32>(tA1 + mine, x);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int j = half * 32 + i;
            const float w = -sgate[j] * x[i];
            acc_k[i] += w;
            tau[i] = w * kq_at<NQ, KP>(sm + L::oKq, j, row);
          }
          tmem_row<32>(tA3 + mine, x);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int j = half * 32 + i;
            const float w = a.scale * sgate[j] * x[i];
            acc_q[i] += w;
            tau[i] = fmaf(w, kq_at<NQ, KP>(sm + L::oKq, 64 + j, row), tau[i]);
          }
        }
        stau[quad * 64 + half * 32 + lane] = lane_column_sum(tau, lane);
        if (row < KP * 64) {
          float x[32];
          tmem_row<32>(tA2 + mine, x);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int j = half * 32 + i;
            acc_k[i] = fmaf(sgate[64 + j], x[i], acc_k[i]);
            kap[i] = x[i] * kq_at<NQ, KP>(sm + L::oKq, j, row);
          }
        }
        skap[quad * 64 + half * 32 + lane] = lane_column_sum(kap, lane);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0) sdot[warp] = dot;
      }
      wait(done, done_phase);
      done_phase ^= 1;
      tmem_fence_after_sync();
      if (copier && !L::kOwnM) refill((hh + 1) * tiles - 1);  // M lay in the stage
      {
        float x[32];
        tmem_row<32>(tCK + mine, x);
#pragma unroll
        for (int i = 0; i < 32; ++i) acc_k[i] += x[i];
        tmem_row<32>(tCQ + mine, x);
#pragma unroll
        for (int i = 0; i < 32; ++i) acc_q[i] += x[i];
      }
      tmem_fence_before_sync();
      named_barrier(1, 256);
      if (warp == 0) {
        // tokens 2 lane and 2 lane + 1
        float dg[2], end = 0.0f;
        const float g_last = sgate[192 + 63], l_last = sgate[256 + 63];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int j = 2 * lane + i;
          const float kap = (skap[j] + skap[64 + j]) + (skap[128 + j] + skap[192 + j]);
          const float tau = (stau[j] + stau[64 + j]) + (stau[128 + j] + stau[192 + j]);
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
      if (hh + 1 < rep) named_barrier(1, 256);  // before the next head's gates and sums
    }

    if (row < a.K) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const int j = half * 32 + i;
        if (j < len) {
          const int64_t at = ((start + j) * a.Hk + kh) * a.K + row;
          static_cast<T*>(a.dk)[at] = from_f<T>(acc_k[i]);
          static_cast<T*>(a.dq)[at] = from_f<T>(acc_q[i]);
        }
      }
    }
  }
  tmem_fence_before_sync();
  __syncthreads();
  if (warp == 0) tmem_dealloc<512>(tm);
}

template <IO kIO, int KP>
cudaError_t run_grads(const DeltaArgs& a, cudaStream_t st) {
  constexpr size_t bytes = GradSmem<kIO, KP>::kBytes;
  static_assert(bytes <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> done{0};
  cudaError_t e = set_smem(reinterpret_cast<const void*>(delta_grad_kernel<kIO, KP>), bytes, done);
  if (e != cudaSuccess) return e;
  delta_grad_kernel<kIO, KP><<<(unsigned)(a.max_chunks * a.Hk), 256, bytes, st>>>(a);
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
