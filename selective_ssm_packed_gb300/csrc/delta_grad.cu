// delta_grad.cu -- the gated delta rule's gradients that need no walk: dq,
// dk, dg and dbeta of a chunk from the states and state gradients around it.
#include "delta.cuh"

namespace vssm {
namespace {

// One CTA of 256 threads per chunk and key head; the value heads that share
// the key head follow each other, and dq and dk are summed over them in
// registers and tensor memory, in that order.  Products over the state's
// columns (panel by panel) and over the chunk's tokens; dq and dk appear
// transposed, state row by token, so that every product fills the matrix
// unit's 128 rows:
//   A1 = S0 dV^T   A2 = dS1 E^T   A3 = S0 dO^T   (rows: state rows)
//   Wa = dV E^T (rows 0-63)       Wb = dO E^T (rows 64-127)
//   QK = [K; Q] K^T
//   CK = K^T M2^T + K^T M2 + Q^T M1               CQ = K^T M1^T
// All eight are 64 columns wide: the SM's whole tensor memory.
template <IO kIO, int KP>
struct GradSmem {
  using D = DeltaTerms<kIO>;
  static constexpr int kRow = D::kCols * 2;
  static constexpr int kKq = D::kIn * KP * 16384;
  static constexpr int kSTerm = KP * 64 * kRow, kRTerm = 64 * kRow;
  static constexpr int kS = D::kMid * kSTerm, kR = D::kMid * kRTerm, kM = D::kMid * 8192;
  // S0 and dS1, later M2 and M1
  static constexpr int kShared = 2 * kS > 2 * kM ? 2 * kS : 2 * kM;
  static constexpr int oKq = 0, oS0 = kKq, oDs = oS0 + kS, oM2 = oS0, oM1 = oS0 + kM;
  static constexpr int oE = oS0 + kShared, oDv = oE + kR, oDo = oDv + kR;
  static constexpr int oF = oDo + D::kIn * kRTerm;  // floats below
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
  constexpr int NQ = DeltaTerms<kIO>::kIn, NT = DeltaTerms<kIO>::kMid, BV = DeltaTerms<kIO>::kCols;
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
  uint64_t* done = full + 1;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(done + 1);

  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, quad = warp & 3, half = warp >> 2;
  const int row = quad * 32 + lane, r = row & 63;
  const bool is_k = row < 64;
  const int kh = blockIdx.x % a.Hk;
  const int64_t c = blockIdx.x / a.Hk;
  if (c >= a.info[0]) return;
  const int4 chunk = a.table[c];
  const int64_t start = chunk.y;
  const int len = chunk.z;
  const int rep = a.Hv / a.Hk;
  const int panels = (a.V + BV - 1) / BV;

  if (t == 0) {
    mbar_init(full, 1);
    mbar_init(done, 1);
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc<512>(tmem_at);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tm = *tmem_at;
  const uint32_t tA1 = tm, tA2 = tm + 64, tA3 = tm + 128, tWa = tm + 192, tWb = tm + 256, tQK = tm + 320, tCK = tm + 384,
                 tCQ = tm + 448;
  const uint32_t mine = ((uint32_t)(quad * 32) << 16) + half * 32;
  const uint32_t kq = smem_u32(sm + L::oKq);
  Waiter wait{a.wait_ns, a.status};
  uint32_t full_phase = 0, done_phase = 0;

  float acc_k[32], acc_q[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) acc_k[i] = acc_q[i] = 0.0f;

  for (int hh = 0; hh < rep; ++hh) {
    const int h = kh * rep + hh;
    const int64_t ch = c * a.Hv + h;
    float dot = 0.0f;
    for (int i = t; i < 320; i += 256) sgate[i] = a.gates[ch * kDeltaGates + i];
    for (int p = 0; p < panels; ++p) {
      if (t == 0) {
        const bool first = hh == 0 && p == 0;
        mbar_arrive_expect_tx(full, (first ? L::kKq : 0) + 2 * L::kS + 2 * L::kR);
        if (first) bulk_load_1d(sm + L::oKq, a.kq + (size_t)(c * a.Hk + kh) * L::kKq, L::kKq, full);
        const size_t at = ch * panels + p;
        bulk_load_1d(sm + L::oS0, a.s0 + at * L::kS, L::kS, full);
        bulk_load_1d(sm + L::oDs, a.ds + at * L::kS, L::kS, full);
        bulk_load_1d(sm + L::oE, a.e + at * L::kR, L::kR, full);
        bulk_load_1d(sm + L::oDv, a.dvi + at * L::kR, L::kR, full);
      }
      {  // dO: a quarter of a token's columns for each thread
        const int tr = t >> 2, q = t & 3, col = p * BV + q * (BV / 4);
        const T* src = static_cast<const T*>(a.dout) + ((start + tr) * a.Hv + h) * a.V + col;
#pragma unroll
        for (int i = 0; i < BV / 32; ++i) {
          float w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
          if (tr < len && col + 8 * i < a.V) ld_io8(src + 8 * i, w);
          put_chunk<NQ, L::kRow>(sm + L::oDo, L::kRTerm, tr, q * (BV / 32) + i, w);
        }
      }
      fence_async_smem();
      __syncthreads();
      wait(full, full_phase);
      full_phase ^= 1;
      if (t == 0) {
        tmem_fence_after_sync();
        constexpr int kSteps = BV / 16;
        using Rows = Operand<L::kRow, kKMajor, NT, L::kRTerm>;
        const Operand<L::kRow, kKMajor, NT, L::kSTerm> S0(smem_u32(sm + L::oS0)), dS(smem_u32(sm + L::oDs));
        const Rows E(smem_u32(sm + L::oE)), dV(smem_u32(sm + L::oDv));
        // the 64 rows before dO fill the instruction's first half and are not read back
        const Operand<L::kRow, kKMajor, NQ, L::kRTerm> dO(smem_u32(sm + L::oDo)), dO64(smem_u32(sm + L::oDo) - L::kRTerm);
        if (hh == 0 && p == 0) {
          const Operand<128, kKMajor, NQ, KP * 16384, 16384> KQ(kq);
          umma_terms<64, KP * 4, NQ>(tQK, KQ, KQ, false);
        }
        umma_terms<64, kSteps, NT>(tWa, dV, E, p > 0);
        umma_terms<64, kSteps, NT>(tWb, dO64, E, p > 0);
        umma_terms<64, kSteps, NT>(tA1, S0, dV, p > 0);
        umma_terms<64, kSteps, NT>(tA3, S0, dO, p > 0);
        umma_terms<64, kSteps, NT>(tA2, dS, E, p > 0);
        umma_commit(done);
      }
      // <dS1, S0> over the panel: both images are permuted alike
      for (int i = t; i < L::kSTerm / 16; i += 256) {
        float x[8], y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = y[j] = 0.0f;
#pragma unroll
        for (int k = NT - 1; k >= 0; --k) {
          float w[8];
          ld_io8(reinterpret_cast<const __nv_bfloat16*>(sm + L::oS0 + k * L::kSTerm + i * 16), w);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] += w[j];
          ld_io8(reinterpret_cast<const __nv_bfloat16*>(sm + L::oDs + k * L::kSTerm + i * 16), w);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] += w[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) dot = fmaf(x[j], y[j], dot);
      }
      wait(done, done_phase);
      done_phase ^= 1;
      tmem_fence_after_sync();
      fence_async_smem();  // the reads above, before the next copies overwrite what they read
      __syncthreads();
    }

    // M1 and M2, and what their elements add to dg and dbeta
    {
      float m[32], qk[32];
      tmem_row<32>((is_k ? tWa : tWb) + mine, m);
      tmem_row<32>(tQK + mine, qk);
      const float gi = sgate[192 + r], gl = sgate[256 + r];
      float rows = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const int j = half * 32 + i;
        const float d = exp_f((gi - sgate[192 + j]) + (gl - sgate[256 + j]));
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
      put_row<NT, 128>(sm + (is_k ? L::oM2 : L::oM1), 8192, r, half * 4, m);
      srow[half * 128 + row] = rows;
      scol[quad * 64 + half * 32 + lane] = lane_column_sum(qk, lane);
    }
    fence_async_smem();
    tmem_fence_before_sync();
    __syncthreads();
    if (t == 0) {
      tmem_fence_after_sync();
      const Operand<128, kMnMajor, NQ, KP * 16384, 0, 16384> K(kq), Q(kq + 64 * 128);
      const Operand<128, kKMajor, NT, 8192> M2t(smem_u32(sm + L::oM2)), M1t(smem_u32(sm + L::oM1));
      const Operand<128, kMnMajor, NT, 8192> M2(smem_u32(sm + L::oM2)), M1(smem_u32(sm + L::oM1));
      umma_terms<64, 4, NT>(tCK, K, M2t, hh > 0);
      umma_terms<64, 4, NT>(tCK, K, M2, true);
      umma_terms<64, 4, NT>(tCK, Q, M1, true);
      umma_terms<64, 4, NT>(tCQ, K, M1t, hh > 0);
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
        tmem_row<32>(tA2 + mine, x);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int j = half * 32 + i;
          acc_k[i] = fmaf(sgate[64 + j], x[i], acc_k[i]);
          kap[i] = x[i] * kq_at<NQ, KP>(sm + L::oKq, j, row);
        }
      }
      stau[quad * 64 + half * 32 + lane] = lane_column_sum(tau, lane);
      skap[quad * 64 + half * 32 + lane] = lane_column_sum(kap, lane);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if (lane == 0) sdot[warp] = dot;
    }
    __syncthreads();
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
        const float dec = exp_f((g_last - sgate[192 + j]) + (l_last - sgate[256 + j]));
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
    wait(done, done_phase);
    done_phase ^= 1;
    tmem_fence_after_sync();
    __syncthreads();
  }

  float ck[32], cq[32];
  tmem_row<32>(tCK + mine, ck);
  tmem_row<32>(tCQ + mine, cq);
  if (row < a.K) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int j = half * 32 + i;
      if (j < len) {
        const int64_t at = ((start + j) * a.Hk + kh) * a.K + row;
        static_cast<T*>(a.dk)[at] = from_f<T>(acc_k[i] + ck[i]);
        static_cast<T*>(a.dq)[at] = from_f<T>(acc_q[i] + cq[i]);
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
  cudaError_t e = set_smem(reinterpret_cast<const void*>(delta_grad_kernel<kIO, KP>), bytes);
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
