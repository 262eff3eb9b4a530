// delta_bwd.cu -- the gated delta rule's walk back over the chunks of a
// sequence: the gradient of the state, and dV.
#include "delta.cuh"

namespace vssm {
namespace {

// One CTA of 256 threads per (sequence, value head, panel of kCols state
// columns), as the forward walk: dS in registers (FP32) and as bf16 terms in
// shared memory.  A chunk is
//   D1 = [K; Q] dS1                     rows 0-63, times dec beta, become Z
//   D2 = X^T [Z; dO] = dV               (64 rows; 64 to 127 are not used)
//   D3 = [K; Q]^T [-exp(G) dV; scale exp(G) dO] and dS0 = exp(G_63) dS1 + D3
// Threads of rows 64-127 bring dO in: as it is for D2, and scaled, as the
// lower half of D3's operand, whose upper half first holds Z.  dS1 of every
// chunk and dV leave as images for the gradients that need no walk.
template <IO kIO, int KP>
struct BwdSmem {
  using D = DeltaTerms<kIO>;
  static constexpr int kRow = D::kCols * 2;
  static constexpr int kKq = D::kIn * KP * 16384, kX = D::kMid * 16384;
  static constexpr int kSTerm = KP * 64 * kRow, kRTerm = 64 * kRow, kZTerm = 128 * kRow;
  static constexpr int oKq = 0, oX = oKq + D::kStages * kKq, oS = oX + D::kStages * kX;
  static constexpr int oZ = oS + D::kMid * kSTerm, oDo = oZ + D::kMid * kZTerm;
  static constexpr int oBar = oDo + D::kIn * kRTerm;
  static constexpr int kBytes = oBar + 128 + 1024;
};

template <IO kIO, int KP>
__global__ void __launch_bounds__(256, 1) delta_bwd_kernel(DeltaArgs a) {
  using T = typename IoType<kIO>::type;
  using L = BwdSmem<kIO, KP>;
  constexpr int NQ = DeltaTerms<kIO>::kIn, NT = DeltaTerms<kIO>::kMid, BV = DeltaTerms<kIO>::kCols,
                ST = DeltaTerms<kIO>::kStages, HC = BV / 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  uint64_t* kq_full = reinterpret_cast<uint64_t*>(sm + L::oBar);
  uint64_t* x_full = kq_full + ST;
  uint64_t* done = x_full + ST;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(done + 1);

  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, quad = warp & 3, half = warp >> 2;
  const int row = quad * 32 + lane;
  const int panels = (a.V + BV - 1) / BV;
  const int panel = blockIdx.x % panels;
  const int h = blockIdx.x / panels % a.Hv;
  const int s = blockIdx.x / panels / a.Hv;
  if (a.info[0] < 0) return;
  const int c0 = a.first[s], n = a.first[s + 1] - c0;
  const int col0 = panel * BV + half * HC;
  const int64_t state_at = (((int64_t)s * a.Hv + h) * a.K + row) * a.V + col0;
  const int kh = h / (a.Hv / a.Hk);

  float S[HC];
#pragma unroll
  for (int i = 0; i < HC; ++i) S[i] = 0.0f;
  if (a.d_final && row < a.K) {
#pragma unroll
    for (int i = 0; i < HC; i += 4)
      if (col0 + i < a.V) {
        const float4 f = *reinterpret_cast<const float4*>(a.d_final + state_at + i);
        S[i] = f.x; S[i + 1] = f.y; S[i + 2] = f.z; S[i + 3] = f.w;
      }
  }

  if (n > 0) {
    // i counts the chunks walked: chunk n - 1 - i
    auto load_kq = [&](int i) {
      const int st = i % ST;
      mbar_arrive_expect_tx(&kq_full[st], L::kKq);
      bulk_load_1d(sm + L::oKq + st * L::kKq, a.kq + ((size_t)(c0 + n - 1 - i) * a.Hk + kh) * L::kKq, L::kKq,
                   &kq_full[st]);
    };
    auto load_x = [&](int i) {
      const int st = i % ST;
      mbar_arrive_expect_tx(&x_full[st], L::kX);
      bulk_load_1d(sm + L::oX + st * L::kX, a.x + ((size_t)(c0 + n - 1 - i) * a.Hv + h) * L::kX, L::kX, &x_full[st]);
    };
    if (t == 0) {
      for (int i = 0; i < ST; ++i) {
        mbar_init(&kq_full[i], 1);
        mbar_init(&x_full[i], 1);
      }
      mbar_init(done, 1);
      fence_mbar_init();
      for (int i = 0; i < ST && i < n; ++i) {
        load_kq(i);
        load_x(i);
      }
    }
    if (warp == 0) tmem_alloc<256>(tmem_at);
    if (row < KP * 64) put_row<NT, L::kRow>(sm + L::oS, L::kSTerm, row, half * HC / 8, S);
    fence_async_smem();
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tm = *tmem_at;
    const uint32_t mine = tm + ((uint32_t)(quad * 32) << 16) + half * HC;
    Waiter wait{a.wait_ns, a.status};
    uint32_t phase = 0;

    for (int i = 0; i < n; ++i) {
      const int st = i % ST, parity = (i / ST) & 1;
      const bool has_state = i > 0 || a.d_final != nullptr;
      const bool last = i + 1 == n;
      const int64_t c = c0 + n - 1 - i;
      const int64_t ch = c * a.Hv + h;
      const uint32_t kq = smem_u32(sm + L::oKq + st * L::kKq);
      if (t == 0) {
        bulk_store_1d(a.ds + (ch * panels + panel) * (size_t)(NT * L::kSTerm), sm + L::oS, NT * L::kSTerm);
        bulk_commit();
        wait(&kq_full[st], parity);
        if (has_state) {
          const Operand<128, kKMajor, NQ, KP * 16384, 16384> A(kq);
          const Operand<L::kRow, kMnMajor, NT, L::kSTerm> B(smem_u32(sm + L::oS));
          umma_terms<BV, KP * 4, NT>(tm, A, B, false);
          umma_commit(done);
        }
      }
      const int4 chunk = a.table[c];
      const int r = row & 63;
      const bool valid = r < chunk.z;
      const int64_t tok = (int64_t)chunk.y + r;
      const float* gates = a.gates + ch * kDeltaGates;
      const float gam = gates[r], decb = gates[64 + r], gam_end = gates[63];
      float d[HC];
      if (row >= 64) {
#pragma unroll
        for (int k = 0; k < HC; ++k) d[k] = 0.0f;
        if (valid) {
          const T* p = static_cast<const T*>(a.dout) + (tok * a.Hv + h) * a.V + col0;
#pragma unroll
          for (int k = 0; k < HC; k += 8)
            if (col0 + k < a.V) {
              float w[8];
              ld_io8(p + k, w);
#pragma unroll
              for (int j = 0; j < 8; ++j) d[k + j] = w[j];
            }
        }
        put_row<NQ, L::kRow>(sm + L::oDo, L::kRTerm, r, half * HC / 8, d);
        const float f = a.scale * gam;
#pragma unroll
        for (int k = 0; k < HC; ++k) d[k] *= f;
        put_row<NT, L::kRow>(sm + L::oZ, L::kZTerm, row, half * HC / 8, d);
      }
      if (has_state) {
        wait(done, phase);
        phase ^= 1;
        tmem_fence_after_sync();
        if (row < 64) tmem_row<HC>(mine, d);
      } else if (row < 64) {
#pragma unroll
        for (int k = 0; k < HC; ++k) d[k] = 0.0f;
      }
      if (row < 64) {
#pragma unroll
        for (int k = 0; k < HC; ++k) d[k] *= decb;
        put_row<NT, L::kRow>(sm + L::oZ, L::kZTerm, row, half * HC / 8, d);
      }
      fence_async_smem();
      tmem_fence_before_sync();
      __syncthreads();
      if (t == 0) {
        tmem_fence_after_sync();
        wait(&x_full[st], parity);
        const uint32_t x = smem_u32(sm + L::oX + st * L::kX);
        // X^T: 64 rows; the instruction's other 64 come from whatever lies 8 KB further and are not read back
        const Operand<128, kMnMajor, NT, 16384, 0, 8192> A0(x), A1(x + 64 * 128);
        const Operand<L::kRow, kMnMajor, NT, L::kZTerm> B0(smem_u32(sm + L::oZ));
        const Operand<L::kRow, kMnMajor, NQ, L::kRTerm> B1(smem_u32(sm + L::oDo));
        umma_terms<BV, 4, NT>(tm + BV, A0, B0, false);
        umma_terms<BV, 4, NT>(tm + BV, A1, B1, true);
        umma_commit(done);
      }
      wait(done, phase);
      phase ^= 1;
      tmem_fence_after_sync();
      if (t == 0 && i + ST < n) load_x(i + ST);
      if (row < 64) {
        tmem_row<HC>(mine + BV, d);
        put_row<NT, L::kRow>(a.dvi + (ch * panels + panel) * (size_t)(NT * L::kRTerm), L::kRTerm, row, half * HC / 8, d);
        if (valid) {
          T* p = static_cast<T*>(a.dv) + (tok * a.Hv + h) * a.V + col0;
#pragma unroll
          for (int k = 0; k < HC; k += 8)
            if (col0 + k < a.V) st_io8(p + k, d + k);
        }
#pragma unroll
        for (int k = 0; k < HC; ++k) d[k] *= -gam;
        put_row<NT, L::kRow>(sm + L::oZ, L::kZTerm, row, half * HC / 8, d);
      }
      if (last && !a.d_initial) break;
      fence_async_smem();
      tmem_fence_before_sync();
      if (t == 0) bulk_wait_read();
      __syncthreads();
      if (t == 0) {
        tmem_fence_after_sync();
        const Operand<128, kMnMajor, NQ, KP * 16384, 0, 16384> A(kq);
        const Operand<L::kRow, kMnMajor, NT, L::kZTerm> B(smem_u32(sm + L::oZ));
        umma_terms<BV, 8, NT>(tm + 2 * BV, A, B, false);
        umma_commit(done);
      }
      wait(done, phase);
      phase ^= 1;
      tmem_fence_after_sync();
      if (t == 0 && i + ST < n) load_kq(i + ST);
      tmem_row<HC>(mine + 2 * BV, d);
      if (row < KP * 64) {
#pragma unroll
        for (int k = 0; k < HC; ++k) S[k] = fmaf(gam_end, S[k], d[k]);
        if (!last) put_row<NT, L::kRow>(sm + L::oS, L::kSTerm, row, half * HC / 8, S);
      }
      fence_async_smem();
      tmem_fence_before_sync();
      __syncthreads();
      if (t == 0) tmem_fence_after_sync();
    }
    if (t == 0) bulk_wait_all();
    tmem_fence_before_sync();
    __syncthreads();
    if (warp == 0) tmem_dealloc<256>(tm);
  }

  if (a.d_initial && row < a.K) {
#pragma unroll
    for (int i = 0; i < HC; i += 4)
      if (col0 + i < a.V)
        *reinterpret_cast<float4*>(a.d_initial + state_at + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
  }
}

template <IO kIO, int KP>
cudaError_t run_bwd(const DeltaArgs& a, cudaStream_t st) {
  constexpr size_t bytes = BwdSmem<kIO, KP>::kBytes;
  static_assert(bytes <= 227 * 1024, "shared memory");
  cudaError_t e = set_smem(reinterpret_cast<const void*>(delta_bwd_kernel<kIO, KP>), bytes);
  if (e != cudaSuccess) return e;
  const int panels = (a.V + DeltaTerms<kIO>::kCols - 1) / DeltaTerms<kIO>::kCols;
  delta_bwd_kernel<kIO, KP><<<(unsigned)((int64_t)a.num_seqs * a.Hv * panels), 256, bytes, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_bwd(const DeltaArgs& a, IO io, cudaStream_t st) {
  if (a.num_seqs == 0) return cudaSuccess;
  const bool two = delta_panels_k(a.K) == 2;
  if (io == IO::BF16) return two ? run_bwd<IO::BF16, 2>(a, st) : run_bwd<IO::BF16, 1>(a, st);
  return two ? run_bwd<IO::F32, 2>(a, st) : run_bwd<IO::F32, 1>(a, st);
}

}  // namespace vssm
