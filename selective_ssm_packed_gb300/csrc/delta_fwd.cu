// delta_fwd.cu -- the gated delta rule's walk over the chunks of a sequence.
#include "delta.cuh"

namespace vssm {
namespace {

// One CTA of 256 threads per (sequence, value head, panel of kCols state
// columns; the columns of S never mix).  The state lives in registers (FP32,
// thread = one row, half a panel) and as bf16 terms in shared memory.  A chunk
// is three products on the matrix unit, each read back from tensor memory by
// all threads (warp w: lanes 32 (w % 4) .., column half w / 4):
//   D1 = [K; Q] S0        rows 0-63 become R, rows 64-127 wait as exp(G) Q S0
//   D2 = [Tm; P Tm] R     rows 0-63 are E, rows 64-127 finish O
//   D3 = K^T (dec beta E) and S1 = exp(G_63) S0 + D3
// The images of [K; Q] and X arrive by bulk copies, kStages ahead.  bf16 I/O
// holds 160 KB of shared memory and FP32 I/O 180 KB, so one CTA has the SM.
template <IO kIO, int KP>
struct FwdSmem {
  using D = DeltaTerms<kIO>;
  static constexpr int kRow = D::kCols * 2;  // bytes of an image row of a panel
  static constexpr int kKq = D::kIn * KP * 16384, kX = D::kMid * 16384;
  static constexpr int kSTerm = KP * 64 * kRow, kRTerm = 64 * kRow;
  static constexpr int oKq = 0, oX = oKq + D::kStages * kKq, oS = oX + D::kStages * kX;
  static constexpr int oR = oS + D::kMid * kSTerm, oBar = oR + D::kMid * kRTerm;
  static constexpr int kBytes = oBar + 128 + 1024;
};

template <IO kIO, int KP>
__global__ void __launch_bounds__(256, 1) delta_fwd_kernel(DeltaArgs a) {
  using T = typename IoType<kIO>::type;
  using L = FwdSmem<kIO, KP>;
  constexpr int NQ = DeltaTerms<kIO>::kIn, NT = DeltaTerms<kIO>::kMid, BV = DeltaTerms<kIO>::kCols,
                ST = DeltaTerms<kIO>::kStages, HC = BV / 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  uint64_t* kq_full = reinterpret_cast<uint64_t*>(sm + L::oBar);
  uint64_t* x_full = kq_full + ST;
  uint64_t* done = x_full + ST;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(done + 1);

  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, quad = warp & 3, half = warp >> 2;
  const int row = quad * 32 + lane;  // of a product: token (K rows, then Q rows) or state row
  const int panels = (a.V + BV - 1) / BV;
  const int panel = blockIdx.x % panels;
  const int h = blockIdx.x / panels % a.Hv;
  const int s = blockIdx.x / panels / a.Hv;
  if (a.info[0] < 0) return;
  const int c0 = a.first[s], n = a.first[s + 1] - c0;
  const int col0 = panel * BV + half * HC;  // this thread's first state column
  const int64_t state_at = (((int64_t)s * a.Hv + h) * a.K + row) * a.V + col0;
  const int kh = h / (a.Hv / a.Hk);

  float S[HC];
#pragma unroll
  for (int i = 0; i < HC; ++i) S[i] = 0.0f;
  if (a.initial && row < a.K) {
#pragma unroll
    for (int i = 0; i < HC; i += 4)
      if (col0 + i < a.V) {
        const float4 f = *reinterpret_cast<const float4*>(a.initial + state_at + i);
        S[i] = f.x; S[i + 1] = f.y; S[i + 2] = f.z; S[i + 3] = f.w;
      }
  }

  if (n > 0) {
    auto load_kq = [&](int c) {
      const int st = c % ST;
      mbar_arrive_expect_tx(&kq_full[st], L::kKq);
      bulk_load_1d(sm + L::oKq + st * L::kKq, a.kq + ((size_t)(c0 + c) * a.Hk + kh) * L::kKq, L::kKq, &kq_full[st]);
    };
    auto load_x = [&](int c) {
      const int st = c % ST;
      mbar_arrive_expect_tx(&x_full[st], L::kX);
      bulk_load_1d(sm + L::oX + st * L::kX, a.x + ((size_t)(c0 + c) * a.Hv + h) * L::kX, L::kX, &x_full[st]);
    };
    if (t == 0) {
      for (int i = 0; i < ST; ++i) {
        mbar_init(&kq_full[i], 1);
        mbar_init(&x_full[i], 1);
      }
      mbar_init(done, 1);
      fence_mbar_init();
      for (int c = 0; c < ST && c < n; ++c) {
        load_kq(c);
        load_x(c);
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

    for (int c = 0; c < n; ++c) {
      const int st = c % ST, parity = (c / ST) & 1;
      const bool has_state = c > 0 || a.initial != nullptr;
      const bool last = c + 1 == n;
      const int64_t ch = (int64_t)(c0 + c) * a.Hv + h;
      const uint32_t kq = smem_u32(sm + L::oKq + st * L::kKq);
      if (t == 0) {
        if (a.s0) {
          bulk_store_1d(a.s0 + (ch * panels + panel) * (size_t)(NT * L::kSTerm), sm + L::oS, NT * L::kSTerm);
          bulk_commit();
        }
        wait(&kq_full[st], parity);
        if (has_state) {
          const Operand<128, kKMajor, NQ, KP * 16384, 16384> A(kq);
          const Operand<L::kRow, kMnMajor, NT, L::kSTerm> B(smem_u32(sm + L::oS));
          umma_terms<BV, KP * 4, NT>(tm, A, B, false);
          umma_commit(done);
        }
      }
      // while that runs: the chunk's gates and this row's v
      const int4 chunk = a.table[c0 + c];
      const int r = row & 63;
      const bool valid = r < chunk.z;
      const int64_t tok = (int64_t)chunk.y + r;
      const float* gates = a.gates + ch * kDeltaGates;
      const float gam = gates[r], decb = gates[64 + r], gam_end = gates[63];
      float v[HC];
#pragma unroll
      for (int i = 0; i < HC; ++i) v[i] = 0.0f;
      if (row < 64 && valid) {
        const T* vp = static_cast<const T*>(a.v) + tok * a.sv + (int64_t)h * a.V + col0;
#pragma unroll
        for (int i = 0; i < HC; i += 8)
          if (col0 + i < a.V) {
            float w[8];
            ld_io8(vp + i, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i + j] = w[j];
          }
      }
      float d[HC];
      if (has_state) {
        wait(done, phase);
        phase ^= 1;
        tmem_fence_after_sync();
        tmem_row<HC>(mine, d);
      } else {
#pragma unroll
        for (int i = 0; i < HC; ++i) d[i] = 0.0f;
      }
      if (row < 64) {
#pragma unroll
        for (int i = 0; i < HC; ++i) v[i] = valid ? fmaf(-gam, d[i], v[i]) : 0.0f;
        put_row<NT, L::kRow>(sm + L::oR, L::kRTerm, row, half * HC / 8, v);
      } else {
#pragma unroll
        for (int i = 0; i < HC; ++i) v[i] = a.scale * gam * d[i];
      }
      fence_async_smem();
      tmem_fence_before_sync();
      __syncthreads();
      if (t == 0) {
        tmem_fence_after_sync();
        wait(&x_full[st], parity);
        const Operand<128, kKMajor, NT, 16384> A(smem_u32(sm + L::oX + st * L::kX));
        const Operand<L::kRow, kMnMajor, NT, L::kRTerm> B(smem_u32(sm + L::oR));
        umma_terms<BV, 4, NT>(tm + BV, A, B, false);
        umma_commit(done);
      }
      wait(done, phase);
      phase ^= 1;
      tmem_fence_after_sync();
      if (t == 0 && c + ST < n) load_x(c + ST);
      tmem_row<HC>(mine + BV, d);
      if (row < 64) {
        if (a.e)
          put_row<NT, L::kRow>(a.e + (ch * panels + panel) * (size_t)(NT * L::kRTerm), L::kRTerm, row, half * HC / 8, d);
#pragma unroll
        for (int i = 0; i < HC; ++i) d[i] *= decb;
        put_row<NT, L::kRow>(sm + L::oR, L::kRTerm, row, half * HC / 8, d);
      } else if (valid) {
        T* op = static_cast<T*>(a.out) + (tok * a.Hv + h) * a.V + col0;
#pragma unroll
        for (int i = 0; i < HC; ++i) v[i] += d[i];
#pragma unroll
        for (int i = 0; i < HC; i += 8)
          if (col0 + i < a.V) st_io8(op + i, v + i);
      }
      if (last && !a.final_states) break;
      fence_async_smem();
      tmem_fence_before_sync();
      if (t == 0) bulk_wait_read();  // S0's images are free to be overwritten
      __syncthreads();
      if (t == 0) {
        tmem_fence_after_sync();
        const Operand<128, kMnMajor, NQ, KP * 16384, 0, 16384> A(kq);  // K^T: the first 64 rows
        const Operand<L::kRow, kMnMajor, NT, L::kRTerm> B(smem_u32(sm + L::oR));
        umma_terms<BV, 4, NT>(tm + 2 * BV, A, B, false);
        umma_commit(done);
      }
      wait(done, phase);
      phase ^= 1;
      tmem_fence_after_sync();
      if (t == 0 && c + ST < n) load_kq(c + ST);
      tmem_row<HC>(mine + 2 * BV, d);
      if (row < KP * 64) {
#pragma unroll
        for (int i = 0; i < HC; ++i) S[i] = fmaf(gam_end, S[i], d[i]);
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

  if (a.final_states && row < a.K) {
#pragma unroll
    for (int i = 0; i < HC; i += 4)
      if (col0 + i < a.V)
        *reinterpret_cast<float4*>(a.final_states + state_at + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
  }
}

template <IO kIO, int KP>
cudaError_t run_fwd(const DeltaArgs& a, cudaStream_t st) {
  constexpr size_t bytes = FwdSmem<kIO, KP>::kBytes;
  static_assert(bytes <= 227 * 1024, "shared memory");
  cudaError_t e = set_smem(reinterpret_cast<const void*>(delta_fwd_kernel<kIO, KP>), bytes);
  if (e != cudaSuccess) return e;
  const int panels = (a.V + DeltaTerms<kIO>::kCols - 1) / DeltaTerms<kIO>::kCols;
  delta_fwd_kernel<kIO, KP><<<(unsigned)((int64_t)a.num_seqs * a.Hv * panels), 256, bytes, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_fwd(const DeltaArgs& a, IO io, cudaStream_t st) {
  if (a.num_seqs == 0) return cudaSuccess;
  const bool two = delta_panels_k(a.K) == 2;
  if (io == IO::BF16) return two ? run_fwd<IO::BF16, 2>(a, st) : run_fwd<IO::BF16, 1>(a, st);
  return two ? run_fwd<IO::F32, 2>(a, st) : run_fwd<IO::F32, 1>(a, st);
}

}  // namespace vssm
