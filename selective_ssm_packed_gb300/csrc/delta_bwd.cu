// delta_bwd.cu -- the gated delta rule's walk back over the chunks of a
// sequence: the gradient of the state, and dV.
#include "delta.cuh"

namespace vssm {
namespace {

// CTAs and walks as in the forward (four walks spill 28 bytes a thread, 36 for
// K <= 64; 661 us at 32768 tokens of 32 heads, 128 x 128).  dS lives in registers (FP32) and as bf16
// terms in shared memory; a chunk is
//   D1 = [K; Q] dS1                     rows 0-63, times dec beta, become Z
//   D2 = (P Tm)^T dO                    beside it
//   D2 += Tm^T Z = dV                   (64 rows; 64 to 127 are not used)
//   D1 = [K; Q]^T [-exp(G) dV; scale exp(G) dO] and dS0 = exp(G_63) dS1 + D1
// sZ holds 128 rows: dO as it is, then Z, then -exp(G) dV in the upper 64, and
// dO scaled in the lower 64; sS dS1, then dV on its way out.  dS1, dO and dV of
// every chunk leave as images for the gradients that need no walk.
template <IO kIO, int KP, int kWalks>
struct BwdSmem {
  using D = DeltaTerms<kIO>;
  static constexpr int kKq = D::kIn * KP * 16384, kX = D::kMid * 16384;
  static constexpr int kSTile = KP * 64 * 64, kZTile = 128 * 64;
  static constexpr int kS = D::kMid * kSTile, kZ = D::kMid * kZTile;
  static constexpr int oKq = 0, oX = oKq + D::kStages * kKq, oWalk = oX + kX;
  static constexpr int kWalk = kS + kZ;
  static constexpr int oBar = oWalk + kWalks * kWalk;
  static constexpr int kBytes = oBar + 128 + 1024;
};

template <IO kIO, int KP, int kWalks>
__global__ void __launch_bounds__(walk_threads<kWalks>(), 1) delta_bwd_kernel(DeltaArgs a) {
  using T = typename IoType<kIO>::type;
  using R = WalkRow<T, kWalks>;
  using L = BwdSmem<kIO, KP, kWalks>;
  constexpr int NQ = DeltaTerms<kIO>::kIn, NT = DeltaTerms<kIO>::kMid, ST = DeltaTerms<kIO>::kStages, BV = kDeltaTile, HP = R::kCols / 2;
  constexpr int kTmemUsed = 2 * kWalks * NT * BV;
  constexpr int kTmemCols = kTmemUsed > 256 ? 512 : kTmemUsed > 128 ? 256 : 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  uint64_t* kq_full = reinterpret_cast<uint64_t*>(sm + L::oBar);
  uint64_t* x_full = kq_full + ST;
  uint64_t* done_all = x_full + 1;
  uint64_t* drained = done_all + kWalks;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(drained + 1);
  int* kq_used = reinterpret_cast<int*>(tmem_at + 1);  // walks that are through with what a buffer holds
  int* x_used = kq_used + ST;
  volatile int* stop = x_used + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = delta_tiles(a.V), groups = (tiles + kWalks - 1) / kWalks;
  const int group = blockIdx.x % groups;
  const int h = blockIdx.x / groups % a.Hv;
  if (a.info[1] != a.key || a.info[0] < 0) {
    if (threadIdx.x == 0) atomicOr(a.status, a.info[1] != a.key ? kStatusBadSaved : kStatusBadCu);
    return;
  }
  const int4 sequence = a.order[blockIdx.x / groups / a.Hv];
  const int s = sequence.x, c0 = sequence.w, n = (sequence.z + kDeltaChunk - 1) / kDeltaChunk;
  const int64_t seq_start = sequence.y, seq_len = sequence.z;
  const int kh = h / (a.Hv / a.Hk);
  const int walks = min(kWalks, tiles - group * kWalks);
  if (n == 0 && !a.d_initial) return;

  // i counts the chunks walked: chunk n - 1 - i
  auto load_kq = [&](int i) {
    const int st = i % ST;
    mbar_arrive_expect_tx(&kq_full[st], L::kKq);
    bulk_load_1d(sm + L::oKq + st * L::kKq, a.kq + ((size_t)(c0 + n - 1 - i) * a.Hk + kh) * L::kKq, L::kKq, &kq_full[st]);
  };
  auto load_x = [&](int i) {
    mbar_arrive_expect_tx(x_full, L::kX);
    bulk_load_1d(sm + L::oX, a.x + ((size_t)(c0 + n - 1 - i) * a.Hv + h) * L::kX, L::kX, x_full);
  };
  // a walk's leader is through with a buffer: the last one may have it filled again
  auto last_user = [&](int* used) {
    __threadfence_block();
    const bool last = (atomicAdd(used, 1) + 1) % walks == 0;
    __threadfence_block();
    return last;
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&kq_full[i], 1);
      kq_used[i] = 0;
    }
    mbar_init(x_full, 1);
    *x_used = *stop = 0;
    mbar_init(drained, walks);
    for (int i = 0; i < kWalks; ++i) mbar_init(&done_all[i], 2);  // the products, and the porter
    fence_mbar_init();
    for (int i = 0; i < ST && i < n; ++i) load_kq(i);
    if (n > 0) load_x(0);
  }
  if (warp == 0) tmem_alloc<kTmemCols>(tmem_at);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tm = *tmem_at;
  Waiter wait{a, stop};
  if (threadIdx.x == 96 && n > 0 && forced_here(a)) wait(&kq_full[0], 0, true);  // the first walk's leader

  if ((int)threadIdx.x / R::kThreads < walks) {
    const int walk = threadIdx.x / R::kThreads, quad = warp & 3, half = warp / 4 % R::kHalves;
    const int row = quad * 32 + lane, r = row & 63;
    const bool leader = threadIdx.x % R::kThreads == 96, porter = threadIdx.x % R::kThreads == 64;  // as in the forward
    const int tile = group * kWalks + walk;
    const int col0 = tile * BV + half * R::kCols, step0 = half * R::kSteps;  // this thread's columns
    uint8_t* sS = sm + L::oWalk + walk * L::kWalk;
    uint8_t* sZ = sS + L::kS;
    uint64_t* done = done_all + walk;
    const uint32_t tD1 = tm + walk * 2 * NT * BV, tD2 = tD1 + NT * BV;
    const uint32_t lane_at = (uint32_t)(quad * 32) << 16;
    const int64_t state_at = (((int64_t)s * a.Hv + h) * a.K + row) * a.V + col0;

    float2 S[HP];
#pragma unroll
    for (int i = 0; i < HP; ++i) S[i] = splat2(0.0f);
    if (a.d_final && row < a.K) {
#pragma unroll
      for (int i = 0; i < HP; i += 2)
        if (col0 + 2 * i < a.V) {
          const float4 f = *reinterpret_cast<const float4*>(a.d_final + state_at + 2 * i);
          S[i] = make_float2(f.x, f.y);
          S[i + 1] = make_float2(f.z, f.w);
        }
    }
    // the next chunk's dO, raw, and gates: read a chunk ahead
    typename R::Raw raw;
    float gam, decb, gam_end;
    auto prefetch = [&](int c) {
      const float* gates = a.gates + ((int64_t)(c0 + c) * a.Hv + h) * kDeltaGates;
      gam = gates[r];
      decb = gates[64 + r];
      gam_end = gates[63];
      const int64_t at = (int64_t)c * kDeltaChunk + (quad & 1) * 32;  // the warp's first token
      if (row >= 64)
        R::load(static_cast<const T*>(a.dout) + ((seq_start + at) * a.Hv + h) * a.V + col0, (int64_t)a.Hv * a.V, seq_len - at,
                a.V - col0, lane, raw);
    };
    // rows 64-127: dO into sZ, as it is and scaled
    auto put_dout = [&]() {
#pragma unroll
      for (int i = 0; i < R::kParts; ++i) transpose(raw[i], lane);
#pragma unroll
      for (int u = 0; u < R::kSteps; ++u) {
        float2 d[8];
        R::each(raw, u, [&](int k, float2 w) { d[k] = w; });
        put_row<NQ, 64>(sZ, L::kZTile, r, 2 * (step0 + u), d);
        scale_row(d, a.scale * gam);
        put_row<NT, 64>(sZ, L::kZTile, row, 2 * (step0 + u), d);
      }
    };
    if (n > 0) {
      prefetch(n - 1);
      if (row >= 64) put_dout();
    }
    if (row < KP * 64) put_row<NT, 64>(sS, L::kSTile, row, 2 * step0, S);
    fence_async_smem();
    named_barrier(1 + walk, R::kThreads);
    uint32_t phase = 0;

    for (int i = 0; i < n; ++i) {
      const int st = i % ST, c = n - 1 - i;
      const bool has_state = i > 0 || a.d_final != nullptr;
      const bool last = i + 1 == n;
      const int64_t ch = (int64_t)(c0 + c) * a.Hv + h;
      const uint32_t kq = smem_u32(sm + L::oKq + st * L::kKq), x = smem_u32(sm + L::oX);
      if (porter) {

#pragma unroll
        for (int j = 0; j < NQ; ++j)
          bulk_store_1d(a.doi + ((ch * tiles + tile) * NQ + j) * (size_t)kRowTile, sZ + j * L::kZTile, kRowTile);
        bulk_commit();
        bulk_store_1d(a.ds + (ch * tiles + tile) * (size_t)(NT * L::kSTile), sS, NT * L::kSTile);
        bulk_commit();
        asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        if (wait.ok) mbar_arrive(done);  // dO's image has left, before Z takes its place
      }
      if (leader) {
        wait(&kq_full[st], (i / ST) & 1);
        tmem_fence_after_sync();
        if (has_state && wait.ok) {
          const Operand<128, kKMajor, NQ, KP * 16384, 16384> A(kq);
          const Operand<64, kMnMajor, NT, L::kSTile, 0, L::kSTile> B(smem_u32(sS));
          umma_blocks<BV, KP * 4, NT, true>(tD1, A, B);
        }
        if (wait(x_full, i & 1)) {
          // (P Tm)^T: 64 rows; the instruction's other 64 come from whatever lies 8 KB further and are not read back
          const Operand<128, kMnMajor, NT, 16384, 0, 8192> A(x + 64 * 128);
          const Operand<64, kMnMajor, NQ, L::kZTile, 0, L::kZTile> B(smem_u32(sZ));
          umma_blocks<BV, 4, NT, true>(tD2, A, B);
          umma_commit(done);
        }
      }
      const float g_row = gam, db_row = decb, g_end = gam_end;
      wait(done, phase);
      phase ^= 1;
      tmem_fence_after_sync();
      if (row < 64) {
#pragma unroll
        for (int u = 0; u < R::kSteps; ++u) {
          float2 d[8];
          if (has_state) {
            tmem_sum<NT>(tD1 + lane_at + 16 * (step0 + u), BV, d);
            scale_row(d, db_row);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) d[k] = splat2(0.0f);
          }
          put_row<NT, 64>(sZ, L::kZTile, row, 2 * (step0 + u), d);
        }
      }
      fence_async_smem();
      tmem_fence_before_sync();
      if (porter) {
        bulk_wait_read();  // dS1's image has left too, before dV takes its place
        if (wait.ok) mbar_arrive(done);
      }
      named_barrier(1 + walk, R::kThreads);
      if (leader && wait.ok) {
        tmem_fence_after_sync();
        const Operand<128, kMnMajor, NT, 16384, 0, 8192> A(x);
        const Operand<64, kMnMajor, NT, L::kZTile, 0, L::kZTile> B(smem_u32(sZ));
        umma_blocks<BV, 4, NT, false>(tD2, A, B);
        umma_commit(done);
      }
      if (!last) prefetch(c - 1);
      wait(done, phase);
      phase ^= 1;
      tmem_fence_after_sync();
      if (porter && wait.ok && i + 1 < n && last_user(x_used)) load_x(i + 1);
      if (row < 64) {
        typename R::Raw q;
#pragma unroll
        for (int u = 0; u < R::kSteps; ++u) {
          float2 d[8];
          tmem_sum<NT>(tD2 + lane_at + 16 * (step0 + u), BV, d);
          put_row<NT, 64>(sS, kRowTile, row, 2 * (step0 + u), d);  // dS1's images have been read
          R::put(q, u, d);
          scale_row(d, -g_row);
          put_row<NT, 64>(sZ, L::kZTile, row, 2 * (step0 + u), d);
        }
        const int64_t at = (int64_t)c * kDeltaChunk + quad * 32;
        R::store(static_cast<T*>(a.dv) + ((seq_start + at) * a.Hv + h) * a.V + col0, (int64_t)a.Hv * a.V, seq_len - at,
                 a.V - col0, lane, q);
      }
      fence_async_smem();
      tmem_fence_before_sync();
      named_barrier(1 + walk, R::kThreads);
      if (porter) {
        bulk_store_1d(a.dvi + (ch * tiles + tile) * (size_t)(NT * kRowTile), sS, NT * kRowTile);
        bulk_commit();
        if (!(last && !a.d_initial)) {
          bulk_wait_read();
          if (wait.ok) mbar_arrive(done);  // dV's image has left, before dS0 takes its place
        }
      }
      if (last && !a.d_initial) break;
      if (leader && wait.ok) {
        tmem_fence_after_sync();
        const Operand<128, kMnMajor, NQ, KP * 16384, 0, 16384> A(kq);
        const Operand<64, kMnMajor, NT, L::kZTile, 0, L::kZTile> B(smem_u32(sZ));
        umma_blocks<BV, 8, NT, true>(tD1, A, B);
        umma_commit(done);
      }
      wait(done, phase);
      phase ^= 1;
      tmem_fence_after_sync();
      if (porter && wait.ok && i + ST < n && last_user(&kq_used[st])) load_kq(i + ST);
      if (row < KP * 64) {
#pragma unroll
        for (int u = 0; u < R::kSteps; ++u) {
          float2 d[8];
          tmem_sum<NT>(tD1 + lane_at + 16 * (step0 + u), BV, d);
#pragma unroll
          for (int k = 0; k < 8; ++k) S[8 * u + k] = d[k] = fma2(splat2(g_end), S[8 * u + k], d[k]);
          if (!last) put_row<NT, 64>(sS, L::kSTile, row, 2 * (step0 + u), d);
        }
      }
      if (!last && row >= 64) put_dout();
      fence_async_smem();
      tmem_fence_before_sync();
      if (!vote(1 + walk, R::kThreads, wait.ok)) break;
    }
    if (porter) bulk_wait_all();
    if (a.d_initial && row < a.K) {
#pragma unroll
      for (int i = 0; i < HP; i += 2)
        if (col0 + 2 * i < a.V)
          *reinterpret_cast<float4*>(a.d_initial + state_at + 2 * i) = make_float4(S[i].x, S[i].y, S[i + 1].x, S[i + 1].y);
    }
  }
  tmem_fence_before_sync();
  if (!__syncthreads_and(wait.ok)) {
    // nobody asks for anything any more: what is on its way comes in before the memory is given back
    if ((int)threadIdx.x / R::kThreads < walks && threadIdx.x % R::kThreads == 96) umma_commit(drained);
    if (threadIdx.x == 0) {
      for (int i = 0; i < ST; ++i) drain_copies(&kq_full[i], (i < n) + kq_used[i] / walks);
      drain_copies(x_full, (n > 0) + *x_used / walks);
      mbar_wait(drained, 0, kCopyDrainNs);
    }
    __syncthreads();
  }
  if (warp == 0) tmem_dealloc<kTmemCols>(tm);
}

template <IO kIO, int KP, int kWalks>
cudaError_t run_bwd(const DeltaArgs& a, cudaStream_t st) {
  constexpr size_t bytes = BwdSmem<kIO, KP, kWalks>::kBytes;
  static_assert(bytes <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> done{0};
  cudaError_t e = set_smem(reinterpret_cast<const void*>(delta_bwd_kernel<kIO, KP, kWalks>), bytes, done);
  if (e != cudaSuccess) return e;
  const int groups = (delta_tiles(a.V) + kWalks - 1) / kWalks;
  delta_bwd_kernel<kIO, KP, kWalks>
      <<<(unsigned)((int64_t)a.num_seqs * a.Hv * groups), walk_threads<kWalks>(), bytes, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_bwd(const DeltaArgs& a, IO io, cudaStream_t st) {
  if (a.num_seqs == 0) return cudaSuccess;
  const bool two = delta_panels_k(a.K) == 2;
  if (io == IO::BF16) {
    const int walks = delta_walks(a, io);
    if (walks == 4) return two ? run_bwd<IO::BF16, 2, 4>(a, st) : run_bwd<IO::BF16, 1, 4>(a, st);
    if (walks == 2) return two ? run_bwd<IO::BF16, 2, 2>(a, st) : run_bwd<IO::BF16, 1, 2>(a, st);
    return two ? run_bwd<IO::BF16, 2, 1>(a, st) : run_bwd<IO::BF16, 1, 1>(a, st);
  }
  return two ? run_bwd<IO::F32, 2, 1>(a, st) : run_bwd<IO::F32, 1, 1>(a, st);
}

}  // namespace vssm
