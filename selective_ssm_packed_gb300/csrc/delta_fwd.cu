// delta_fwd.cu -- the gated delta rule's walk over the chunks of a sequence.
#include "delta.cuh"

namespace vssm {
namespace {

// One CTA per (sequence, value head, kWalks tiles of the state's columns; the
// columns never mix).  A walk is one tile and 128 threads, or 256 where at most
// two share a CTA: the state lives in registers (FP32; thread = one row or
// half of one) and as bf16 terms in shared memory.  A chunk is three products
// on the matrix unit, each read back from tensor memory by the walk's threads:
//   D1 = [K; Q] S0        rows 0-63 become R, rows 64-127 wait in tensor memory
//   D2 = [Tm; P Tm] R     rows 0-63 are E, rows 64-127 with D1's make O
//   D1 = K^T (dec beta E) and S1 = exp(G_63) S0 + D1
// The chain product - read back - product bounds a walk, not the matrix unit
// (25% busy), so up to four walks share a CTA, its [K; Q] and its X: one
// multiplies while others read back.  Wider tiles would read [K; Q] and X from
// shared memory less often, but a step of 128 columns took two walks of 64 8900
// cycles and four of 32 7600: with as many instructions to issue there were
// fewer chains to issue them from.  [K; Q] and X come by bulk copies, ahead of
// the walks, asked for by whichever walk is through with the buffer last.  Four
// walks leave a thread 128 registers, so they read back 16 columns at a time:
// a register spilled within a step is a trip to L2, shared memory having taken
// nearly all of L1 (a build that spilled 28 bytes took 560 us at 32768 tokens,
// this one, with 4, takes 500; with 28 for K <= 64 444).  CTAs that stay, with a
// fixed deal of the items and the next one's operands already on their way, took
// 726 us at 32768 tokens where these take 446: sequences are unequal, and the
// hardware hands the next CTA to the SM that is free.  Two threads to a row
// shorten the read-backs of a chain that has little else to wait for: the walk
// of a 3001-token f32 pack took 122 us with one and 108 with two (the walk back
// 168 and 134), of one 32768-token bf16 sequence 1150 and 1096.  The checks of
// waits and of values that are not finite cost these walks 2%, 0 and 3%.
template <IO kIO, int KP, int kWalks>
struct FwdSmem {
  using D = DeltaTerms<kIO>;
  static constexpr int kKq = D::kIn * KP * 16384, kX = D::kMid * 16384;
  static constexpr int kSTile = KP * 64 * 64;
  static constexpr int kS = D::kMid * kSTile, kR = D::kMid * kRowTile;
  static constexpr int oKq = 0, oX = oKq + D::kStages * kKq, oWalk = oX + kX;
  static constexpr int kWalk = kS + 2 * kR;  // S, R, E
  static constexpr int oBar = oWalk + kWalks * kWalk;
  static constexpr int oBad = oBar + 128;  // of a walk's columns: the first token that is not finite
  static constexpr int oAnyBad = oBad + kWalks * kDeltaTile * 4;  // whether a walk has met one
  static constexpr int kBytes = oAnyBad + 16 + 1024;
};

// What is not finite stays out of the products, where 0 times it, above Tm's
// diagonal, would reach earlier tokens: a walk takes 0 in its place, keeps each
// column's first token that has it, and in the end writes NaN from there on.
// Both are calls that find their places anew, so that the walk, which has no
// register to spare, keeps nothing for them.
template <IO kIO, int KP, int kWalks>
__device__ __forceinline__ int* bad_tokens() {  // of this thread's columns
  extern __shared__ uint8_t smem_raw[];
  using R = WalkRow<typename IoType<kIO>::type, kWalks>;
  const int walk = threadIdx.x / R::kThreads, half = threadIdx.x / 128 % R::kHalves;
  return reinterpret_cast<int*>(align1024(smem_raw) + FwdSmem<kIO, KP, kWalks>::oBad) + walk * kDeltaTile + half * R::kCols;
}

template <IO kIO, int KP, int kWalks>
__device__ __forceinline__ volatile int* any_bad_token() {  // of this thread's walk
  extern __shared__ uint8_t smem_raw[];
  using R = WalkRow<typename IoType<kIO>::type, kWalks>;
  return reinterpret_cast<int*>(align1024(smem_raw) + FwdSmem<kIO, KP, kWalks>::oAnyBad) + threadIdx.x / R::kThreads;
}

// This thread's columns of its row of R, in chunk c.
template <IO kIO, int KP, int kWalks>
__device__ __noinline__ void clear_row(int c) {
  extern __shared__ uint8_t smem_raw[];
  using R = WalkRow<typename IoType<kIO>::type, kWalks>;
  using L = FwdSmem<kIO, KP, kWalks>;
  const int walk = threadIdx.x / R::kThreads, half = threadIdx.x / 128 % R::kHalves, row = threadIdx.x % 128;
  uint8_t* image = align1024(smem_raw) + L::oWalk + walk * L::kWalk + L::kS;
  int* bad = bad_tokens<kIO, KP, kWalks>();
#pragma unroll 1
  for (int i = 0; i < R::kCols; ++i) {
    const int col = half * R::kCols + i;
    uint8_t* p = image + image_chunk<64>(row, col / 8) + col % 8 * 2;
    if ((*reinterpret_cast<const uint16_t*>(p) & 0x7f80) != 0x7f80) continue;
    for (int k = 0; k < DeltaTerms<kIO>::kMid; ++k) *reinterpret_cast<uint16_t*>(p + k * kRowTile) = 0;
    atomicMin(bad + i, c * kDeltaChunk + row);
    *any_bad_token<kIO, KP, kWalks>() = 1;
  }
}

// NaN for this thread's columns from their bad tokens on: in out, in the saved images of E and S0, in the final state.
template <IO kIO, int KP, int kWalks>
__device__ __noinline__ void spoil_columns(const DeltaArgs& a) {
  using T = typename IoType<kIO>::type;
  using R = WalkRow<T, kWalks>;
  using L = FwdSmem<kIO, KP, kWalks>;
  constexpr int NT = DeltaTerms<kIO>::kMid;
  const int tiles = delta_tiles(a.V), groups = (tiles + kWalks - 1) / kWalks;
  const int tile = blockIdx.x % groups * kWalks + threadIdx.x / R::kThreads, half = threadIdx.x / 128 % R::kHalves;
  const int h = blockIdx.x / groups % a.Hv, row = threadIdx.x % 128, r = row & 63;
  const int4 sequence = a.order[blockIdx.x / groups / a.Hv];
  const int n = (sequence.z + kDeltaChunk - 1) / kDeltaChunk;
  const int* bad = bad_tokens<kIO, KP, kWalks>();
  const float nan = __int_as_float(0x7fffffff);
#pragma unroll 1
  for (int i = 0; i < R::kCols; ++i) {
    const int from = bad[i], in_tile = half * R::kCols + i, col = tile * kDeltaTile + in_tile;
    if (from == 0x7fffffff || col >= a.V) continue;
    const int in_image = in_tile % 8 * 2;
#pragma unroll 1
    for (int c = from / kDeltaChunk; c < n; ++c) {
      const int token = c * kDeltaChunk + r;
      const int64_t image = ((int64_t)(sequence.w + c) * a.Hv + h) * tiles + tile;
      if (row >= 64 && token >= from && token < sequence.z)
        static_cast<T*>(a.out)[(((int64_t)sequence.y + token) * a.Hv + h) * a.V + col] = from_f<T>(nan);
      if (a.e && row < 64 && token >= from)
        *reinterpret_cast<uint16_t*>(a.e + image * (NT * kRowTile) + image_chunk<64>(row, in_tile / 8) + in_image) = 0x7fff;
      if (a.s0 && row < KP * 64 && c * kDeltaChunk > from)
        *reinterpret_cast<uint16_t*>(a.s0 + image * (NT * L::kSTile) + image_chunk<64>(row, in_tile / 8) + in_image) = 0x7fff;
    }
    if (a.final_states && row < a.K) a.final_states[(((int64_t)sequence.x * a.Hv + h) * a.K + row) * a.V + col] = nan;
  }
}

template <IO kIO, int KP, int kWalks>
__global__ void __launch_bounds__(walk_threads<kWalks>(), 1) delta_fwd_kernel(const __grid_constant__ DeltaArgs a) {
  using T = typename IoType<kIO>::type;
  using R = WalkRow<T, kWalks>;
  using L = FwdSmem<kIO, KP, kWalks>;
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
  if (a.info[0] < 0) return;
  const int4 sequence = a.order[blockIdx.x / groups / a.Hv];
  const int s = sequence.x, c0 = sequence.w, n = (sequence.z + kDeltaChunk - 1) / kDeltaChunk;
  const int64_t seq_start = sequence.y, seq_len = sequence.z;
  const int kh = h / (a.Hv / a.Hk);
  const int walks = min(kWalks, tiles - group * kWalks);  // tiles there are for this CTA
  if (n == 0 && !a.final_states) return;

  auto load_kq = [&](int c) {
    const int st = c % ST;
    mbar_arrive_expect_tx(&kq_full[st], L::kKq);
    bulk_load_1d(sm + L::oKq + st * L::kKq, a.kq + ((size_t)(c0 + c) * a.Hk + kh) * L::kKq, L::kKq, &kq_full[st]);
  };
  auto load_x = [&](int c) {
    mbar_arrive_expect_tx(x_full, L::kX);
    bulk_load_1d(sm + L::oX, a.x + ((size_t)(c0 + c) * a.Hv + h) * L::kX, L::kX, x_full);
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
    for (int i = 0; i < kWalks; ++i) mbar_init(&done_all[i], 1);
    fence_mbar_init();
    for (int i = 0; i < ST && i < n; ++i) load_kq(i);
    if (n > 0) load_x(0);
  }
  if (threadIdx.x < kWalks * BV) reinterpret_cast<int*>(sm + L::oBad)[threadIdx.x] = 0x7fffffff;
  if (threadIdx.x < kWalks) reinterpret_cast<int*>(sm + L::oAnyBad)[threadIdx.x] = 0;
  if (warp == 0) tmem_alloc<kTmemCols>(tmem_at);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tm = *tmem_at;
  Waiter wait{a, stop};
  if (threadIdx.x == 96 && n > 0 && forced_here(a)) wait(&kq_full[0], 0, true);  // the first walk's leader

  if ((int)threadIdx.x / R::kThreads < walks) {
    const int walk = threadIdx.x / R::kThreads, quad = warp & 3, half = warp / 4 % R::kHalves;
    const int row = quad * 32 + lane, r = row & 63;  // of a product: token (K rows, then Q rows) or state row
    // one thread issues the products, another the bulk copies: in warps of Q rows, whose read-backs are the shorter ones
    const bool leader = threadIdx.x % R::kThreads == 96, porter = threadIdx.x % R::kThreads == 64;
    const int tile = group * kWalks + walk;
    const int col0 = tile * BV + half * R::kCols, step0 = half * R::kSteps;  // this thread's columns
    uint8_t* sS = sm + L::oWalk + walk * L::kWalk;
    uint8_t* sR = sS + L::kS;
    uint8_t* sE = sR + L::kR;
    uint64_t* done = done_all + walk;
    volatile int* leave = stop + 1 + walk;  // the porter's word on whether this chunk is the last
    const uint32_t tD1 = tm + walk * 2 * NT * BV, tD2 = tD1 + NT * BV;
    const uint32_t lane_at = (uint32_t)(quad * 32) << 16;
    const int64_t state_at = (((int64_t)s * a.Hv + h) * a.K + row) * a.V + col0;

    float2 S[HP];
#pragma unroll
    for (int i = 0; i < HP; ++i) S[i] = splat2(0.0f);
    if (a.initial && row < a.K) {
#pragma unroll
      for (int i = 0; i < HP; i += 2)
        if (col0 + 2 * i < a.V) {
          const float4 f = *reinterpret_cast<const float4*>(a.initial + state_at + 2 * i);
          S[i] = make_float2(f.x, f.y);
          S[i + 1] = make_float2(f.z, f.w);
        }
    }
    const float2 trace = trace_row(S, splat2(0.0f));
    if (trace.x + trace.y != 0.0f && n > 0) {  // a column that is not finite is 0 for the walk, and NaN in the end
      *any_bad_token<kIO, KP, kWalks>() = 1;
#pragma unroll
      for (int i = 0; i < HP; ++i) {
        if (S[i].x * 0.0f != 0.0f) bad_tokens<kIO, KP, kWalks>()[2 * i] = -1;
        if (S[i].y * 0.0f != 0.0f) bad_tokens<kIO, KP, kWalks>()[2 * i + 1] = -1;
        S[i] = make_float2(S[i].x * 0.0f != 0.0f ? 0.0f : S[i].x, S[i].y * 0.0f != 0.0f ? 0.0f : S[i].y);
      }
    }
    // the next chunk's v, raw, and gates: read a chunk ahead
    typename R::Raw raw;
    float gam, decb, gam_end;
    auto prefetch = [&](int c) {
      const float* gates = a.gates + ((int64_t)(c0 + c) * a.Hv + h) * kDeltaGates;
      gam = gates[r];
      decb = gates[64 + r];
      gam_end = gates[63];
      const int64_t at = (int64_t)c * kDeltaChunk + quad * 32;  // the warp's first token
      if (row < 64)
        R::load(static_cast<const T*>(a.v) + (seq_start + at) * a.sv + (int64_t)h * a.V + col0, a.sv, seq_len - at,
                a.V - col0, lane, raw);
    };
    if (n > 0) prefetch(0);
    if (row < KP * 64) put_row<NT, 64>(sS, L::kSTile, row, 2 * step0, S);
    fence_async_smem();
    named_barrier(1 + walk, R::kThreads);
    uint32_t phase = 0;

    for (int c = 0; c < n; ++c) {
      const int st = c % ST;
      const bool has_state = c > 0 || a.initial != nullptr;
      const bool last = c + 1 == n;
      const int64_t ch = (int64_t)(c0 + c) * a.Hv + h;
      const uint32_t kq = smem_u32(sm + L::oKq + st * L::kKq);
      if (porter) *leave = *stop;
      if (porter && a.s0) {
        bulk_store_1d(a.s0 + (ch * tiles + tile) * (size_t)(NT * L::kSTile), sS, NT * L::kSTile);
        bulk_commit();
      }
      if (leader) {
        wait(&kq_full[st], (c / ST) & 1);
        tmem_fence_after_sync();
        if (has_state && wait.ok) {
          const Operand<128, kKMajor, NQ, KP * 16384, 16384> A(kq);
          const Operand<64, kMnMajor, NT, L::kSTile, 0, L::kSTile> B(smem_u32(sS));
          umma_blocks<BV, KP * 4, NT, true>(tD1, A, B);
          umma_commit(done);
        }
      }
      const float g_row = gam, db_row = decb, g_end = gam_end;
      bool odd = false;  // whether this row of R may hold what is not finite, by v or by the chunk's keys and gates
      if (row < 64) {
#pragma unroll
        for (int i = 0; i < R::kParts; ++i) transpose(raw[i], lane);
        float2 trace = splat2(0.0f);
#pragma unroll
        for (int u = 0; u < R::kSteps; ++u) R::each(raw, u, [&](int, float2 w) { trace = fma2(w, splat2(0.0f), trace); });
        odd = fmaf(g_end, 0.0f, trace.x + trace.y) != 0.0f;
      }
      if (has_state) {
        wait(done, phase);
        phase ^= 1;
        tmem_fence_after_sync();
      }
      if (row < 64) {
        // past the chunk's end v and the rows of K are zero, and so is R
#pragma unroll
        for (int u = 0; u < R::kSteps; ++u) {
          float2 d[8];
          if (has_state) tmem_sum<NT>(tD1 + lane_at + 16 * (step0 + u), BV, d);
          R::each(raw, u, [&](int k, float2 w) { d[k] = has_state ? fma2(splat2(-g_row), d[k], w) : w; });
          put_row<NT, 64>(sR, kRowTile, row, 2 * (step0 + u), d);
        }
        if (odd) clear_row<kIO, KP, kWalks>(c);
      }
      fence_async_smem();
      tmem_fence_before_sync();
      if (porter && a.s0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");  // the last chunk's E has left
      named_barrier(1 + walk, R::kThreads);
      if (leader) {
        tmem_fence_after_sync();
        if (wait(x_full, c & 1)) {
          const Operand<128, kKMajor, NT, 16384> A(smem_u32(sm + L::oX));
          const Operand<64, kMnMajor, NT, kRowTile, 0, kRowTile> B(smem_u32(sR));
          umma_blocks<BV, 4, NT, true>(tD2, A, B);
          umma_commit(done);
        }
      }
      if (!last) prefetch(c + 1);
      wait(done, phase);
      phase ^= 1;
      tmem_fence_after_sync();
      if (porter && wait.ok && c + 1 < n && last_user(x_used)) load_x(c + 1);
      if (row < 64) {
#pragma unroll
        for (int u = 0; u < R::kSteps; ++u) {
          float2 d[8];
          tmem_sum<NT>(tD2 + lane_at + 16 * (step0 + u), BV, d);
          if (a.e) put_row<NT, 64>(sE, kRowTile, row, 2 * (step0 + u), d);
          scale_row(d, db_row);
          put_row<NT, 64>(sR, kRowTile, row, 2 * (step0 + u), d);
        }
      } else {
        typename R::Raw q;
#pragma unroll
        for (int u = 0; u < R::kSteps; ++u) {
          float2 d[8], o[8];
          tmem_sum<NT>(tD2 + lane_at + 16 * (step0 + u), BV, d);
          if (has_state) {
            tmem_sum<NT>(tD1 + lane_at + 16 * (step0 + u), BV, o);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = fma2(splat2(a.scale * g_row), o[i], d[i]);
          }
          R::put(q, u, d);
        }
        const int64_t at = (int64_t)c * kDeltaChunk + (quad & 1) * 32;
        R::store(static_cast<T*>(a.out) + ((seq_start + at) * a.Hv + h) * a.V + col0, (int64_t)a.Hv * a.V, seq_len - at,
                 a.V - col0, lane, q);
      }
      const bool stop = last && !a.final_states;
      if (stop && !a.e) break;
      fence_async_smem();
      tmem_fence_before_sync();
      if (porter && a.s0) bulk_wait_read();  // S0's images are free to be overwritten
      named_barrier(1 + walk, R::kThreads);
      if (porter && a.e) {
        bulk_store_1d(a.e + (ch * tiles + tile) * (size_t)(NT * kRowTile), sE, NT * kRowTile);
        bulk_commit();
      }
      if (stop) break;
      if (leader && wait.ok) {
        tmem_fence_after_sync();
        const Operand<128, kMnMajor, NQ, KP * 16384, 0, 16384> A(kq);  // K^T: the first 64 rows
        const Operand<64, kMnMajor, NT, kRowTile, 0, kRowTile> B(smem_u32(sR));
        umma_blocks<BV, 4, NT, true>(tD1, A, B);
        umma_commit(done);
      }
      const int left = kWalks < 4 ? *leave : 0;  // four walks rather vote: a vote needs no register
      wait(done, phase);
      phase ^= 1;
      tmem_fence_after_sync();
      if (porter && wait.ok && c + ST < n && last_user(&kq_used[st])) load_kq(c + ST);
      if (row < KP * 64) {
#pragma unroll
        for (int u = 0; u < R::kSteps; ++u) {
          float2 d[8];
          tmem_sum<NT>(tD1 + lane_at + 16 * (step0 + u), BV, d);
#pragma unroll
          for (int i = 0; i < 8; ++i) S[8 * u + i] = d[i] = fma2(splat2(g_end), S[8 * u + i], d[i]);
          if (!last) put_row<NT, 64>(sS, L::kSTile, row, 2 * (step0 + u), d);
        }
      }
      fence_async_smem();
      tmem_fence_before_sync();
      if (kWalks < 4) named_barrier(1 + walk, R::kThreads);
      if (kWalks < 4 ? left != 0 : !vote(1 + walk, R::kThreads, wait.ok)) break;
    }
    if (porter) bulk_wait_all();
    if (a.final_states && row < a.K) {
#pragma unroll
      for (int i = 0; i < HP; i += 2)
        if (col0 + 2 * i < a.V)
          *reinterpret_cast<float4*>(a.final_states + state_at + 2 * i) = make_float4(S[i].x, S[i].y, S[i + 1].x, S[i + 1].y);
    }
    if (*any_bad_token<kIO, KP, kWalks>()) {  // said before a barrier that all of the walk have passed
      named_barrier(1 + walk, R::kThreads);
      spoil_columns<kIO, KP, kWalks>(a);
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
cudaError_t run_fwd(const DeltaArgs& a, cudaStream_t st) {
  constexpr size_t bytes = FwdSmem<kIO, KP, kWalks>::kBytes;
  static_assert(bytes <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> done{0};
  cudaError_t e = set_smem(reinterpret_cast<const void*>(delta_fwd_kernel<kIO, KP, kWalks>), bytes, done);
  if (e != cudaSuccess) return e;
  const int groups = (delta_tiles(a.V) + kWalks - 1) / kWalks;
  delta_fwd_kernel<kIO, KP, kWalks>
      <<<(unsigned)((int64_t)a.num_seqs * a.Hv * groups), walk_threads<kWalks>(), bytes, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_fwd(const DeltaArgs& a, IO io, cudaStream_t st) {
  if (a.num_seqs == 0) return cudaSuccess;
  const bool two = delta_panels_k(a.K) == 2;
  if (io == IO::BF16) {
    const int walks = delta_walks(a, io);
    if (walks == 4) return two ? run_fwd<IO::BF16, 2, 4>(a, st) : run_fwd<IO::BF16, 1, 4>(a, st);
    if (walks == 2) return two ? run_fwd<IO::BF16, 2, 2>(a, st) : run_fwd<IO::BF16, 1, 2>(a, st);
    return two ? run_fwd<IO::BF16, 2, 1>(a, st) : run_fwd<IO::BF16, 1, 1>(a, st);
  }
  return two ? run_fwd<IO::F32, 2, 1>(a, st) : run_fwd<IO::F32, 1, 1>(a, st);
}

}  // namespace vssm
