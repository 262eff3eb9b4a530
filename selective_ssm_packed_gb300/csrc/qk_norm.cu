// qk_norm.cu -- queries and keys normalised for each head, and rotated by
// their position, in one pass; and the gradients.
#include "delta.cuh"

namespace vssm {
namespace {

// A row is one head of one token: K values.  A lane holds two chunks of 8
// neighbouring values, kLanes lanes a row, and a warp works on 32 / kLanes
// heads of one token at a time, keeping the token's cosines and sines in
// registers over all of them.  The rotation turns value i of the first half of
// the rotated width with value i + half, so a lane's two chunks lie half a
// rotated width apart there (kPaired: every chunk then has its partner in its
// own lane) and side by side past it.  Where half is no multiple of 8, or the
// chunks do not come in pairs, a lane holds neighbouring chunks and reads its
// partners' values once more, from L1.  q and k are separate CTAs, so that a
// lane needs one set of weights.  Every value is read from and written to
// DRAM once, which bounds the pass: kUnroll rows of a lane are in flight, and
// four CTAs an SM (32768 x 48 heads of 128 in bf16: 139 us, 5.8 TB/s, although
// 64 registers a thread spill 56 bytes, 20 in f32; twice the rows and three CTAs
// an SM 152 us; asking for the rows ahead of the cosines 146 to 170 us).  Pairs
// that are read again cost more than twice as much: 367 us with 24 or 40 of the
// 128 values rotated, and 815 us with the backward, which spills 200 bytes there,
// against 398.
constexpr int kNormThreads = 256, kNormWarps = kNormThreads / 32;

template <typename T>
struct NormSide {  // q or k
  const T *x, *dy;
  T *out;
  const float* w;
  int64_t stride;
  int H;
};

template <typename T>
__device__ __forceinline__ NormSide<T> norm_side(const QkNormArgs& a, bool is_q, bool bwd) {
  NormSide<T> s;
  s.x = static_cast<const T*>(is_q ? a.q : a.k);
  s.dy = static_cast<const T*>(is_q ? a.dq_out : a.dk_out);
  s.out = static_cast<T*>(bwd ? (is_q ? a.dq : a.dk) : (is_q ? a.q_out : a.k_out));
  s.w = is_q ? a.qw : a.kw;
  s.stride = is_q ? a.sq : a.sk;
  s.H = is_q ? a.Hq : a.Hk;
  return s;
}

// Where lane l's chunks of a row start (past the row: no such chunk).
template <bool kPaired>
__device__ __forceinline__ void chunk_places(int l, int rot, int (&d)[2]) {
  const int turned = kPaired ? rot / 16 : 0;  // lanes whose chunks turn with each other
  d[0] = l < turned ? 8 * l : 16 * l;
  d[1] = l < turned ? d[0] + rot / 2 : d[0] + 8;
}

// The token's cosines and sines at the places of a lane: a turned value is
// x c - partner s in the first half, x c + partner s in the second.
template <bool kPaired>
struct Turn {
  float c[kPaired ? 1 : 2][8], s[kPaired ? 1 : 2][8];
};

template <bool kPaired>
__device__ __forceinline__ void load_turn(const QkNormArgs& a, int64_t tok, const int (&d)[2], Turn<kPaired>& t) {
  const int half = a.rot / 2;
  const int64_t p = a.pos[tok];
  const bool inside = p >= 0 && p < a.positions;
  if (!inside && a.status && d[0] == 0) atomicOr(a.status, kStatusBadIndex);
  const float nan = __int_as_float(0x7fffffff);
#pragma unroll
  for (int k = 0; k < (kPaired ? 1 : 2); ++k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = d[k] + i;
      t.c[k][i] = 1.0f;
      t.s[k][i] = 0.0f;
      if (e < a.rot) {
        const int64_t at = p * half + (e < half ? e : e - half);
        t.c[k][i] = inside ? a.cos[at] : nan;
        t.s[k][i] = inside ? (kPaired || e >= half ? a.sin[at] : -a.sin[at]) : nan;
      }
    }
  }
}

// A lane's pair of chunks turned by t, or back.
template <bool kBack>
__device__ __forceinline__ void turn_pair(const Turn<true>& t, float (&v)[2][8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = v[0][i], y = v[1][i], c = t.c[0][i], s = kBack ? -t.s[0][i] : t.s[0][i];
    v[0][i] = x * c - y * s;
    v[1][i] = y * c + x * s;
  }
}

template <typename T>
__device__ __forceinline__ float partner(const T* row, int e, int half) {
  return to_f(row[e < half ? e + half : e - half]);
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// blockIdx.x: kNormWarps tokens (one a warp); blockIdx.y: a share of the heads
// of q, then of k.
template <typename T, int kLanes, bool kPaired>
__global__ void __launch_bounds__(kNormThreads, kPaired ? 4 : 2) qk_norm_fwd_kernel(QkNormArgs a, int heads_per_block, int q_shares) {
  constexpr int kRows = 32 / kLanes, kUnroll = 4 / (int)sizeof(T);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t tok = (int64_t)blockIdx.x * kNormWarps + warp;
  if (tok >= a.T) return;
  const bool is_q = (int)blockIdx.y < q_shares;
  const NormSide<T> side = norm_side<T>(a, is_q, false);
  const int mine = lane / kLanes;
  int d[2];
  chunk_places<kPaired>(lane % kLanes, a.rot, d);
  const int half = a.rot / 2;
  const bool turns = a.rot && d[0] < a.rot;
  Turn<kPaired> t;
  if (turns) load_turn<kPaired>(a, tok, d, t);
  float w[2][8];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) w[k][i] = side.w && d[k] < a.K ? side.w[d[k] + i] : 1.0f;
  const float inv_count = a.l2 ? 1.0f : 1.0f / (float)a.K;
  const int h0 = ((int)blockIdx.y - (is_q ? 0 : q_shares)) * heads_per_block, h1 = min(side.H, h0 + heads_per_block);
  const T* rows = side.x + tok * side.stride;
  T* outs = side.out + tok * (int64_t)side.H * a.K;
  for (int hb = h0; hb < h1; hb += kRows * kUnroll) {
    Chunk8<T> raw[kUnroll][2];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = hb + u * kRows + mine;
#pragma unroll
      for (int k = 0; k < 2; ++k) raw[u][k].load(rows + (int64_t)h * a.K + d[k], h < h1 && d[k] < a.K);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = hb + u * kRows + mine;
      float x[2][8];
      raw[u][0].get(x[0]);
      raw[u][1].get(x[1]);
      float sq = 0.0f;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) sq = fmaf(x[k][i], x[k][i], sq);
      sq = row_sum<kLanes>(sq);
      const float r = 1.0f / sqrtf(fmaf(sq, inv_count, a.eps));
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] *= r * w[k][i];
      if constexpr (kPaired) {
        if (turns) turn_pair<false>(t, x);
      } else if (turns && h < h1) {
        const T* row = rows + (int64_t)h * a.K;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int e = d[k] + i;
            if (e < a.rot) {
              const float pw = side.w ? side.w[e < half ? e + half : e - half] : 1.0f;
              x[k][i] = x[k][i] * t.c[k][i] + partner(row, e, half) * (r * pw) * t.s[k][i];
            }
          }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (h < h1 && d[k] < a.K) st_io8(outs + (int64_t)h * a.K + d[k], x[k]);
    }
  }
}

// Persistent CTAs stride over the tokens, the first q_blocks of them for q:
// the weights' gradients add up in registers (a lane's places are the same in
// every row it meets), then over the CTA's rows and warps in shared memory, and
// one row of sums per CTA goes to `partial`, which a second kernel adds in CTA
// order: no atomics, the same bits every time.
constexpr int kNormBwdBlocks = 152 * 4;

template <typename T, int kLanes, bool kPaired>
__global__ void __launch_bounds__(kNormThreads, 2) qk_norm_bwd_kernel(QkNormArgs a, int q_blocks) {
  constexpr int kRows = 32 / kLanes, kUnroll = 4 / (int)sizeof(T);
  __shared__ float sums[kNormWarps][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool is_q = (int)blockIdx.x < q_blocks;
  const NormSide<T> side = norm_side<T>(a, is_q, true);
  const int mine = lane / kLanes;
  int d[2];
  chunk_places<kPaired>(lane % kLanes, a.rot, d);
  const int half = a.rot / 2;
  const bool turns = a.rot && d[0] < a.rot;
  float w[2][8], gw[2][8];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[k][i] = side.w && d[k] < a.K ? side.w[d[k] + i] : 1.0f;
      gw[k][i] = 0.0f;
    }
  const float inv_count = a.l2 ? 1.0f : 1.0f / (float)a.K;
  // a warp takes one token's share of the heads: small packs split the heads too
  const int groups = (side.H + kRows - 1) / kRows;
  const int64_t warps = (int64_t)(is_q ? q_blocks : gridDim.x - q_blocks) * kNormWarps;
  int64_t splits = warps / (a.T > 0 ? a.T : 1);
  splits = splits < 1 ? 1 : splits > groups ? groups : splits;
  const int per = splits ? (int)((groups + splits - 1) / splits) * kRows : 0;
  for (int64_t item = (int64_t)(blockIdx.x - (is_q ? 0 : q_blocks)) * kNormWarps + warp; item < a.T * splits; item += warps) {
    const int64_t tok = item / splits;
    const int h0 = (int)(item - tok * splits) * per, h1 = min(side.H, h0 + per);
    Turn<kPaired> t;
    if (turns) load_turn<kPaired>(a, tok, d, t);
    const T* rows = side.x + tok * side.stride;
    const int64_t tok_at = tok * (int64_t)side.H * a.K;
    for (int hb = h0; hb < h1; hb += kRows * kUnroll) {
      Chunk8<T> rx[kUnroll][2], rg[kUnroll][2];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = hb + u * kRows + mine;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const bool there = h < h1 && d[k] < a.K;
          rx[u][k].load(rows + (int64_t)h * a.K + d[k], there);
          rg[u][k].load(side.dy + tok_at + (int64_t)h * a.K + d[k], there);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = hb + u * kRows + mine;
        float x[2][8], g[2][8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          rx[u][k].get(x[k]);
          rg[u][k].get(g[k]);
        }
        if constexpr (kPaired) {
          if (turns) turn_pair<true>(t, g);
        } else if (turns && h < h1) {
          const T* row = side.dy + tok_at + (int64_t)h * a.K;
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int e = d[k] + i;
              if (e < a.rot) g[k][i] = g[k][i] * t.c[k][i] - partner(row, e, half) * t.s[k][i];
            }
        }
        float sq = 0.0f, dot = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            sq = fmaf(x[k][i], x[k][i], sq);
            dot = fmaf(g[k][i] * w[k][i], x[k][i], dot);
          }
        sq = row_sum<kLanes>(sq);
        dot = row_sum<kLanes>(dot);
        const float r = 1.0f / sqrtf(fmaf(sq, inv_count, a.eps));
        const float f = dot * r * r * inv_count;  // (dn . n) / count, over r
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (h < h1) gw[k][i] = fmaf(g[k][i], x[k][i] * r, gw[k][i]);
            o[i] = r * (g[k][i] * w[k][i] - x[k][i] * f);
          }
          if (h < h1 && d[k] < a.K) st_io8(side.out + tok_at + (int64_t)h * a.K + d[k], o);
        }
      }
    }
  }
  if (!(is_q ? a.dqw : a.dkw)) return;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) gw[k][i] += __shfl_xor_sync(0xffffffffu, gw[k][i], o);
      if (lane < kLanes && d[k] < a.K) sums[warp][d[k] + i] = gw[k][i];
    }
  __syncthreads();
  for (int e = threadIdx.x; e < a.K; e += kNormThreads) {
    float v = 0.0f;
    for (int i = 0; i < kNormWarps; ++i) v += sums[i][e];
    a.partial[(int64_t)blockIdx.x * a.K + e] = v;
  }
}

// One CTA per (weight, 32 places): 8 threads along the CTAs' rows, each adding
// its own stretch in order, then the eight in order.
__global__ void __launch_bounds__(256) qk_norm_sum_kernel(QkNormArgs a, int q_blocks) {
  __shared__ float s[8][32];
  const int which = blockIdx.y, e = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  float* out = which ? a.dkw : a.dqw;
  if (!out) return;
  const int b0 = which ? q_blocks : 0, b1 = which ? kNormBwdBlocks : q_blocks, per = (b1 - b0 + 7) / 8;
  float v = 0.0f;
  if (e < a.K && a.T > 0)
    for (int b = b0 + part * per; b < min(b1, b0 + (part + 1) * per); ++b) v += a.partial[(int64_t)b * a.K + e];
  s[part][threadIdx.x & 31] = v;
  __syncthreads();
  if (part == 0 && e < a.K) {
    for (int p = 1; p < 8; ++p) v += s[p][threadIdx.x & 31];
    out[e] = v;
  }
}

template <typename T, int kLanes, bool kPaired>
cudaError_t run_norm(const QkNormArgs& a, bool bwd, cudaStream_t st) {
  constexpr int kRows = 32 / kLanes;
  if (bwd) {
    int q_blocks = (int)((int64_t)kNormBwdBlocks * a.Hq / (a.Hq + a.Hk));
    if (a.Hq && q_blocks == 0) q_blocks = 1;
    if (a.Hk && q_blocks == kNormBwdBlocks) q_blocks = kNormBwdBlocks - 1;
    if (a.T > 0) qk_norm_bwd_kernel<T, kLanes, kPaired><<<kNormBwdBlocks, kNormThreads, 0, st>>>(a, q_blocks);
    if (a.dqw || a.dkw) qk_norm_sum_kernel<<<dim3((a.K + 31) / 32, 2), 256, 0, st>>>(a, q_blocks);
    return cudaGetLastError();
  }
  if (a.T == 0) return cudaSuccess;
  // few tokens: the heads are split over CTAs as well, down to one pass of a warp
  const int H = a.Hq > a.Hk ? a.Hq : a.Hk, groups = (H + kRows - 1) / kRows;
  const int64_t blocks = (a.T + kNormWarps - 1) / kNormWarps;
  int64_t splits = 152 * 8 / blocks;
  splits = splits < 1 ? 1 : splits > groups ? groups : splits;
  const int per = (int)((groups + splits - 1) / splits) * kRows;
  const int q_shares = (a.Hq + per - 1) / per, k_shares = (a.Hk + per - 1) / per;
  qk_norm_fwd_kernel<T, kLanes, kPaired>
      <<<dim3((unsigned)blocks, (unsigned)(q_shares + k_shares)), kNormThreads, 0, st>>>(a, per, q_shares);
  return cudaGetLastError();
}

template <typename T, bool kPaired>
cudaError_t pick_lanes(const QkNormArgs& a, bool bwd, cudaStream_t st) {
  const int lanes = (a.K + 15) / 16;
  if (lanes <= 2) return run_norm<T, 2, kPaired>(a, bwd, st);
  if (lanes <= 4) return run_norm<T, 4, kPaired>(a, bwd, st);
  if (lanes <= 8) return run_norm<T, 8, kPaired>(a, bwd, st);
  return run_norm<T, 16, kPaired>(a, bwd, st);
}

template <typename T>
cudaError_t pick_norm(const QkNormArgs& a, bool bwd, cudaStream_t st) {
  // chunks come in pairs where the rotated half is whole chunks
  return a.rot % 16 == 0 ? pick_lanes<T, true>(a, bwd, st) : pick_lanes<T, false>(a, bwd, st);
}

}  // namespace

int qk_norm_partial_rows() { return kNormBwdBlocks; }

cudaError_t launch_qk_norm_fwd(const QkNormArgs& a, IO io, cudaStream_t st) {
  return io == IO::BF16 ? pick_norm<__nv_bfloat16>(a, false, st) : pick_norm<float>(a, false, st);
}
cudaError_t launch_qk_norm_bwd(const QkNormArgs& a, IO io, cudaStream_t st) {
  return io == IO::BF16 ? pick_norm<__nv_bfloat16>(a, true, st) : pick_norm<float>(a, true, st);
}

}  // namespace vssm
