// qk_norm.cu -- queries and keys normalised for each head, and rotated by
// their position, in one pass; and the gradients.
#include "delta.cuh"

namespace vssm {
namespace {

// A row is one head of one token: K values.  Lanes hold 8 neighbouring values
// each, kLanes lanes a row, so a warp works on 32 / kLanes heads of one token
// at a time and keeps the token's cosines and sines in registers over all of
// them.  The rotation turns value i of the first half of the rotated width
// with value i + half; each lane reads its partners' values for itself (they
// are in L1: the row is being read anyway) instead of exchanging normalised
// ones, so the reads of a row all start at once.  Every value is read from
// and written to DRAM once, which bounds the pass.
template <typename T>
__device__ __forceinline__ void partner8(const T* row, int d, int half, bool aligned, float (&v)[8]) {
  // values d .. d + 7 of the row's other half, where d + i < 2 half
  if (aligned) {
    ld_io8(row + (d < half ? d + half : d - half), v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = d + i;
      v[i] = e < 2 * half ? to_f(row[e < half ? e + half : e - half]) : 0.0f;
    }
  }
}

// The token's cosines and signed sines at this lane's 8 places: the rotated
// value is x c + partner s.  Places past the rotated width get 1 and 0.
__device__ __forceinline__ void load_turn(const QkNormArgs& a, int64_t tok, int d, float (&c)[8], float (&s)[8]) {
  const int half = a.rot / 2;
  const int64_t p = a.pos[tok];
  const bool inside = p >= 0 && p < a.positions;
  if (!inside && a.status && d == 0) atomicOr(a.status, kStatusBadIndex);
  const float nan = __int_as_float(0x7fffffff);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = d + i;
    c[i] = 1.0f;
    s[i] = 0.0f;
    if (e < a.rot) {
      const int64_t at = p * half + (e < half ? e : e - half);
      c[i] = inside ? a.cos[at] : nan;
      s[i] = inside ? (e < half ? -a.sin[at] : a.sin[at]) : nan;
    }
  }
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

constexpr int kNormThreads = 256;

// blockIdx.x: 8 tokens (one a warp), blockIdx.y: a share of the heads.
template <typename T, int kLanes>
__global__ void __launch_bounds__(kNormThreads) qk_norm_fwd_kernel(QkNormArgs a, int heads_per_block) {
  constexpr int kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t tok = (int64_t)blockIdx.x * (kNormThreads / 32) + warp;
  if (tok >= a.T) return;
  const int H = a.Hq + a.Hk;
  const int d = (lane % kLanes) * 8, mine = lane / kLanes;
  const bool in = d < a.K;
  const int half = a.rot / 2;
  const bool turns = in && d < a.rot, aligned = half % 8 == 0;
  float c[8], s[8], wq[8], wk[8];
  if (a.rot && in) load_turn(a, tok, d, c, s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    wq[i] = a.qw && in ? a.qw[d + i] : 1.0f;
    wk[i] = a.kw && in ? a.kw[d + i] : 1.0f;
  }
  const float count = a.l2 ? 1.0f : (float)a.K;
  const int h0 = blockIdx.y * heads_per_block, h1 = min(H, h0 + heads_per_block);
#pragma unroll 2
  for (int hb = h0; hb < h1; hb += kRows) {
    const int h = hb + mine;
    const bool live = h < h1 && in;
    const bool is_q = h < a.Hq;
    const T* src = is_q ? static_cast<const T*>(a.q) + tok * a.sq + (int64_t)h * a.K
                        : static_cast<const T*>(a.k) + tok * a.sk + (int64_t)(h - a.Hq) * a.K;
    T* dst = is_q ? static_cast<T*>(a.q_out) + (tok * a.Hq + h) * a.K
                  : static_cast<T*>(a.k_out) + (tok * a.Hk + (h - a.Hq)) * a.K;
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0}, y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (live) ld_io8(src + d, x);
    if (live && turns) partner8(src, d, half, aligned, y);
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fmaf(x[i], x[i], sq);
    sq = row_sum<kLanes>(sq);
    const float r = 1.0f / sqrtf(sq / count + a.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= r * (is_q ? wq[i] : wk[i]);
    if (live && turns) {
      const float* wp = is_q ? a.qw : a.kw;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = d + i;
        if (e < a.rot) {
          const float pw = wp ? wp[e < half ? e + half : e - half] : 1.0f;
          x[i] = x[i] * c[i] + y[i] * (r * pw) * s[i];
        }
      }
    }
    if (live) st_io8(dst + d, x);
  }
}

// Persistent CTAs stride over the tokens: the weights' gradients add up in
// registers (a lane's 8 places are the same in every row it meets), then over
// the CTA's rows and warps in shared memory, and one row of sums per CTA goes
// to `partial`, which a second kernel adds in CTA order: no atomics, the same
// bits every time.
constexpr int kNormBwdBlocks = 152 * 4;

template <typename T, int kLanes>
__global__ void __launch_bounds__(kNormThreads) qk_norm_bwd_kernel(QkNormArgs a) {
  constexpr int kRows = 32 / kLanes, kWarps = kNormThreads / 32;
  __shared__ float sums[kWarps][2][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = a.Hq + a.Hk;
  const int d = (lane % kLanes) * 8, mine = lane / kLanes;
  const bool in = d < a.K;
  const int half = a.rot / 2;
  const bool turns = in && d < a.rot, aligned = half % 8 == 0;
  float gq[8], gk[8], wq[8], wk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    gq[i] = gk[i] = 0.0f;
    wq[i] = a.qw && in ? a.qw[d + i] : 1.0f;
    wk[i] = a.kw && in ? a.kw[d + i] : 1.0f;
  }
  const float inv_count = a.l2 ? 1.0f : 1.0f / (float)a.K;
  // a warp takes one token's share of the heads: small packs split the heads too
  const int groups = (H + kRows - 1) / kRows;
  const int64_t warps = (int64_t)gridDim.x * kWarps;
  int64_t splits = warps / (a.T > 0 ? a.T : 1);
  splits = splits < 1 ? 1 : splits > groups ? groups : splits;
  const int per = (int)((groups + splits - 1) / splits) * kRows;
  for (int64_t item = (int64_t)blockIdx.x * kWarps + warp; item < a.T * splits; item += warps) {
    const int64_t tok = item / splits;
    const int h0 = (int)(item - tok * splits) * per, h1 = min(H, h0 + per);
    float c[8], s[8];
    if (a.rot && in) load_turn(a, tok, d, c, s);
#pragma unroll 2
    for (int hb = h0; hb < h1; hb += kRows) {
      const int h = hb + mine;
      const bool live = h < h1 && in;
      const bool is_q = h < a.Hq;
      const int64_t at = is_q ? (tok * a.Hq + h) * a.K : (tok * a.Hk + (h - a.Hq)) * a.K;
      const T* src = is_q ? static_cast<const T*>(a.q) + tok * a.sq + (int64_t)h * a.K
                          : static_cast<const T*>(a.k) + tok * a.sk + (int64_t)(h - a.Hq) * a.K;
      const T* dsrc = (is_q ? static_cast<const T*>(a.dq_out) : static_cast<const T*>(a.dk_out)) + at;
      float x[8] = {0, 0, 0, 0, 0, 0, 0, 0}, g[8] = {0, 0, 0, 0, 0, 0, 0, 0}, y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (live) {
        ld_io8(src + d, x);
        ld_io8(dsrc + d, g);
      }
      if (live && turns) {
        partner8(dsrc, d, half, aligned, y);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (d + i < a.rot) g[i] = g[i] * c[i] - y[i] * s[i];  // turned back
      }
      float sq = 0.0f, dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sq = fmaf(x[i], x[i], sq);
        dot = fmaf(g[i] * (is_q ? wq[i] : wk[i]), x[i], dot);
      }
      sq = row_sum<kLanes>(sq);
      dot = row_sum<kLanes>(dot);
      const float r = 1.0f / sqrtf(sq * inv_count + a.eps);
      const float f = dot * r * r * inv_count;  // (dn . n) / count, over r
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float gn = g[i] * (x[i] * r);
        if (live) (is_q ? gq[i] : gk[i]) += gn;
        o[i] = r * (g[i] * (is_q ? wq[i] : wk[i]) - x[i] * f);
      }
      if (live) st_io8((is_q ? static_cast<T*>(a.dq) : static_cast<T*>(a.dk)) + at + d, o);
    }
  }
  if (!a.dqw && !a.dkw) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1) {
      gq[i] += __shfl_xor_sync(0xffffffffu, gq[i], o);
      gk[i] += __shfl_xor_sync(0xffffffffu, gk[i], o);
    }
    if (lane < kLanes) {
      sums[warp][0][d + i] = gq[i];
      sums[warp][1][d + i] = gk[i];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.K; i += kNormThreads) {
    const int which = i / a.K, e = i - which * a.K;
    float v = 0.0f;
    for (int w = 0; w < kWarps; ++w) v += sums[w][which][e];
    a.partial[((int64_t)blockIdx.x * 2 + which) * a.K + e] = v;
  }
}

// One CTA per (weight, 32 places): 8 threads along the CTAs' rows, each adding
// its own stretch in order, then the eight in order.
__global__ void __launch_bounds__(256) qk_norm_sum_kernel(QkNormArgs a) {
  __shared__ float s[8][32];
  const int which = blockIdx.y, e = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  float* out = which ? a.dkw : a.dqw;
  if (!out) return;
  constexpr int kPer = kNormBwdBlocks / 8;
  float v = 0.0f;
  if (e < a.K && a.T > 0)
    for (int b = part * kPer; b < (part + 1) * kPer; ++b) v += a.partial[((int64_t)b * 2 + which) * a.K + e];
  s[part][threadIdx.x & 31] = v;
  __syncthreads();
  if (part == 0 && e < a.K) {
    for (int p = 1; p < 8; ++p) v += s[p][threadIdx.x & 31];
    out[e] = v;
  }
}

template <typename T, int kLanes>
cudaError_t run_norm(const QkNormArgs& a, bool bwd, cudaStream_t st) {
  constexpr int kRows = 32 / kLanes;
  if (bwd) {
    if (a.T > 0) qk_norm_bwd_kernel<T, kLanes><<<kNormBwdBlocks, kNormThreads, 0, st>>>(a);
    if (a.dqw || a.dkw) qk_norm_sum_kernel<<<dim3((a.K + 31) / 32, 2), 256, 0, st>>>(a);
    return cudaGetLastError();
  }
  if (a.T == 0) return cudaSuccess;
  // few tokens: the heads are split over CTAs as well, down to one pass of a warp
  const int H = a.Hq + a.Hk, groups = (H + kRows - 1) / kRows;
  const int64_t blocks = (a.T + kNormThreads / 32 - 1) / (kNormThreads / 32);
  int64_t splits = 152 * 8 / blocks;
  splits = splits < 1 ? 1 : splits > groups ? groups : splits;
  const int per = (int)((groups + splits - 1) / splits) * kRows;
  qk_norm_fwd_kernel<T, kLanes><<<dim3((unsigned)blocks, (unsigned)((H + per - 1) / per)), kNormThreads, 0, st>>>(a, per);
  return cudaGetLastError();
}

template <typename T>
cudaError_t pick_norm(const QkNormArgs& a, bool bwd, cudaStream_t st) {
  const int lanes = a.K / 8;
  if (lanes <= 2) return run_norm<T, 2>(a, bwd, st);
  if (lanes <= 4) return run_norm<T, 4>(a, bwd, st);
  if (lanes <= 8) return run_norm<T, 8>(a, bwd, st);
  if (lanes <= 16) return run_norm<T, 16>(a, bwd, st);
  return run_norm<T, 32>(a, bwd, st);
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
