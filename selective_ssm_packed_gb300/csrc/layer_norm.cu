// layer_norm.cu -- layer norm over a token's channels or over each group of
// them, with the addition to the residual stream in the same pass; and the
// gradients.
#include "delta.cuh"
#include "linear.h"

namespace vssm {
namespace {

// A row is one group of one token.  kTeam threads share it, 16 values each as
// two chunks of 8 (chunk i of thread l at 8 (l + i kTeam), so that neighbours
// read neighbouring chunks): part of a warp for rows of up to 512 values, a
// whole CTA for longer ones.  The row stays in registers: its mean first, then
// the sum of the squared differences from it (a sum of squares would lose them
// where the mean is far from 0), both in f32.  A team walks over rows of one
// group, so that its weights, and in the backward their gradients, are
// registers too; the next row is on its way while one is worked on.
// The mean that is taken from a row is itself rounded, by up to 2^-20 of a mean
// that may be a thousand deviations away.  What it leaves is the same in all of
// the row: the mean of the centred row, whose sum is exact to 2^-20 of its own
// small size and comes with the squares' in one pass over the team.  It is taken
// from the row, and its square from the variance.
// Everything is read and written once, which bounds the pass: 32768 x 2048 in
// bf16 with the f32 stream 117 us (6.9 TB/s, some of it left in L2), 32 groups of 128 in 4096
// channels 84 us (6.4 TB/s), one row of 2048 4 us.
template <int kTeam>
struct Team {
  static constexpr int kThreads = kTeam <= 32 ? 128 : kTeam, kUnits = kThreads / kTeam;
};
constexpr int kNormSms = 152;
// Threads an SM, which bound a thread's registers (65536 between them): as many
// as leave it enough for two rows on their way and its weights.
template <typename T, bool kRes>
constexpr int fwd_threads() { return sizeof(T) == 2 && !kRes ? 768 : 512; }
template <int kTeam>
constexpr int bwd_threads() { return kTeam >= 256 ? 512 : 384; }

// v[i] summed over the team, in a fixed order.  Over several warps each part of
// a warp's lanes takes one of the sums after the first steps, which spares half
// the shuffles (8192 x 4096 in f32, backward: 145 -> 132 us).  flip: which half of
// the scratch is this sum's; one barrier a sum is enough with two.
template <int kTeam, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], float (*scratch)[4][16], int& flip) {
  static_assert(N == 1 || N == 2 || N == 4, "");
  if constexpr (kTeam <= 32) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int o = kTeam / 2; o >= 1; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  } else {
    constexpr int kWarps = kTeam / 32;
    const int lane = threadIdx.x & 31;
    const bool up = lane & 16, up2 = lane & 8;
    float own = v[0];
    if constexpr (N == 4) {
      const float a = (up ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16);
      const float b = (up ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 16);
      own = (up2 ? b : a) + __shfl_xor_sync(0xffffffffu, up2 ? a : b, 8);
    } else if constexpr (N == 2) {
      own = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16);
    }
#pragma unroll
    for (int o = 16 / N; o >= 1; o >>= 1) own += __shfl_xor_sync(0xffffffffu, own, o);
    if (lane % (32 / N) == 0) scratch[flip][lane / (32 / N)][threadIdx.x >> 5] = own;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += scratch[flip][i][w];
      v[i] = s;
    }
    flip ^= 1;
  }
}

template <int kTeam>
struct Place {  // of a thread: its group's first channel, its chunks in the row, whether they exist
  int local, col0, d[2];
  bool in[2];
  __device__ __forceinline__ Place(const LayerNormArgs& a, int64_t slot) {
    const int l = threadIdx.x % kTeam, width = a.D / a.groups;
    local = threadIdx.x / kTeam;
    col0 = (int)(slot % a.groups) * width;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      d[i] = (l + i * kTeam) * 8;
      in[i] = d[i] < width;
    }
  }
};

// Channels' f32 parameters, or `none` where there are none.
template <int kTeam>
__device__ __forceinline__ void load_params(const float* p, const Place<kTeam>& at, float none, float (&v)[2][8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    Chunk8<float> c;
    c.load(p + at.col0 + at.d[i], p != nullptr && at.in[i]);
    c.get(v[i]);
    if (!p)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = none;
  }
}

// The row's centred values, but for the mean's own rounding.
template <int kTeam>
__device__ __forceinline__ void centre(float (&h)[2][8], const Place<kTeam>& at, float inv_count, float (*scratch)[4][16], int& flip) {
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) s[0] += h[i][j];  // 0 past the row
  team_sum<kTeam>(s, scratch, flip);
  const float mean = s[0] * inv_count;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i][j] = at.in[i] ? h[i][j] - mean : 0.0f;
}

// 1 / the standard deviation, from the centred row's sum of squares and its own mean.
__device__ __forceinline__ float inv_std(float squares, float rest, float inv_count, float eps) {
  const float var = fmaf(-rest, rest, squares * inv_count);
  return 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps);  // below 0 by rounding only; NaN stays
}

template <typename T, bool kRes, int kTeam>
__global__ void __launch_bounds__(Team<kTeam>::kThreads, fwd_threads<T, kRes>() / Team<kTeam>::kThreads)
    layer_norm_fwd_kernel(LayerNormArgs a, int64_t slots) {
  __shared__ float scratch[2][4][16];
  const int64_t slot = (int64_t)blockIdx.x * Team<kTeam>::kUnits + threadIdx.x / kTeam;
  const Place<kTeam> at(a, slot);
  const float inv_count = 1.0f / (float)(a.D / a.groups);
  const int64_t units = a.T * a.groups, tokens = slots / a.groups;  // tokens a step of the team moves on
  float w[2][8], b[2][8];
  load_params(a.weight, at, 1.0f, w);
  load_params(a.bias, at, 0.0f, b);
  Chunk8<T> rx[2];
  Chunk8<float> rr[2];
  int64_t tok = slot / a.groups;
  bool there = slot < slots && tok < a.T;
  auto load = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      rx[i].load(static_cast<const T*>(a.x) + tok * a.sx + at.col0 + at.d[i], there && at.in[i]);
      if (kRes) rr[i].load(a.residual + tok * a.D + at.col0 + at.d[i], there && at.in[i]);
    }
  };
  load();
  int flip = 0;
  for (int64_t base = (int64_t)blockIdx.x * Team<kTeam>::kUnits; base < units; base += slots) {  // the same turns for all of the CTA
    float h[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      rx[i].get(h[i]);
      if (kRes) {
        float r[8];
        rr[i].get(r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] += r[j];
      }
    }
    const int64_t row = tok * a.D + at.col0;
    const bool mine = there;
    tok += tokens;
    there = slot < slots && tok < a.T;
    load();
    if (kRes && a.sum)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (mine && at.in[i]) st_io8(a.sum + row + at.d[i], h[i]);
    centre(h, at, inv_count, scratch, flip);
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[0] = fmaf(h[i][j], h[i][j], s[0]);
        s[1] += h[i][j];
      }
    team_sum<kTeam>(s, scratch, flip);
    const float rest = s[1] * inv_count, r = inv_std(s[0], rest, inv_count, a.eps);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = fmaf((h[i][j] - rest) * r, w[i][j], b[i][j]);
      if (mine && at.in[i]) st_io8(static_cast<T*>(a.out) + row + at.d[i], h[i]);
    }
  }
}

// With c the centred row without its own mean, r = 1 / its standard deviation, n = c r and u = dy w:
//   dh = r (u - mean(u) - n mean(u n)) + dsum
//   dweight = sum over tokens of dy n,  dbias = sum of dy
// One row of sums per team goes to `partial`, which a second kernel adds in
// the teams' order: no atomics, the same bits every time.  32768 x 2048 with the
// stream 152 us (6.2 TB/s), 32 groups of 128 in 4096 channels 145 us (5.5 TB/s: five sums
// a row of 8 threads keep the issue slots 60% busy), the teams' sums 8 us.
template <typename T, typename H, int kTeam>
__global__ void __launch_bounds__(Team<kTeam>::kThreads, bwd_threads<kTeam>() / Team<kTeam>::kThreads)
    layer_norm_bwd_kernel(LayerNormArgs a, int64_t slots) {
  __shared__ float scratch[2][4][16];
  const int64_t slot = (int64_t)blockIdx.x * Team<kTeam>::kUnits + threadIdx.x / kTeam;
  const Place<kTeam> at(a, slot);
  const int width = a.D / a.groups;
  const float inv_count = 1.0f / (float)width;
  const int64_t units = a.T * a.groups, tokens = slots / a.groups;
  float w[2][8], gw[2][8], gb[2][8];
  load_params(a.weight, at, 1.0f, w);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) gw[i][j] = gb[i][j] = 0.0f;
  Chunk8<H> rx[2];
  Chunk8<T> rg[2];
  int64_t tok = slot / a.groups;
  bool there = slot < slots && tok < a.T;
  auto load = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      rx[i].load(static_cast<const H*>(a.x) + tok * a.sx + at.col0 + at.d[i], there && at.in[i]);
      rg[i].load(static_cast<const T*>(a.dout) + tok * a.D + at.col0 + at.d[i], there && at.in[i]);
    }
  };
  load();
  int flip = 0;
  for (int64_t base = (int64_t)blockIdx.x * Team<kTeam>::kUnits; base < units; base += slots) {
    float h[2][8], g[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      rx[i].get(h[i]);
      rg[i].get(g[i]);
    }
    const int64_t row = tok * a.D + at.col0;
    const bool mine = there;
    tok += tokens;
    there = slot < slots && tok < a.T;
    load();
    Chunk8<float> rs[2];
    if (a.dsum)
#pragma unroll
      for (int i = 0; i < 2; ++i) rs[i].load(a.dsum + row + at.d[i], mine && at.in[i]);
    centre(h, at, inv_count, scratch, flip);
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = g[i][j] * w[i][j];
        s[0] = fmaf(h[i][j], h[i][j], s[0]);
        s[1] += u;
        s[2] = fmaf(u, h[i][j], s[2]);
        s[3] += h[i][j];
      }
    team_sum<kTeam>(s, scratch, flip);
    const float rest = s[3] * inv_count, r = inv_std(s[0], rest, inv_count, a.eps);
    const float mean_u = s[1] * inv_count, f = fmaf(-rest, s[1], s[2]) * inv_count * r * r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[i][j] -= rest;
        if (mine) {
          gw[i][j] = fmaf(g[i][j], h[i][j] * r, gw[i][j]);
          gb[i][j] += g[i][j];
        }
        o[j] = r * (fmaf(g[i][j], w[i][j], -mean_u) - h[i][j] * f);
      }
      if (a.dsum) {
        float d[8];
        rs[i].get(d);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] += d[j];
      }
      if (mine && at.in[i]) {
        st_io8(static_cast<T*>(a.dx) + row + at.d[i], o);
        if (a.dresidual) st_io8(a.dresidual + row + at.d[i], o);
      }
    }
  }
  if (slot >= slots || !(a.dweight || a.dbias)) return;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (at.in[i]) {
      float* p = a.partial + slot * 2 * width + at.d[i];
      st_io8(p, gw[i]);
      st_io8(p + width, gb[i]);
    }
}

// blockIdx.x: 32 channels; blockIdx.y: weight or bias.  The teams of a group in
// kSumParts stretches, each added up in order by a warp, then those in order.
constexpr int kSumParts = 32;

__global__ void __launch_bounds__(32 * kSumParts) layer_norm_sum_kernel(LayerNormArgs a, int64_t slots) {
  __shared__ float s[kSumParts][32];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5, width = a.D / a.groups;
  float* out = blockIdx.y ? a.dbias : a.dweight;
  if (!out) return;
  const int64_t rows = a.T > 0 ? slots / a.groups : 0, per = (rows + kSumParts - 1) / kSumParts;
  float v = 0.0f;
  if (col < a.D) {
    const int group = col / width;
    const float* p = a.partial + blockIdx.y * width + (col - group * width);
    const int64_t end = rows < (part + 1) * per ? rows : (part + 1) * per;
#pragma unroll 8
    for (int64_t i = part * per; i < end; ++i) v += p[(i * a.groups + group) * 2 * width];
  }
  s[part][threadIdx.x & 31] = v;
  __syncthreads();
  if (part == 0 && col < a.D) {
#pragma unroll
    for (int p = 1; p < kSumParts; ++p) v += s[p][threadIdx.x & 31];
    out[col] = v;
  }
}

int team_of(int width) {
  int t = 4;
  while (t * 16 < width) t *= 2;
  return t;
}

// Teams that walk, a multiple of the groups: as many as an SM's threads allow, no more than there are rows.
int64_t slots_of(int64_t T, int D, int groups, int sm_threads) {
  const int64_t most = (int64_t)kNormSms * sm_threads / team_of(D / groups), units = T * groups;
  const int64_t use = units < most ? units : most;
  return use < groups ? groups : use / groups * groups;
}

}  // namespace

int64_t layer_norm_slots(int64_t T, int D, int groups) {
  return slots_of(T, D, groups, team_of(D / groups) >= 256 ? bwd_threads<256>() : bwd_threads<128>());
}

namespace {

template <typename F>
cudaError_t with_team(int width, F f) {
  switch (team_of(width)) {
    case 4: return f(std::integral_constant<int, 4>());
    case 8: return f(std::integral_constant<int, 8>());
    case 16: return f(std::integral_constant<int, 16>());
    case 32: return f(std::integral_constant<int, 32>());
    case 64: return f(std::integral_constant<int, 64>());
    case 128: return f(std::integral_constant<int, 128>());
    case 256: return f(std::integral_constant<int, 256>());
    default: return f(std::integral_constant<int, 512>());
  }
}

template <typename T, bool kRes>
cudaError_t run_fwd(const LayerNormArgs& a, cudaStream_t st) {
  return with_team(a.D / a.groups, [&](auto team) {
    constexpr int kTeam = decltype(team)::value, kUnits = Team<kTeam>::kUnits;
    const int64_t slots = slots_of(a.T, a.D, a.groups, fwd_threads<T, kRes>());
    layer_norm_fwd_kernel<T, kRes, kTeam><<<(unsigned)((slots + kUnits - 1) / kUnits), Team<kTeam>::kThreads, 0, st>>>(a, slots);
    return cudaGetLastError();
  });
}

template <typename T, typename H>
cudaError_t run_bwd(const LayerNormArgs& a, cudaStream_t st) {
  return with_team(a.D / a.groups, [&](auto team) {
    constexpr int kTeam = decltype(team)::value, kUnits = Team<kTeam>::kUnits;
    const int64_t slots = layer_norm_slots(a.T, a.D, a.groups);
    if (a.T > 0)
      layer_norm_bwd_kernel<T, H, kTeam><<<(unsigned)((slots + kUnits - 1) / kUnits), Team<kTeam>::kThreads, 0, st>>>(a, slots);
    if (a.dweight || a.dbias) layer_norm_sum_kernel<<<dim3((unsigned)((a.D + 31) / 32), 2), 32 * kSumParts, 0, st>>>(a, slots);
    return cudaGetLastError();
  });
}

}  // namespace


cudaError_t launch_layer_norm_fwd(const LayerNormArgs& a, IO io, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  if (io == IO::BF16) return a.residual ? run_fwd<__nv_bfloat16, true>(a, st) : run_fwd<__nv_bfloat16, false>(a, st);
  return a.residual ? run_fwd<float, true>(a, st) : run_fwd<float, false>(a, st);
}

cudaError_t launch_layer_norm_bwd(const LayerNormArgs& a, IO io, bool x_f32, cudaStream_t st) {
  if (io == IO::F32) return run_bwd<float, float>(a, st);
  return x_f32 ? run_bwd<__nv_bfloat16, float>(a, st) : run_bwd<__nv_bfloat16, __nv_bfloat16>(a, st);
}

}  // namespace vssm
