// linear_plan.cu -- linear attention: the plan of a pack, the scan over a
// sequence's segments, the decays' gradient, and the sum over shared heads.
#include "linear.cuh"

namespace vssm {
namespace {

// ------------------------------------------------------------------ plan
// One CTA: a pack has a few thousand sequences.  Running sums of the segments
// and inner segments give each sequence its places; the order is by length
// class (of 64, longest first) and within a class left to chance: it decides
// when a segment is walked, not how.  5 us, of which 2 to 3 are a launch's.
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int length_class(int len, int seg) {
  return 63 - min(63, (int)((int64_t)len * 63 / seg));
}

__global__ void __launch_bounds__(kPlanThreads) lin_plan_kernel(LinArgs a) {
  __shared__ int2 warp_sum[kPlanThreads / 32];
  __shared__ int carry_segs, carry_inner, splits, bad, classes[64];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, S = a.num_seqs, seg = a.seg;
  if (t == 0) carry_segs = carry_inner = splits = bad = 0;
  if (t < 64) classes[t] = 0;
  __syncthreads();
  for (int base = 0; base < S; base += kPlanThreads) {
    const int s = base + t;
    if (s < S) {
      const int64_t lo = a.cu[s], hi = a.cu[s + 1];
      if ((s == 0 && lo != 0) || hi < lo || lo < 0 || hi > a.T || (s == S - 1 && hi != a.T)) bad = 1;
    }
  }
  __syncthreads();
  if (bad || (S == 0 && a.T > 0)) {
    if (t == 0) {
      a.info[0] = a.info[1] = a.info[2] = -1;
      *a.status = kStatusBadCu;
    }
    return;
  }
  for (int base = 0; base < S; base += kPlanThreads) {
    const int s = base + t;
    int n = 0, lo = 0, len = 0;
    if (s < S) {
      lo = a.cu[s];
      len = a.cu[s + 1] - lo;
      n = len > 0 ? (len - 1) / seg + 1 : 1;  // an empty sequence still has a state
      atomicAdd(&classes[length_class(len - (n - 1) * seg, seg)], 1);
      if (n > 1) atomicAdd(&classes[0], n - 1);
    }
    int2 incl = make_int2(n, s < S ? n - 1 : 0);
    const int2 own = incl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
      if (lane >= o) {
        incl.x += x;
        incl.y += y;
      }
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int first = carry_segs + incl.x - own.x, inner = carry_inner + incl.y - own.y;
    for (int w = 0; w < warp; ++w) {
      first += warp_sum[w].x;
      inner += warp_sum[w].y;
    }
    if (s < S) {
      for (int p = 0; p < n; ++p) {
        a.table[first + p] = make_int4(s, lo + p * seg, min(seg, len - p * seg),
                                       (p == 0 ? kLinFirst : 0) | (p + 1 == n ? kLinLast : 0) |
                                           (int)((unsigned)(inner + p) << kLinPlaceShift));
        if (p + 1 < n) a.inner[inner + p] = first + p;
      }
      if (n > 1) a.split[atomicAdd(&splits, 1)] = make_int2(inner, n - 1);
    }
    __syncthreads();
    if (t == kPlanThreads - 1) {
      carry_segs = first + own.x;
      carry_inner = inner + own.y;
    }
    __syncthreads();
  }
  if (t == 0) {
    a.info[0] = carry_segs;
    a.info[1] = carry_inner;
    a.info[2] = splits;
    *a.status = 0;
    int at = 0;
    for (int i = 0; i < 64; ++i) {
      const int k = classes[i];
      classes[i] = at;
      at += k;
    }
  }
  __threadfence_block();
  __syncthreads();
  for (int i = t; i < carry_segs; i += kPlanThreads) a.order[atomicAdd(&classes[length_class(a.table[i].z, seg)], 1)] = i;
}

// ------------------------------------------------------------------ scan over segments
// A thread has four elements of one (sequence, head, role): the state before
// each segment (or, in reversed time, its gradient behind it) from what each
// adds.  blockIdx.x: sequence of several segments, blocks of the state;
// blockIdx.y: head; blockIdx.z: role.
constexpr int kScanAhead = 4;

__global__ void __launch_bounds__(256) lin_scan_kernel(LinArgs a, int blocks) {
  const int s = blockIdx.x / blocks, h = blockIdx.y;
  if (s >= a.info[2]) return;
  const LinRole& role = a.role[blockIdx.z];
  const int64_t size = (int64_t)a.K * a.V, at = ((int64_t)(blockIdx.x % blocks) * 256 + threadIdx.x) * 4;
  if (at >= size) return;
  const int2 split = a.split[s];
  const int step = role.back ? -1 : 1;
  const int64_t from = role.back ? split.x + split.y - 1 : split.x;
  auto place = [&](int i) { return reinterpret_cast<float4*>(role.slots + ((from + (int64_t)i * step) * a.Hv + h) * size + at); };
  float4 run = *place(0);
  for (int i = 1; i < split.y; i += kScanAhead) {
    float4 add[kScanAhead];
    float f[kScanAhead];
#pragma unroll
    for (int u = 0; u < kScanAhead; ++u)
      if (i + u < split.y) {
        add[u] = *place(i + u);
        f[u] = role.decay[(from + (int64_t)(i + u) * step) * a.Hv + h];
      }
#pragma unroll
    for (int u = 0; u < kScanAhead; ++u)
      if (i + u < split.y) {
        run = make_float4(fmaf(f[u], run.x, add[u].x), fmaf(f[u], run.y, add[u].y), fmaf(f[u], run.z, add[u].z),
                          fmaf(f[u], run.w, add[u].w));
        *place(i + u) = run;
      }
  }
}

// ------------------------------------------------------------------ gradient of the decays
// One CTA per (segment, head): a thread has a stretch of the segment's tokens,
// which it sums up first and then walks from its end.  Sums are of two floats: a
// token's dg is the sum of all later differences, in which most cancels.
// 32768 tokens, 32 heads: 25 us for 21 MB, two CTAs an SM (44 with rows of all heads and two heads to a
// CTA of 1024, 37 with a CTA alone on its SM).
constexpr int kDgThreads = 512, kDgWarps = kDgThreads / 32, kDgPer = kLinMaxSegment / kDgThreads;

__device__ __forceinline__ Pair shfl_down(Pair v, int o) {
  return Pair{__shfl_down_sync(0xffffffffu, v.hi, o), __shfl_down_sync(0xffffffffu, v.lo, o)};
}
__device__ __forceinline__ float sum_behind(float v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float w = __shfl_down_sync(0xffffffffu, v, o);
    if (lane + o < 32) v += w;
  }
  return v;
}
// The sum over this lane and those behind it.
__device__ __forceinline__ Pair sum_behind(Pair v, int lane) {
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const Pair w = shfl_down(v, o);
    if (lane + o < 32) v = add(v, w);
  }
  return v;
}

template <int kParts>
__global__ void __launch_bounds__(kDgThreads, 2) lin_dg_kernel(LinArgs a, int tiles) {
  __shared__ Pair sums[kDgWarps];
  __shared__ float sizes[kDgWarps];
  const int seg = blockIdx.x, h = blockIdx.y;
  if (seg >= a.info[0]) return;
  const int4 entry = a.table[seg];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int per = (entry.z + kDgThreads - 1) / kDgThreads, lo = min(entry.z, t * per), n = min(entry.z - lo, per);
  const int64_t plane = a.T * a.Hv, first = h * a.T + entry.y + lo;
  Pair d[kDgPer], own{0.0f, 0.0f};
  float size[kDgPer], own_size = 0.0f;  // |rho| + |sigma|
#pragma unroll
  for (int i = 0; i < kDgPer; ++i) {
    d[i] = Pair{0.0f, 0.0f};
    size[i] = 0.0f;
    if (i >= n) continue;
    const int64_t at = first + i;
#pragma unroll
    for (int p = 0; p < kParts; ++p) d[i] = add(d[i], Pair{a.role[0].dots[p * plane + at], 0.0f});
    size[i] = fabsf(d[i].hi);
    Pair sigma{0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < kParts; ++p) sigma = add(sigma, Pair{-a.role[1].dots[p * plane + at], 0.0f});
    size[i] += fabsf(sigma.hi);
    d[i] = add(d[i], sigma);
  }
#pragma unroll
  for (int i = kDgPer - 1; i >= 0; --i) {
    own = add(own, d[i]);
    own_size += size[i];
  }
  const Pair incl = sum_behind(own, lane);
  const float incl_size = sum_behind(own_size, lane);
  if (lane == 0) sums[warp] = incl;
  if (lane == 0) sizes[warp] = incl_size;
  __syncthreads();
  if (warp == 0) {
    const Pair v = sum_behind(lane < kDgWarps ? sums[lane] : Pair{0.0f, 0.0f}, lane);
    const float w = sum_behind(lane < kDgWarps ? sizes[lane] : 0.0f, lane);
    if (lane < kDgWarps) sums[lane] = v;
    if (lane < kDgWarps) sizes[lane] = w;
  }
  __syncthreads();
  Pair run = shfl_down(incl, 1), total{0.0f, 0.0f}, gap = sums[0];  // gap: what the sum over all tokens is off by
  if (lane == 31) run = Pair{0.0f, 0.0f};
  if (warp + 1 < kDgWarps) run = add(run, sums[warp + 1]);
  float behind = __shfl_down_sync(0xffffffffu, incl_size, 1);
  if (lane == 31) behind = 0.0f;
  if (warp + 1 < kDgWarps) behind += sizes[warp + 1];
  const float *at_end = a.role[0].cross + ((int64_t)seg * a.Hv + h) * tiles;
  const float *at_begin = !(entry.w & kLinFirst) ? at_end - (int64_t)a.Hv * tiles
                          : a.role[1].cross      ? a.role[1].cross + ((int64_t)seg * a.Hv + h) * tiles
                                                 : nullptr;
  for (int i = 0; i < tiles; ++i) {
    run = add(run, Pair{at_end[i], 0.0f});
    gap = add(gap, Pair{at_end[i], 0.0f});
    if (at_begin) gap = add(gap, Pair{-at_begin[i], 0.0f});
  }
  // A token's part in it goes by the size of its terms: one without any has no error, and one of 1000 times the others'
  // size has it all.
  float share = (gap.hi + gap.lo) / sizes[0];
  if (!isfinite(share)) share = 0.0f;  // tokens behind what is not finite keep their sums
#pragma unroll
  for (int i = kDgPer - 1; i >= 0; --i) {
    if (i >= n) continue;
    run = add(run, d[i]);
    behind += size[i];
    const float off = share * behind;
    if (a.g_token) a.dg[((int64_t)entry.y + lo + i) * a.Hv + h] = run.hi + (run.lo - off);
    else total = add(total, Pair{run.hi, run.lo - off});
  }
  if (a.g_token) return;
  total = sum_behind(total, lane);
  __syncthreads();
  if (lane == 0) sums[warp] = total;
  __syncthreads();
  if (warp == 0) {
    total = sum_behind(lane < kDgWarps ? sums[lane] : Pair{0.0f, 0.0f}, lane);
    if (lane == 0) a.seg_dg[(int64_t)seg * a.Hv + h] = (double)total.hi + (double)total.lo;
  }
}

// One decay a head: the segments' sums, in order.
__global__ void __launch_bounds__(256) lin_dg_head_kernel(LinArgs a) {
  __shared__ double sums[8][32];
  const int h = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5, n = max(a.info[0], 0), per = (n + 7) / 8;
  double v = 0.0;
  if (h < a.Hv)
    for (int i = part * per; i < min(n, (part + 1) * per); ++i) v += a.seg_dg[(int64_t)i * a.Hv + h];
  sums[part][threadIdx.x & 31] = v;
  __syncthreads();
  if (part == 0 && h < a.Hv && a.info[0] >= 0) {
    for (int p = 1; p < 8; ++p) v += sums[p][threadIdx.x & 31];
    a.dg[h] = (float)v;
  }
}

// ------------------------------------------------------------------ shared heads
// dq and dk: the value heads' parts that share a head, added in order.
// blockIdx.y: dq or dk.  A thread has four values.  16384 tokens, 64 value heads on 8
// of 128: 163 us for 1.1 GB, 6.9 TB/s.
template <typename T>
__global__ void __launch_bounds__(256) lin_head_sum_kernel(LinArgs a, int64_t count) {
  if (a.info[0] < 0) return;
  const float* part = blockIdx.y ? a.dk_part : a.dq_part;
  T* out = static_cast<T*>(blockIdx.y ? a.dk : a.dq);
  const int rep = a.Hv / a.Hk;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    const int64_t head = i * 4 / a.K, d = i * 4 - head * a.K;  // (token, shared head)
    const float* p = part + head * rep * a.K + d;
    float4 v = *reinterpret_cast<const float4*>(p);
    for (int r = 1; r < rep; ++r) {
      const float4 f = *reinterpret_cast<const float4*>(p + (int64_t)r * a.K);
      v.x += f.x; v.y += f.y; v.z += f.z; v.w += f.w;
    }
    st_io2(out + i * 4, make_float2(v.x, v.y));
    st_io2(out + i * 4 + 2, make_float2(v.z, v.w));
  }
}

}  // namespace

cudaError_t launch_lin_plan(const LinArgs& a, cudaStream_t st) {
  lin_plan_kernel<<<1, kPlanThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_lin_scan(const LinArgs& a, int roles, cudaStream_t st) {
  if (a.max_inner == 0) return cudaSuccess;
  const int blocks = (a.K * a.V / 4 + 255) / 256;
  lin_scan_kernel<<<dim3((unsigned)(a.max_inner * blocks), (unsigned)a.Hv, (unsigned)roles), 256, 0, st>>>(a, blocks);
  return cudaGetLastError();
}

cudaError_t launch_lin_dg(const LinArgs& a, IO io, cudaStream_t st) {
  const dim3 grid((unsigned)a.max_segs, (unsigned)a.Hv);
  const int tiles = lin_ctas(io, a.K);
  if (a.max_segs > 0) {
    if (io == IO::BF16) lin_dg_kernel<2><<<grid, kDgThreads, 0, st>>>(a, tiles);
    else if (tiles == 1) lin_dg_kernel<kLinParts><<<grid, kDgThreads, 0, st>>>(a, tiles);
    else lin_dg_kernel<2 * kLinParts><<<grid, kDgThreads, 0, st>>>(a, tiles);
  }
  if (!a.g_token) lin_dg_head_kernel<<<(unsigned)((a.Hv + 31) / 32), 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_lin_head_sum(const LinArgs& a, IO io, cudaStream_t st) {
  const int64_t count = a.T * a.Hk * a.K / 4;
  if (count == 0) return cudaSuccess;
  const dim3 grid((unsigned)grid_stride_blocks(count), 2);
  if (io == IO::BF16) lin_head_sum_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a, count);
  else lin_head_sum_kernel<float><<<grid, 256, 0, st>>>(a, count);
  return cudaGetLastError();
}

}  // namespace vssm
