// linear_step.cu -- one token of linear attention with a decay for each head,
// for each of many sequences, against a pool of states.
#include "delta.cuh"
#include "linear.h"

namespace vssm {
namespace {

// One CTA of 256 threads per (token, value head, kCols state columns): kCols / 4
// threads along the columns (float4 each), the others along the state rows, so
// that a thread has its whole share of the state (up to 8 rows) in flight at
// once and in registers until it is written back:
//   S = exp(g) S + k v^T,  o = scale S^T q.
// The state is read and written once, which is all the traffic that counts: 256
// tokens, 32 heads of 128 x 128, 177 us, 6.1 TB/s; one token 6 us.
constexpr int kStepThreads = 256;

template <typename T, int kCols>
__global__ void __launch_bounds__(kStepThreads, 4) lin_step_kernel(LinStepArgs a) {
  constexpr int kAlong = kCols / 4, kStep = kStepThreads / kAlong, kPer = kLinMaxK / kStep;
  __shared__ float part[8][kCols];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int cx = t % kAlong, ry = t / kAlong;
  const int slabs = (a.V + kCols - 1) / kCols;
  const int slab = blockIdx.x % slabs;
  const int h = blockIdx.x / slabs % a.Hv;
  const int64_t b = blockIdx.x / slabs / a.Hv;
  const int col = slab * kCols + cx * 4;
  T* out = static_cast<T*>(a.out) + (b * a.Hv + h) * a.V;
  const int64_t slot = a.indices ? (int64_t)a.indices[b] : b;
  if (slot < 0 || slot >= a.slots) {  // a padded entry, or an index outside the pool
    const bool outside = slot >= a.slots;
    if (outside && t == 0 && a.status) atomicOr(a.status, kStatusBadIndex);
    const int c = slab * kCols + t;
    if (t < kCols && c < a.V) out[c] = from_f<T>(outside ? __int_as_float(0x7fffffff) : 0.0f);
    return;
  }
  float* state = a.states + (slot * a.Hv + h) * (int64_t)a.K * a.V;
  const int kh = h / (a.Hv / a.Hk);
  const T* kp = static_cast<const T*>(a.k) + b * a.sk + (int64_t)kh * a.K;
  const T* qp = static_cast<const T*>(a.q) + b * a.sq + (int64_t)kh * a.K;

  float4 s[kPer];
  float kv[kPer], qv[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int row = ry + kStep * i;
    s[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    kv[i] = qv[i] = 0.0f;
    if (row < a.K) {
      if (col < a.V) s[i] = __ldcs(reinterpret_cast<const float4*>(state + (int64_t)row * a.V + col));
      kv[i] = to_f(kp[row]);
      qv[i] = to_f(qp[row]);
    }
  }
  const float alpha = exp_f(a.g[b * a.g_token + h]);
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f), o = v;
  if (col < a.V) v = ld_io4(static_cast<const T*>(a.v) + b * a.sv + (int64_t)h * a.V + col);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    s[i].x = fmaf(kv[i], v.x, s[i].x * alpha); s[i].y = fmaf(kv[i], v.y, s[i].y * alpha);
    s[i].z = fmaf(kv[i], v.z, s[i].z * alpha); s[i].w = fmaf(kv[i], v.w, s[i].w * alpha);
    o.x = fmaf(qv[i], s[i].x, o.x); o.y = fmaf(qv[i], s[i].y, o.y);
    o.z = fmaf(qv[i], s[i].z, o.z); o.w = fmaf(qv[i], s[i].w, o.w);
    const int row = ry + kStep * i;
    if (row < a.K && col < a.V) __stcs(reinterpret_cast<float4*>(state + (int64_t)row * a.V + col), s[i]);
  }
  // over the warp's row groups, then over the warps
#pragma unroll
  for (int d = kAlong; d <= 16; d <<= 1) {
    o.x += __shfl_xor_sync(0xffffffffu, o.x, d); o.y += __shfl_xor_sync(0xffffffffu, o.y, d);
    o.z += __shfl_xor_sync(0xffffffffu, o.z, d); o.w += __shfl_xor_sync(0xffffffffu, o.w, d);
  }
  if (lane < kAlong) *reinterpret_cast<float4*>(&part[warp][cx * 4]) = o;
  __syncthreads();
  if (ry == 0 && col < a.V) {
    o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(&part[i][cx * 4]);
      o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
    }
    st_io2(out + col, make_float2(a.scale * o.x, a.scale * o.y));
    st_io2(out + col + 2, make_float2(a.scale * o.z, a.scale * o.w));
  }
}

}  // namespace

cudaError_t launch_lin_step(const LinStepArgs& a, IO io, cudaStream_t st) {
  if (a.B == 0) return cudaSuccess;
  // wide CTAs have twice the bytes in flight, once there are enough of them
  const int64_t heads = a.B * a.Hv, wide = heads * ((a.V + 63) / 64), narrow = heads * ((a.V + 31) / 32);
  const bool use_wide = wide >= 152 * 4;
  const unsigned blocks = (unsigned)(use_wide ? wide : narrow);
  if (io == IO::BF16) {
    if (use_wide) lin_step_kernel<__nv_bfloat16, 64><<<blocks, kStepThreads, 0, st>>>(a);
    else lin_step_kernel<__nv_bfloat16, 32><<<blocks, kStepThreads, 0, st>>>(a);
  } else {
    if (use_wide) lin_step_kernel<float, 64><<<blocks, kStepThreads, 0, st>>>(a);
    else lin_step_kernel<float, 32><<<blocks, kStepThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace vssm
