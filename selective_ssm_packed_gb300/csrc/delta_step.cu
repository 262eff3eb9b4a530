// delta_step.cu -- one token of the gated delta rule for each of many
// sequences, against a pool of states.
#include "delta.cuh"

namespace vssm {
namespace {

// One CTA of 256 threads per (token, value head, kCols state columns): kCols / 4
// threads along the columns (float4 each), the others along the state rows, so
// that a thread has its whole share of the state (16 to 64 bytes a row, up to 8
// rows) in flight at once and in registers until it is written back.  With S' = exp(g) S, both sums
// over the state rows come from S' in one pass:
//   p = S'^T k, w = S'^T q;  u = beta (v - p);  S = S' + k u^T;
//   o = scale (w + (k . q) u)
// since S^T q = S'^T q + u (k . q).  The state is read and written once, which
// is all the traffic that counts: 187 us for 256 sequences of 32 heads of
// 128 x 128, 5.8 TB/s.  Four CTAs an SM leave 64 registers, of which 64 columns
// spill 12 bytes in bf16 and 20 in f32.
constexpr int kStepThreads = 256;

template <typename T, int kCols>
__global__ void __launch_bounds__(kStepThreads, 4) delta_step_kernel(DeltaStepArgs a) {
  constexpr int kAlong = kCols / 4, kStep = kStepThreads / kAlong, kPer = kDeltaMaxK / kStep;
  __shared__ float part[8][2][kCols];
  __shared__ float part_kq[8];
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
  const float alpha = exp_f(a.g[b * a.Hv + h]), beta = a.beta[b * a.Hv + h];
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (col < a.V) v = ld_io4(static_cast<const T*>(a.v) + b * a.sv + (int64_t)h * a.V + col);

  float4 p = make_float4(0.0f, 0.0f, 0.0f, 0.0f), w = p;
  float kq = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    s[i].x *= alpha; s[i].y *= alpha; s[i].z *= alpha; s[i].w *= alpha;
    p.x = fmaf(kv[i], s[i].x, p.x); p.y = fmaf(kv[i], s[i].y, p.y);
    p.z = fmaf(kv[i], s[i].z, p.z); p.w = fmaf(kv[i], s[i].w, p.w);
    w.x = fmaf(qv[i], s[i].x, w.x); w.y = fmaf(qv[i], s[i].y, w.y);
    w.z = fmaf(qv[i], s[i].z, w.z); w.w = fmaf(qv[i], s[i].w, w.w);
    kq = fmaf(kv[i], qv[i], kq);
  }
  // over the warp's row groups, then over the warps
#pragma unroll
  for (int o = kAlong; o <= 16; o <<= 1) {
    p.x += __shfl_xor_sync(0xffffffffu, p.x, o); p.y += __shfl_xor_sync(0xffffffffu, p.y, o);
    p.z += __shfl_xor_sync(0xffffffffu, p.z, o); p.w += __shfl_xor_sync(0xffffffffu, p.w, o);
    w.x += __shfl_xor_sync(0xffffffffu, w.x, o); w.y += __shfl_xor_sync(0xffffffffu, w.y, o);
    w.z += __shfl_xor_sync(0xffffffffu, w.z, o); w.w += __shfl_xor_sync(0xffffffffu, w.w, o);
    kq += __shfl_xor_sync(0xffffffffu, kq, o);
  }
  if (lane < kAlong) {
    *reinterpret_cast<float4*>(&part[warp][0][cx * 4]) = p;
    *reinterpret_cast<float4*>(&part[warp][1][cx * 4]) = w;
    if (lane == 0) part_kq[warp] = kq;
  }
  __syncthreads();
  p = w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  kq = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 x = *reinterpret_cast<const float4*>(&part[i][0][cx * 4]);
    p.x += x.x; p.y += x.y; p.z += x.z; p.w += x.w;
    kq += part_kq[i];
  }
  const float4 u = make_float4(beta * (v.x - p.x), beta * (v.y - p.y), beta * (v.z - p.z), beta * (v.w - p.w));
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int row = ry + kStep * i;
    if (row < a.K && col < a.V)
      __stcs(reinterpret_cast<float4*>(state + (int64_t)row * a.V + col),
             make_float4(fmaf(kv[i], u.x, s[i].x), fmaf(kv[i], u.y, s[i].y), fmaf(kv[i], u.z, s[i].z),
                         fmaf(kv[i], u.w, s[i].w)));
  }
  if (ry == 0 && col < a.V) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(&part[i][1][cx * 4]);
      w.x += x.x; w.y += x.y; w.z += x.z; w.w += x.w;
    }
    st_io2(out + col, make_float2(a.scale * fmaf(kq, u.x, w.x), a.scale * fmaf(kq, u.y, w.y)));
    st_io2(out + col + 2, make_float2(a.scale * fmaf(kq, u.z, w.z), a.scale * fmaf(kq, u.w, w.w)));
  }
}

}  // namespace

cudaError_t launch_delta_step(const DeltaStepArgs& a, IO io, cudaStream_t st) {
  if (a.B == 0) return cudaSuccess;
  // wide CTAs have twice the bytes in flight, once there are enough of them
  const int64_t heads = a.B * a.Hv, wide = heads * ((a.V + 63) / 64), narrow = heads * ((a.V + 31) / 32);
  const bool use_wide = wide >= 152 * 4;
  const unsigned blocks = (unsigned)(use_wide ? wide : narrow);
  if (io == IO::BF16) {
    if (use_wide) delta_step_kernel<__nv_bfloat16, 64><<<blocks, kStepThreads, 0, st>>>(a);
    else delta_step_kernel<__nv_bfloat16, 32><<<blocks, kStepThreads, 0, st>>>(a);
  } else {
    if (use_wide) delta_step_kernel<float, 64><<<blocks, kStepThreads, 0, st>>>(a);
    else delta_step_kernel<float, 32><<<blocks, kStepThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace vssm
