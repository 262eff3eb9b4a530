// delta_prep.cu -- the gated delta rule's plan of a pack and everything of a
// chunk that no earlier chunk enters: gates, the images of [K; Q], and X.
#include "delta.cuh"

namespace vssm {
namespace {

// ------------------------------------------------------------------ plan
// Every block sums the sequences' chunk counts for itself (a pack has a few
// thousand sequences, so that costs less than a second launch), block 0
// writes the sums, and each block fills its share of the chunk table.  Block 0
// also orders the sequences by length for the walks, whose CTAs start in that
// order: a long one that starts last would be walked alone.  The order is
// exact to 16 chunks and to a quarter of a power of two above, and within a
// class left to chance: it decides when a sequence is walked, not how.
constexpr int kPlanThreads = 512;

// Length class, longest first, of a sequence of n chunks.
__device__ __forceinline__ int length_class(int n) {
  if (n < 16) return 63 - n;
  const int e = 31 - __clz(n);
  return 63 - min(63, 16 + 4 * (e - 4) + ((n >> (e - 2)) & 3));
}

__global__ void __launch_bounds__(kPlanThreads) delta_plan_kernel(DeltaArgs a) {
  __shared__ int warp_sum[kPlanThreads / 32];
  __shared__ int carry, bad, classes[64];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, S = a.num_seqs;
  if (t == 0) carry = bad = 0;
  if (t < 64) classes[t] = 0;
  __syncthreads();
  for (int base = 0; base < S; base += kPlanThreads) {
    const int s = base + t;
    int n = 0;
    if (s < S) {
      const int64_t lo = a.cu[s], hi = a.cu[s + 1];
      if ((s == 0 && lo != 0) || hi < lo || lo < 0 || hi > a.T || (s == S - 1 && hi != a.T)) {
        bad = 1;
      } else {
        n = (int)((hi - lo + kDeltaChunk - 1) / kDeltaChunk);
      }
      if (blockIdx.x == 0) atomicAdd(&classes[length_class(n)], 1);
    }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    // every block writes the same values: the later fill reads its own block's
    if (s < S) a.first[s] = before + incl - n;
    __syncthreads();
    if (t == kPlanThreads - 1) carry = before + incl;
    __syncthreads();
  }
  const bool ok = !bad && carry <= a.max_chunks && (S > 0 || a.T == 0);
  const int total = ok ? carry : -1;
  if (t == 0) {
    a.first[S] = carry;
    if (blockIdx.x == 0) {
      a.info[0] = total;
      a.info[1] = a.key;
      *a.status = ok ? 0 : kStatusBadCu;  // the call's first word on it
    }
  }
  __threadfence_block();
  __syncthreads();
  if (blockIdx.x == 0 && ok) {
    if (t == 0) {
      int at = 0;
      for (int i = 0; i < 64; ++i) {
        const int k = classes[i];
        classes[i] = at;
        at += k;
      }
    }
    __syncthreads();
    for (int s = t; s < S; s += kPlanThreads)
      a.order[atomicAdd(&classes[length_class(a.first[s + 1] - a.first[s])], 1)] =
          make_int4(s, a.cu[s], a.cu[s + 1] - a.cu[s], a.first[s]);
  }
  for (int c = blockIdx.x * kPlanThreads + t; c < total; c += gridDim.x * kPlanThreads) {
    int lo = 0, hi = S - 1;  // the last sequence whose first chunk is at or before c
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.first[mid] <= c) lo = mid; else hi = mid - 1;
    }
    const int place = c - a.first[lo];
    const int start = a.cu[lo] + place * kDeltaChunk;
    a.table[c] = make_int4(lo, start, min(kDeltaChunk, a.cu[lo + 1] - start), place);
  }
}

// ------------------------------------------------------------------ prep
// One CTA of 256 threads per chunk and key head; the value heads that share
// the key head follow each other, or go to `split` CTAs where there are too few
// of them to fill the GPU.  Rows 0-63 of a product are K K^T, N and Tm,
// rows 64-127 Q K^T, P and P Tm; a thread has half a row.
// Tm = (I + N)^-1 in place of N, in shared memory: the four 16 x 16 blocks of
// the diagonal by substitution, then twice two neighbouring blocks' inverses
// T1, T2 and the block N21 below T1 are joined by T21 = -T2 N21 T1 (16, then
// 32 wide), in FP32.  The sum of powers of N would take fewer steps, but powers
// grow without bound for keys that resemble each other, while Tm's entries do
// not.  Substitution over all 64 columns took one warp 8300 cycles, most of
// them waiting for itself.
// P Tm is a product on the matrix unit, from and into X's own images.
// Four CTAs fit an SM (bf16; two or three in f32), so that one's waits hide
// behind the others; four leave 64 registers, of which 12 bytes spill (f32, K <=
// 64: 28; beyond, none).  336 us at 32768 tokens of 16 + 32 heads in bf16, 55 us
// at 4096 of 12 in f32 (K = 128).
constexpr int kNPitch = 68;    // floats a row of N: 16-byte writes of a warp's rows hit all banks
constexpr int kPrepHeads = 4;  // value heads whose gates are made at once, one a warp

template <IO kIO, int KP>
struct PrepSmem {
  using D = DeltaTerms<kIO>;
  static constexpr int kKq = D::kIn * KP * 16384, kX = D::kMid * 16384;
  static constexpr int kImages = kKq > kX ? kKq : kX;  // [K; Q], later X
  // N, too, in the place of [K; Q] where X leaves room: two CTAs an SM then for K > 64 in f32, not one
  static constexpr int kN = 64 * kNPitch * 4, oN = kX + kN <= kImages ? kX : kImages;
  static constexpr int oG = oN + kN > kImages ? oN + kN : kImages, oBeta = oG + kPrepHeads * 64 * 8;
  static constexpr int oBar = oBeta + kPrepHeads * 64 * 4;
  static constexpr int kBytes = oBar + 64 + 1024;
  static constexpr int kCtas = kIO == IO::BF16 ? 4 : KP == 1 ? 3 : 2;  // that fit an SM
  static_assert(kCtas * (kBytes + 1024) <= 228 * 1024, "shared memory");
};

// Rows i0 .. i0 + kRows - 1, columns c .. c + 3 of -A B or A B, for A and B in
// shared memory, row pitches pa and pb, kDepth deep.
template <int kRows, int kDepth, bool kNegate>
__device__ __forceinline__ void small_product(const float* A, int pa, const float* B, int pb, float* out, int po) {
  float2 acc[kRows][2];
#pragma unroll
  for (int i = 0; i < kRows; ++i) acc[i][0] = acc[i][1] = splat2(0.0f);
#pragma unroll 2
  for (int k = 0; k < kDepth; k += 4) {
    float4 f[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) f[i] = *reinterpret_cast<const float4*>(A + i * pa + k);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 b = *reinterpret_cast<const float4*>(B + (k + j) * pb);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const float a = j == 0 ? f[i].x : j == 1 ? f[i].y : j == 2 ? f[i].z : f[i].w;
        acc[i][0] = fma2(splat2(a), make_float2(b.x, b.y), acc[i][0]);
        acc[i][1] = fma2(splat2(a), make_float2(b.z, b.w), acc[i][1]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const float s = kNegate ? -1.0f : 1.0f;
    *reinterpret_cast<float4*>(out + i * po) =
        make_float4(s * acc[i][0].x, s * acc[i][0].y, s * acc[i][1].x, s * acc[i][1].y);
  }
}

// (I + N)^-1 over N (64 rows, kNPitch floats apart, zero above the diagonal),
// by 256 threads numbered t in any order of whole warps; y: 32 x 36 floats of
// scratch.  N's rows from len on are zero, so a short chunk has nothing to join.
__device__ __forceinline__ void invert(float* n, float* y, int t, int len) {
  if (t < 64) {
    const int r = t & 15;
    const float* block = n + (t & ~15) * (kNPitch + 1);
    float2 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = make_float2(2 * i == r ? 1.0f : 0.0f, 2 * i + 1 == r ? 1.0f : 0.0f);
    // x_j is final, then x_l -= x_j N_jl for l < j
#pragma unroll
    for (int j = 15; j >= 1; --j) {
      const float2 m = splat2(-((j & 1) ? x[j / 2].y : x[j / 2].x));
      const float4* row = reinterpret_cast<const float4*>(block + j * kNPitch);
#pragma unroll
      for (int q = 0; q <= (j - 1) / 4; ++q) {
        const float4 f = row[q];
        x[2 * q] = fma2(m, make_float2(f.x, f.y), x[2 * q]);
        if (4 * q + 2 < j) x[2 * q + 1] = fma2(m, make_float2(f.z, f.w), x[2 * q + 1]);
      }
    }
    __syncwarp();  // a warp holds whole blocks: all of its rows have been read
    float* out = n + t * kNPitch + (t & ~15);
#pragma unroll
    for (int i = 0; i < 8; i += 2) *reinterpret_cast<float4*>(out + 2 * i) = make_float4(x[i].x, x[i].y, x[i + 1].x, x[i + 1].y);
  }
  __syncthreads();
  if (len <= 16) return;
  // Products of 4 x 4 values a thread: shared memory serves one float of a
  // vector read a cycle, repeated or not, and its cycles bound this kernel.
  {
    const int at = (t >> 4) * 32, i = (t >> 2 & 3) * 4, c = (t & 3) * 4;  // pair of blocks, rows, columns
    float* y1 = y + (t >> 4) * 16 * 20;
    if (t < 32)
      small_product<4, 16, false>(n + (at + 16 + i) * kNPitch + at, kNPitch, n + at * kNPitch + at + c, kNPitch,
                                  y1 + i * 20 + c, 20);
    __syncwarp();
    if (t < 32)
      small_product<4, 16, true>(n + (at + 16 + i) * kNPitch + at + 16, kNPitch, y1 + c, 20,
                                 n + (at + 16 + i) * kNPitch + at + c, kNPitch);
    __syncthreads();
  }
  if (len <= 32) return;
  const int i = (t >> 3) * 4, c = (t & 7) * 4;
  if (t < 64) small_product<4, 32, false>(n + (32 + i) * kNPitch, kNPitch, n + c, kNPitch, y + i * 36 + c, 36);
  __syncthreads();
  if (t < 64)
    small_product<4, 32, true>(n + (32 + i) * kNPitch + 32, kNPitch, y + c, 36, n + (32 + i) * kNPitch + c, kNPitch);
  __syncthreads();
}

template <IO kIO, int KP>
__global__ void __launch_bounds__(256, PrepSmem<kIO, KP>::kCtas) delta_prep_kernel(DeltaArgs a, int split) {
  using T = typename IoType<kIO>::type;
  using L = PrepSmem<kIO, KP>;
  constexpr int NQ = DeltaTerms<kIO>::kIn, NT = DeltaTerms<kIO>::kMid;
  constexpr int kTerm = KP * 16384;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* images = align1024(smem_raw);
  float* sn = reinterpret_cast<float*>(images + L::oN);
  float2* sg_all = reinterpret_cast<float2*>(images + L::oG);  // running sum of g over ln 2, in two floats
  float* sbeta_all = reinterpret_cast<float*>(images + L::oBeta);
  uint64_t* bar = reinterpret_cast<uint64_t*>(images + L::oBar);
  uint64_t* drained = bar + 1;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* stop = reinterpret_cast<int*>(tmem_at + 1);
  int* bad = const_cast<int*>(stop) + 1;  // the first row of N that is not finite

  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, quad = warp & 3, half = warp >> 2;
  const int share = blockIdx.x % split, kh = blockIdx.x / split % a.Hk;
  const int64_t c = blockIdx.x / split / a.Hk;
  if (c >= a.info[0]) return;
  const int4 chunk = a.table[c];
  const int64_t start = chunk.y;
  const int len = chunk.z;
  const int rep = a.Hv / a.Hk;
  const int h0 = kh * rep + rep * share / split, h1 = kh * rep + rep * (share + 1) / split;  // value heads

  if (t == 0) {
    mbar_init(bar, 1);
    mbar_init(drained, 1);
    *stop = 0;
    *bad = 64;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc<128>(tmem_at);

  // warp w: the gates of value head h + w
  auto make_gates = [&](int h) {
    const int hw = h + warp;
    if (warp >= kPrepHeads || hw >= h1) return;
    // the running sum of g, in double: differences of it enter exp
    float g[2], b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 2 * lane + i;
      const int64_t at = (start + r) * a.Hv + hw;
      g[i] = r < len ? a.g[at] : 0.0f;
      b[i] = r < len ? a.beta[at] : 0.0f;
      g[i] = g[i] < -256.0f ? -256.0f : g[i];  // exp of either is 0; -inf would leave inf - inf
    }
    double incl = (double)g[0] + (double)g[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const double last = __shfl_sync(0xffffffffu, incl, 31);
    double before = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane == 0) before = 0.0;
    const double G[2] = {before + (double)g[0], incl};
    float* gates = a.gates + (c * a.Hv + hw) * kDeltaGates;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 2 * lane + i;
      const double G2 = G[i] * 1.4426950408889634;
      const float hi = (float)G2, lo = (float)(G2 - (double)hi);
      sg_all[warp * 64 + r] = make_float2(hi, lo);
      sbeta_all[warp * 64 + r] = b[i];
      const float gh = (float)G[i], dh = (float)(last - G[i]);
      gates[r] = exp_f(gh) * (1.0f + (float)(G[i] - (double)gh));
      gates[64 + r] = exp_f(dh) * (1.0f + (float)(last - G[i] - (double)dh)) * b[i];
      gates[128 + r] = b[i];
      gates[192 + r] = hi;
      gates[256 + r] = lo;
    }
  };
  // the images of [K; Q]: rows past the chunk's end and columns past K are zero
  const T* kbase = static_cast<const T*>(a.k) + start * a.sk + (int64_t)kh * a.K;
  const T* qbase = static_cast<const T*>(a.q) + start * a.sq + (int64_t)kh * a.K;
  if constexpr (kIO == IO::BF16) {
#pragma unroll
    for (int u = 0; u < KP * 4; ++u) {
      const int i = t + u * 256, row = i / (KP * 8), ch = i % (KP * 8), r = row & 63;
      const bool in = r < len && ch * 8 < a.K;
      const T* src = in ? (row < 64 ? kbase + r * a.sk : qbase + r * a.sq) + ch * 8 : kbase;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                       smem_u32(images + (ch >> 3) * 16384 + image_chunk<128>(row, ch & 7))),
                   "l"(src), "r"(in ? 16 : 0)
                   : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  } else {
    constexpr int kBatch = 4;  // reads in flight
    for (int u = 0; u < KP * 4; u += kBatch) {
      float4 f[kBatch][2];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = t + (u + k) * 256, row = i / (KP * 8), ch = i % (KP * 8), r = row & 63;
        f[k][0] = f[k][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < len && ch * 8 < a.K) {
          const float4* src = reinterpret_cast<const float4*>((row < 64 ? kbase + r * a.sk : qbase + r * a.sq) + ch * 8);
          f[k][0] = src[0];
          f[k][1] = src[1];
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = t + (u + k) * 256, row = i / (KP * 8), ch = i % (KP * 8);
        const float2 v[4] = {make_float2(f[k][0].x, f[k][0].y), make_float2(f[k][0].z, f[k][0].w),
                             make_float2(f[k][1].x, f[k][1].y), make_float2(f[k][1].z, f[k][1].w)};
        put_chunk<NQ, 128>(images + (ch >> 3) * 16384, kTerm, row, ch & 7, v);
      }
    }
  }
  make_gates(h0);  // while [K; Q] is on its way
  if constexpr (kIO == IO::BF16) asm volatile("cp.async.wait_group 0;" ::: "memory");
  fence_async_smem();
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tm = *tmem_at;
  const int row = quad * 32 + lane, r = row & 63;
  const bool is_k = row < 64;
  const bool empty = half && !(quad & 1);  // rows 0-31 end before column 32
  const uint32_t mine = tm + ((uint32_t)(quad * 32) << 16) + half * 32;
  if (t == 0) {
    const Operand<128, kKMajor, NQ, kTerm, 16384> kq(smem_u32(images));
    umma_terms<64, KP * 4, NQ>(tm, kq, kq, false);  // B: the K rows
    umma_commit(bar);
    if (share == 0) bulk_store_1d(a.kq + (size_t)(c * a.Hk + kh) * L::kKq, images, L::kKq);
    bulk_commit();
  }
  uint32_t phase = 0;

  for (int h = h0; h < h1; ++h) {
    const int64_t ch = c * a.Hv + h;
    if (h > h0 && (h - h0) % kPrepHeads == 0) make_gates(h);
    if (t == 0) bulk_wait_read();  // [K; Q], or the last head's X, has left
    __syncthreads();
    if (h == h0) {
      wait_or_stop(a, stop, bar, phase, t == 0 && forced_here(a));
      phase ^= 1;
      tmem_fence_after_sync();
      if (t < 32)  // N's upper right quarter, which nothing else writes
#pragma unroll
        for (int i = 0; i < 8; ++i) *reinterpret_cast<float4*>(sn + t * kNPitch + 32 + 4 * i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    const float2* sg = sg_all + ((h - h0) % kPrepHeads) * 64;
    const float* sbeta = sbeta_all + ((h - h0) % kPrepHeads) * 64;
    if (!empty) {
      const float2 gi = sg[r];
      const float f = is_k ? 1.0f : a.scale;
      const int end = is_k ? r : r + 1;  // columns j < end
      float2 trace = splat2(0.0f);  // not 0 once there is a value that is not finite
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float d[16];
        tmem_row(mine + u * 16, d);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = half * 32 + u * 16 + i;
          const float2 gj = sg[j];
          const float w = ex2((gi.x - gj.x) + (gi.y - gj.y)) * (sbeta[j] * f) * d[i];
          d[i] = j < end ? w : 0.0f;
        }
        if (is_k) {
#pragma unroll
          for (int i = 0; i < 16; i += 2) trace = fma2(make_float2(d[i], d[i + 1]), splat2(0.0f), trace);
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4*>(sn + r * kNPitch + half * 32 + u * 16 + i) = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
        } else {
          float2 p[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) p[i] = make_float2(d[2 * i], d[2 * i + 1]);
          put_row<NT, 128>(images, 16384, row, half * 4 + 2 * u, p);
        }
      }
      if (trace.x + trace.y != 0.0f) atomicMin(bad, r);
    } else if (!is_k) {
#pragma unroll
      for (int k = 0; k < 4 * NT; ++k)
        *reinterpret_cast<uint4*>(images + k / 4 * 16384 + image_chunk<128>(row, 4 + k % 4)) = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    if (*bad < 64) {
      // From this token on nothing of the head is finite.  Its rows leave N, so that the products of the inverse (0
      // times them) do not carry them to earlier tokens, and NaN takes their place where they would have come out.
      const float nan = __int_as_float(0x7fffffff);
      const int first = *bad;
      for (int i = t; i < 64 * 64; i += 256)
        if (i / 64 >= first) sn[i / 64 * kNPitch + i % 64] = 0.0f;
      if (t >= first && t < 64) {
        *reinterpret_cast<uint16_t*>(images + image_chunk<128>(64 + t, 0)) = 0x7fff;
        a.gates[ch * kDeltaGates + t] = nan;  // exp(G), the last of which scales the state
      }
      __syncthreads();
      if (t == 0) *bad = 64;
    }
    invert(sn, reinterpret_cast<float*>(images), (t + 64 * blockIdx.x) & 255, len);  // scratch: where the rows of Tm go next
    {
      const int tr = t >> 2, side = t & 3;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4* src = reinterpret_cast<const float4*>(sn + tr * kNPitch + side * 16 + q * 8);
        const float4 f = src[0], g = src[1];
        const float2 v[4] = {make_float2(f.x, f.y), make_float2(f.z, f.w), make_float2(g.x, g.y), make_float2(g.z, g.w)};
        put_chunk<NT, 128>(images, 16384, tr, side * 2 + q, v);
      }
    }
    fence_async_smem();
    tmem_fence_before_sync();
    __syncthreads();
    if (t == 0 && !*stop) {
      tmem_fence_after_sync();
      const Operand<128, kKMajor, NT, 16384> A(smem_u32(images));
      const Operand<128, kMnMajor, NT, 16384> B(smem_u32(images));  // the rows of Tm
      umma_terms<64, 4, NT>(tm + 64, A, B, false);
      umma_commit(bar);
    }
    wait_or_stop(a, stop, bar, phase);
    phase ^= 1;
    tmem_fence_after_sync();
    if (!is_k && !empty) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float2 d[8];
        tmem_sum<1>(mine + 64 + u * 16, 0, d);
        put_row<NT, 128>(images, 16384, row, half * 4 + 2 * u, d);
      }
    }
    fence_async_smem();
    tmem_fence_before_sync();
    if (!__syncthreads_and(!*stop)) break;  // a wait ran out: one that did has said so before it came here
    if (t == 0) {
      bulk_store_1d(a.x + (size_t)ch * L::kX, images, L::kX);
      bulk_commit();
    }
  }
  if (t == 0) {
    bulk_wait_all();
    if (*stop) {  // products that were not waited for
      umma_commit(drained);
      mbar_wait(drained, 0, kCopyDrainNs);
    }
  }
  tmem_fence_before_sync();
  __syncthreads();
  if (warp == 0) tmem_dealloc<128>(tm);
}

template <IO kIO, int KP>
cudaError_t run_prep(const DeltaArgs& a, cudaStream_t st) {
  constexpr size_t bytes = PrepSmem<kIO, KP>::kBytes;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = set_smem(reinterpret_cast<const void*>(delta_prep_kernel<kIO, KP>), bytes, done);
  if (e != cudaSuccess) return e;
  const int64_t blocks = a.max_chunks * a.Hk, rep = a.Hv / a.Hk, free = 152 * 2 / blocks;
  const int split = (int)(free < 1 ? 1 : free < rep ? free : rep);
  delta_prep_kernel<kIO, KP><<<(unsigned)(blocks * split), 256, bytes, st>>>(a, split);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_plan(const DeltaArgs& a, cudaStream_t st) {
  int64_t blocks = (a.max_chunks + kPlanThreads - 1) / kPlanThreads;
  blocks = blocks < 1 ? 1 : blocks > 64 ? 64 : blocks;
  delta_plan_kernel<<<(unsigned)blocks, kPlanThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_delta_prep(const DeltaArgs& a, IO io, cudaStream_t st) {
  if (a.max_chunks == 0) return cudaSuccess;
  const bool two = delta_panels_k(a.K) == 2;
  if (io == IO::BF16) return two ? run_prep<IO::BF16, 2>(a, st) : run_prep<IO::BF16, 1>(a, st);
  return two ? run_prep<IO::F32, 2>(a, st) : run_prep<IO::F32, 1>(a, st);
}

}  // namespace vssm
