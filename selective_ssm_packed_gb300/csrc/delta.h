// delta.h -- the gated delta rule's internal interface: arguments, the arrays
// the kernels pass on to each other, launchers.  Not part of the public ABI.
//
// Per value head, with a_t = exp(g_t):
//   S_t = a_t S_{t-1} + k_t u_t^T,  u_t = beta_t e_t,  e_t = v_t - a_t S_{t-1}^T k_t,  o_t = scale S_t^T q_t.
//
// A chunk of 64 tokens in matrices (rows are tokens; G the running sum of g in
// the chunk, D_ij = exp(G_i - G_j), S0 the state before it, S1 after it):
//   N  = strictly lower part of (K K^T * D) diag(beta)      Tm = (I + N)^-1
//   R  = V - diag(exp G) K S0                               E  = Tm R
//   P  = lower part of scale (Q K^T * D) diag(beta)         X  = [Tm; P Tm]
//   O  = scale diag(exp G) Q S0 + (P Tm) R
//   S1 = exp(G_63) S0 + K^T diag(dec beta) E,  dec_i = exp(G_63 - G_i)
// and backwards, from dO and dS1:
//   dV  = X^T [diag(dec beta) K dS1; dO]
//   dS0 = exp(G_63) dS1 + K^T (-diag(exp G) dV) + Q^T (scale diag(exp G) dO)
//   M1  = lower part of scale (dO E^T * D) diag(beta);  M2 = -strictly lower part of (dV E^T * D) diag(beta)
//   dQ  = scale diag(exp G) dO S0^T + M1 K
//   dK  = -diag(exp G) dV S0^T + diag(dec beta) E dS1^T + M2 K + M2^T K + M1^T Q
//   kappa_j = dec_j k_j . (E dS1^T)_j;  W = M1 * Q K^T + M2 * K K^T
//   dbeta_j = (column sum of W / beta_j) + kappa_j
//   dG_i = scale exp(G_i) q_i.(dO S0^T)_i - exp(G_i) k_i.(dV S0^T)_i + row sum of W - beta_i dbeta_i,
//          where W's diagonal, in both sums, is left out of both
//   dg_t = sum of dG_i, i >= t, + exp(G_63) <dS1, S0> + sum_j beta_j kappa_j
// Only R, E, O and the two states depend on earlier chunks, so everything
// else is computed for all chunks at once.
#pragma once

#include "kernels.h"

namespace vssm {

constexpr int kDeltaChunk = 64;      // tokens of a chunk
constexpr int kDeltaGates = 5 * 64;  // floats a chunk and value head keep: exp(G), dec beta, beta, G / ln 2 high, low
constexpr int kDeltaMaxK = 128, kDeltaMaxV = 1024;

// The state's columns are cut into tiles of 32, the unit in which states and
// per-token vectors pass from kernel to kernel as images of 64-byte rows.
constexpr int kDeltaTile = 32;
constexpr int kRowTile = 64 * 64;  // bytes of one term of 64 token rows of a tile

// bf16 terms of an input and of an FP32 intermediate, and how many chunks of
// [K; Q] the walks hold.  bf16 inputs are exact in one term
// and their intermediates carry two (16 bits, far below the rounding of the
// outputs to bf16, and about 5e-6 on the FP32 ones); FP32 I/O carries three,
// all 24 bits.
template <IO kIO> struct DeltaTerms;
template <> struct DeltaTerms<IO::BF16> { static constexpr int kIn = 1, kMid = 2, kStages = 2; };
template <> struct DeltaTerms<IO::F32> { static constexpr int kIn = 3, kMid = 3, kStages = 1; };
inline int delta_in_terms(IO io) { return io == IO::BF16 ? 1 : 3; }
inline int delta_mid_terms(IO io) { return io == IO::BF16 ? 2 : 3; }
__host__ __device__ inline int delta_tiles(int V) { return (V + kDeltaTile - 1) / kDeltaTile; }
inline int delta_panels_k(int K) { return (K + 63) / 64; }

struct DeltaArgs {
  const void *q, *k, *v;  // (T, Hk, K), (T, Hk, K), (T, Hv, V), token strides in elements
  int64_t sq, sk, sv;
  const float *g, *beta;  // (T, Hv)
  const int32_t* cu;
  int64_t T;
  int num_seqs, Hk, Hv, K, V;
  float scale;
  void* out;                  // fwd
  const float* initial;       // (S, Hv, K, V), nullable
  float* final_states;        // nullable
  const void* dout;           // bwd, (T, Hv, V)
  const float* d_final;       // nullable
  float* d_initial;           // nullable
  void *dq, *dk, *dv;         // (T, Hk, K) x2, (T, Hv, V)
  float *dg, *dbeta;          // (T, Hv)
  // the plan of the pack and what the chunks keep (see DeltaLayout)
  int* info;      // [0]: chunks in the pack, -1 when cu_seqlens is malformed; [1]: key
  int key;        // what says that a plan is this shape's
  int* first;     // (S + 1): each sequence's first chunk
  int4* order;    // (S): sequence, first token, tokens, first chunk; longest (about) first
  int4* table;    // per chunk: sequence, first token, tokens, place in the sequence
  float* gates;   // (chunks, Hv, kDeltaGates)
  uint8_t* kq;    // (chunks, Hk, in terms, K panels) images of [K; Q], 128 rows of 64
  uint8_t* x;     // (chunks, Hv, mid terms) images of X, 128 rows of 64
  uint8_t* s0;    // (chunks, Hv, tiles, mid terms) images of S0, 64 or 128 rows of a tile, or null
  uint8_t* e;     // (chunks, Hv, tiles, mid terms) images of E, 64 rows of a tile, or null
  uint8_t* ds;    // bwd: images of dS1, laid out as s0
  uint8_t* dvi;   // bwd: images of dV, laid out as e
  uint8_t* doi;   // bwd: images of dO, (chunks, Hv, tiles, in terms)
  float* partial; // bwd: the value heads' parts of dk and dq, (chunks, Hv, 2, 64, K), or null
  int* status;
  unsigned long long wait_ns;
  long long force_timeout_cta;  // test knob: this CTA reports its first wait as run out
  int64_t max_chunks;
};

// The most chunks a pack of T tokens in num_seqs sequences can have.
inline int64_t delta_max_chunks(int64_t T, int64_t num_seqs) {
  return T / kDeltaChunk + (num_seqs < T ? num_seqs : T);
}

// Whether the gradients' value heads go to CTAs of their own: where that
// spares a third of the rounds of 152 CTAs, each of which takes a CTA 16 us a
// value head in f32 and 8.5 us in bf16 (128 x 128), while the parts are added
// up in 3 to 7 us.  Four heads of one chunk: 63 -> 20 + 4 us in f32, 32 ->
// 12 + 4 us in bf16; a quarter spared (192 chunks and key heads of four):
// 145 -> 126 + 7 us and 72 -> 66 + 7 us.  The parts are 80 MB at most.
inline bool delta_split_grads(int64_t max_chunks, int Hk, int Hv) {
  const int64_t whole = (max_chunks * Hk + 151) / 152 * (Hv / Hk), split = (max_chunks * Hv + 151) / 152;
  return 3 * split <= 2 * whole && split <= 8;
}

// Tiles a CTA of the bf16 walks takes, which share what they read.  A step of
// one, two or four walks on an SM took 2.1, 3.1 or 4.0 us (one sequence of
// 32768 tokens, 32 heads of 128 x 128; the first is 2.2 with the checks of its
// waits and values): four are the fastest way through much
// work, one is the fastest way along a sequence.  What a pack takes is about
// the longer of all its steps over the SMs and of its longest sequence, which
// only the GPU knows and which is taken for four times the mean.
inline int delta_walks(const DeltaArgs& a, IO io) {
  if (io == IO::F32) return 1;  // three terms fill shared memory
  const double chunks = (double)a.T / kDeltaChunk + 1.0, longest = 4.0 * chunks / (a.num_seqs > 0 ? a.num_seqs : 1) + 1.0;
  const int tiles = delta_tiles(a.V);
  const double step[3] = {2.1, 3.1, 4.0};
  int best = 1;
  double least = 0.0;
  for (int i = 0; i < 3 && (i == 0 || (1 << i) / 2 < tiles); ++i) {
    const int groups = (tiles + (1 << i) - 1) >> i;
    const double all = chunks * a.Hv * groups / 152.0, along = longest < chunks ? longest : chunks;
    const double time = step[i] * (all > along ? all : along);
    if (i == 0 || time < least) {
      best = 1 << i;
      least = time;
    }
  }
  return best;
}

cudaError_t launch_delta_plan(const DeltaArgs& a, cudaStream_t st);
cudaError_t launch_delta_prep(const DeltaArgs& a, IO io, cudaStream_t st);
cudaError_t launch_delta_fwd(const DeltaArgs& a, IO io, cudaStream_t st);
cudaError_t launch_delta_bwd(const DeltaArgs& a, IO io, cudaStream_t st);
cudaError_t launch_delta_grads(const DeltaArgs& a, IO io, cudaStream_t st);

// ---------------------------------------------------------------- one token for each sequence
struct DeltaStepArgs {
  const void *q, *k, *v;
  int64_t sq, sk, sv;
  const float *g, *beta;      // (B, Hv)
  float* states;              // (slots, Hv, K, V), updated in place
  const int32_t* indices;     // (B), nullable: the identity
  void* out;                  // (B, Hv, V)
  int64_t B, slots;
  int Hk, Hv, K, V;
  float scale;
  int* status;                // nullable
};
cudaError_t launch_delta_step(const DeltaStepArgs& a, IO io, cudaStream_t st);

// ---------------------------------------------------------------- norm and rotation of queries and keys
struct QkNormArgs {
  const void *q, *k;            // (T, Hq, K), (T, Hk, K), token strides sq, sk
  int64_t sq, sk;
  const float *qw, *kw;         // (K), nullable
  const float *cos, *sin;       // (positions, rot / 2), nullable
  const int32_t* pos;           // (T)
  int64_t T, positions;
  int Hq, Hk, K, rot, l2;
  float eps;
  void *q_out, *k_out;          // fwd
  const void *dq_out, *dk_out;  // bwd, contiguous
  void *dq, *dk;                // contiguous
  float *dqw, *dkw;             // (K), null without weights
  float* partial;               // bwd: per CTA sums of the weights' gradients
  int* status;
};
// Rows of K floats the backward's partial sums need.
int qk_norm_partial_rows();
cudaError_t launch_qk_norm_fwd(const QkNormArgs& a, IO io, cudaStream_t st);
cudaError_t launch_qk_norm_bwd(const QkNormArgs& a, IO io, cudaStream_t st);

}  // namespace vssm
