// linear.h -- internal interface of linear attention with a decay for each
// head, and of layer norm: arguments, arrays the kernels pass on, launchers.
// Not part of the public ABI.
//
// Per value head, with a_t = exp(g_t):  S_t = a_t S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t.
//
// A chunk in matrices (rows are tokens; G the running sum of g in the chunk, S0
// the state before it, S1 after it):
//   P  = lower part of scale (Q K^T * exp(G_i - G_j))
//   O  = diag(scale exp G) Q S0 + P V
//   S1 = exp(G_end) S0 + K^T diag(exp(G_end - G)) V
// The gradients are three operators of this form.  With Z_t = scale q_t do_t^T +
// a_{t+1} Z_{t+1}, dq_t = scale S_t do_t, dv_t = Z_t^T k_t and dk_t = Z_t v_t:
//            rows X   columns Y   values W   state
//   out        q         k           v        S
//   dq         do        v           k        S^T
//   dv         k         q           do       Z     time reversed
//   dk         v         do          q        Z^T   time reversed
// In reversed time P is the upper part, and the weights of the state on the
// rows and of the rows in the state change places:
//   O = diag(exp(G_end - G)) X Z1 + P W,   Z0 = exp(G_end) Z1 + Y^T diag(scale exp G) W
// (Z1 and Z0 with the decay towards the earlier chunk, that is, as gradients of
// the states S1 and S0.)  A pair of tokens s < t adds W_ts = scale exp(..) (q_t.k_s)
// (do_t.v_s) to dg of every token in (s, t], so
//   dg_t = sum over i >= t of (rho_i - sigma_i) + <gradient of S_end, S_end>,
//   rho_t = q_t . (dq_t without s = t),  sigma_s = k_s . (dk_s without t = s),
// the sum over the rest of the token's segment, S_end the state at its end.  Both
// walks have the same A = do v^T and, but for a float's last bits, the same P,
// so what is rounded off a pair of one chunk leaves the sum again behind both its
// tokens (the other choice for sigma, v_s . dv_s, has a P of its own: rounded to
// two bf16 terms, dg was then 1.6e-5 off over sequences of 4096 tokens).
// The token's own pair is in none of them: it goes to dq and dk by itself, behind
// the dots.  It does not decay, where dg falls as exp(g): with its rounding in rho
// and sigma dg of a constant g of -6 was 7e-4 of its norm off, of -12 17%.
// That sum is known at a segment's first token as well: <gradient of S_begin,
// S_begin>, the product at the end of the segment before, or that with the
// initial state, or nothing.  What it is off by there has piled up over the
// segment, with each token's part going by |rho| + |sigma|, and each token takes
// back the parts of those from it on.
//
// Segments.  A sequence is cut into segments of at most `seg` tokens, which are
// walked by CTAs of their own once the state before each is known: a first
// walk of each segment but the last gives what it adds to the state, and a
// scan over a sequence's segments adds them up.
#pragma once

#include <cuda.h>

#include "kernels.h"

namespace vssm {

constexpr int kLinTile = 64;   // columns of the state that an f32 walk's CTA has
constexpr int kLinMaxK = 128, kLinMaxV = 128;
constexpr int kLinRoles = 3;
constexpr int kLinMaxSegment = 4096;  // tokens
constexpr int kLinParts = 4;   // f32: threads to a row, 16 columns of the tile each

// CTAs that share the columns of a state: in bf16 one walks them all.
inline int lin_ctas(IO io, int n2) { return io == IO::BF16 ? 1 : (n2 + kLinTile - 1) / kLinTile; }
// Parts that rho and sigma come in: the threads that share a row.
inline int lin_dot_parts(IO io, int n2) { return io == IO::BF16 ? 2 : kLinParts * lin_ctas(io, n2); }
inline int lin_chunk(IO io) { return io == IO::BF16 ? 128 : 64; }  // tokens
__host__ __device__ inline int lin_tiles(int n) { return (n + kLinTile - 1) / kLinTile; }

// One operator of the form above.
struct LinRole {
  const void *x, *y, *w;   // tokens sx, sy, sw elements apart
  int64_t sx, sy, sw;
  int rx, ry, rw;          // value heads that share a head of each
  int n1, n2;              // widths of x and y, and of w
  int mx, my, mw;          // bf16: their tensor maps
  void* out;               // contiguous (T, Hv, n2), io or, where part, f32; null: the state only
  int part;
  const void* dot;         // rho's or sigma's partner rows, or null
  int64_t sdot;
  int rdot;
  float* dots;             // (lin_dot_parts, Hv, T)
  int back;                // reversed time
  int64_t srow, scol;      // a state's element (row of n1, column of n2) in memory
  const float* first;      // states that the sequences come with, (S, Hv, ., .), or null
  float* last;             // states that they leave, or null (bf16: of the state-only walks)
  float* slots;            // states between segments, (inner segments, Hv, ., .)
  float* decay;            // (inner segments, Hv): exp of the segment's sum of g (the state-only walks write it)
  const float* against;    // gradients of the states at the segments' ends, as `slots` of a reversed role, or null
  const float* against_last;  // of those that a sequence leaves; of a reversed role, the states it comes with; or null
  float* cross;            // (segments, Hv, lin_ctas): their products with the states, or null
};

struct LinArgs {
  LinRole role[kLinRoles];
  const float* g;
  int64_t g_token;         // Hv, or 0 where a head has one decay
  const int32_t* cu;
  int64_t T;
  int num_seqs, Hk, Hv, K, V, seg;
  float scale;
  // the plan
  int* info;               // [0] segments (-1: malformed cu_seqlens), [1] inner segments, [2] sequences of several
  int4* table;             // per segment: sequence, first token, tokens, place (see kLinFirst)
  int* order;              // segments, longest (about) first
  int* inner;              // segments that others follow
  int2* split;             // per sequence of several segments: its first inner segment, how many
  int64_t max_segs, max_inner;
  // backward
  const void* dout;
  float *dq_part, *dk_part;  // (T, Hv, K) where heads are shared
  void *dq, *dk;
  float* dg;               // (T, Hv) or (Hv)
  double* seg_dg;          // (segments, Hv), for one decay a head
  int* status;
  unsigned long long wait_ns;
  long long force_timeout_cta;
};
// The tensor maps of the calls' bf16 rows: (width, heads, tokens), boxes of 64 x 1 x 128.
struct LinMaps {
  CUtensorMap m[4];
};
// A table entry's w: flags and, above them, the inner segments before it.
constexpr int kLinFirst = 1, kLinLast = 2, kLinPlaceShift = 2;

cudaError_t launch_lin_plan(const LinArgs& a, cudaStream_t st);
// state_only: the inner segments of roles [0, roles), otherwise all segments.
cudaError_t launch_lin_walk(const LinArgs& a, const LinMaps& maps, int roles, bool state_only, IO io, cudaStream_t st);
cudaError_t launch_lin_walk_bf16(const LinArgs& a, const LinMaps& maps, int roles, cudaStream_t st);
// bf16, ends: the states that the sequences leave (the f32 walk writes them as it goes).
cudaError_t launch_lin_state_bf16(const LinArgs& a, const LinMaps& maps, int roles, bool ends, cudaStream_t st);
cudaError_t launch_lin_scan(const LinArgs& a, int roles, cudaStream_t st);
cudaError_t launch_lin_dg(const LinArgs& a, IO io, cudaStream_t st);
cudaError_t launch_lin_head_sum(const LinArgs& a, IO io, cudaStream_t st);

struct LinStepArgs {
  const void *q, *k, *v;
  int64_t sq, sk, sv;
  const float* g;
  int64_t g_token;
  float* states;              // (slots, Hv, K, V), updated in place
  const int32_t* indices;     // (B), nullable: the identity
  void* out;                  // (B, Hv, V)
  int64_t B, slots;
  int Hk, Hv, K, V;
  float scale;
  int* status;                // nullable
};
cudaError_t launch_lin_step(const LinStepArgs& a, IO io, cudaStream_t st);

// ---------------------------------------------------------------- layer norm
constexpr int kLayerNormMaxWidth = 8192;

struct LayerNormArgs {
  const void* x;              // fwd: (T, D) io; bwd: what was normalised, io or f32; rows sx apart
  int64_t sx;
  const float* residual;      // fwd: (T, D) f32, nullable
  const float *weight, *bias; // (D), nullable
  int64_t T;
  int D, groups;
  float eps;
  void* out;                  // fwd
  float* sum;                 // fwd: x + residual, nullable
  const void* dout;           // bwd
  const float* dsum;          // bwd, nullable
  void* dx;
  float* dresidual;           // bwd, nullable
  float *dweight, *dbias;     // bwd, nullable
  float* partial;             // bwd: (slots, 2, D / groups)
  int* status;
};
// Rows of D / groups float pairs the backward's partial sums need.
int64_t layer_norm_slots(int64_t T, int D, int groups);
cudaError_t launch_layer_norm_fwd(const LayerNormArgs& a, IO io, cudaStream_t st);
// x_f32: x holds f32 rows whatever the io type.
cudaError_t launch_layer_norm_bwd(const LayerNormArgs& a, IO io, bool x_f32, cudaStream_t st);

}  // namespace vssm
