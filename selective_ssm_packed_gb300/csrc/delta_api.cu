// delta_api.cu -- the C ABI of the gated delta rule and of the norm and
// rotation of queries and keys: argument checks, workspace layout, launches.
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include <nvtx3/nvToolsExt.h>

#include "delta.h"
#include "varlen_ssm.h"

using namespace vssm;

namespace {

struct Range {
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
};

int bad(int code, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return record_error(code, buf);
}

int check(cudaError_t e, const char* what) {
  return e == cudaSuccess ? VSSM_OK : bad(VSSM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

#define TRY(expr)                   \
  do {                              \
    const int rc_ = (expr);         \
    if (rc_ != VSSM_OK) return rc_; \
  } while (0)

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_dtype(vssm_dtype dt, IO* io) {
  if (dt != VSSM_F32 && dt != VSSM_BF16) return bad(VSSM_ERR_DTYPE, "dtype %d is neither VSSM_F32 nor VSSM_BF16", (int)dt);
  *io = dt == VSSM_F32 ? IO::F32 : IO::BF16;
  return VSSM_OK;
}

// A tensor that has to be there when the call has rows.
int check_ptr(const void* p, const char* name, bool needed) {
  if (!p) return needed ? bad(VSSM_ERR_ARG, "%s is NULL", name) : VSSM_OK;
  return al16(p) ? VSSM_OK : bad(VSSM_ERR_ALIGN, "%s is not 16-byte aligned", name);
}

int check_stride(int64_t stride, int64_t row, IO io, const char* name) {
  if (stride < row) return bad(VSSM_ERR_ARG, "%s %lld is below the row's %lld values", name, (long long)stride, (long long)row);
  if (stride % (16 / io_bytes(io))) return bad(VSSM_ERR_ALIGN, "%s %lld is not a multiple of 16 bytes", name, (long long)stride);
  return VSSM_OK;
}

int check_room(const void* p, size_t have, size_t need, const char* name) {
  if (have < need) return bad(VSSM_ERR_WORKSPACE, "%s has %zu bytes, needs %zu", name, have, need);
  if (!p) return bad(VSSM_ERR_WORKSPACE, "%s is NULL", name);
  return al16(p) ? VSSM_OK : bad(VSSM_ERR_ALIGN, "%s is not 16-byte aligned", name);
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

// ---------------------------------------------------------------- gated delta rule
int check_heads(int32_t Hk, int32_t Hv, int32_t K, int32_t V) {
  if (Hv > 65535) return bad(VSSM_ERR_UNSUPPORTED, "Hv = %d is above 65535", Hv);  // sizes then stay within 64 bits
  if (Hk < 1 || Hv < 1 || Hv % Hk) return bad(VSSM_ERR_ARG, "Hv = %d must be a positive multiple of Hk = %d", Hv, Hk);
  if (K < 8 || K > kDeltaMaxK || K % 8) return bad(VSSM_ERR_UNSUPPORTED, "K = %d is not a multiple of 8 in 8..%d", K, kDeltaMaxK);
  if (V < 8 || V > kDeltaMaxV || V % 8) return bad(VSSM_ERR_UNSUPPORTED, "V = %d is not a multiple of 8 in 8..%d", V, kDeltaMaxV);
  return VSSM_OK;
}

int check_pack(int64_t T, int32_t S, const int32_t* cu, int32_t Hk, int32_t Hv, int32_t K, int32_t V) {
  if (T < 0 || T > 2147483647LL) return bad(VSSM_ERR_ARG, "total_tokens %lld out of range", (long long)T);
  if (S < 0) return bad(VSSM_ERR_ARG, "num_seqs must be >= 0 (got %d)", S);
  if (T > 0 && S < 1) return bad(VSSM_ERR_ARG, "%lld tokens but num_seqs = %d", (long long)T, S);
  if (!cu) return bad(VSSM_ERR_ARG, "cu_seqlens is NULL");
  TRY(check_heads(Hk, Hv, K, V));
  if ((int64_t)S * Hv * delta_tiles(V) > 2147483647LL || delta_max_chunks(T, S) * Hk > 2147483647LL)
    return bad(VSSM_ERR_UNSUPPORTED, "too many sequences, chunks and heads for one call");
  return VSSM_OK;
}

// What the chunks keep for each other, one after the other:
// [info][first chunks][order][chunk table][gates][images of [K; Q]][images of X], and
// in a saved array [images of S0][images of E] behind them.
struct DeltaLayout {
  size_t first, order, table, gates, kq, x, plan_end, s0, e, saved_end, ds, dvi, doi, partial, bwd_end;
};

DeltaLayout delta_layout(int64_t T, int64_t S, int Hk, int Hv, int K, int V, IO io) {
  DeltaLayout l;
  const size_t nc = (size_t)delta_max_chunks(T, S);
  const size_t mid = delta_mid_terms(io), kp = delta_panels_k(K), tiles = nc * Hv * delta_tiles(V);
  const size_t rows = tiles * mid * kRowTile, states = rows * kp;
  size_t o = 256;
  l.first = o; o += up((S + 1) * sizeof(int));
  l.order = o; o += up(S * sizeof(int4));
  l.table = o; o += up(nc * sizeof(int4));
  l.gates = o; o += up(nc * Hv * kDeltaGates * sizeof(float));
  l.kq = o; o += up(nc * Hk * delta_in_terms(io) * kp * 16384);
  l.x = o; o += up(nc * Hv * mid * 16384);
  l.plan_end = o;
  l.s0 = o; o += up(states);
  l.e = o; o += up(rows);
  l.saved_end = o;
  l.ds = 256;
  l.dvi = l.ds + up(states);
  l.doi = l.dvi + up(rows);
  l.partial = l.doi + up(tiles * delta_in_terms(io) * kRowTile);
  l.bwd_end = l.partial + (delta_split_grads((int64_t)nc, Hk, Hv) ? up(nc * Hv * 128 * K * sizeof(float)) : 0);
  return l;
}

bool sizes_ok(int64_t T, int32_t S, int32_t Hk, int32_t Hv, int32_t K, int32_t V, vssm_dtype dt) {
  IO io;
  const int32_t cu = 0;
  return check_dtype(dt, &io) == VSSM_OK && check_pack(T, S, &cu, Hk, Hv, K, V) == VSSM_OK;
}

// Tells the plan of one shape from another's, and both from memory that holds none.
int plan_key(int64_t T, int64_t S, int Hk, int Hv, int K, int V, IO io) {
  uint64_t h = 0x9e3779b97f4a7c15ull;
  for (int64_t v : {T, S, (int64_t)Hk, (int64_t)Hv, (int64_t)K, (int64_t)V, (int64_t)io}) h = (h ^ (uint64_t)v) * 0x100000001b3ull;
  return (int)(h >> 16 | 1);
}

void set_plan(DeltaArgs& a, const void* base, const DeltaLayout& l, bool saved) {
  char* p = const_cast<char*>(static_cast<const char*>(base));
  a.info = reinterpret_cast<int*>(p) + 32;  // past the status word
  a.first = reinterpret_cast<int*>(p + l.first);
  a.order = reinterpret_cast<int4*>(p + l.order);
  a.table = reinterpret_cast<int4*>(p + l.table);
  a.gates = reinterpret_cast<float*>(p + l.gates);
  a.kq = reinterpret_cast<uint8_t*>(p + l.kq);
  a.x = reinterpret_cast<uint8_t*>(p + l.x);
  a.s0 = saved ? reinterpret_cast<uint8_t*>(p + l.s0) : nullptr;
  a.e = saved ? reinterpret_cast<uint8_t*>(p + l.e) : nullptr;
}

}  // namespace

extern "C" {

size_t varlen_gated_delta_saved_size(int64_t T, int32_t S, int32_t Hk, int32_t Hv, int32_t K, int32_t V, vssm_dtype dt) {
  return sizes_ok(T, S, Hk, Hv, K, V, dt) ? delta_layout(T, S, Hk, Hv, K, V, dt == VSSM_F32 ? IO::F32 : IO::BF16).saved_end : 0;
}

size_t varlen_gated_delta_fwd_workspace_size(int64_t T, int32_t S, int32_t Hk, int32_t Hv, int32_t K, int32_t V,
                                             vssm_dtype dt) {
  return sizes_ok(T, S, Hk, Hv, K, V, dt) ? delta_layout(T, S, Hk, Hv, K, V, dt == VSSM_F32 ? IO::F32 : IO::BF16).plan_end : 0;
}

size_t varlen_gated_delta_bwd_workspace_size(int64_t T, int32_t S, int32_t Hk, int32_t Hv, int32_t K, int32_t V,
                                             vssm_dtype dt) {
  return sizes_ok(T, S, Hk, Hv, K, V, dt) ? delta_layout(T, S, Hk, Hv, K, V, dt == VSSM_F32 ? IO::F32 : IO::BF16).bwd_end : 0;
}

int vssm_gated_delta_walks(int64_t T, int32_t S, int32_t Hk, int32_t Hv, int32_t K, int32_t V, vssm_dtype dt) {
  if (!sizes_ok(T, S, Hk, Hv, K, V, dt)) return VSSM_ERR_ARG;
  DeltaArgs a{};
  a.T = T; a.num_seqs = S; a.Hv = Hv; a.V = V;
  return delta_walks(a, dt == VSSM_F32 ? IO::F32 : IO::BF16);
}

int varlen_gated_delta_fwd(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                           int64_t v_stride, const float* g, const float* beta, float scale,
                           const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens, int32_t Hk,
                           int32_t Hv, int32_t K, int32_t V, vssm_dtype dtype, void* out,
                           const float* initial_states, float* final_states, void* saved, size_t saved_bytes,
                           void* workspace, size_t workspace_bytes, void* stream) {
  Range range_("varlen_gated_delta_fwd");
  IO io;
  TRY(check_dtype(dtype, &io));
  const int64_t T = total_tokens;
  TRY(check_pack(T, num_seqs, cu_seqlens, Hk, Hv, K, V));
  TRY(check_ptr(q, "q", T > 0));
  TRY(check_ptr(k, "k", T > 0));
  TRY(check_ptr(v, "v", T > 0));
  TRY(check_ptr(out, "out", T > 0));
  TRY(check_stride(q_stride, (int64_t)Hk * K, io, "q_stride"));
  TRY(check_stride(k_stride, (int64_t)Hk * K, io, "k_stride"));
  TRY(check_stride(v_stride, (int64_t)Hv * V, io, "v_stride"));
  if (T > 0 && (!g || !beta)) return bad(VSSM_ERR_ARG, "g and beta must be non-NULL");
  TRY(check_ptr(initial_states, "initial_states", false));
  TRY(check_ptr(final_states, "final_states", false));
  const DeltaLayout l = delta_layout(T, num_seqs, Hk, Hv, K, V, io);
  if (saved) TRY(check_room(saved, saved_bytes, l.saved_end, "saved"));
  TRY(check_room(workspace, workspace_bytes, saved ? 256 : l.plan_end, "workspace"));

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  DeltaArgs a{};
  a.q = q; a.k = k; a.v = v; a.sq = q_stride; a.sk = k_stride; a.sv = v_stride;
  a.g = g; a.beta = beta; a.cu = cu_seqlens; a.T = T; a.num_seqs = num_seqs;
  a.Hk = Hk; a.Hv = Hv; a.K = K; a.V = V; a.scale = scale; a.out = out;
  a.initial = initial_states; a.final_states = final_states;
  a.status = static_cast<int*>(workspace);
  a.wait_ns = debug_knobs().wait_ns;
  a.force_timeout_cta = debug_knobs().force_copy_timeout;
  a.max_chunks = delta_max_chunks(T, num_seqs);
  a.key = plan_key(T, num_seqs, Hk, Hv, K, V, io);
  set_plan(a, saved ? saved : workspace, l, saved != nullptr);
  TRY(check(launch_delta_plan(a, st), "gated delta plan launch"));
  TRY(check(launch_delta_prep(a, io, st), "gated delta chunk launch"));
  TRY(check(launch_delta_fwd(a, io, st), "gated delta forward launch"));
  const void* outs[] = {out, final_states};
  const int64_t counts[] = {T * Hv * V, (int64_t)num_seqs * Hv * K * V};
  const bool f32[] = {io == IO::F32, true};
  return check_outputs_finite(a.status, st, outs, counts, f32, final_states ? 2 : 1);
}

int varlen_gated_delta_bwd(const void* dout, float scale, const int32_t* cu_seqlens, int32_t num_seqs,
                           int64_t total_tokens, int32_t Hk, int32_t Hv, int32_t K, int32_t V, vssm_dtype dtype,
                           const void* saved, size_t saved_bytes, const float* d_final_states,
                           float* d_initial_states, void* dq, void* dk, void* dv, float* dg, float* dbeta,
                           void* workspace, size_t workspace_bytes, void* stream) {
  Range range_("varlen_gated_delta_bwd");
  IO io;
  TRY(check_dtype(dtype, &io));
  const int64_t T = total_tokens;
  TRY(check_pack(T, num_seqs, cu_seqlens, Hk, Hv, K, V));
  TRY(check_ptr(dout, "dout", T > 0));
  TRY(check_ptr(dq, "dq", T > 0));
  TRY(check_ptr(dk, "dk", T > 0));
  TRY(check_ptr(dv, "dv", T > 0));
  if (T > 0 && (!dg || !dbeta)) return bad(VSSM_ERR_ARG, "dg and dbeta must be non-NULL");
  TRY(check_ptr(d_final_states, "d_final_states", false));
  TRY(check_ptr(d_initial_states, "d_initial_states", false));
  const DeltaLayout l = delta_layout(T, num_seqs, Hk, Hv, K, V, io);
  TRY(check_room(saved, saved_bytes, l.saved_end, "saved"));
  TRY(check_room(workspace, workspace_bytes, l.bwd_end, "workspace"));

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  DeltaArgs a{};
  a.T = T; a.num_seqs = num_seqs;
  a.Hk = Hk; a.Hv = Hv; a.K = K; a.V = V; a.scale = scale; a.dout = dout;
  a.d_final = d_final_states; a.d_initial = d_initial_states;
  a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta;
  a.status = static_cast<int*>(workspace);
  a.wait_ns = debug_knobs().wait_ns;
  a.force_timeout_cta = debug_knobs().force_copy_timeout;
  a.max_chunks = delta_max_chunks(T, num_seqs);
  a.key = plan_key(T, num_seqs, Hk, Hv, K, V, io);
  set_plan(a, saved, l, true);
  a.ds = reinterpret_cast<uint8_t*>(static_cast<char*>(workspace) + l.ds);
  a.dvi = reinterpret_cast<uint8_t*>(static_cast<char*>(workspace) + l.dvi);
  a.doi = reinterpret_cast<uint8_t*>(static_cast<char*>(workspace) + l.doi);
  a.partial = l.bwd_end > l.partial ? reinterpret_cast<float*>(static_cast<char*>(workspace) + l.partial) : nullptr;
  TRY(check(cudaMemsetAsync(workspace, 0, 128, st), "clearing the status word"));
  TRY(check(launch_delta_bwd(a, io, st), "gated delta backward launch"));
  TRY(check(launch_delta_grads(a, io, st), "gated delta gradients launch"));
  const void* outs[] = {dq, dk, dv, dg, dbeta, d_initial_states};
  const int64_t counts[] = {T * Hk * K, T * Hk * K, T * Hv * V, T * Hv, T * Hv, (int64_t)num_seqs * Hv * K * V};
  const bool w = io == IO::F32;
  const bool f32[] = {w, w, w, true, true, true};
  return check_outputs_finite(a.status, st, outs, counts, f32, d_initial_states ? 6 : 5);
}

int varlen_gated_delta_step(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                            int64_t v_stride, const float* g, const float* beta, float scale, float* states,
                            const int32_t* state_indices, int64_t num_slots, int64_t batch, int32_t Hk, int32_t Hv,
                            int32_t K, int32_t V, vssm_dtype dtype, void* out, int32_t* status, void* stream) {
  Range range_("varlen_gated_delta_step");
  IO io;
  TRY(check_dtype(dtype, &io));
  if (batch < 0 || num_slots < 0) return bad(VSSM_ERR_ARG, "batch and num_slots must be >= 0");
  TRY(check_heads(Hk, Hv, K, V));
  if (batch > 2147483647LL || batch * Hv * ((V + 31) / 32) > 2147483647LL) return bad(VSSM_ERR_UNSUPPORTED, "batch %lld too large", (long long)batch);
  if (!state_indices && batch > num_slots)
    return bad(VSSM_ERR_ARG, "batch %lld exceeds num_slots %lld and state_indices is NULL", (long long)batch, (long long)num_slots);
  const bool any = batch > 0;
  TRY(check_ptr(q, "q", any));
  TRY(check_ptr(k, "k", any));
  TRY(check_ptr(v, "v", any));
  TRY(check_ptr(out, "out", any));
  TRY(check_ptr(states, "states", any && num_slots > 0));
  TRY(check_stride(q_stride, (int64_t)Hk * K, io, "q_stride"));
  TRY(check_stride(k_stride, (int64_t)Hk * K, io, "k_stride"));
  TRY(check_stride(v_stride, (int64_t)Hv * V, io, "v_stride"));
  if (any && (!g || !beta)) return bad(VSSM_ERR_ARG, "g and beta must be non-NULL");
  DeltaStepArgs a{q, k, v, q_stride, k_stride, v_stride, g, beta, states, state_indices, out, batch, num_slots,
                  Hk, Hv, K, V, scale, status};
  return check(launch_delta_step(a, io, static_cast<cudaStream_t>(stream)), "gated delta step launch");
}

// ---------------------------------------------------------------- norm and rotation
static int check_norm(const QkNormArgs& a, IO io) {
  if (a.T < 0 || a.T > 2147483647LL) return bad(VSSM_ERR_ARG, "total_tokens %lld out of range", (long long)a.T);
  if (a.Hq < 0 || a.Hk < 0 || (int64_t)a.Hq + a.Hk < 1 || (int64_t)a.Hq + a.Hk > 65535)
    return bad(VSSM_ERR_ARG, "Hq = %d and Hk = %d heads", a.Hq, a.Hk);
  if (a.K < 8 || a.K > 256 || a.K % 8) return bad(VSSM_ERR_UNSUPPORTED, "K = %d is not a multiple of 8 in 8..256", a.K);
  if (a.rot < 0 || a.rot > a.K || a.rot % 2) return bad(VSSM_ERR_ARG, "rot = %d is not even in 0..K", a.rot);
  if (!(a.eps >= 0.0f)) return bad(VSSM_ERR_ARG, "eps must be >= 0");
  const bool q = a.T > 0 && a.Hq > 0, k = a.T > 0 && a.Hk > 0;
  TRY(check_ptr(a.q, "q", q));
  TRY(check_ptr(a.k, "k", k));
  if (a.Hq) TRY(check_stride(a.sq, (int64_t)a.Hq * a.K, io, "q_stride"));
  if (a.Hk) TRY(check_stride(a.sk, (int64_t)a.Hk * a.K, io, "k_stride"));
  if (a.rot && a.T > 0 && (!a.cos || !a.sin || !a.pos)) return bad(VSSM_ERR_ARG, "rot = %d needs cos, sin and positions", a.rot);
  if (a.rot && a.positions < 0) return bad(VSSM_ERR_ARG, "table_rows must be >= 0");
  return VSSM_OK;
}

int varlen_qk_norm_rope_fwd(const void* q, const void* k, int64_t q_stride, int64_t k_stride,
                            const float* q_weight, const float* k_weight, const float* cos, const float* sin,
                            const int32_t* positions, int64_t table_rows, int64_t total_tokens, int32_t Hq,
                            int32_t Hk, int32_t K, int32_t rot, int32_t l2, float eps, vssm_dtype dtype,
                            void* q_out, void* k_out, int32_t* status, void* stream) {
  Range range_("varlen_qk_norm_rope_fwd");
  IO io;
  TRY(check_dtype(dtype, &io));
  QkNormArgs a{};
  a.q = q; a.k = k; a.sq = q_stride; a.sk = k_stride; a.qw = q_weight; a.kw = k_weight;
  a.cos = cos; a.sin = sin; a.pos = positions; a.T = total_tokens; a.positions = table_rows;
  a.Hq = Hq; a.Hk = Hk; a.K = K; a.rot = rot; a.l2 = l2; a.eps = eps; a.q_out = q_out; a.k_out = k_out;
  a.status = status;
  TRY(check_norm(a, io));
  TRY(check_ptr(q_out, "q_out", a.T > 0 && Hq > 0));
  TRY(check_ptr(k_out, "k_out", a.T > 0 && Hk > 0));
  return check(launch_qk_norm_fwd(a, io, static_cast<cudaStream_t>(stream)), "q/k norm launch");
}

size_t varlen_qk_norm_rope_bwd_workspace_size(int32_t K) {
  return K < 8 || K > 256 || K % 8 ? 0 : 256 + sizeof(float) * (size_t)K * qk_norm_partial_rows();
}

int varlen_qk_norm_rope_bwd(const void* q, const void* k, int64_t q_stride, int64_t k_stride,
                            const float* q_weight, const float* k_weight, const float* cos, const float* sin,
                            const int32_t* positions, int64_t table_rows, const void* dq_out, const void* dk_out,
                            int64_t total_tokens, int32_t Hq, int32_t Hk, int32_t K, int32_t rot, int32_t l2,
                            float eps, vssm_dtype dtype, void* dq, void* dk, float* dq_weight, float* dk_weight,
                            void* workspace, size_t workspace_bytes, void* stream) {
  Range range_("varlen_qk_norm_rope_bwd");
  IO io;
  TRY(check_dtype(dtype, &io));
  QkNormArgs a{};
  a.q = q; a.k = k; a.sq = q_stride; a.sk = k_stride; a.qw = q_weight; a.kw = k_weight;
  a.cos = cos; a.sin = sin; a.pos = positions; a.T = total_tokens; a.positions = table_rows;
  a.Hq = Hq; a.Hk = Hk; a.K = K; a.rot = rot; a.l2 = l2; a.eps = eps;
  a.dq_out = dq_out; a.dk_out = dk_out; a.dq = dq; a.dk = dk; a.dqw = dq_weight; a.dkw = dk_weight;
  TRY(check_norm(a, io));
  const bool any_q = a.T > 0 && Hq > 0, any_k = a.T > 0 && Hk > 0;
  TRY(check_ptr(dq_out, "dq_out", any_q));
  TRY(check_ptr(dk_out, "dk_out", any_k));
  TRY(check_ptr(dq, "dq", any_q));
  TRY(check_ptr(dk, "dk", any_k));
  TRY(check_room(workspace, workspace_bytes, varlen_qk_norm_rope_bwd_workspace_size(K), "workspace"));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  a.status = static_cast<int*>(workspace);
  a.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + 256);
  TRY(check(cudaMemsetAsync(workspace, 0, 128, st), "clearing the status word"));
  TRY(check(launch_qk_norm_bwd(a, io, st), "q/k norm backward launch"));
  const void* outs[] = {dq, dk};
  const int64_t counts[] = {any_q ? a.T * Hq * K : 0, any_k ? a.T * Hk * K : 0};
  const bool f32[] = {io == IO::F32, io == IO::F32};
  return check_outputs_finite(a.status, st, outs, counts, f32, 2);
}

}  // extern "C"
