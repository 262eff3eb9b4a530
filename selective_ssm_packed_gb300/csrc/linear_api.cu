// linear_api.cu -- the C ABI of linear attention with a decay for each head
// and of layer norm: argument checks, workspace layout, launches.
#include "api_checks.h"
#include "linear.h"

namespace {

// ---------------------------------------------------------------- linear attention
int check_lin_heads(int32_t Hk, int32_t Hv, int32_t K, int32_t V) {
  if (Hv > 65535) return bad(VSSM_ERR_UNSUPPORTED, "Hv = %d is above 65535", Hv);  // sizes then stay within 64 bits
  if (Hk < 1 || Hv < 1 || Hv % Hk) return bad(VSSM_ERR_ARG, "Hv = %d must be a positive multiple of Hk = %d", Hv, Hk);
  if (K < 8 || K > kLinMaxK || K % 8) return bad(VSSM_ERR_UNSUPPORTED, "K = %d is not a multiple of 8 in 8..%d", K, kLinMaxK);
  if (V < 8 || V > kLinMaxV || V % 8) return bad(VSSM_ERR_UNSUPPORTED, "V = %d is not a multiple of 8 in 8..%d", V, kLinMaxV);
  return VSSM_OK;
}

// Tokens of a segment, at most 4096 (whose state is 3% of the data, and over
// which dg's sums run).  An SM has `share` tokens to walk in a launch of `ctas`
// for a segment's head; where no sequence is likely to be longer than that (the
// longest is taken for four times the mean: only the GPU knows it) they are
// better left whole, which spares the walk before and the scan (32768 packed
// tokens of 32 heads in bf16: 282 us, and 361 in segments of 1792).  Otherwise a
// quarter of it fills the GPU evenly, but no fewer than 256 tokens (3001 of 6 heads
// in f32: 75 us, 85 with 128, 93 with 384; 4000 of 8 in bf16: 50 us, 67 with 128, 58
// with 512), and no pack of 512 is worth it (500 tokens in bf16: 28 us, 40 with 256).
// The bf16 backward walks two roles for the states before, and each role in a
// launch of its own: it takes all of the share (32768 tokens of 8 heads in sequences
// of up to 4096 415 us, share 1724; 523 with 512, 628 whole; 9000 of 16 heads 250,
// share 947; 388 with 256, 454 whole; one sequence of 16384, 8 heads, 286, share 862;
// 404 with 256), and leaves sequences of half as much again whole (32768 of 16 heads,
// share 3449: 592 us, 641 with 3584; of 12, share 2586: 640, and 571 with 2048).
int lin_segment(int64_t T, int64_t S, int Hv, int ctas, int parts, IO io) {
  const int64_t chunk = lin_chunk(io), share = T * Hv * ctas / 152, longest = 4 * T / (S > 0 ? S : 1);
  if (longest <= (parts == 1 ? share * 3 / 2 : share)) return kLinMaxSegment;
  const int64_t step = parts == 1 ? 2 * chunk : chunk;
  int64_t seg = (share / parts + step - 1) / step * step;
  const int64_t least = T <= 512 ? 512 : 256;
  return (int)(seg < least ? least : seg > kLinMaxSegment ? kLinMaxSegment : seg);
}

struct LinLayout {
  int seg;
  int64_t max_segs, max_inner;
  size_t table, order, inner, split, slots, decay, fwd_end;
  size_t slots_back, decay_back, rho, sigma, cross, cross_back, seg_dg, dq_part, dk_part, bwd_end;
};

LinLayout lin_layout(int64_t T, int64_t S, int Hk, int Hv, int K, int V, IO io, bool bwd) {
  LinLayout l;
  const int tk = lin_ctas(io, K), tv = lin_ctas(io, V);
  l.seg = io == IO::BF16 ? lin_segment(T, S, Hv, 1, bwd ? 1 : 4, io) : lin_segment(T, S, Hv, bwd ? 2 * tk + tv : tv, 4, io);
  l.max_inner = T > l.seg ? T / l.seg : 0;
  l.max_segs = T / l.seg + S;
  const size_t segs = (size_t)l.max_segs, inner = (size_t)l.max_inner, state = (size_t)Hv * K * V * sizeof(float);
  size_t o = 256;
  l.table = o; o += up(segs * sizeof(int4));
  l.order = o; o += up(segs * sizeof(int));
  l.inner = o; o += up(inner * sizeof(int));
  l.split = o; o += up(inner * sizeof(int2));
  l.slots = o; o += up(inner * state);
  l.decay = o; o += up(inner * Hv * sizeof(float));
  l.fwd_end = o;
  const size_t tokens = (size_t)T * Hv * sizeof(float);
  l.slots_back = o; o += up(inner * state);
  l.decay_back = o; o += up(inner * Hv * sizeof(float));
  l.rho = o; o += up(lin_dot_parts(io, K) * tokens);
  l.sigma = o; o += up(lin_dot_parts(io, K) * tokens);
  l.cross = o; o += up(segs * Hv * tk * sizeof(float));
  l.cross_back = o; o += up(segs * Hv * tk * sizeof(float));
  l.seg_dg = o; o += up(segs * Hv * sizeof(double));
  l.dq_part = o; o += Hk == Hv ? 0 : up(tokens * K);
  l.dk_part = o; o += Hk == Hv ? 0 : up(tokens * K);
  l.bwd_end = o;
  return l;
}

int check_lin_pack(int64_t T, int32_t S, const int32_t* cu, int32_t Hk, int32_t Hv, int32_t K, int32_t V) {
  if (T < 0 || T > 2147483647LL) return bad(VSSM_ERR_ARG, "total_tokens %lld out of range", (long long)T);
  if (S < 0) return bad(VSSM_ERR_ARG, "num_seqs must be >= 0 (got %d)", S);
  if (T > 0 && S < 1) return bad(VSSM_ERR_ARG, "%lld tokens but num_seqs = %d", (long long)T, S);
  if (!cu) return bad(VSSM_ERR_ARG, "cu_seqlens is NULL");
  TRY(check_lin_heads(Hk, Hv, K, V));
  // segments (at least 256 tokens each but the sequences' last), heads and tiles of three roles
  if ((T / 256 + S) * Hv * 6 > 2147483647LL)
    return bad(VSSM_ERR_UNSUPPORTED, "too many sequences, tokens and heads for one call");
  return VSSM_OK;
}

bool lin_sizes_ok(int64_t T, int32_t S, int32_t Hk, int32_t Hv, int32_t K, int32_t V, vssm_dtype dt, IO* io) {
  const int32_t cu = 0;
  return check_dtype(dt, io) == VSSM_OK && check_lin_pack(T, S, &cu, Hk, Hv, K, V) == VSSM_OK;
}

// What the two packed calls share.
LinArgs lin_args(const float* g, int32_t g_per_token, float scale, const int32_t* cu, int32_t S, int64_t T, int32_t Hk,
                 int32_t Hv, int32_t K, int32_t V, void* workspace, const LinLayout& l) {
  LinArgs a{};
  char* p = static_cast<char*>(workspace);
  a.g = g; a.g_token = g_per_token ? Hv : 0; a.cu = cu; a.T = T; a.num_seqs = S;
  a.Hk = Hk; a.Hv = Hv; a.K = K; a.V = V; a.seg = l.seg; a.scale = scale;
  a.info = reinterpret_cast<int*>(p) + 32;  // past the status word
  a.table = reinterpret_cast<int4*>(p + l.table);
  a.order = reinterpret_cast<int*>(p + l.order);
  a.inner = reinterpret_cast<int*>(p + l.inner);
  a.split = reinterpret_cast<int2*>(p + l.split);
  a.max_segs = l.max_segs; a.max_inner = l.max_inner;
  a.status = static_cast<int*>(workspace);
  a.wait_ns = debug_knobs().wait_ns;
  a.force_timeout_cta = debug_knobs().force_copy_timeout;
  return a;
}

// rows (T, H, n) of bf16, their tokens `stride` apart
int lin_map(CUtensorMap* m, const void* base, int64_t T, int H, int n, int64_t stride, IO io) {
  if (io != IO::BF16 || T == 0) return VSSM_OK;
  return encode_heads_map(m, base, T, H, n, stride, 64, 128);
}

int check_lin_inputs(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                     const float* g, bool any, int32_t Hk, int32_t Hv, int32_t K, int32_t V, IO io) {
  TRY(check_ptr(q, "q", any));
  TRY(check_ptr(k, "k", any));
  TRY(check_ptr(v, "v", any));
  TRY(check_stride(q_stride, (int64_t)Hk * K, io, "q_stride"));
  TRY(check_stride(k_stride, (int64_t)Hk * K, io, "k_stride"));
  TRY(check_stride(v_stride, (int64_t)Hv * V, io, "v_stride"));
  if (any && !g) return bad(VSSM_ERR_ARG, "g is NULL");
  return VSSM_OK;
}

// ---------------------------------------------------------------- layer norm
int check_norm_shape(int64_t T, int32_t D, int32_t groups) {
  if (T < 0 || T > 2147483647LL) return bad(VSSM_ERR_ARG, "total_tokens %lld out of range", (long long)T);
  if (groups < 1 || groups > 65535 || D < 1 || D % groups)
    return bad(VSSM_ERR_ARG, "D = %d must be a positive multiple of groups = %d", D, groups);
  const int width = D / groups;
  if (width % 8 || width > kLayerNormMaxWidth)
    return bad(VSSM_ERR_UNSUPPORTED, "D / groups = %d is not a multiple of 8 in 8..%d", width, kLayerNormMaxWidth);
  return VSSM_OK;
}

int check_layer_norm(const LayerNormArgs& a, IO x_io) {
  TRY(check_norm_shape(a.T, a.D, a.groups));
  if (!(a.eps >= 0.0f)) return bad(VSSM_ERR_ARG, "eps must be >= 0");
  TRY(check_ptr(a.x, "x", a.T > 0));
  TRY(check_stride(a.sx, a.D, x_io, "x_stride"));
  TRY(check_ptr(a.weight, "weight", false));
  TRY(check_ptr(a.bias, "bias", false));
  return VSSM_OK;
}

}  // namespace

extern "C" {

size_t varlen_linear_attn_fwd_workspace_size(int64_t T, int32_t S, int32_t Hk, int32_t Hv, int32_t K, int32_t V,
                                             vssm_dtype dt) {
  IO io;
  return lin_sizes_ok(T, S, Hk, Hv, K, V, dt, &io) ? lin_layout(T, S, Hk, Hv, K, V, io, false).fwd_end : 0;
}

size_t varlen_linear_attn_bwd_workspace_size(int64_t T, int32_t S, int32_t Hk, int32_t Hv, int32_t K, int32_t V,
                                             vssm_dtype dt) {
  IO io;
  return lin_sizes_ok(T, S, Hk, Hv, K, V, dt, &io) ? lin_layout(T, S, Hk, Hv, K, V, io, true).bwd_end : 0;
}

int vssm_linear_attn_segment(int64_t T, int32_t S, int32_t Hk, int32_t Hv, int32_t K, int32_t V, vssm_dtype dt,
                             int32_t backward) {
  IO io;
  return lin_sizes_ok(T, S, Hk, Hv, K, V, dt, &io) ? lin_layout(T, S, Hk, Hv, K, V, io, backward != 0).seg : VSSM_ERR_ARG;
}

int varlen_linear_attn_fwd(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                           int64_t v_stride, const float* g, int32_t g_per_token, float scale,
                           const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens, int32_t Hk, int32_t Hv,
                           int32_t K, int32_t V, vssm_dtype dtype, void* out, const float* initial_states,
                           float* final_states, void* workspace, size_t workspace_bytes, void* stream) {
  Range range_("varlen_linear_attn_fwd");
  IO io;
  TRY(check_dtype(dtype, &io));
  const int64_t T = total_tokens;
  TRY(check_lin_pack(T, num_seqs, cu_seqlens, Hk, Hv, K, V));
  TRY(check_lin_inputs(q, k, v, q_stride, k_stride, v_stride, g, T > 0, Hk, Hv, K, V, io));
  TRY(check_ptr(out, "out", T > 0));
  TRY(check_ptr(initial_states, "initial_states", false));
  TRY(check_ptr(final_states, "final_states", false));
  const LinLayout l = lin_layout(T, num_seqs, Hk, Hv, K, V, io, false);
  if (io == IO::F32 && final_states && final_states == initial_states && l.max_inner > 0)
    return bad(VSSM_ERR_ARG, "final_states are initial_states, which the walks of a sequence's segments (%d tokens) read meanwhile", l.seg);
  TRY(check_room(workspace, workspace_bytes, l.fwd_end, "workspace"));

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LinArgs a = lin_args(g, g_per_token, scale, cu_seqlens, num_seqs, T, Hk, Hv, K, V, workspace, l);
  char* p = static_cast<char*>(workspace);
  const int rep = Hv / Hk;
  LinRole& r = a.role[0];
  r.x = q; r.y = k; r.w = v; r.sx = q_stride; r.sy = k_stride; r.sw = v_stride;
  r.rx = r.ry = rep; r.rw = 1; r.n1 = K; r.n2 = V; r.out = out;
  r.srow = V; r.scol = 1; r.first = initial_states; r.last = final_states;
  r.slots = reinterpret_cast<float*>(p + l.slots);
  r.decay = reinterpret_cast<float*>(p + l.decay);
  r.mx = 0; r.my = 1; r.mw = 2;
  LinMaps maps{};
  TRY(lin_map(maps.m + 0, q, T, Hk, K, q_stride, io));
  TRY(lin_map(maps.m + 1, k, T, Hk, K, k_stride, io));
  TRY(lin_map(maps.m + 2, v, T, Hv, V, v_stride, io));
  TRY(check(launch_lin_plan(a, st), "linear attention plan launch"));
  TRY(check(launch_lin_walk(a, maps, 1, true, io, st), "linear attention state launch"));
  TRY(check(launch_lin_scan(a, 1, st), "linear attention scan launch"));
  TRY(check(launch_lin_walk(a, maps, 1, false, io, st), "linear attention forward launch"));
  if (io == IO::BF16 && final_states) TRY(check(launch_lin_state_bf16(a, maps, 1, true, st), "linear attention final state launch"));
  const void* outs[] = {out, final_states};
  const int64_t counts[] = {T * Hv * V, (int64_t)num_seqs * Hv * K * V};
  const bool f32[] = {io == IO::F32, true};
  return check_outputs_finite(a.status, st, outs, counts, f32, final_states ? 2 : 1);
}

int varlen_linear_attn_bwd(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                           int64_t v_stride, const float* g, int32_t g_per_token, const void* dout, float scale,
                           const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens, int32_t Hk, int32_t Hv,
                           int32_t K, int32_t V, vssm_dtype dtype, const float* initial_states,
                           const float* d_final_states, float* d_initial_states, void* dq, void* dk, void* dv,
                           float* dg, void* workspace, size_t workspace_bytes, void* stream) {
  Range range_("varlen_linear_attn_bwd");
  IO io;
  TRY(check_dtype(dtype, &io));
  const int64_t T = total_tokens;
  TRY(check_lin_pack(T, num_seqs, cu_seqlens, Hk, Hv, K, V));
  TRY(check_lin_inputs(q, k, v, q_stride, k_stride, v_stride, g, T > 0, Hk, Hv, K, V, io));
  TRY(check_ptr(dout, "dout", T > 0));
  TRY(check_ptr(initial_states, "initial_states", false));
  TRY(check_ptr(d_final_states, "d_final_states", false));
  TRY(check_ptr(d_initial_states, "d_initial_states", false));
  TRY(check_ptr(dq, "dq", T > 0));
  TRY(check_ptr(dk, "dk", T > 0));
  TRY(check_ptr(dv, "dv", T > 0));
  const LinLayout l = lin_layout(T, num_seqs, Hk, Hv, K, V, io, true);
  if (io == IO::F32 && d_initial_states && (d_initial_states == d_final_states || d_initial_states == initial_states))
    return bad(VSSM_ERR_ARG, "d_initial_states is an array of states that the walks of other gradients read meanwhile");
  TRY(check_room(workspace, workspace_bytes, l.bwd_end, "workspace"));

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LinArgs a = lin_args(g, g_per_token, scale, cu_seqlens, num_seqs, T, Hk, Hv, K, V, workspace, l);
  char* p = static_cast<char*>(workspace);
  const int rep = Hv / Hk;
  const int64_t so = (int64_t)Hv * V;  // tokens of dout
  float* slots = reinterpret_cast<float*>(p + l.slots);
  float* slots_back = reinterpret_cast<float*>(p + l.slots_back);
  a.dg = dg;
  a.seg_dg = reinterpret_cast<double*>(p + l.seg_dg);
  a.dq = dq; a.dk = dk;
  a.dq_part = reinterpret_cast<float*>(p + l.dq_part);
  a.dk_part = reinterpret_cast<float*>(p + l.dk_part);
  LinMaps maps{};
  TRY(lin_map(maps.m + 0, q, T, Hk, K, q_stride, io));
  TRY(lin_map(maps.m + 1, k, T, Hk, K, k_stride, io));
  TRY(lin_map(maps.m + 2, v, T, Hv, V, v_stride, io));
  TRY(lin_map(maps.m + 3, dout, T, Hv, V, so, io));
  TRY(check(launch_lin_plan(a, st), "linear attention plan launch"));

  LinArgs s = a;  // the states before the segments and their gradients behind them
  LinRole& fs = s.role[0];
  fs.y = k; fs.w = v; fs.sy = k_stride; fs.sw = v_stride; fs.rx = 1; fs.ry = rep; fs.rw = 1; fs.n1 = K; fs.n2 = V;
  fs.srow = V; fs.scol = 1; fs.first = initial_states; fs.slots = slots;
  fs.decay = reinterpret_cast<float*>(p + l.decay);
  fs.my = 1; fs.mw = 2;
  LinRole& bs = s.role[1];
  bs = fs;
  bs.y = q; bs.w = dout; bs.sy = q_stride; bs.sw = so; bs.back = 1; bs.first = d_final_states; bs.slots = slots_back;
  bs.decay = reinterpret_cast<float*>(p + l.decay_back);
  bs.my = 0; bs.mw = 3;
  TRY(check(launch_lin_walk(s, maps, 2, true, io, st), "linear attention state launch"));
  TRY(check(launch_lin_scan(s, 2, st), "linear attention scan launch"));

  LinRole& rq = a.role[0];
  rq.x = dout; rq.y = v; rq.w = k; rq.sx = so; rq.sy = v_stride; rq.sw = k_stride;
  rq.rx = rq.ry = 1; rq.rw = rep; rq.n1 = V; rq.n2 = K;
  rq.out = rep > 1 ? a.dq_part : dq; rq.part = rep > 1;
  rq.srow = 1; rq.scol = V; rq.first = initial_states; rq.slots = slots;
  LinRole& rv = a.role[2];
  rv.x = k; rv.y = q; rv.w = dout; rv.sx = k_stride; rv.sy = q_stride; rv.sw = so;
  rv.rx = rv.ry = rep; rv.rw = 1; rv.n1 = K; rv.n2 = V; rv.out = dv; rv.back = 1;
  rv.srow = V; rv.scol = 1; rv.first = d_final_states; rv.last = d_initial_states; rv.slots = slots_back;
  LinRole& rk = a.role[1];
  rk.x = v; rk.y = dout; rk.w = q; rk.sx = v_stride; rk.sy = so; rk.sw = q_stride;
  rk.rx = rk.ry = 1; rk.rw = rep; rk.n1 = V; rk.n2 = K;
  rk.out = rep > 1 ? a.dk_part : dk; rk.part = rep > 1; rk.back = 1;
  rk.srow = 1; rk.scol = V; rk.first = d_final_states; rk.slots = slots_back;
  rq.mx = 3; rq.my = 2; rq.mw = 1;
  rv.mx = 1; rv.my = 0; rv.mw = 3;
  rk.mx = 2; rk.my = 3; rk.mw = 0;
  if (dg) {
    rq.dot = q; rq.sdot = q_stride; rq.rdot = rep; rq.dots = reinterpret_cast<float*>(p + l.rho);
    rq.against = slots_back; rq.against_last = d_final_states; rq.cross = reinterpret_cast<float*>(p + l.cross);
    if (initial_states) {
      rk.against_last = initial_states;
      rk.cross = reinterpret_cast<float*>(p + l.cross_back);
    }
    rk.dot = k; rk.sdot = k_stride; rk.rdot = rep; rk.dots = reinterpret_cast<float*>(p + l.sigma);
  }
  TRY(check(launch_lin_walk(a, maps, 3, false, io, st), "linear attention backward launch"));
  if (io == IO::BF16 && d_initial_states) {
    s.role[0] = s.role[1];
    s.role[0].last = d_initial_states;
    TRY(check(launch_lin_state_bf16(s, maps, 1, true, st), "linear attention initial state launch"));
  }
  if (dg) TRY(check(launch_lin_dg(a, io, st), "linear attention decay gradient launch"));
  if (rep > 1) TRY(check(launch_lin_head_sum(a, io, st), "linear attention head sum launch"));
  const void* outs[] = {dq, dk, dv, dg, d_initial_states};
  const int64_t counts[] = {T * Hk * K, T * Hk * K, T * Hv * V, dg ? (g_per_token ? T * Hv : Hv) : 0,
                            d_initial_states ? (int64_t)num_seqs * Hv * K * V : 0};
  const bool w = io == IO::F32;
  const bool f32[] = {w, w, w, true, true};
  return check_outputs_finite(a.status, st, outs, counts, f32, 5);
}

int varlen_linear_attn_step(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                            int64_t v_stride, const float* g, int32_t g_per_token, float scale, float* states,
                            const int32_t* state_indices, int64_t num_slots, int64_t batch, int32_t Hk, int32_t Hv,
                            int32_t K, int32_t V, vssm_dtype dtype, void* out, int32_t* status, void* stream) {
  Range range_("varlen_linear_attn_step");
  IO io;
  TRY(check_dtype(dtype, &io));
  if (batch < 0 || num_slots < 0) return bad(VSSM_ERR_ARG, "batch and num_slots must be >= 0");
  TRY(check_lin_heads(Hk, Hv, K, V));
  if (batch > 2147483647LL || batch * Hv * ((V + 31) / 32) > 2147483647LL)
    return bad(VSSM_ERR_UNSUPPORTED, "batch %lld too large", (long long)batch);
  if (!state_indices && batch > num_slots)
    return bad(VSSM_ERR_ARG, "batch %lld exceeds num_slots %lld and state_indices is NULL", (long long)batch, (long long)num_slots);
  const bool any = batch > 0;
  TRY(check_lin_inputs(q, k, v, q_stride, k_stride, v_stride, g, any, Hk, Hv, K, V, io));
  TRY(check_ptr(out, "out", any));
  TRY(check_ptr(states, "states", any && num_slots > 0));
  LinStepArgs a{q, k, v, q_stride, k_stride, v_stride, g, g_per_token ? Hv : 0, states, state_indices, out, batch,
                num_slots, Hk, Hv, K, V, scale, status};
  return check(launch_lin_step(a, io, static_cast<cudaStream_t>(stream)), "linear attention step launch");
}

// ---------------------------------------------------------------- layer norm
int varlen_layer_norm_fwd(const void* x, int64_t x_stride, const float* residual, const float* weight,
                          const float* bias, int64_t total_tokens, int32_t D, int32_t groups, float eps,
                          vssm_dtype dtype, void* out, float* sum, void* stream) {
  Range range_("varlen_layer_norm_fwd");
  IO io;
  TRY(check_dtype(dtype, &io));
  LayerNormArgs a{};
  a.x = x; a.sx = x_stride; a.residual = residual; a.weight = weight; a.bias = bias; a.T = total_tokens;
  a.D = D; a.groups = groups; a.eps = eps; a.out = out; a.sum = sum;
  TRY(check_layer_norm(a, io));
  TRY(check_ptr(residual, "residual", false));
  TRY(check_ptr(out, "out", a.T > 0));
  TRY(check_ptr(sum, "sum", false));
  if (sum && !residual && a.T > 0) return bad(VSSM_ERR_ARG, "sum needs a residual");
  return check(launch_layer_norm_fwd(a, io, static_cast<cudaStream_t>(stream)), "layer norm launch");
}

size_t varlen_layer_norm_bwd_workspace_size(int64_t T, int32_t D, int32_t groups) {
  if (check_norm_shape(T, D, groups) != VSSM_OK) return 0;
  return 256 + up(2 * sizeof(float) * (size_t)layer_norm_slots(T, D, groups) * (D / groups));
}

int varlen_layer_norm_bwd(const void* x, int64_t x_stride, int32_t x_f32, const float* weight, const void* dout,
                          const float* dsum, int64_t total_tokens, int32_t D, int32_t groups, float eps,
                          vssm_dtype dtype, void* dx, float* dresidual, float* dweight, float* dbias,
                          void* workspace, size_t workspace_bytes, void* stream) {
  Range range_("varlen_layer_norm_bwd");
  IO io;
  TRY(check_dtype(dtype, &io));
  LayerNormArgs a{};
  a.x = x; a.sx = x_stride; a.weight = weight; a.dout = dout; a.dsum = dsum; a.T = total_tokens; a.D = D;
  a.groups = groups; a.eps = eps; a.dx = dx; a.dresidual = dresidual; a.dweight = dweight; a.dbias = dbias;
  const bool wide = x_f32 || io == IO::F32;
  TRY(check_layer_norm(a, wide ? IO::F32 : io));
  TRY(check_ptr(dout, "dout", a.T > 0));
  TRY(check_ptr(dsum, "dsum", false));
  TRY(check_ptr(dx, "dx", a.T > 0));
  TRY(check_ptr(dresidual, "dresidual", false));
  TRY(check_room(workspace, workspace_bytes, varlen_layer_norm_bwd_workspace_size(a.T, D, groups), "workspace"));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  a.status = static_cast<int*>(workspace);
  a.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + 256);
  TRY(check(cudaMemsetAsync(workspace, 0, 128, st), "clearing the status word"));
  TRY(check(launch_layer_norm_bwd(a, io, wide, st), "layer norm backward launch"));
  const int64_t rows = a.T * D;
  const void* outs[] = {dx, dresidual, dweight, dbias};
  const int64_t counts[] = {rows, dresidual ? rows : 0, dweight ? D : 0, dbias ? D : 0};
  const bool f32[] = {io == IO::F32, true, true, true};
  return check_outputs_finite(a.status, st, outs, counts, f32, 4);
}

}  // extern "C"
