"""The gated delta rule and the q/k norm on the GPU against the oracle.

Tolerances, from the arithmetic (errors and references as 2-norms over a
tensor).  An FP32 operand of a product carries 24 bits with FP32 I/O and at
least 16 with bf16 I/O (relative rounding up to 2^-16); a value passes through
at most five such operands per chunk (state, R, X, E, dV) and the rule is a
contraction for unit keys, so errors do not grow from chunk to chunk beyond
the few chunks the state remembers: 8 * 2^-16 = 1.2e-4 on FP32 outputs of bf16
calls.  FP32 calls are bounded by FP32 sums of up to 128 products in the
matrix unit (128 * 2^-24 = 8e-6) over the same steps: 4e-5.  bf16 outputs add
one rounding, 2^-8 at most of each value (8 significant bits, half a unit of
the last).
"""
import os

import numpy as np
import pytest
import torch

import selective_ssm_packed_gb300 as vs
from oracle import gated_delta as od
from selective_ssm_packed_gb300 import binding

pytestmark = pytest.mark.gpu

TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
NET = {"f32": 4e-5, "bf16": 1.2e-4}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from selective_ssm_packed_gb300 import build
    build.build()
    binding.lib()


def close(name, got, ref, dtype):
    """got: a GPU tensor of a call with I/O type dtype."""
    tol = NET[dtype] + (2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0)
    g = got.double().cpu().numpy()
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    if not ref.size:
        return
    assert np.all(np.isfinite(g)), name
    err, size = np.linalg.norm(g - ref), np.linalg.norm(ref)
    assert err <= tol * max(size, 1e-20), f"{name}: {err / max(size, 1e-20):.3e} > {tol:.1e}"


def inputs(lens, Hk, Hv, K, V, dtype, seed, states=False, bias=0.3, wide=False):
    """Seeded inputs as the device holds them.  wide: q, k, v are slices of wider rows."""
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])

    def dev(a):
        a = torch.from_numpy(np.ascontiguousarray(a)).cuda().to(TDT[dtype])
        if not wide:
            return a
        rows = torch.full((T, a.shape[1] * a.shape[2] + 24), float("nan"), device="cuda", dtype=a.dtype)
        rows[:, 8:8 + a.shape[1] * a.shape[2]] = a.flatten(1)
        return rows[:, 8:8 + a.shape[1] * a.shape[2]].unflatten(1, a.shape[1:])

    def unit(x):
        return x / np.linalg.norm(x, axis=-1, keepdims=True)

    f32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()  # noqa: E731
    x = dict(q=dev(unit(r.standard_normal((T, Hk, K)) + bias)), k=dev(unit(r.standard_normal((T, Hk, K)) + bias)),
             v=dev(r.standard_normal((T, Hv, V))), g=f32(-np.exp(r.uniform(np.log(1e-3), np.log(2.0), (T, Hv)))),
             beta=f32(r.random((T, Hv))), dout=dev(r.standard_normal((T, Hv, V))).contiguous(),
             cu=torch.from_numpy(cu).cuda())
    x["init"] = f32(0.3 * r.standard_normal((len(lens), Hv, K, V))) if states else None
    x["dfinal"] = f32(0.1 * r.standard_normal((len(lens), Hv, K, V))) if states else None
    return x


def host(t):
    return None if t is None else t.double().cpu().numpy()


def run(x, scale=None, states=False, bwd=True):
    r = vs.varlen_gated_delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], scale=scale, saved=bwd,
                                  initial_states=x["init"], final_states=states)
    res = dict(out=r[0])
    if states:
        res["final"] = r[2]
    if bwd:
        g = vs.varlen_gated_delta_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["dout"], x["cu"], r[1], scale=scale,
                                      d_final_states=x["dfinal"], d_initial_states=states)
        res.update({n: t for n, t in g.items() if t is not None})
    torch.cuda.synchronize()
    return res


def check(x, res, dtype, scale=None):
    scale = x["q"].shape[2] ** -0.5 if scale is None else scale
    a = [host(x[n]) for n in ("q", "k", "v", "g", "beta")]
    cu = x["cu"].cpu().numpy()
    out, final = od.delta_fwd(*a, cu, scale, host(x["init"]))
    close("out", res["out"], out, dtype)
    if "final" in res:
        close("final", res["final"], final, dtype)
    if "dq" in res:
        g = od.delta_bwd(*a, host(x["dout"]), cu, scale, host(x["init"]), host(x["dfinal"]))
        for n in ("dq", "dk", "dv", "dg", "dbeta"):
            close(n, res[n], g[n], dtype)
        if "d_initial_states" in res:
            close("dinit", res["d_initial_states"], g["dinit"], dtype)


LENS = {"one": [1], "tiny": [4, 2, 3, 7], "edges": [0, 1, 63, 64, 0, 65, 128, 129, 0], "ones": [1] * 70,
        "long": [700], "mix": [5, 300, 0, 77, 64, 1, 190]}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,Hk,Hv,K,V,states", [
    ("one", 1, 1, 8, 8, False), ("one", 2, 2, 128, 128, True), ("tiny", 2, 4, 64, 64, False), ("edges", 1, 2, 64, 40, True),
    ("edges", 2, 2, 128, 64, False), ("ones", 1, 3, 24, 72, True), ("long", 1, 1, 128, 128, False),
    ("long", 1, 2, 72, 32, True), ("mix", 3, 6, 96, 80, True), ("mix", 1, 4, 128, 200, False), ("mix", 1, 1, 16, 264, True),
    ("mix", 2, 2, 56, 8, False)])
def test_forward_and_backward(lens, Hk, Hv, K, V, states, dtype):
    x = inputs(LENS[lens], Hk, Hv, K, V, dtype, seed=len(lens) + K + V, states=states)
    check(x, run(x, states=states), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_inputs_and_scale(dtype):
    x = inputs(LENS["mix"], 2, 4, 64, 48, dtype, 3, states=True, wide=True)
    assert not x["q"].is_contiguous()
    check(x, run(x, scale=0.7, states=True), dtype, scale=0.7)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_keys_that_resemble_each_other(dtype):
    # nearly equal keys, slow decay: powers of the chunk's triangular matrix would grow without bound
    x = inputs([300], 1, 2, 64, 64, dtype, 4, bias=4.0)
    x["g"].fill_(-1e-3)
    x["beta"].fill_(0.95)
    check(x, run(x), dtype)


def test_gates_at_their_ends():
    # beta 0 and 1, g 0 (no decay), strong decay, and a full reset inside a sequence
    x = inputs([200, 130], 1, 2, 32, 40, "f32", 5, states=True)
    x["beta"][::3] = 0.0
    x["beta"][1::3] = 1.0
    x["g"][:64] = 0.0
    x["g"][70:90] = -30.0
    x["g"][100] = -1e30
    x["g"][250] = -float("inf")
    res = run(x, states=True)
    x["g"].clamp_(min=-700)  # the oracle's exponential of either is zero
    check(x, res, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sequences_do_not_meet(dtype):
    # a neighbour full of NaN and infinities changes no bit of the others
    lens = [37, 100, 64, 5]
    x = inputs(lens, 1, 2, 64, 72, dtype, 6, states=True)
    ref = run(x, states=True)
    lo, hi = 37, 137
    for n in ("q", "k", "v", "dout"):
        x[n][lo:hi] = float("nan")
        x[n][lo + 1:hi:2] = float("inf")
    x["g"][lo:hi] = float("nan")
    x["init"][1] = float("nan")
    x["dfinal"][1] = float("inf")
    res = run(x, states=True)
    for n, t in res.items():
        rows = [0, 2, 3] if n in ("final", "d_initial_states") else list(range(lo)) + list(range(hi, 206))
        assert torch.equal(t[rows], ref[n][rows]), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_repeats_streams_and_given_buffers(dtype):
    x = inputs([130, 70, 300], 2, 4, 64, 72, dtype, 7, states=True)
    ref = run(x, states=True)
    side = torch.cuda.Stream()
    T, Hk, K = x["q"].shape
    Hv, V = x["v"].shape[1:]
    sizes = (T, 3, Hk, Hv, K, V, 0 if dtype == "f32" else 1)
    saved = torch.full((binding.gated_delta_saved_size(*sizes),), 255, dtype=torch.uint8, device="cuda")
    ws = torch.full((binding.gated_delta_bwd_workspace_size(*sizes),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full_like(x["v"], float("nan"))
    grads = {n: torch.full_like(x[n], float("nan")) for n in ("q", "k", "v", "g", "beta")}
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        vs.varlen_gated_delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], out=out, saved=saved, workspace=ws,
                                  initial_states=x["init"])
        g = vs.varlen_gated_delta_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["dout"], x["cu"], saved, workspace=ws,
                                      grads={"d" + n: t for n, t in grads.items()}, d_final_states=x["dfinal"],
                                      d_initial_states=True)
    side.synchronize()
    assert binding.read_status(ws) == 0
    assert torch.equal(out, ref["out"])
    for n in ("dq", "dk", "dv", "dg", "dbeta", "d_initial_states"):
        assert torch.equal(g[n], ref[n]), n
    # without the saved array the forward is the same
    o2, none, f2 = vs.varlen_gated_delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], saved=False,
                                             initial_states=x["init"], final_states=True)
    assert none is None and torch.equal(o2, ref["out"]) and torch.equal(f2, ref["final"])


def test_new_memory_belongs_to_the_calls_stream():
    # the calls wait behind a busy stream while their workspaces' memory, were it the current stream's, is written
    # over by that one
    x = inputs([130, 70, 300], 2, 4, 64, 72, "bf16", 11, states=True)
    w, cos = torch.ones(64, device="cuda"), torch.ones(500, 16, device="cuda")
    pos = torch.arange(500, dtype=torch.int32, device="cuda")
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    side = torch.cuda.Stream()

    def calls(stream):
        pool = x["init"].clone()
        idx = torch.arange(3, dtype=torch.int32, device="cuda")
        if stream is not None:
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                torch.cuda._sleep(40_000_000)
        out, saved, final = vs.varlen_gated_delta_fwd(*a, x["cu"], initial_states=x["init"], final_states=True, stream=stream)
        again = vs.varlen_gated_delta_fwd(*a, x["cu"], saved=False, stream=stream)[0]
        g = vs.varlen_gated_delta_bwd(*a, x["dout"], x["cu"], saved, d_initial_states=True, stream=stream)
        qo, ko = vs.varlen_qk_norm_rope_fwd(x["q"], x["k"], w, w, cos, cos, pos, stream=stream)
        gn = vs.varlen_qk_norm_rope_bwd(x["q"], x["k"], w, w, cos, cos, pos, x["q"], x["k"], stream=stream)
        o1 = vs.varlen_gated_delta_step(*(t[:3] for t in a), pool, idx, stream=stream)
        res = dict(out=out, saved=saved, final=final, again=again, qo=qo, ko=ko, o1=o1, pool=pool,
                   **{k: t for k, t in g.items()}, **{"n" + k: t for k, t in gn.items()})
        if stream is not None:
            junk = [torch.full((1 << n,), 255, dtype=torch.uint8, device="cuda") for n in range(9, 25) for _ in range(4)]
            torch.cuda.synchronize()
            del junk
        return res

    ref = calls(None)
    got = calls(side)
    torch.cuda.synchronize()
    mine = [(s["address"], s["address"] + s["total_size"]) for s in torch.cuda.memory_snapshot()
            if s["stream"] == side.cuda_stream]
    for n, t in got.items():
        if n != "pool":
            assert any(lo <= t.data_ptr() < hi for lo, hi in mine), n
        if n != "saved":
            assert torch.equal(t, ref[n]), n


def test_a_sequence_has_the_same_bits_in_packs_of_any_size():
    # few chunks spread their value heads over CTAs, many do not
    r = []
    for lens in ([100], [100, 64 * 40], [100, 64 * 400]):
        x = inputs(lens, 2, 8, 64, 40, "bf16", 12)
        small = inputs([100], 2, 8, 64, 40, "bf16", 13)
        for n in ("q", "k", "v", "g", "beta", "dout"):
            x[n][:100] = small[n]
        r.append({n: t[:100] for n, t in run(x).items()})
    for other in r[1:]:
        for n, t in other.items():
            assert torch.equal(t, r[0][n]), n


def test_binding_refuses_what_has_no_three_axes():
    x = inputs([4], 1, 2, 16, 16, "f32", 31)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    for i, bad in ((0, a[0].flatten(1)), (2, a[2].flatten(1)), (1, a[1][0])):
        with pytest.raises(ValueError, match="tokens, "):
            vs.varlen_gated_delta_fwd(*a[:i], bad, *a[i + 1:], x["cu"])
    with pytest.raises(TypeError):
        vs.varlen_gated_delta_fwd(None, *a[1:], x["cu"])
    with pytest.raises(ValueError):
        vs.varlen_gated_delta_fwd(*a, x["cu"][:0])
    with pytest.raises(ValueError, match="tokens, "):
        vs.varlen_qk_norm_rope_fwd(a[0].flatten(1), a[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_cut_sequence_continues_from_its_state(dtype):
    x = inputs([257], 1, 2, 64, 64, dtype, 8, states=True)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    whole, _, final = vs.varlen_gated_delta_fwd(*a, x["cu"], saved=False, initial_states=x["init"], final_states=True)
    cut, state, parts = 100, x["init"], []
    for lo, hi in ((0, cut), (cut, 257)):
        p = [t[lo:hi] for t in a]
        o, _, state = vs.varlen_gated_delta_fwd(*p, torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda"),
                                                saved=False, initial_states=state, final_states=True)
        parts.append(o)
    close("out", torch.cat(parts), host(whole), dtype)
    close("final", state, host(final), dtype)


def test_gradient_against_differences():
    # the GPU's gradient along a direction against differences of the double-precision forward
    x = inputs([70, 0, 33], 1, 2, 16, 24, "f32", 9, states=True)
    res = run(x, states=True)
    a = {n: host(x[n]) for n in ("q", "k", "v", "g", "beta", "init")}
    cu, dout, dfinal = x["cu"].cpu().numpy(), host(x["dout"]), host(x["dfinal"])

    def f(y):
        o, s = od.delta_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], cu, 0.25, y["init"])
        return (o * dout).sum() + (s * dfinal).sum()

    r = np.random.default_rng(1)
    for n in a:
        d = r.standard_normal(a[n].shape)
        h = 1e-6
        diff = (f(dict(a, **{n: a[n] + h * d})) - f(dict(a, **{n: a[n] - h * d}))) / (2 * h)
        g = host(res["d_initial_states" if n == "init" else "d" + n])
        assert abs(diff - (g * d).sum()) <= NET["f32"] * np.linalg.norm(g) * np.linalg.norm(d), n


def test_no_tokens_and_empty_sequences():
    x = inputs([0, 0], 1, 2, 16, 16, "f32", 10, states=True)
    res = run(x, states=True)
    assert torch.equal(res["final"], x["init"]) and torch.equal(res["d_initial_states"], x["dfinal"])
    x["init"] = x["dfinal"] = None
    res = run(x, states=True)
    assert not res["final"].any() and not res["d_initial_states"].any()


@pytest.mark.parametrize("cu", [[0, 10, 5, 20], [1, 20], [0, 30], [0, 19], [0, -5, 20]])
def test_malformed_cu_seqlens_is_reported(cu):
    x = inputs([20], 1, 1, 16, 16, "f32", 11)
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    sizes = (20, cu.numel() - 1, 1, 1, 16, 16, 0)
    ws = torch.empty(binding.gated_delta_bwd_workspace_size(*sizes), dtype=torch.uint8, device="cuda")
    _, saved = vs.varlen_gated_delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], cu, workspace=ws)
    assert binding.read_status(ws) == -16
    vs.varlen_gated_delta_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["dout"], cu, saved, workspace=ws)
    torch.cuda.synchronize()


def test_a_saved_array_of_another_call_is_reported():
    x = inputs([20], 1, 1, 16, 16, "f32", 13)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    size = binding.gated_delta_saved_size(20, 1, 1, 1, 16, 16, 0)
    ws = torch.empty(binding.gated_delta_bwd_workspace_size(20, 1, 1, 1, 16, 16, 0), dtype=torch.uint8, device="cuda")
    for saved in (torch.zeros(size, dtype=torch.uint8, device="cuda"),
                  torch.full((size,), 255, dtype=torch.uint8, device="cuda")):
        vs.varlen_gated_delta_bwd(*a, x["dout"], x["cu"], saved, workspace=ws)
        assert binding.read_status(ws) == -21
    y = inputs([10, 10], 1, 1, 16, 16, "f32", 13)
    _, saved = vs.varlen_gated_delta_fwd(*(y[n] for n in ("q", "k", "v", "g", "beta")), y["cu"])
    vs.varlen_gated_delta_bwd(*a, x["dout"], x["cu"], saved, workspace=ws)
    assert binding.read_status(ws) == -21


def test_the_calls_can_be_captured_in_a_graph():
    x = inputs([70, 130], 1, 2, 64, 64, "bf16", 14, states=True)
    ref = run(x, states=True)  # also sizes the kernels' shared memory, before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, saved, final = vs.varlen_gated_delta_fwd(*(x[n] for n in ("q", "k", "v", "g", "beta")), x["cu"],
                                                      initial_states=x["init"], final_states=True)
        g = vs.varlen_gated_delta_bwd(*(x[n] for n in ("q", "k", "v", "g", "beta")), x["dout"], x["cu"], saved,
                                      d_final_states=x["dfinal"], d_initial_states=True)
    for t in (out, final, g["dq"]):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref["out"]) and torch.equal(final, ref["final"])
    for n in ("dq", "dk", "dv", "dg", "dbeta", "d_initial_states"):
        assert torch.equal(g[n], ref[n]), n


def test_non_finite_outputs_are_reported_when_asked():
    x = inputs([20], 1, 1, 16, 16, "f32", 12)
    ws = torch.empty(binding.gated_delta_fwd_workspace_size(20, 1, 1, 1, 16, 16, 0), dtype=torch.uint8, device="cuda")
    binding.debug_set(binding.VSSM_DBG_CHECK_FINITE, 1)
    try:
        vs.varlen_gated_delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], saved=False, workspace=ws)
        assert binding.read_status(ws) == 0
        x["v"][3] = float("inf")
        vs.varlen_gated_delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], saved=False, workspace=ws)
        assert binding.read_status(ws) == -18
    finally:
        binding.debug_set(binding.VSSM_DBG_CHECK_FINITE, 0)


@pytest.mark.slow
def test_offsets_past_32_bits():
    # 2.3e9 output values: the last sequence's bits are those of a call of its own
    T, H, K, V, tail = 140_000, 128, 16, 128, 100
    gen = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(T, 1, K, device="cuda", generator=gen).mul_(0.25).bfloat16()
    v = torch.empty(T, H, V, device="cuda", dtype=torch.bfloat16).normal_(generator=gen)
    g, beta = -torch.rand(T, H, device="cuda", generator=gen), torch.rand(T, H, device="cuda", generator=gen)
    lens = [4096] * ((T - tail) // 4096) + [(T - tail) % 4096, tail]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    out, _ = vs.varlen_gated_delta_fwd(q, q, v, g, beta, cu, saved=False)
    one = torch.tensor([0, tail], dtype=torch.int32, device="cuda")
    ref, _ = vs.varlen_gated_delta_fwd(q[-tail:], q[-tail:], v[-tail:], g[-tail:], beta[-tail:], one, saved=False)
    assert torch.equal(out[-tail:], ref)


# ------------------------------------------------------------------ one token at a time
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,slots,Hk,Hv,K,V", [(1, 1, 1, 1, 8, 8), (3, 5, 2, 4, 64, 64), (7, 7, 1, 3, 40, 72),
                                               (33, 40, 2, 2, 128, 136), (2, 3, 1, 2, 128, 1024)])
def test_step(B, slots, Hk, Hv, K, V, dtype):
    x = inputs([B], Hk, Hv, K, V, dtype, B + K + V, wide=True)
    r = np.random.default_rng(B)
    states = torch.from_numpy(r.standard_normal((slots, Hv, K, V)).astype(np.float32)).cuda()
    idx = r.permutation(slots)[:B].astype(np.int32)
    if B > 2:
        idx[1] = -1
    before = host(states)
    out = vs.varlen_gated_delta_step(x["q"], x["k"], x["v"], x["g"], x["beta"], states,
                                     state_indices=torch.from_numpy(idx).cuda())
    want, ref = np.zeros((B, Hv, V)), before.copy()
    for b in range(B):
        if idx[b] >= 0:
            o, f = od.delta_fwd(*(host(x[n])[b:b + 1] for n in ("q", "k", "v", "g", "beta")), [0, 1], K ** -0.5,
                                before[idx[b]][None])
            want[b], ref[idx[b]] = o[0], f[0]
    close("out", out, want, dtype)
    close("states", states, ref, "f32")
    untouched = np.setdiff1d(np.arange(slots), idx)
    assert np.array_equal(host(states)[untouched], before[untouched])


def test_steps_follow_the_packed_forward():
    x = inputs([65], 2, 4, 64, 64, "f32", 20, states=True)
    out, _, final = vs.varlen_gated_delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], saved=False,
                                              initial_states=x["init"], final_states=True)
    states = x["init"].clone()
    rows = [vs.varlen_gated_delta_step(*(x[n][t:t + 1] for n in ("q", "k", "v", "g", "beta")), states) for t in range(65)]
    close("out", torch.cat(rows), host(out), "f32")
    close("final", states, host(final), "f32")


def test_step_reports_an_index_outside_the_pool():
    x = inputs([3], 1, 1, 16, 16, "f32", 21)
    states = torch.ones(2, 1, 16, 16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = torch.tensor([0, 2, -1], dtype=torch.int32, device="cuda")
    out = vs.varlen_gated_delta_step(x["q"], x["k"], x["v"], x["g"], x["beta"], states, state_indices=idx, status=status)
    assert binding.status_code(status.item()) == -20
    assert torch.isnan(out[1]).all() and not out[2].any() and torch.isfinite(out[0]).all()
    assert torch.equal(states[1], torch.ones_like(states[1]))


def test_step_pool_past_32_bits():
    K = V = 128
    slots = 2 ** 31 // (K * V) + 2
    states = torch.empty(slots, 1, K, V, device="cuda")
    states[-1].normal_()
    small = states[-1:].clone()
    x = inputs([1], 1, 1, K, V, "f32", 22)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o1 = vs.varlen_gated_delta_step(*a, states, state_indices=torch.tensor([slots - 1], dtype=torch.int32, device="cuda"))
    o2 = vs.varlen_gated_delta_step(*a, small)
    assert torch.equal(o1, o2) and torch.equal(states[-1:], small)


# ------------------------------------------------------------------ norm and rotation
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,Hq,Hk,K,rot,l2,weights", [
    (1, 1, 1, 8, 8, False, True), (1, 16, 16, 128, 128, False, True), (5, 3, 2, 64, 0, True, False),
    (37, 4, 1, 72, 72, False, True), (300, 6, 3, 96, 40, True, True), (1025, 2, 2, 256, 64, False, True),
    (64, 1, 5, 24, 2, True, False), (9, 40, 0, 128, 64, False, True), (9, 0, 7, 16, 16, True, True),
    (3000, 2, 1, 40, 24, False, True)])
def test_norm_and_rotation(T, Hq, Hk, K, rot, l2, weights, dtype):
    r = np.random.default_rng(T + K)
    H = Hq + Hk
    rows = torch.from_numpy(r.standard_normal((T, (H + 1) * K)) * np.exp(r.standard_normal((H + 1) * K))).cuda().to(TDT[dtype])
    q, k = rows[:, :Hq * K].unflatten(1, (Hq, K)), rows[:, Hq * K:H * K].unflatten(1, (Hk, K))
    f32 = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
    qw, kw = (f32(r.standard_normal(K)), f32(r.standard_normal(K))) if weights else (None, None)
    cos = sin = pos = None
    if rot:
        ang = r.uniform(-3, 3, (50, rot // 2))
        cos, sin, pos = f32(np.cos(ang)), f32(np.sin(ang)), torch.from_numpy(r.integers(0, 50, T).astype(np.int32)).cuda()
    mode = "l2" if l2 else "rms"
    a = (q, k, qw, kw, cos, sin, pos)
    out = vs.varlen_qk_norm_rope_fwd(*a, mode=mode)
    dq, dk = (torch.from_numpy(r.standard_normal((T, h, K))).cuda().to(TDT[dtype]) for h in (Hq, Hk))
    g = vs.varlen_qk_norm_rope_bwd(*a, dq, dk, mode=mode)
    g2 = vs.varlen_qk_norm_rope_bwd(*a, dq, dk, mode=mode)
    table = [host(t) for t in (cos, sin)] + [None if pos is None else pos.cpu().numpy()]
    for x, w, y, dy, n in ((q, qw, out[0], dq, "q"), (k, kw, out[1], dk, "k")):
        ref, dx, dw = od.qk_norm(host(x), host(w), *table, l2, 1e-6, host(dy))
        close(n, y, ref, dtype)
        close("d" + n, g["d" + n], dx, dtype)
        if weights:
            close("dw " + n, g[f"d{n}_weight"], dw, "f32")
            assert torch.equal(g[f"d{n}_weight"], g2[f"d{n}_weight"])
        else:
            assert g[f"d{n}_weight"] is None


def test_norm_of_zero_and_huge_rows():
    x = torch.zeros(3, 2, 16, device="cuda")
    x[1] = 1e-20
    x[2] = 1e15
    for mode in ("rms", "l2"):
        y, _ = vs.varlen_qk_norm_rope_fwd(x, x, mode=mode)
        assert torch.isfinite(y).all() and not y[0].any()
        close("rows", y, od.qk_norm(host(x), l2=mode == "l2"), "f32")


def test_norm_positions_of_a_pack_and_outside_the_table():
    lens = [4, 2, 3, 7]
    cu = torch.tensor([0, 4, 6, 9, 16], dtype=torch.int32, device="cuda")
    pos = vs.varlen_position_indices(cu, 16)
    ang = np.arange(7)[:, None] * np.array([1.0, 0.1])
    cos, sin = (torch.from_numpy(f(ang).astype(np.float32)).cuda() for f in (np.cos, np.sin))
    x = torch.ones(16, 1, 8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, _ = vs.varlen_qk_norm_rope_fwd(x, x, None, None, cos, sin, pos, status=status)
    assert status.item() == 0
    start = 0
    for n in lens:  # every sequence starts at position 0 again
        assert torch.equal(y[start:start + n], y[9:9 + n])
        start += n
    pos[5] = 7
    pos[6] = -1
    y, _ = vs.varlen_qk_norm_rope_fwd(x, x, None, None, cos, sin, pos, status=status)
    assert binding.status_code(status.item()) == -20
    assert torch.isnan(y[5:7, :, :4]).all() and torch.isfinite(y[5:7, :, 4:]).all() and torch.isfinite(y[7:]).all()


def test_binding_refuses():
    x = inputs([4], 1, 2, 16, 16, "f32", 30)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    with pytest.raises(TypeError):
        vs.varlen_gated_delta_fwd(a[0].half(), *a[1:], x["cu"])
    with pytest.raises(TypeError):
        vs.varlen_gated_delta_fwd(a[0], a[1].bfloat16(), *a[2:], x["cu"])
    with pytest.raises(ValueError):
        vs.varlen_gated_delta_fwd(a[0].transpose(1, 2), *a[1:], x["cu"])
    with pytest.raises(ValueError):
        vs.varlen_gated_delta_fwd(*a[:3], a[3][:3], a[4], x["cu"])
    with pytest.raises(TypeError):
        vs.varlen_gated_delta_fwd(*a, x["cu"].long())
    with pytest.raises(vs.VssmError):
        vs.varlen_gated_delta_fwd(*a, x["cu"][:1])  # four tokens, no sequence
    with pytest.raises(ValueError):
        vs.varlen_qk_norm_rope_fwd(a[0], a[1], mode="layer")
    with pytest.raises(ValueError):
        vs.varlen_qk_norm_rope_fwd(a[0], a[1], cos=torch.ones(4, 4, device="cuda"), sin=torch.ones(4, 4, device="cuda"))
    with pytest.raises(ValueError):
        vs.varlen_gated_delta_step(*a, torch.zeros(4, 2, 16, 8, device="cuda"))


def test_example_trains_and_serves():
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "gated_delta_layer.py"), "--steps", "30"],
                       capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0, r.stdout + r.stderr
