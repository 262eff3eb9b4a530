"""Linear attention with a decay for each head on the GPU against the oracle.

Tolerances, from the arithmetic (errors and references as 2-norms over a
tensor).  An FP32 operand of a product carries 24 bits with FP32 I/O and at
least 16 with bf16 I/O (relative rounding up to 2^-16); a value passes through
at most three such operands (the weighted rows, the state, P), each of them
once a chunk, and the decays are at most 1: 8 * 2^-16 = 1.2e-4 on FP32
outputs of bf16 calls.  FP32 calls are bounded by FP32 sums of up to 128
products in the matrix unit (128 * 2^-24 = 8e-6) over the same steps: 4e-5.
bf16 outputs add one rounding, 2^-8 of each value at most.
dg sums rho - sigma over the rest of a segment, of at most 385 tokens here,
each with an error of its own: sqrt(385) times the bound on one, 2^-16 and
8e-6, is 3.0e-4 and 1.6e-4 of the size of rho, which is no larger than dg's (of
all pairs of tokens across t, rho has those that end at t); sigma doubles the
variance: 4.3e-4 and 2.3e-4.  With one decay a head these are added up: an error
of rho or sigma counts once for every token before it in its segment of n, so
the sum is off by sqrt(2 sum of i^2 over i < n) = 0.82 n^1.5 of them a segment, 0.82 n
sqrt(T) in all, that is 0.82 * 385 * 2^-16 = 4.8e-3 (bf16) or 0.82 * 385 * 8e-6 =
2.5e-3 (f32) of the 2-norm of the tokens' dg, against which it is held.
In bf16 the weights of pairs and the state that a row meets are rounded to bf16
once on the way to out and dv, 2^-9 of each value on the average of its binade and
2^-8 at most, besides the result's own rounding: 2 * 2^-8.
"""
import numpy as np
import pytest
import torch

import selective_ssm_packed_gb300 as vs
from oracle import linear_attn as ol
from selective_ssm_packed_gb300 import binding

pytestmark = pytest.mark.gpu

TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
CODE = {"f32": binding.VSSM_F32, "bf16": binding.VSSM_BF16}
NET = {"f32": 4e-5, "bf16": 1.2e-4}
DG = {"f32": 2.3e-4, "bf16": 4.3e-4}
DG_HEAD = {"f32": 2.5e-3, "bf16": 4.8e-3}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from selective_ssm_packed_gb300 import build
    build.build()
    binding.lib()


def close(name, got, ref, dtype, size=None):
    tol = {"dg": DG, "dg_head": DG_HEAD}.get(name, NET)[dtype]
    if got.dtype == torch.bfloat16:
        tol += (2 if name in ("out", "dv") else 1) * 2.0 ** -8
    g = got.double().cpu().numpy()
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    if not ref.size:
        return
    assert np.all(np.isfinite(g)), name
    err, size = np.linalg.norm(g - ref), np.linalg.norm(ref) if size is None else size
    assert err <= tol * max(size, 1e-20), f"{name}: {err / max(size, 1e-20):.3e} > {tol:.1e}"


def inputs(lens, Hk, Hv, K, V, dtype, seed, states=False, decay="token", wide=False):
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

    f32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()  # noqa: E731
    x = dict(q=dev(r.standard_normal((T, Hk, K)) + 0.3), k=dev((r.standard_normal((T, Hk, K)) + 0.3) * K ** -0.5),
             v=dev(r.standard_normal((T, Hv, V))),
             g=f32(-np.exp(r.uniform(np.log(1e-3), np.log(2.0), (T, Hv) if decay == "token" else (Hv,)))),
             dout=dev(r.standard_normal((T, Hv, V))).contiguous(), cu=torch.from_numpy(cu).cuda())
    x["init"] = f32(0.3 * r.standard_normal((len(lens), Hv, K, V))) if states else None
    x["dfinal"] = f32(0.1 * r.standard_normal((len(lens), Hv, K, V))) if states else None
    return x


def host(t):
    return None if t is None else t.double().cpu().numpy()


def run(x, scale=None, states=False, bwd=True, **kw):
    args = (x["q"], x["k"], x["v"], x["g"])
    res = vs.varlen_linear_attn_fwd(*args, x["cu"], scale=scale, initial_states=x["init"], final_states=states, **kw)
    out = {"out": res[0], "final": res[1]} if states else {"out": res}
    if bwd:
        g = vs.varlen_linear_attn_bwd(*args, x["dout"], x["cu"], scale=scale, initial_states=x["init"],
                                      d_final_states=x["dfinal"], d_initial_states=states, **kw)
        out.update({n: g[n] for n in ("dq", "dk", "dv", "dg")})
        if states:
            out["dinit"] = g["d_initial_states"]
    return out


def reference(x, scale=None, bwd=True):
    a = [host(x[n]) for n in ("q", "k", "v", "g")]
    cu, scale = x["cu"].cpu().numpy(), x["q"].shape[2] ** -0.5 if scale is None else scale
    out, final = ol.linear_fwd(*a, cu, scale, host(x["init"]))
    ref = {"out": out, "final": final}
    if bwd:
        ref.update(ol.linear_bwd(*a, host(x["dout"]), cu, scale, host(x["init"]), host(x["dfinal"])))
    return ref


def check(x, dtype, states=False, scale=None, bwd=True):
    got, ref = run(x, scale, states, bwd), reference(x, scale, bwd)
    if "dg" in got and x["g"].dim() == 1:
        got = dict(got, dg_head=got.pop("dg"))
        tokens = reference(dict(x, g=x["g"].expand(x["q"].shape[0], -1)), scale)["dg"]
        ref["dg_head"], ref["size"] = ref["dg"], np.linalg.norm(tokens)
    for n, t in got.items():
        close(n, t, ref[n], dtype, ref.get("size") if n == "dg_head" else None)


CASES = [
    # lens, Hk, Hv, K, V, states
    ([4, 2, 3, 7], 2, 4, 64, 64, False),
    ([1], 1, 1, 8, 8, True),
    ([0, 5, 0, 1, 130, 0], 1, 3, 24, 72, True),
    ([64, 65, 127, 128, 129, 63], 1, 2, 128, 128, False),
    ([700], 1, 1, 96, 80, True),
    ([513, 3, 900], 2, 2, 128, 64, True),
    ([31, 385], 1, 2, 64, 128, False),
]


@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_forward(i, dtype, decay):
    lens, Hk, Hv, K, V, states = CASES[i]
    check(inputs(lens, Hk, Hv, K, V, dtype, i, states, decay), dtype, states, bwd=False)


@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_gradients(i, dtype, decay):
    lens, Hk, Hv, K, V, states = CASES[i]
    check(inputs(lens, Hk, Hv, K, V, dtype, 10 + i, states, decay), dtype, states)


def test_a_sequence_across_segments():
    for dtype in ("f32", "bf16"):
        for back in (False, True):
            T = 789
            seg = binding.linear_attn_segment(T, 2, 1, 2, 64, 64, CODE[dtype], back)
            assert seg == 256  # the first sequence has four of them
        check(inputs([784, 5], 1, 2, 64, 64, dtype, 31, True), dtype, True)


@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decays_gradient_between_segments(dtype, decay):
    """The bf16 walks' operands have two terms, rounded by 2^-18 of a value at most and half of that on the average; dg
    sums the two walks' difference of that over a segment, from a known value at either end: with the 2^-17 of a
    pair's weight, 2^-16 = 1.5e-5 of the tokens' dg (in f32 2^-20, by three terms and FP32 sums).  A sum over T tokens is
    off by sqrt(T) times that at most."""
    x = inputs([2100, 300], 2, 4, 128, 64, dtype, 21, True, decay)
    seg = binding.linear_attn_segment(2400, 2, 2, 4, 128, 64, CODE[dtype], True)
    assert seg < 2100
    got, ref = run(x, states=True)["dg"], reference(x)["dg"]
    tokens = reference(dict(x, g=x["g"].expand(2400, -1)))["dg"] if decay == "head" else ref
    size = np.linalg.norm(tokens) * (2400 ** 0.5 if decay == "head" else 1.0)
    assert np.linalg.norm(host(got) - ref) <= {"f32": 2.0 ** -20, "bf16": 2.0 ** -16}[dtype] * size


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_states_carry_a_sequence_over_calls(dtype):
    # a sequence in two calls, the second from the first's state, and in one
    x = inputs([300], 2, 4, 72, 40, dtype, 5, True)
    whole = run(x, states=True, bwd=False)
    cut = 173
    parts, state = [], x["init"]
    for a, b in ((0, cut), (cut, 300)):
        part = {n: x[n][a:b] for n in ("q", "k", "v", "g")}
        cu = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        o, state = vs.varlen_linear_attn_fwd(*part.values(), cu, initial_states=state, final_states=True)
        parts.append(o)
    close("out", torch.cat(parts), host(whole["out"]), dtype)
    close("final", state, host(whole["final"]), dtype)


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def same(a, b):
    assert a.keys() == b.keys()
    for n in a:
        assert torch.equal(bits(a[n]), bits(b[n])), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128), (24, 40)])
def test_slices_of_wider_rows_and_repeated_calls_have_equal_bits(K, V, dtype):
    lens = [130, 1, 0, 300]
    x = inputs(lens, 2, 4, K, V, dtype, 7, True)
    first = run(x, states=True)
    same(first, run(x, states=True))
    same(first, run(inputs(lens, 2, 4, K, V, dtype, 7, True, wide=True), states=True))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_sequence_has_the_bits_it_has_alone(dtype):
    lens = [17, 200, 128, 1]
    x = inputs(lens, 2, 4, 96, 64, dtype, 8, True)
    pack = run(x, states=True)
    at = 0
    for i, n in enumerate(lens):
        one = dict(x, cu=torch.tensor([0, n], dtype=torch.int32, device="cuda"), init=x["init"][i:i + 1].contiguous(),
                   dfinal=x["dfinal"][i:i + 1].contiguous())
        one.update({k: x[k][at:at + n].contiguous() for k in ("q", "k", "v", "g", "dout")})
        alone = run(one, states=True)
        for name, t in alone.items():
            part = pack[name][i:i + 1] if name in ("final", "dinit") else pack[name][at:at + n]
            assert torch.equal(bits(part), bits(t)), (name, i)
        at += n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_what_is_asked_for_changes_no_other_bits(dtype):
    x = inputs([150, 60], 1, 2, 64, 72, dtype, 9, True)
    full = run(x, states=True)
    a = (x["q"], x["k"], x["v"], x["g"])
    assert torch.equal(bits(full["out"]), bits(vs.varlen_linear_attn_fwd(*a, x["cu"], initial_states=x["init"])))
    g = vs.varlen_linear_attn_bwd(*a, x["dout"], x["cu"], initial_states=x["init"], d_final_states=x["dfinal"])
    assert g["d_initial_states"] is None
    for n in ("dq", "dk", "dv", "dg"):
        assert torch.equal(bits(g[n]), bits(full[n])), n
    g = vs.varlen_linear_attn_bwd(*a, x["dout"], x["cu"], initial_states=x["init"], d_final_states=x["dfinal"], dg=False)
    assert g["dg"] is None
    for n in ("dq", "dk", "dv"):  # without dg, bf16 dq and dv have the rounding that dk has
        close("dk" if dtype == "bf16" else n, g[n], host(full[n]), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["steep", "very steep", "zero", "none", "mixed", "growing"])
def test_decays_of_every_size(kind, dtype):
    x = inputs([300, 40], 1, 3, 64, 64, dtype, 12, True)
    g, r = x["g"], np.random.default_rng(1)
    if kind == "steep":
        g.fill_(-6.0)
    elif kind == "very steep":  # a float's range within a few tokens
        g.copy_(torch.from_numpy(-np.exp(r.uniform(2, 5.5, g.shape))).float())
    elif kind == "zero":
        g.zero_()
    elif kind == "none":  # what went before is forgotten at single tokens
        g[r.integers(0, 340, 20)] = float("-inf")
        g[r.integers(0, 340, 20)] = -1e30
    elif kind == "mixed":
        g[100:140] = -40.0
        g[150:160] = 0.0
        g[200] = -300.0
    else:
        g.copy_(torch.from_numpy(r.uniform(-0.05, 0.04, g.shape)).float())
    got, ref = run(x, states=True), reference(x)
    for n, t in got.items():
        # dg of tokens that let through nothing is nothing: its size is that of the pairs beside it
        close(n, t, ref[n], dtype, max(np.linalg.norm(ref[n]), 0.05 * np.linalg.norm(ref["dv"])) if n == "dg" else None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_a_value_that_is_not_finite_reaches_what_the_formula_carries_it_to(name, bad, dtype):
    lens, t, c = [50, 300, 20], 50 + 140, 5
    x = inputs(lens, 1, 2, 64, 64, dtype, 13, True)
    clean = run(x, states=True, bwd=False)
    x[name][t, 0, c] = bad
    got = run(x, states=True, bwd=False)
    o, ref = got["out"], clean["out"]
    heads = [0] if name == "v" else [0, 1]  # a query and key head has two value heads
    touched = torch.zeros_like(o, dtype=torch.bool)
    for h in heads:
        if name == "q":
            touched[t, h] = True
        elif name == "k":
            touched[t:350, h] = True
        else:
            touched[t:350, h, c] = True
    assert not torch.isfinite(o[touched]).any()
    assert torch.equal(bits(o)[~touched], bits(ref)[~touched])
    f, fr = got["final"], clean["final"]
    hit = torch.zeros_like(f, dtype=torch.bool)
    for h in heads:
        if name == "k":
            hit[1, h, c] = True
        elif name == "v":
            hit[1, h, :, c] = True
    assert not torch.isfinite(f[hit]).any()
    assert torch.equal(bits(f)[~hit], bits(fr)[~hit])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["q", "k", "v", "dout"])
def test_gradients_of_other_tokens_and_sequences_stay(name, dtype):
    lens, t, c = [50, 300, 20], 50 + 140, 5
    x = inputs(lens, 1, 2, 64, 64, dtype, 14)
    clean = run(x)
    x[name][t, 0, c] = float("nan")
    got = run(x)
    for n in ("dq", "dk", "dv", "dg"):
        for a, b in ((0, 50), (350, 370)):
            assert torch.equal(bits(got[n][a:b]), bits(clean[n][a:b])), n
    # dq looks back, dk and dv look ahead
    if name in ("k", "v"):
        assert torch.equal(bits(got["dq"][50:t]), bits(clean["dq"][50:t]))
        assert not torch.isfinite(got["dq"][t:350, 0]).all(-1).any()
    if name in ("q", "dout"):
        for n in ("dk", "dv"):
            assert torch.equal(bits(got[n][t + 1:350]), bits(clean[n][t + 1:350])), n
            assert not torch.isfinite(got[n][50:t + 1, 0]).all(-1).any(), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_g_that_is_not_finite_spoils_what_follows_only(bad, dtype):
    """Earlier tokens of the chunk keep their values, not their bits: a pair's weight is exp(G_i - m) exp(m - G_j) with
    m half of the whole chunk's sum where both are normal numbers, so its rounding goes by every g of the chunk."""
    x = inputs([50, 300, 20], 1, 2, 64, 64, dtype, 15, True)
    ref = reference(x, bwd=False)["out"]
    clean = run(x, states=True, bwd=False)["out"]
    x["g"][50 + 140, 1] = bad
    o = run(x, states=True, bwd=False)["out"]
    assert not torch.isfinite(o[190:350, 1]).any()
    close("out", o[178:190, 1], ref[178:190, 1], dtype)  # the chunk starts 128 tokens into its sequence
    kept = torch.ones_like(o, dtype=torch.bool)
    kept[178:350, 1] = False
    assert torch.equal(bits(o)[kept], bits(clean)[kept])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_tokens_and_empty_sequences(dtype):
    for decay in ("token", "head"):
        x = inputs([0, 0, 0], 1, 2, 64, 64, dtype, 16, True, decay)
        got = run(x, states=True)
        assert torch.equal(got["final"], x["init"]) and torch.equal(got["dinit"], x["dfinal"])
        assert got["out"].numel() == 0 and (decay == "token" or torch.equal(got["dg"], torch.zeros(2, device="cuda")))
    x = inputs([], 1, 2, 64, 64, dtype, 16)
    assert run(x)["out"].shape == (0, 2, 64)


def test_many_short_sequences():
    lens = np.random.default_rng(0).integers(0, 4, 2500).tolist()
    check(inputs(lens, 1, 2, 16, 24, "f32", 17, True), "f32", True)
    check(inputs(lens, 1, 2, 16, 24, "bf16", 17, True), "bf16", True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_malformed_packs_are_reported_and_nothing_is_written(dtype):
    for cu in ([0, 9, 7, 12], [1, 5, 9, 12], [0, 5, 9, 11], [0, 5, 9, 13]):
        x = inputs([5, 4, 3], 1, 2, 64, 64, dtype, 18)
        x["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        out = torch.full_like(x["v"], 7.0)
        n = binding.linear_attn_bwd_workspace_size(12, 3, 1, 2, 64, 64, CODE[dtype])
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        a = (x["q"], x["k"], x["v"], x["g"])
        vs.varlen_linear_attn_fwd(*a, x["cu"], out=out, workspace=ws)
        assert vs.read_status(ws) == -16 and (out == 7).all()
        grads = {m: torch.full_like(t, 7.0) for m, t in (("dq", a[0]), ("dk", a[1]), ("dv", a[2]), ("dg", a[3]))}
        vs.varlen_linear_attn_bwd(*a, x["dout"], x["cu"], grads=grads, workspace=ws)
        assert vs.read_status(ws) == -16 and all((t == 7).all() for t in grads.values())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [40, 700])  # one segment, several
def test_a_wait_that_runs_out_is_reported(T, dtype):
    x = inputs([T], 1, 2, 64, 64, dtype, 19)
    a = (x["q"], x["k"], x["v"], x["g"])
    n = binding.linear_attn_bwd_workspace_size(T, 1, 1, 2, 64, 64, CODE[dtype])
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    binding.debug_set(binding.VSSM_DBG_FORCE_COPY_TIMEOUT, 0)
    try:
        vs.varlen_linear_attn_fwd(*a, x["cu"], workspace=ws)
        assert vs.read_status(ws) == -17
        vs.varlen_linear_attn_bwd(*a, x["dout"], x["cu"], workspace=ws)
        assert vs.read_status(ws) == -17
    finally:
        binding.debug_set(binding.VSSM_DBG_FORCE_COPY_TIMEOUT, -1)
    vs.varlen_linear_attn_fwd(*a, x["cu"], workspace=ws)
    assert vs.read_status(ws) == 0
    check(x, dtype)


def test_outputs_that_are_not_finite_are_reported_when_asked():
    x = inputs([30], 1, 1, 64, 64, "f32", 20)
    n = binding.linear_attn_fwd_workspace_size(30, 1, 1, 1, 64, 64, 0)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    binding.debug_set(binding.VSSM_DBG_CHECK_FINITE, 1)
    try:
        vs.varlen_linear_attn_fwd(x["q"], x["k"], x["v"], x["g"], x["cu"], workspace=ws)
        assert vs.read_status(ws) == 0
        x["v"][3, 0, 1] = float("nan")
        vs.varlen_linear_attn_fwd(x["q"], x["k"], x["v"], x["g"], x["cu"], workspace=ws)
        assert vs.read_status(ws) == -18
    finally:
        binding.debug_set(binding.VSSM_DBG_CHECK_FINITE, 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_calls_take_new_inputs(dtype):
    x, y = (inputs([90, 200], 2, 4, 64, 64, dtype, s, True) for s in (21, 22))
    want = run(y, states=True)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(x, states=True)  # warm-up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(x, states=True)
    for n in ("q", "k", "v", "g", "dout", "init", "dfinal"):
        x[n].copy_(y[n])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    same(got, want)


def test_calls_on_a_given_stream():
    x = inputs([300], 1, 2, 64, 64, "bf16", 23)
    want = run(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(x, stream=side)
    side.synchronize()
    same(got, want)


def test_two_calls_at_once():
    x, y = inputs([400], 1, 2, 64, 64, "bf16", 24), inputs([10, 500], 1, 3, 64, 128, "bf16", 25)
    want = run(x), run(y)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (a, b):
        s.wait_stream(torch.cuda.current_stream())
    got = [(run(x, stream=a), run(y, stream=b)) for _ in range(10)]
    torch.cuda.synchronize()
    for p, q in got:
        same(p, want[0])
        same(q, want[1])


def test_offsets_past_32_bits():
    # more than 2^31 values of v: the last sequence has the bits that it has alone
    Hv, V, n = 136, 128, 200
    lens = [4096] * 31 + [n]
    T = sum(lens)
    assert T * Hv * V > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(0)
    v = torch.randn((T, Hv, V), generator=gen, device="cuda", dtype=torch.bfloat16)
    q, k = (torch.randn((T, 1, 64), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    g = -torch.rand((Hv,), generator=gen, device="cuda")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    out = vs.varlen_linear_attn_fwd(q, k, v, g, cu)
    tail = [t[-n:].contiguous() for t in (q, k, v)]
    one = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    assert torch.equal(bits(out[-n:]), bits(vs.varlen_linear_attn_fwd(*tail, g, one)))
    del out
    grads = vs.varlen_linear_attn_bwd(q, k, v, g.expand(T, Hv).contiguous(), v, cu)
    alone = vs.varlen_linear_attn_bwd(*tail, g.expand(n, Hv).contiguous(), tail[2], one)
    for name in ("dq", "dk", "dv", "dg"):
        assert torch.equal(bits(grads[name][-n:]), bits(alone[name])), name


# ------------------------------------------------------------------ one token
def step_inputs(B, slots, Hk, Hv, K, V, dtype, seed, decay, wide=False):
    x = inputs([B], Hk, Hv, K, V, dtype, seed, decay=decay, wide=wide)
    r = np.random.default_rng(seed)
    x["states"] = torch.from_numpy(r.standard_normal((slots, Hv, K, V)).astype(np.float32)).cuda()
    x["slots"] = torch.from_numpy(r.permutation(slots)[:B].astype(np.int32)).cuda()
    return x


@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,slots,Hk,Hv,K,V,wide", [(1, 1, 1, 1, 8, 8, False), (3, 7, 2, 4, 128, 128, False),
                                                    (70, 80, 1, 8, 64, 40, True), (5, 5, 3, 3, 24, 72, True),
                                                    (200, 300, 1, 4, 128, 64, False)])
def test_step(B, slots, Hk, Hv, K, V, wide, dtype, decay):
    x = step_inputs(B, slots, Hk, Hv, K, V, dtype, B, decay, wide)
    before = x["states"].clone()
    at = x["slots"].long()
    g = host(x["g"]) if decay == "token" else np.broadcast_to(host(x["g"]), (B, Hv))
    out, final = ol.linear_fwd(host(x["q"]), host(x["k"]), host(x["v"]), g, np.arange(B + 1), 0.7, host(before[at]))
    got = vs.varlen_linear_attn_step(x["q"], x["k"], x["v"], x["g"], x["states"], state_indices=x["slots"], scale=0.7)
    # f32 sums of up to 128 products, K / 8 of them in a row: well under 4e-5
    close("step", got, out, "f32")
    close("states", x["states"][at], final, "f32")
    rest = torch.ones(slots, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(x["states"][rest], before[rest])


def test_steps_follow_a_prompt():
    x = inputs([60], 2, 4, 64, 64, "f32", 26, decay="head")
    whole = run(x, bwd=False)["out"]
    a = (x["q"], x["k"], x["v"])
    cu = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    _, states = vs.varlen_linear_attn_fwd(*(t[:40] for t in a), x["g"], cu, final_states=True)
    for t in range(40, 60):
        o = vs.varlen_linear_attn_step(*(y[t:t + 1] for y in a), x["g"], states)
        close("out", o, host(whole[t:t + 1]), "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_pads_and_reports_indices(dtype):
    x = step_inputs(4, 6, 1, 2, 64, 64, dtype, 27, "token")
    idx = torch.tensor([3, -1, 6, 0], dtype=torch.int32, device="cuda")
    before, status = x["states"].clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    o = vs.varlen_linear_attn_step(x["q"], x["k"], x["v"], x["g"], x["states"], state_indices=idx, status=status)
    assert binding.status_code(int(status)) == -20
    assert (o[1] == 0).all() and torch.isnan(o[2]).all() and torch.isfinite(o[[0, 3]]).all()
    for s in (1, 2, 4, 5):
        assert torch.equal(x["states"][s], before[s])
    assert not torch.equal(x["states"][3], before[3]) and not torch.equal(x["states"][0], before[0])


def test_captured_step():
    x = step_inputs(8, 8, 1, 2, 64, 64, "bf16", 28, "head")
    start, want = x["states"].clone(), x["states"].clone()
    a = (x["q"], x["k"], x["v"], x["g"])
    outs = [vs.varlen_linear_attn_step(*a, want, state_indices=x["slots"]) for _ in range(3)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = vs.varlen_linear_attn_step(*a, x["states"], state_indices=x["slots"])
    x["states"].copy_(start)
    for w in outs:
        graph.replay()
        assert torch.equal(bits(o), bits(w))
    assert torch.equal(x["states"], want)


def test_binding_refuses():
    x = inputs([12], 2, 4, 64, 64, "f32", 29)
    a = (x["q"], x["k"], x["v"], x["g"])
    with pytest.raises(ValueError):
        vs.varlen_linear_attn_fwd(*a[:3], x["g"][:, :3].contiguous(), x["cu"])
    with pytest.raises(ValueError):
        vs.varlen_linear_attn_fwd(*a[:3], x["g"].t(), x["cu"])
    with pytest.raises(TypeError):
        vs.varlen_linear_attn_fwd(*a[:3], x["g"].double(), x["cu"])
    with pytest.raises(TypeError):
        vs.varlen_linear_attn_fwd(a[0], a[1].bfloat16(), *a[2:], x["cu"])
    with pytest.raises(ValueError):
        vs.varlen_linear_attn_fwd(a[0][:5], *a[1:], x["cu"])
    with pytest.raises(TypeError):
        vs.varlen_linear_attn_fwd(*a, x["cu"].long())
    with pytest.raises(TypeError):
        vs.varlen_linear_attn_fwd(*a, [0, 12])
    with pytest.raises(ValueError):
        vs.varlen_linear_attn_fwd(a[0].transpose(1, 2), *a[1:], x["cu"])
    with pytest.raises(vs.VssmError):
        vs.varlen_linear_attn_fwd(*(t[..., :60].contiguous() for t in a[:2]), *a[2:], x["cu"])
    wide = torch.zeros((12, 4, 136), device="cuda")
    with pytest.raises(vs.VssmError):
        vs.varlen_linear_attn_fwd(*a[:2], wide, a[3], x["cu"])
    with pytest.raises(ValueError):
        vs.varlen_linear_attn_fwd(*a, x["cu"], workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        vs.varlen_linear_attn_bwd(*a, x["dout"][:5], x["cu"])
    with pytest.raises(ValueError):
        vs.varlen_linear_attn_step(*a, torch.zeros((4, 4, 64), device="cuda"))
    with pytest.raises(vs.VssmError):
        vs.varlen_linear_attn_step(*a, torch.zeros((4, 4, 64, 64), device="cuda"))  # 12 tokens, 4 slots
