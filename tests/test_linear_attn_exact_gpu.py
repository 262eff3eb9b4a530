"""How exact linear attention is on the GPU, where its first tests look at a
whole tensor's norm or leave room for more: results in bf16, states and decays'
gradients of bf16 calls, decays that forget, tails without a gradient, values
that are not finite, at the widths of one and of two panels of 64 columns.

Errors and references are 2-norms over what is named.
"""
import numpy as np
import pytest
import torch

import selective_ssm_packed_gb300 as vs
from selective_ssm_packed_gb300 import binding
from test_linear_attn_gpu import bits, close, host, inputs, reference, run

pytestmark = pytest.mark.gpu

WIDTHS = [(64, 64), (128, 128), (128, 64), (64, 128)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from selective_ssm_packed_gb300 import build
    build.build()
    binding.lib()


def rounded(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16).double().numpy()


def off(got, ref):
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("lens", [[500, 130, 3], [3000]])
@pytest.mark.parametrize("K,V", WIDTHS)
def test_bf16_results_lose_no_more_than_their_rounding(K, V, lens):
    """A result that is off by e before it is rounded gets another bf16 value than the exact one with a probability of
    |e| / step, and is then one step off: the squares add up to |e| step, the step being 2^-7 of the value at most.  An
    operand of two terms is 2^-17 off at most, and a result has three of them: e is 3 * 2^-17 < 2^-15 of the size of
    the values, so that what differs is sqrt(2^-15 * 2^-7) = 2^-11."""
    x = inputs(lens, 1, 2, K, V, "bf16", 40, True)
    got, ref = run(x, states=True), reference(x)
    for n in ("out", "dq", "dk", "dv"):
        assert off(host(got[n]), rounded(ref[n])) <= 2.0 ** -11, n
    g = vs.varlen_linear_attn_bwd(x["q"], x["k"], x["v"], x["g"], x["dout"], x["cu"], initial_states=x["init"],
                                  d_final_states=x["dfinal"], dg=False)
    for n in ("dq", "dk", "dv"):
        assert off(host(g[n]), rounded(ref[n])) <= 2.0 ** -11, n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [1e-4, 1e-2, 0.5])
@pytest.mark.parametrize("K,V", WIDTHS)
def test_states_carry_24_bits(K, V, decay, dtype):
    """bf16 inputs and f32 ones: weights are 2^-22 off (the power) and the products' operands 2^-24; sums are of f32, 900
    tokens in steps of 16 and three terms, of which the matrix unit may cut off each time up to 2^-24 of the running
    sum: 168 * 2^-24 = 1e-5 were all of one sign and as large, and sqrt(168) * 2^-24 = 8e-7 as they are of both.  With the
    weights, 2^-20."""
    x = inputs([900, 70], 1, 2, K, V, dtype, 41, True)
    x["g"] = (-decay * torch.exp(0.5 * torch.randn(x["g"].shape, generator=torch.Generator().manual_seed(1)))).cuda()
    got, ref = run(x, states=True), reference(x)
    for n in ("final", "dinit"):
        assert off(host(got[n]), ref[n]) <= 2.0 ** -20, n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", WIDTHS)
def test_dg_of_decays_that_forget_within_a_token(K, V, dtype):
    """dg falls as exp(g), and so do all its terms but the token's own pair, which is none of them.  Two walks make each
    pair's weight, by powers 2^-22 off; what they differ by adds up over a segment as its square root: of 300
    tokens 17 * 2^-22 = 4e-6, and a weight's own rounding to two terms is 2^-17 at most: 2^-16 in all, of each head's own
    size."""
    x = inputs([300, 40], 2, 4, K, V, dtype, 42)
    x["g"] = torch.tensor([-3.0, -6.0, -9.0, -12.0], device="cuda").expand(340, 4).contiguous()
    got, ref = host(run(x)["dg"]), reference(x)["dg"]
    for h in range(4):
        assert off(got[:, h], ref[:, h]) <= 2.0 ** -16, h


@pytest.mark.parametrize("decay", [2e-3, 2e-2, 0.3, 4.0])
@pytest.mark.parametrize("K,V", WIDTHS)
def test_dg_of_bf16_calls_keeps_an_f32_s_digits(K, V, decay):
    """With all operands of three terms what is left is the powers' 2^-22 and the sums' rounding, as in f32 calls: a
    token's rho and sigma are a few 2^-22 off, which over the 600 tokens of a segment add up as their square root, 25 * 2^-22,
    of a rho, and dg of slow decays is a sum of as many of them: 2^-19 of dg at all decays."""
    x = inputs([600, 100], 1, 2, K, V, "bf16", 43)
    x["g"] = (-decay * torch.exp(0.5 * torch.randn(x["g"].shape, generator=torch.Generator().manual_seed(2)))).cuda()
    assert off(host(run(x)["dg"]), reference(x)["dg"]) <= 2.0 ** -19


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", WIDTHS)
def test_dg_of_a_tail_without_gradient_is_zero(K, V, dtype):
    x = inputs([400, 30], 1, 2, K, V, dtype, 44)
    x["dout"][300:400] = 0  # a masked loss
    dg = run(x)["dg"]
    assert (dg[300:400] == 0).all()
    assert (dg[1:300] != 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_dg_behind_a_large_token_keeps_its_own_scale(dtype):
    """Token 100 has a key of 1000 times the others' size, which token 110 forgets.  What the pairs of tokens 101 to 109 are
    off by, a few 2^-22 of 1000 times a pair, is not theirs behind it, of which there are 290: as of decays that forget,
    2^-16 of their own size."""
    x = inputs([400], 1, 2, 64, 64, dtype, 45)
    x["k"][100] *= 1000
    x["g"][110] = -60.0
    got, ref = host(run(x)["dg"]), reference(x)["dg"]
    for h in range(2):
        assert off(got[111:, h], ref[111:, h]) <= 2.0 ** -16, h


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["q", "k", "v", "dout"])
@pytest.mark.parametrize("K,V", WIDTHS)
def test_dg_beside_a_value_that_is_not_finite(K, V, name, bad, dtype):
    """dg_t has the pairs (s, r) with s < t <= r: a bad q or dout at token b reaches dg of b and of what is before it; a bad
    k or v what is behind it, and in a sum over the rest of the segment what is before it, too."""
    for b in (50 + 140, 50 + 290):  # chunks before the last and the last, without gradients of the final states
        x = inputs([50, 300, 20], 1, 2, K, V, dtype, 46)
        clean = run(x)["dg"]
        x[name][b, 0, 5] = bad
        dg = run(x)["dg"]
        for lo, hi in ((0, 50), (350, 370)):
            assert torch.equal(bits(dg[lo:hi]), bits(clean[lo:hi]))
        behind = dg[b + 1:350, 0]
        if name in ("q", "dout"):
            assert not torch.isfinite(dg[b, 0]).any()
            close("dg", behind, host(clean[b + 1:350, 0]), dtype)
        else:
            assert not torch.isfinite(behind).any()


KINDS = ["steep", "very steep", "none", "mixed", "growing"]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("K,V", WIDTHS)
def test_decays_of_every_size(K, V, kind, dtype):
    x = inputs([420, 40], 1, 2, K, V, dtype, 47, True)
    g, r = x["g"], np.random.default_rng(1)
    if kind == "steep":
        g.fill_(-6.0)
    elif kind == "very steep":
        g.copy_(torch.from_numpy(-np.exp(r.uniform(2, 5.5, g.shape))).float())
    elif kind == "none":
        g[r.integers(0, 460, 20)] = float("-inf")
        g[r.integers(0, 460, 20)] = -1e30
    elif kind == "mixed":
        g[100:140] = -40.0
        g[150:160] = 0.0
        g[200] = -300.0
    else:
        g.copy_(torch.from_numpy(r.uniform(-0.05, 0.04, g.shape)).float())
    got, ref = run(x, states=True), reference(x)
    for n, t in got.items():
        close(n, t, ref[n], dtype, max(np.linalg.norm(ref[n]), 0.05 * np.linalg.norm(ref["dv"])) if n == "dg" else None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("name", ["q", "k", "v", "dout"])
@pytest.mark.parametrize("K,V", WIDTHS[1:])
def test_a_value_that_is_not_finite_reaches_what_the_formulas_carry_it_to(K, V, name, bad, dtype):
    lens, t, c = [50, 400, 20], 50 + 140, 5
    x = inputs(lens, 1, 2, K, V, dtype, 48, True)
    clean = run(x, states=True)
    x[name][t, 0, c] = bad
    got = run(x, states=True)
    heads = [0] if name in ("v", "dout") else [0, 1]
    spans = {"out": {"q": (t, t + 1), "k": (t, 450), "v": (t, 450)}, "dq": {"k": (t, 450), "v": (t, 450), "dout": (t, t + 1)},
             "dk": {"q": (50, t + 1), "v": (t, t + 1), "dout": (50, t + 1)}, "dv": {"q": (50, t + 1), "k": (t, t + 1), "dout": (50, t + 1)}}
    column = {("out", "v"), ("dq", "k"), ("dk", "q"), ("dv", "dout")}  # it stays in its column
    for n, by in spans.items():
        hit = torch.zeros_like(got[n], dtype=torch.bool)
        if name in by:
            lo, hi = by[name]
            for h in heads if n in ("out", "dv") else [0]:
                hit[(slice(lo, hi), h, c) if (n, name) in column else (slice(lo, hi), h)] = True
        assert not torch.isfinite(got[n][hit]).any(), n
        assert torch.equal(bits(got[n])[~hit], bits(clean[n])[~hit]), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dg", [True, False])
@pytest.mark.parametrize("T", [300, 900])  # one segment, several; three chunks and more
@pytest.mark.parametrize("K,V", WIDTHS)
def test_a_wait_that_runs_out_is_reported(K, V, T, dg, dtype):
    x = inputs([T], 1, 2, K, V, dtype, 49)
    a = (x["q"], x["k"], x["v"], x["g"])
    code = binding.VSSM_F32 if dtype == "f32" else binding.VSSM_BF16
    ws = torch.zeros(binding.linear_attn_bwd_workspace_size(T, 1, 1, 2, K, V, code), dtype=torch.uint8, device="cuda")
    want = vs.varlen_linear_attn_fwd(*a, x["cu"])
    grads = vs.varlen_linear_attn_bwd(*a, x["dout"], x["cu"], dg=dg)
    binding.debug_set(binding.VSSM_DBG_FORCE_COPY_TIMEOUT, 0)
    try:
        vs.varlen_linear_attn_fwd(*a, x["cu"], workspace=ws)
        assert vs.read_status(ws) == -17
        vs.varlen_linear_attn_bwd(*a, x["dout"], x["cu"], workspace=ws, dg=dg)
        assert vs.read_status(ws) == -17
    finally:
        binding.debug_set(binding.VSSM_DBG_FORCE_COPY_TIMEOUT, -1)
    again = vs.varlen_linear_attn_bwd(*a, x["dout"], x["cu"], workspace=ws, dg=dg)
    assert vs.read_status(ws) == 0
    assert torch.equal(bits(vs.varlen_linear_attn_fwd(*a, x["cu"], workspace=ws)), bits(want))
    for n, t in grads.items():
        assert t is None or torch.equal(bits(t), bits(again[n])), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[300], [900, 0, 40]])
def test_a_wait_that_runs_out_with_states_is_reported(lens, dtype):
    x = inputs(lens, 1, 2, 128, 128, dtype, 51, True)
    a = (x["q"], x["k"], x["v"], x["g"])
    code = binding.VSSM_F32 if dtype == "f32" else binding.VSSM_BF16
    n = binding.linear_attn_bwd_workspace_size(sum(lens), len(lens), 1, 2, 128, 128, code)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    want = run(x, states=True)
    binding.debug_set(binding.VSSM_DBG_FORCE_COPY_TIMEOUT, 0)
    try:
        vs.varlen_linear_attn_fwd(*a, x["cu"], workspace=ws, initial_states=x["init"], final_states=True)
        assert vs.read_status(ws) == -17
        vs.varlen_linear_attn_bwd(*a, x["dout"], x["cu"], workspace=ws, initial_states=x["init"], d_final_states=x["dfinal"],
                                  d_initial_states=True)
        assert vs.read_status(ws) == -17
    finally:
        binding.debug_set(binding.VSSM_DBG_FORCE_COPY_TIMEOUT, -1)
    got = run(x, states=True, workspace=ws)
    for m, t in want.items():
        assert torch.equal(bits(t), bits(got[m])), m
    assert vs.read_status(ws) == 0


@pytest.mark.parametrize("dtype,lens", [("f32", [200, 0, 70]), ("bf16", [200, 0, 70]), ("bf16", [900, 40])])
def test_states_may_take_the_place_of_those_a_call_comes_with(lens, dtype):
    x = inputs(lens, 1, 2, 64, 128, dtype, 52, True)
    a = (x["q"], x["k"], x["v"], x["g"])
    want = run(x, states=True)
    pool = x["init"].clone()
    out, final = vs.varlen_linear_attn_fwd(*a, x["cu"], initial_states=pool, final_states=pool)
    assert final is pool and torch.equal(bits(out), bits(want["out"])) and torch.equal(bits(pool), bits(want["final"]))
    if dtype == "bf16":
        pool = x["dfinal"].clone()
        g = vs.varlen_linear_attn_bwd(*a, x["dout"], x["cu"], initial_states=x["init"], d_final_states=pool, d_initial_states=pool)
        assert torch.equal(bits(pool), bits(want["dinit"]))
        for n in ("dq", "dk", "dv", "dg"):
            assert torch.equal(bits(g[n]), bits(want[n])), n


def test_f32_states_that_other_walks_read_are_not_written():
    x = inputs([900, 40], 1, 2, 64, 64, "f32", 53, True)
    a = (x["q"], x["k"], x["v"], x["g"])
    with pytest.raises(vs.VssmError):
        vs.varlen_linear_attn_fwd(*a, x["cu"], initial_states=x["init"], final_states=x["init"])
    for given in ("init", "dfinal"):
        with pytest.raises(vs.VssmError):
            vs.varlen_linear_attn_bwd(*a, x["dout"], x["cu"], initial_states=x["init"], d_final_states=x["dfinal"], d_initial_states=x[given])


def test_every_tensor_of_a_call_is_looked_at_for_its_device(monkeypatch):
    seen = []
    monkeypatch.setattr(binding, "_together", lambda *t: seen.append({id(x) for x in t}))
    x = inputs([20], 1, 2, 64, 64, "f32", 50, True)
    a = (x["q"], x["k"], x["v"], x["g"])

    def looks(f, *args, **kw):
        seen.clear()
        f(*args, **kw)
        given = [t for t in (*args, *kw.values(), *kw.get("grads", {}).values()) if isinstance(t, torch.Tensor)]
        assert len(seen) == 1 and all(id(t) in seen[0] for t in given), f

    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    looks(vs.varlen_linear_attn_fwd, *a, x["cu"], out=torch.empty_like(x["v"]), workspace=ws, initial_states=x["init"],
          final_states=torch.empty_like(x["init"]))
    looks(vs.varlen_linear_attn_bwd, *a, x["dout"], x["cu"], grads={"dq": torch.empty_like(x["q"])}, workspace=ws,
          initial_states=x["init"], d_final_states=x["dfinal"], d_initial_states=torch.empty_like(x["init"]))
    looks(vs.varlen_linear_attn_step, *a, torch.zeros((20, 2, 64, 64), device="cuda"), out=torch.empty_like(x["v"]),
          state_indices=torch.arange(20, dtype=torch.int32, device="cuda"), status=torch.zeros(1, dtype=torch.int32, device="cuda"))
