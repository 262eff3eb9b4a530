"""The gated delta rule's rarer paths on the GPU: waits that run out, packs of
every walk width, what a call must leave alone."""
import numpy as np
import pytest
import torch

import selective_ssm_packed_gb300 as vs
from selective_ssm_packed_gb300 import binding
from oracle import gated_delta as od
from test_gated_delta_gpu import NET, check, host, inputs, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from selective_ssm_packed_gb300 import build
    build.build()
    binding.lib()


def buffers(x, dtype):
    """(saved, workspace) large enough for both directions."""
    T, Hk, K = x["q"].shape
    Hv, V = x["v"].shape[1:]
    sizes = (T, x["cu"].numel() - 1, Hk, Hv, K, V, 0 if dtype == "f32" else 1)
    size = max(binding.gated_delta_fwd_workspace_size(*sizes), binding.gated_delta_bwd_workspace_size(*sizes))
    return [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in (binding.gated_delta_saved_size(*sizes), size)]


@pytest.mark.parametrize("dtype,lens,Hk,Hv,K,V", [
    ("f32", [5, 300, 0, 77], 2, 4, 96, 80), ("bf16", [700], 1, 2, 128, 128),
    ("bf16", [40, 130, 10, 60] * 10, 4, 12, 64, 72), ("bf16", [64, 200, 30, 90, 16] * 5, 8, 32, 128, 136)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(dtype, lens, Hk, Hv, K, V):
    # the knob has one CTA of each kernel treat its first wait as run out once it is over: nothing is withheld
    x = inputs(lens, Hk, Hv, K, V, dtype, 40, states=True)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    ref = run(x, states=True)
    saved, ws = buffers(x, dtype)
    for cta in (0, 3):
        try:
            binding.debug_set(binding.VSSM_DBG_FORCE_COPY_TIMEOUT, cta)
            vs.varlen_gated_delta_fwd(*a, x["cu"], saved=False, workspace=ws, initial_states=x["init"], final_states=True)
            assert binding.read_status(ws) == -17
            vs.varlen_gated_delta_fwd(*a, x["cu"], saved=saved, workspace=ws, initial_states=x["init"])
            assert binding.read_status(ws) == -17
        finally:
            binding.debug_set(binding.VSSM_DBG_FORCE_COPY_TIMEOUT, -1)
        out, _, final = vs.varlen_gated_delta_fwd(*a, x["cu"], saved=saved, workspace=ws, initial_states=x["init"],
                                                  final_states=True)
        assert binding.read_status(ws) == 0
        assert torch.equal(out, ref["out"]) and torch.equal(final, ref["final"])
        try:
            binding.debug_set(binding.VSSM_DBG_FORCE_COPY_TIMEOUT, cta)
            vs.varlen_gated_delta_bwd(*a, x["dout"], x["cu"], saved, workspace=ws, d_final_states=x["dfinal"],
                                      d_initial_states=True)
            assert binding.read_status(ws) == -17
        finally:
            binding.debug_set(binding.VSSM_DBG_FORCE_COPY_TIMEOUT, -1)
        g = vs.varlen_gated_delta_bwd(*a, x["dout"], x["cu"], saved, workspace=ws, d_final_states=x["dfinal"],
                                      d_initial_states=True)
        assert binding.read_status(ws) == 0
        for n in ("dq", "dk", "dv", "dg", "dbeta", "d_initial_states"):
            assert torch.equal(g[n], ref[n]), n


def bad_case(kind, dtype, lens, Hk, Hv, K, V, states):
    """Inputs with a value that is not finite at one token of a sequence, and the same without it."""
    x = inputs(lens, Hk, Hv, K, V, dtype, 41, states=states)
    s = int(np.argmax(lens))
    start, end = int(sum(lens[:s])), int(sum(lens[:s + 1]))
    at = start + 64 * ((end - start) // 128) + 21  # inside a chunk, others before and behind it
    y = dict(x, **{n: x[n].clone() for n in ("q", "k", "v", "g", "beta")}, init=x["init"].clone() if states else None)
    nan, inf = float("nan"), float("inf")
    if kind == "v":
        y["v"][at, 0, 3], y["v"][at, Hv - 1, V - 1], y["v"][at + 2, 0, 5] = inf, nan, -inf
    elif kind == "k":
        y["k"][at, 0, K - 1] = nan
    elif kind == "k first":
        at = start + 64 * ((end - start) // 128)
        y["k"][at, 0, 0] = inf
    elif kind == "q":
        y["q"][at, 0, 1] = nan
    elif kind == "g":
        y["g"][at, Hv - 1] = nan
    elif kind == "beta":
        y["beta"][at, 0] = nan
    elif kind == "last beta":
        at = start + 64 * ((end - start) // 128) + 63
        y["beta"][at, 0] = inf
    else:
        at = start
        y["init"][s, 0, 0, 2] = nan
    return x, y, at, s


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["v", "k", "k first", "q", "g", "beta", "last beta", "init"])
@pytest.mark.parametrize("lens,Hk,Hv,K,V", [([5, 300, 77], 1, 2, 64, 72), ([40, 130, 10, 60] * 10, 3, 12, 40, 72),
                                            ([64, 200, 30, 90, 16] * 5, 8, 32, 128, 136)])
def test_what_is_not_finite_reaches_later_tokens_only(lens, Hk, Hv, K, V, kind, dtype):
    x, y, at, s = bad_case(kind, dtype, lens, Hk, Hv, K, V, states=True)
    ref, got = run(x, states=True, bwd=False), run(y, states=True, bwd=False)
    assert torch.equal(got["out"][:at], ref["out"][:at])
    # where the recurrence is finite, so are the results, and they are as if the value were not there
    with np.errstate(invalid="ignore"):
        out, final = od.delta_fwd(*(host(y[n]) for n in ("q", "k", "v", "g", "beta")), y["cu"].cpu().numpy(), K ** -0.5,
                                  host(y["init"]))
    for n, want in (("out", out), ("final", final)):
        fine = torch.from_numpy(np.isfinite(want)).cuda()
        assert torch.equal(torch.isfinite(got[n]), fine), n
        assert torch.equal(got[n][fine], ref[n][fine]), n
    assert not np.isfinite(out[at:]).all() and np.isfinite(out[:at]).all()
    # with the saved array the outputs are the same
    saved = run(y, states=True)
    assert torch.equal(saved["out"].nan_to_num(7.0), got["out"].nan_to_num(7.0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["v", "k", "q", "g", "beta", "init", "dout", "dfinal"])
def test_gradients_of_what_is_not_finite_are_nan_or_right(kind, dtype):
    K, V = 64, 72
    if kind.startswith("d"):
        y = inputs([5, 300, 77], 1, 2, K, V, dtype, 41, states=True)
        y["dout"][200, 1, 5] = float("nan") if kind == "dout" else 1.0
        y["dfinal"][1, 0, 3, 7] = float("inf") if kind == "dfinal" else 1.0
    else:
        y = bad_case(kind, dtype, [5, 300, 77], 1, 2, K, V, states=True)[1]
    got = run(y, states=True)
    with np.errstate(invalid="ignore", over="ignore"):
        want = od.delta_bwd(*(host(y[n]) for n in ("q", "k", "v", "g", "beta", "dout")), y["cu"].cpu().numpy(), K ** -0.5,
                            host(y["init"]), host(y["dfinal"]))
    for n in ("dq", "dk", "dv", "dg", "dbeta", "d_initial_states"):
        g, w = host(got[n]), want["dinit" if n == "d_initial_states" else n]
        fine = np.isfinite(g)
        assert np.isfinite(w[fine]).all(), n
        tol = NET[dtype] + (2.0 ** -8 if got[n].dtype == torch.bfloat16 else 0.0)
        assert np.linalg.norm(g[fine] - w[fine]) <= tol * np.linalg.norm(w[fine]), n
        assert fine[np.r_[0:1, 2:3] if n == "d_initial_states" else np.r_[0:5, 305:382]].all(), n  # the other sequences


def test_a_missing_tensor_is_refused_by_name():
    x = inputs([4], 1, 2, 16, 16, "f32", 42)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    out, saved = vs.varlen_gated_delta_fwd(*a, x["cu"], saved=False)
    assert saved is None
    with pytest.raises(TypeError, match="saved"):
        vs.varlen_gated_delta_bwd(*a, x["dout"], x["cu"], saved)
    with pytest.raises(TypeError, match="saved"):
        vs.varlen_gated_delta_bwd(*a, x["dout"], x["cu"], torch.zeros(4, dtype=torch.uint8))
    for call in (lambda cu: vs.varlen_gated_delta_fwd(*a, cu), lambda cu: vs.varlen_gated_delta_bwd(*a, x["dout"], cu, out)):
        with pytest.raises(TypeError, match="cu_seqlens"):
            call(None)
        with pytest.raises(ValueError, match="cu_seqlens"):
            call(x["cu"][:0])
    with pytest.raises(TypeError, match="states"):
        vs.varlen_gated_delta_step(*a, None)
    with pytest.raises(ValueError, match="states"):
        vs.varlen_gated_delta_step(*a, torch.zeros((), device="cuda"))


# packs of every walk width, with CTAs that have fewer tiles than walks (V = 72, 136) and sequences of several chunks
PACKS = {2: [([40, 130, 10, 260] * 8, 4, 12, 64, 72), ([40, 130, 10, 60] * 10, 12, 12, 128, 128)],
         4: [([64, 200, 30, 90, 16] * 5, 8, 32, 40, 136), ([64, 200, 30, 90, 16] * 5, 8, 32, 128, 128)]}


def walks(lens, Hk, Hv, K, V, dtype="bf16"):
    return binding.gated_delta_walks(sum(lens), len(lens), Hk, Hv, K, V, 0 if dtype == "f32" else 1)


@pytest.mark.parametrize("pack", [(w, i) for w in PACKS for i in range(2)], ids=str)
def test_every_walk_width_against_the_oracle(pack):
    # the last pack's gradients are more than two items a CTA as well
    w, i = pack
    assert walks(*PACKS[w][i]) == w and walks(*PACKS[w][i], "f32") == 1
    x = inputs(*PACKS[w][i], "bf16", 43, states=True)
    check(x, run(x, states=True), "bf16")


@pytest.mark.parametrize("w", [2, 4])
def test_every_walk_width_gives_a_sequence_the_same_bits(w):
    for lens, Hk, Hv, K, V in PACKS[w]:
        x = inputs(lens, Hk, Hv, K, V, "bf16", 44, states=True)
        ref = run(x, states=True)
        for _ in range(5):
            again = run(x, states=True)
            assert all(torch.equal(again[n], t) for n, t in ref.items())
        for s in (0, 1, len(lens) // 2, len(lens) - 1):
            lo = sum(lens[:s])
            one = {n: x[n][lo:lo + lens[s]].contiguous() for n in ("q", "k", "v", "g", "beta", "dout")}
            one.update(init=x["init"][s:s + 1], dfinal=x["dfinal"][s:s + 1],
                       cu=torch.tensor([0, lens[s]], dtype=torch.int32, device="cuda"))
            assert walks(lens[s:s + 1], Hk, Hv, K, V) == 1
            for n, t in run(one, states=True).items():
                whole = ref[n][s:s + 1] if n in ("final", "d_initial_states") else ref[n][lo:lo + lens[s]]
                assert torch.equal(t, whole), (n, s)


def test_a_training_pack_gives_its_last_sequence_the_same_bits():
    # 32768 tokens, 32 heads of 128 x 128: two and four walks to a CTA, tens of gradient items to another
    lens, Hk, Hv, K, V = [4096, 700, 3396, 64, 8000, 16000, 212, 300], 16, 32, 128, 128
    assert sum(lens) == 32768
    gen = torch.Generator(device="cuda").manual_seed(5)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    T = sum(lens)
    q, k = (torch.nn.functional.normalize(normal(T, Hk, K), dim=-1).bfloat16() for _ in range(2))
    x = dict(q=q, k=k, v=normal(T, Hv, V).bfloat16(), g=-normal(T, Hv).square(), beta=normal(T, Hv).sigmoid(),
             dout=normal(T, Hv, V).bfloat16(), init=None, dfinal=None)
    for cuts, w in ((lens, 2), ([n // 4 for n in lens for _ in range(4)], 4)):
        assert walks(cuts, Hk, Hv, K, V) == w
        x["cu"] = torch.tensor(np.cumsum([0] + cuts), dtype=torch.int32, device="cuda")
        ref = run(x, states=True)
        one = dict(x, **{n: x[n][-cuts[-1]:] for n in ("q", "k", "v", "g", "beta", "dout")},
                   cu=torch.tensor([0, cuts[-1]], dtype=torch.int32, device="cuda"))
        for n, t in run(one, states=True).items():
            assert torch.equal(t, ref[n][-1:] if n in ("final", "d_initial_states") else ref[n][-cuts[-1]:]), n


@pytest.mark.parametrize("lens,Hk,Hv,K,V", [([700], 1, 2, 128, 128), PACKS[2][0], PACKS[4][1]])
def test_bf16_results_lose_no_more_than_their_rounding(lens, Hk, Hv, K, V):
    # A bf16 result is a value that is NET off, rounded.  Rounding to nearest moves a value by some e that depends on it
    # as if at random, so the errors' squares add: |result - exact|^2 = |bf16(exact) - exact|^2 + (NET |exact|)^2, the
    # latter under (1.2e-4 / 1.66e-3)^2 = 0.6% of the former.  An operand of one term (2^-9 a value, 3e-3 over the whole)
    # would make it four times as much.  10% of the norm is 21% of the squares.
    x = inputs(lens, Hk, Hv, K, V, "bf16", 45, states=True)
    res = run(x, states=True)
    a, cu = [host(x[n]) for n in ("q", "k", "v", "g", "beta")], x["cu"].cpu().numpy()
    want = od.delta_bwd(*a, host(x["dout"]), cu, K ** -0.5, host(x["init"]), host(x["dfinal"]))
    want["out"] = od.delta_fwd(*a, cu, K ** -0.5, host(x["init"]))[0]
    for n in ("out", "dq", "dk", "dv"):
        w = torch.from_numpy(want[n])
        rounded = (w.float().bfloat16().double() - w).norm()
        assert (res[n].double().cpu() - w).norm() <= 1.1 * rounded, n


def sentinels(x):
    """Result tensors full of a value of their own, and a check that they still are."""
    T, Hk, K = x["q"].shape
    Hv, V = x["v"].shape[1:]
    S = x["cu"].numel() - 1
    io = x["q"].dtype
    shapes = {"out": ((T, Hv, V), io), "final": ((S, Hv, K, V), torch.float32), "dq": ((T, Hk, K), io),
              "dk": ((T, Hk, K), io), "dv": ((T, Hv, V), io), "dg": ((T, Hv), torch.float32),
              "dbeta": ((T, Hv), torch.float32), "dinit": ((S, Hv, K, V), torch.float32)}
    t = {n: torch.full(s, -7.0, dtype=d, device="cuda") for n, (s, d) in shapes.items()}
    return t, lambda: all(bool((v == -7.0).all()) for v in t.values())


@pytest.mark.parametrize("dtype,Hv,V", [("f32", 1, 16), ("f32", 4, 40), ("bf16", 2, 136)])
@pytest.mark.parametrize("cu", [[0, 10, 5, 20], [1, 20], [0, 30], [0, 19], [0, -5, 20]])
def test_a_refused_pack_or_saved_array_leaves_every_result_alone(cu, dtype, Hv, V):
    x = inputs([20], 1, Hv, 16, V, dtype, 46)
    x["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    saved, ws = buffers(x, dtype)
    t, untouched = sentinels(x)
    vs.varlen_gated_delta_fwd(*a, x["cu"], out=t["out"], saved=saved, workspace=ws, final_states=t["final"])
    assert binding.read_status(ws) == -16 and untouched()
    vs.varlen_gated_delta_fwd(*a, x["cu"], out=t["out"], saved=False, workspace=ws, final_states=t["final"])
    assert binding.read_status(ws) == -16 and untouched()
    grads = {n: t[n] for n in ("dq", "dk", "dv", "dg", "dbeta")}
    vs.varlen_gated_delta_bwd(*a, x["dout"], x["cu"], saved, grads=grads, workspace=ws, d_initial_states=t["dinit"])
    assert binding.read_status(ws) == -16 and untouched()
    for fill in (0, 255):
        saved.fill_(fill)
        vs.varlen_gated_delta_bwd(*a, x["dout"], x["cu"], saved, grads=grads, workspace=ws, d_initial_states=t["dinit"])
        assert binding.read_status(ws) == -21 and untouched()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_serving_calls_can_be_captured_in_a_graph(dtype):
    # a decode loop's token: norm and rotation of q and k, the step against its pool; and the norm's gradients
    x = inputs([5], 2, 4, 64, 72, dtype, 47)
    pool = torch.randn(7, 4, 64, 72, generator=torch.Generator().manual_seed(1)).cuda()
    at = torch.tensor([3, -1, 0, 6, 2], dtype=torch.int32, device="cuda")
    w = torch.linspace(0.5, 1.5, 64, device="cuda")
    cos, sin = (f(torch.arange(50, device="cuda")[:, None] * torch.rand(32, device="cuda")) for f in (torch.cos, torch.sin))
    pos = torch.tensor([7, 0, 49, 3, 3], dtype=torch.int32, device="cuda")

    def token(states):
        norm = (x["q"], x["k"], w, w, cos, sin, pos)
        q, k = vs.varlen_qk_norm_rope_fwd(*norm)
        out = vs.varlen_gated_delta_step(q, k, x["v"], x["g"], x["beta"], states, state_indices=at)
        g = vs.varlen_qk_norm_rope_bwd(*norm, x["q"], x["k"])
        return dict(q=q, k=k, out=out, **g)

    states = pool.clone()
    ref = [token(states), token(states)]
    mine = pool.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = token(mine)
    assert torch.equal(mine, pool)
    for r in ref:
        for t in got.values():
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], t) for n, t in r.items())
    assert torch.equal(mine, states)


def test_a_gate_near_the_largest_exponential_keeps_its_digits():
    # exp(g) up to 2^128: 2^-22 for the exponential, and four roundings of 2^-24 in it and in the product with the state
    B = 400
    g = torch.cat([torch.linspace(85.0, 88.7, B // 2), torch.linspace(-87.0, 0.0, B // 2)]).cuda()[:, None]
    q = torch.zeros(B, 1, 8, device="cuda")
    q[:, 0, 0] = 1.0
    states = torch.full((B, 1, 8, 8), 0.5, device="cuda")
    zero = torch.zeros_like(q)
    out = vs.varlen_gated_delta_step(q, zero, zero, g, torch.zeros_like(g), states, scale=1.0)
    want = 0.5 * np.exp(host(g))[:, :, None]
    for t in (host(out), host(states)[:, :, 0]):
        assert np.abs(t / want - 1).max() <= 2.0 ** -22 + 4 * 2.0 ** -24
