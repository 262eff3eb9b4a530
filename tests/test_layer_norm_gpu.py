"""Layer norm on the GPU against the oracle.

Tolerances, from the arithmetic (errors and references as 2-norms over a
tensor).  The centred row is off by the mean's rounding and its own
subtraction, 2^-24 of |h|, which the mean may dominate: the inputs' means are
at most three times their deviations, so that |h| / |h - mean| is at most
sqrt(10).  Sums of up to 8192 squares are trees of 16 in a thread and 9 or 13
levels over threads and warps: 29 * 2^-24.  Together, with the square root, the
quotient and the affine step (2^-23 each): (2 * 3.2 + 29 + 6) * 2^-24 = 2.5e-6;
the gradient has three such sums: 1e-5.  dweight and dbias add up to 4000
tokens one after the other, whose roundings grow as the square root of their
number: 64 * 2^-24 = 4e-6 more.  A sum's own error (2^-24) is below these.  bf16
outputs add one rounding, 2^-8 of each value at most.
"""
import numpy as np
import pytest
import torch

import selective_ssm_packed_gb300 as vs
from oracle import linear_attn as ol
from selective_ssm_packed_gb300 import binding

pytestmark = pytest.mark.gpu

TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {"y": 2.5e-6, "sum": 2.5e-6, "dx": 1e-5, "dresidual": 1e-5, "dweight": 1.5e-5, "dbias": 1.5e-5}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from selective_ssm_packed_gb300 import build
    build.build()
    binding.lib()


def host(t):
    return None if t is None else t.double().cpu().numpy()


def close(name, got, ref):
    tol = TOL[name] + (2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0)
    g = host(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    if ref.size:
        assert np.all(np.isfinite(g)), name
        err, size = np.linalg.norm(g - ref), np.linalg.norm(ref)
        assert err <= tol * max(size, 1e-20), f"{name}: {err / max(size, 1e-20):.3e} > {tol:.1e}"


def inputs(T, D, dtype, residual, affine, seed, wide=False):
    r = np.random.default_rng(seed)

    def dev(a, dt=torch.float32):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dt)

    x = dict(x=dev(r.standard_normal((T, D)) + r.uniform(-2, 2, (T, 1)), TDT[dtype]),
             dy=dev(r.standard_normal((T, D)) + 0.2, TDT[dtype]))
    if wide:
        rows = torch.full((T, D + 24), float("nan"), device="cuda", dtype=TDT[dtype])
        rows[:, 8:8 + D] = x["x"]
        x["x"] = rows[:, 8:8 + D]
    x["res"] = dev(r.standard_normal((T, D))) if residual else None
    x["dsum"] = dev(r.standard_normal((T, D))) if residual else None
    x["w"] = dev(1 + 0.2 * r.standard_normal(D)) if affine else None
    x["b"] = dev(r.standard_normal(D)) if affine else None
    return x


def run(x, groups, eps=1e-5, **kw):
    res = vs.varlen_layer_norm_fwd(x["x"], x["w"], x["b"], groups=groups, eps=eps, residual=x["res"], **kw)
    y, h = res if x["res"] is not None else (res, x["x"])
    g = vs.varlen_layer_norm_bwd(h, x["w"], x["b"], x["dy"], groups=groups, eps=eps, residual=x["res"] is not None,
                                 dsum=x["dsum"], **kw)
    return dict(g, y=y, sum=h if x["res"] is not None else None)


def check(x, groups, eps=1e-5):
    got = run(x, groups, eps)
    h = host(x["x"]) + (host(x["res"]) if x["res"] is not None else 0.0)
    y, dx, dw, db = ol.layer_norm(h, host(x["w"]), host(x["b"]), groups, eps, host(x["dy"]))
    if x["dsum"] is not None:
        dx = dx + host(x["dsum"])
    ref = dict(y=y, sum=h, dx=dx, dresidual=dx, dweight=dw, dbias=db)
    for n, t in got.items():
        if t is None:
            assert n == "sum" and x["res"] is None or n == "dresidual" and x["res"] is None or x["w"] is None, n
        else:
            close(n, t, ref[n])


SHAPES = [(1, 8, 1), (1, 2048, 1), (3, 1000, 1), (17, 24, 3), (300, 96, 1), (130, 4096, 32), (41, 8192, 1), (257, 520, 1),
          (64, 1536, 1), (5, 12288, 48), (7, 16384, 2), (2000, 128, 2), (9, 264, 11)]


@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,D,groups", SHAPES)
def test_against_the_oracle(T, D, groups, dtype, residual, affine):
    check(inputs(T, D, dtype, residual, affine, T + D), groups)


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def same(a, b):
    for n in a:
        assert (a[n] is None) == (b[n] is None) and (a[n] is None or torch.equal(bits(a[n]), bits(b[n]))), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("residual", [True, False])
def test_slices_of_wider_rows_and_repeated_calls_have_equal_bits(residual, dtype):
    a = inputs(50, 1536, dtype, residual, True, 3)
    first = run(a, 12)
    same(first, run(a, 12))
    same(first, run(inputs(50, 1536, dtype, residual, True, 3, wide=True), 12))


@pytest.mark.parametrize("mean", [1e3, -3e4])
def test_a_mean_far_from_zero(mean):
    # the mean's rounding, 2^-24 |mean|, and that of its difference are what is lost: 4 * 2^-24 |mean| of a deviation
    x = inputs(20, 2048, "f32", False, False, 4)
    x["x"] += mean
    y = vs.varlen_layer_norm_fwd(x["x"])
    ref = ol.layer_norm(host(x["x"]))
    assert np.linalg.norm(host(y) - ref) <= 4 * 2.0 ** -24 * abs(mean) * np.linalg.norm(ref)


def test_rows_without_variance():
    for dtype in ("f32", "bf16"):
        x = inputs(6, 256, dtype, False, True, 5)
        x["x"][2] = 3.0
        x["x"][4] = 0.0
        check(x, 2)
        check(x, 2, eps=0.25)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_row_that_is_not_finite_stays_alone(bad, dtype):
    x = inputs(40, 512, dtype, True, True, 6)
    clean = run(x, 4)
    x["x"][7, 130] = bad  # the second group
    got = run(x, 4)
    touched = torch.zeros((40, 512), dtype=torch.bool, device="cuda")
    touched[7, 128:256] = True
    for n in ("y", "dx", "dresidual"):
        assert torch.isnan(got[n][touched]).all(), n
        assert torch.equal(bits(got[n])[~touched], bits(clean[n])[~touched]), n
    for n in ("dweight", "dbias"):
        rest = torch.ones(512, dtype=torch.bool, device="cuda")
        if n == "dweight":
            rest[128:256] = False
            assert torch.isnan(got[n][~rest]).all()
        assert torch.equal(bits(got[n])[rest], bits(clean[n])[rest]), n


def test_no_tokens():
    x = inputs(0, 64, "bf16", True, True, 7)
    got = run(x, 2)
    assert got["y"].shape == (0, 64) and (got["dweight"] == 0).all() and (got["dbias"] == 0).all()


def test_the_sum_may_take_the_residual_s_place():
    x = inputs(30, 512, "bf16", True, True, 8)
    y, h = vs.varlen_layer_norm_fwd(x["x"], x["w"], x["b"], residual=x["res"])
    stream = x["res"].clone()
    y2, h2 = vs.varlen_layer_norm_fwd(x["x"], x["w"], x["b"], residual=stream, sum_out=stream)
    assert h2 is stream and torch.equal(bits(h), bits(stream)) and torch.equal(bits(y), bits(y2))
    assert torch.equal(h, x["res"] + x["x"].float())


def test_gradients_asked_for_change_no_other_bits():
    x = inputs(100, 512, "bf16", False, True, 9)
    full = run(x, 2)
    g = vs.varlen_layer_norm_bwd(x["x"], x["w"], None, x["dy"], groups=2)
    assert g["dbias"] is None and torch.equal(g["dweight"], full["dweight"]) and torch.equal(bits(g["dx"]), bits(full["dx"]))


def test_captured_calls_take_new_inputs():
    x, y = (inputs(100, 1000, "bf16", True, True, s) for s in (10, 11))
    want = run(y, 1)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(x, 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(x, 1)
    for n in ("x", "dy", "res", "dsum", "w", "b"):
        x[n].copy_(y[n])
    graph.replay()
    torch.cuda.synchronize()
    same(got, want)


def test_calls_on_a_given_stream():
    x = inputs(100, 1000, "bf16", True, True, 12)
    want = run(x, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(x, 1, stream=side)
    side.synchronize()
    same(got, want)


def test_offsets_past_32_bits():
    T, D = 263000, 8192
    assert T * D > 2 ** 31
    x = torch.zeros((T, D), device="cuda", dtype=torch.bfloat16)
    gen = torch.Generator(device="cuda").manual_seed(0)
    x[-3:] = torch.randn((3, D), generator=gen, device="cuda").bfloat16()
    w = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
    tail = x[-3:].contiguous()
    assert torch.equal(bits(vs.varlen_layer_norm_fwd(x, w)[-3:]), bits(vs.varlen_layer_norm_fwd(tail, w)))
    g = vs.varlen_layer_norm_bwd(x, w, None, x)
    assert torch.equal(bits(g["dx"][-3:]), bits(vs.varlen_layer_norm_bwd(tail, w, None, tail)["dx"]))


def test_status_of_the_backward_when_asked():
    x = inputs(10, 64, "f32", False, True, 13)
    n = binding.lib().varlen_layer_norm_bwd_workspace_size(10, 64, 1)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    binding.debug_set(binding.VSSM_DBG_CHECK_FINITE, 1)
    try:
        vs.varlen_layer_norm_bwd(x["x"], x["w"], x["b"], x["dy"], workspace=ws)
        assert vs.read_status(ws) == 0
        x["dy"][3, 3] = float("inf")
        vs.varlen_layer_norm_bwd(x["x"], x["w"], x["b"], x["dy"], workspace=ws)
        assert vs.read_status(ws) == -18
    finally:
        binding.debug_set(binding.VSSM_DBG_CHECK_FINITE, 0)


def test_binding_refuses():
    x = inputs(10, 64, "bf16", True, True, 14)
    with pytest.raises(TypeError):
        vs.varlen_layer_norm_fwd(x["x"], x["w"], x["b"], residual=x["res"].bfloat16())
    with pytest.raises(ValueError):
        vs.varlen_layer_norm_fwd(x["x"], x["w"][:32])
    with pytest.raises(ValueError):
        vs.varlen_layer_norm_fwd(x["x"], sum_out=x["res"])
    with pytest.raises(ValueError):
        vs.varlen_layer_norm_fwd(x["x"].t())
    with pytest.raises(ValueError):
        vs.varlen_layer_norm_fwd(x["x"][None])
    with pytest.raises(vs.VssmError):
        vs.varlen_layer_norm_fwd(x["x"], groups=3)
    with pytest.raises(vs.VssmError):
        vs.varlen_layer_norm_fwd(x["x"], groups=16)  # groups of 4
    with pytest.raises(vs.VssmError):
        vs.varlen_layer_norm_fwd(x["x"], eps=-1.0)
    with pytest.raises(vs.VssmError):
        vs.varlen_layer_norm_fwd(x["x"][:, :60].contiguous())
    with pytest.raises(TypeError):
        vs.varlen_layer_norm_bwd(x["x"], x["w"], x["b"], x["dy"], residual=True)  # x has to be the sum
    with pytest.raises(TypeError):
        vs.varlen_layer_norm_bwd(x["res"], x["w"], x["b"], x["dy"])
    with pytest.raises(ValueError):
        vs.varlen_layer_norm_bwd(x["x"], x["w"], x["b"], x["dy"], dsum=x["dsum"])
    with pytest.raises(ValueError):
        vs.varlen_layer_norm_bwd(x["x"], x["w"], x["b"], x["dy"][:5])


# ------------------------------------------------------------------ with the attention it stands around
def test_a_layer_of_linear_attention_and_its_gradients():
    """Residual stream -> layer norm -> projections -> q/k norm -> linear attention -> norm of each head -> projection,
    forward and backward through the calls, against 64-bit autograd of the formulas.

    FP32 throughout: each call is within 4e-5 of its formula, and the chain has six of them, none of which
    amplifies a relative error by more than a few times here: 1e-3.
    """
    lens, D, Hk, Hv, K, V = [30, 1, 45], 64, 2, 4, 32, 16
    r = np.random.default_rng(15)
    T, cu = sum(lens), torch.tensor([0, 30, 31, 76], dtype=torch.int32, device="cuda")
    widths = [Hk * K, Hk * K, Hv * V]

    def dev(*shape, s=1.0):
        return torch.from_numpy((s * r.standard_normal(shape)).astype(np.float32)).cuda()

    x, res, W, Wo = dev(T, D), dev(T, D), dev(D, sum(widths), s=D ** -0.5), dev(Hv * V, D, s=(Hv * V) ** -0.5)
    w1, b1, w2, b2 = 1 + dev(D, s=0.1), dev(D, s=0.1), 1 + dev(Hv * V, s=0.1), dev(Hv * V, s=0.1)
    g = -torch.exp(dev(T, Hv) - 1)
    dy, dres = dev(T, D), dev(T, D)

    # the calls
    n1, h = vs.varlen_layer_norm_fwd(x, w1, b1, residual=res)
    p = n1 @ W
    q, k, v = (t.unflatten(1, s) for t, s in zip(p.split(widths, 1), ((Hk, K), (Hk, K), (Hv, V))))
    qn, kn = vs.varlen_qk_norm_rope_fwd(q, k, mode="l2")
    o = vs.varlen_linear_attn_fwd(qn, kn, v, g, cu)
    n2 = vs.varlen_layer_norm_fwd(o.flatten(1), w2, b2, groups=Hv)
    y = n2 @ Wo
    g2 = vs.varlen_layer_norm_bwd(o.flatten(1), w2, b2, dy @ Wo.t(), groups=Hv)
    ga = vs.varlen_linear_attn_bwd(qn, kn, v, g, g2["dx"].unflatten(1, (Hv, V)), cu)
    gq = vs.varlen_qk_norm_rope_bwd(q, k, None, None, None, None, None, ga["dq"], ga["dk"], mode="l2")
    dp = torch.cat([gq["dq"].flatten(1), gq["dk"].flatten(1), ga["dv"].flatten(1)], 1)
    g1 = vs.varlen_layer_norm_bwd(h, w1, b1, dp @ W.t(), residual=True, dsum=dres)
    got = dict(y=y, dx=g1["dx"], dres=g1["dresidual"], dW=n1.t() @ dp, dg=ga["dg"], dw1=g1["dweight"], db1=g1["dbias"],
               dw2=g2["dweight"], db2=g2["dbias"], dWo=n2.t() @ dy)

    # the formulas
    leaf = {n: t.double().cpu().requires_grad_() for n, t in
            dict(x=x, res=res, W=W, Wo=Wo, w1=w1, b1=b1, w2=w2, b2=b2, g=g).items()}

    def norm(t, groups, w, b, eps=1e-5):
        u = t.unflatten(1, (groups, -1))
        u = u - u.mean(-1, keepdim=True)
        return (u / (u.square().mean(-1, keepdim=True) + eps).sqrt()).flatten(1) * w + b

    h64 = leaf["x"] + leaf["res"]
    p64 = norm(h64, 1, leaf["w1"], leaf["b1"]) @ leaf["W"]
    q6, k6, v6 = (t.unflatten(1, s) for t, s in zip(p64.split(widths, 1), ((Hk, K), (Hk, K), (Hv, V))))
    q6, k6 = ((t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt()).repeat_interleave(Hv // Hk, 1) for t in (q6, k6))
    outs, at = [], 0
    for n in lens:
        S = torch.zeros(Hv, K, V, dtype=torch.float64)
        for t in range(at, at + n):
            S = S * leaf["g"][t].exp()[:, None, None] + k6[t][:, :, None] * v6[t][:, None, :]
            outs.append(K ** -0.5 * (q6[t][:, None, :] @ S)[:, 0])
        at += n
    y64 = norm(torch.stack(outs).flatten(1), Hv, leaf["w2"], leaf["b2"]) @ leaf["Wo"]
    ((y64 * dy.double().cpu()).sum() + (h64 * dres.double().cpu()).sum()).backward()
    ref = dict(y=y64.detach(), dx=leaf["x"].grad, dres=leaf["res"].grad, dW=leaf["W"].grad, dg=leaf["g"].grad,
               dw1=leaf["w1"].grad, db1=leaf["b1"].grad, dw2=leaf["w2"].grad, db2=leaf["b2"].grad, dWo=leaf["Wo"].grad)
    for n, t in got.items():
        err = (t.double().cpu() - ref[n]).norm() / ref[n].norm()
        assert err <= 1e-3, (n, float(err))
