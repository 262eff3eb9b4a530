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
