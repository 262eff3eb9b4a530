"""Layer norm on the GPU where rows lie far from zero or have no variance, and
its refusals of a bias in the backward."""
import pytest
import torch

import selective_ssm_packed_gb300 as vs
from selective_ssm_packed_gb300 import binding
from test_layer_norm_gpu import check, host, inputs, run
from oracle import linear_attn as ol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from selective_ssm_packed_gb300 import build
    build.build()
    binding.lib()


@pytest.mark.parametrize("D,groups", [(1000, 1), (264, 1), (96, 1), (5000, 1), (1320, 11)])
@pytest.mark.parametrize("mean,std", [(100.0, 1.0), (1000.0, 1.0), (10.0, 0.01), (-3e4, 30.0)])
def test_a_mean_far_from_zero_costs_no_digits(mean, std, D, groups):
    """The mean that is taken from the row is itself rounded, but what is left of it is the same in all of the row and is
    taken out of the centred row, whose own sum is exact to 2^-24 of its small size: the bounds are those of rows
    around zero."""
    x = inputs(24, D, "f32", False, True, 30)
    x["x"] = x["x"] * std + mean
    check(x, groups)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [30.0, -0.1, 3e5])
@pytest.mark.parametrize("D,groups", [(1000, 1), (264, 1), (5000, 1), (1320, 11)])
def test_constant_rows_have_no_output(D, groups, value, dtype):
    """The centred row is a rounding of the mean, 2^-20 of the value at most, the same in all channels; its own mean takes it
    out but for 2^-20 of it: 2^-40 of the value, over sqrt(eps) = 2^-8.3 at least, 2^-31 of it.  The output is the bias."""
    x = inputs(3, D, dtype, False, True, 31)
    x["x"][:] = value
    got = run(x, groups)
    y, dx, dw, db = ol.layer_norm(host(x["x"]), host(x["w"]), host(x["b"]), groups, dy=host(x["dy"]))
    step = 0.0 if dtype == "f32" else 2.0 ** -8 * abs(host(x["b"])).max()
    assert abs(host(got["y"]) - host(x["b"])).max() <= 2.0 ** -30 * abs(value) + 2.0 ** -22 + step
    size = abs(dx).max()
    assert abs(host(got["dx"]) - dx).max() <= (1e-5 + (0.0 if dtype == "f32" else 2.0 ** -8)) * size
    assert abs(host(got["dweight"])).max() <= 2.0 ** -28 * abs(value)


def test_the_backward_looks_at_the_bias():
    x = inputs(5, 64, "f32", False, True, 32)
    a = (x["x"], x["w"])
    for bias, error in ((x["b"][:32].contiguous(), ValueError), (x["b"].double(), TypeError), (object(), TypeError), (x["b"].cpu(), TypeError)):
        with pytest.raises(error):
            vs.varlen_layer_norm_fwd(*a, bias)
        with pytest.raises(error):
            vs.varlen_layer_norm_bwd(*a, bias, x["dy"])


def test_every_tensor_of_a_call_is_looked_at_for_its_device(monkeypatch):
    seen = []
    monkeypatch.setattr(binding, "_together", lambda *t: seen.append({id(x) for x in t}))
    y, w = torch.zeros((5, 64), device="cuda"), torch.ones(64, device="cuda")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    fwd = dict(x=y, weight=w, bias=w.clone(), residual=y.clone(), out=y.clone(), sum_out=y.clone())
    bwd = dict(x=y, weight=w, bias=w.clone(), dout=y.clone(), dsum=y.clone(), workspace=ws)
    dx = y.clone()
    vs.varlen_layer_norm_fwd(**fwd)
    vs.varlen_layer_norm_bwd(**bwd, residual=True, grads={"dx": dx})
    for at, given in zip(seen, (fwd, dict(bwd, dx=dx)), strict=True):
        assert all(id(t) in at for t in given.values())
