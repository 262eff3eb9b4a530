"""Host side of linear attention and layer norm: the oracle is pinned by closed
forms and differences, and the calls refuse what they cannot do before they
touch the GPU."""
import numpy as np
import pytest

from oracle import gated_delta as od
from oracle import linear_attn as ol
from selective_ssm_packed_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def case(seed=0, lens=(3, 0, 5, 1), Hk=1, Hv=2, K=8, V=8):
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    return dict(q=r.standard_normal((T, Hk, K)), k=r.standard_normal((T, Hk, K)), v=r.standard_normal((T, Hv, V)),
                g=-r.random((T, Hv)), cu=cu, scale=0.3, init=r.standard_normal((len(lens), Hv, K, V)))


def test_oracle_attention_without_decay_is_a_masked_product():
    c = case(lens=(7,), Hk=2, Hv=2)
    out, final = ol.linear_fwd(c["q"], c["k"], c["v"], np.zeros(2), c["cu"], 1.0)
    for h in range(2):
        q, k, v = c["q"][:, h], c["k"][:, h], c["v"][:, h]
        np.testing.assert_allclose(out[:, h], np.tril(q @ k.T) @ v, atol=1e-12)
        np.testing.assert_allclose(final[0, h], k.T @ v, atol=1e-12)


def test_oracle_attention_decays_a_pair_by_the_tokens_between():
    c = case(lens=(6,))
    G = np.cumsum(c["g"], 0)
    out, final = ol.linear_fwd(c["q"], c["k"], c["v"], c["g"], c["cu"], 1.0, c["init"])
    for h in range(2):
        P = np.tril((c["q"][:, 0] @ c["k"][:, 0].T) * np.exp(G[:, h, None] - G[None, :, h]))
        ref = P @ c["v"][:, h] + np.exp(G[:, h])[:, None] * (c["q"][:, 0] @ c["init"][0, h])
        np.testing.assert_allclose(out[:, h], ref, atol=1e-12)


def test_oracle_attention_is_the_delta_rule_without_its_correction():
    # for keys that are orthogonal to all earlier ones the correction is nothing
    r = np.random.default_rng(1)
    k, q, v = np.eye(8)[:, None], r.standard_normal((8, 1, 8)), r.standard_normal((8, 2, 8))
    g = -r.random((8, 2))
    a = ol.linear_fwd(q, k, v, g, [0, 8], 0.5)
    b = od.delta_fwd(q, k, v, g, np.ones((8, 2)), [0, 8], 0.5)
    for x, y in zip(a, b):
        np.testing.assert_allclose(x, y, atol=1e-12)


@pytest.mark.parametrize("head", [False, True])
def test_oracle_attention_gradient_against_differences(head):
    c = case(Hk=2, Hv=4)
    if head:
        c["g"] = c["g"][0]
    r = np.random.default_rng(5)
    dout, dfinal = r.standard_normal(c["v"].shape), r.standard_normal(c["init"].shape)

    def f(x):
        o, s = ol.linear_fwd(x["q"], x["k"], x["v"], x["g"], c["cu"], c["scale"], x["init"])
        return (o * dout).sum() + (s * dfinal).sum()

    grads = ol.linear_bwd(c["q"], c["k"], c["v"], c["g"], dout, c["cu"], c["scale"], c["init"], dfinal)
    for name in ("q", "k", "v", "g", "init"):
        d, h = r.standard_normal(c[name].shape), 1e-6
        diff = (f(dict(c, **{name: c[name] + h * d})) - f(dict(c, **{name: c[name] - h * d}))) / (2 * h)
        assert grads["d" + name].shape == c[name].shape
        assert abs(diff - (grads["d" + name] * d).sum()) <= 1e-7 * max(1.0, abs(diff)), name


@pytest.mark.parametrize("groups", [1, 3])
def test_oracle_norm_has_mean_zero_and_variance_one_and_its_gradient(groups):
    r = np.random.default_rng(2)
    x, w, b, dy = r.standard_normal((4, 12)) + 3, r.standard_normal(12), r.standard_normal(12), r.standard_normal((4, 12))
    n = ol.layer_norm(x, groups=groups, eps=0.0).reshape(4, groups, -1)
    np.testing.assert_allclose(n.mean(-1), 0, atol=1e-12)
    np.testing.assert_allclose(n.var(-1), 1, atol=1e-12)
    _, dx, dw, db = ol.layer_norm(x, w, b, groups, 1e-3, dy)
    for name, a, d in (("x", x, dx), ("w", w, dw), ("b", b, db)):
        e, h = r.standard_normal(a.shape), 1e-6
        up, down = (ol.layer_norm(**dict(dict(x=x, w=w, b=b), **{name: a + s * h * e}), groups=groups, eps=1e-3) for s in (1, -1))
        diff = ((up - down) * dy).sum() / (2 * h)
        assert abs(diff - (d * e).sum()) <= 1e-7 * max(1.0, abs(diff)), name


# ------------------------------------------------------------------ refusals (pointers are never dereferenced)
def fwd(lib, **kw):
    a = dict(q=16, k=16, v=16, sq=64, sk=64, sv=128, g=16, per_token=1, scale=1.0, cu=16, S=1, T=16, Hk=1, Hv=2, K=64, V=64,
             dt=0, out=16, init=None, final=None, ws=16, wsb=1 << 40, st=None)
    a.update(kw)
    return lib.varlen_linear_attn_fwd(*a.values())


def test_forward_refuses(lib):
    assert fwd(lib, dt=5) == -2
    assert fwd(lib, T=-1) == -1 and fwd(lib, T=2**31) == -1
    assert fwd(lib, S=0) == -1 and fwd(lib, S=-1) == -1
    assert fwd(lib, cu=None) == -1
    assert fwd(lib, Hk=3) == -1 and fwd(lib, Hk=0) == -1 and fwd(lib, Hv=65536, sv=2**22) == -6
    assert fwd(lib, K=60, sq=64, sk=64) == -6 and fwd(lib, K=136, sq=136, sk=136) == -6 and fwd(lib, K=0) == -6
    assert fwd(lib, V=136, sv=4096) == -6 and fwd(lib, V=4) == -6
    assert fwd(lib, q=None) == -1 and fwd(lib, out=None) == -1 and fwd(lib, g=None) == -1
    assert fwd(lib, v=8) == -3 and fwd(lib, init=4) == -3 and fwd(lib, final=8) == -3
    assert fwd(lib, sq=63) == -1 and fwd(lib, sk=66) == -3 and fwd(lib, sv=64) == -1
    assert fwd(lib, wsb=255) == -4 and fwd(lib, ws=None) == -4 and fwd(lib, ws=8) == -3
    assert "workspace" in binding.last_error() or fwd(lib, wsb=0) == -4
    assert fwd(lib, T=2**31 - 1, S=2**31 - 1, Hv=4, sv=256) == -6
    assert fwd(lib, T=0, S=2**30, Hk=2**30, Hv=2**30, sq=2**40, sk=2**40, sv=2**40) == -6
    assert fwd(lib, sq=2**62 + 1) == -3


def test_backward_refuses(lib):
    def bwd(**kw):
        a = dict(q=16, k=16, v=16, sq=64, sk=64, sv=128, g=16, per_token=0, dout=16, scale=1.0, cu=16, S=1, T=16, Hk=1, Hv=2,
                 K=64, V=64, dt=0, init=None, df=None, di=None, dq=16, dk=16, dv=16, dg=None, ws=16, wsb=1 << 40, st=None)
        a.update(kw)
        return lib.varlen_linear_attn_bwd(*a.values())

    assert bwd(dout=None) == -1 and bwd(dq=None) == -1 and bwd(dk=4) == -3 and bwd(dv=None) == -1 and bwd(dout=8) == -3
    assert bwd(df=8) == -3 and bwd(di=8) == -3 and bwd(init=2) == -3 and bwd(wsb=0) == -4 and bwd(K=7) == -6 and bwd(dt=9) == -2
    assert bwd(g=None) == -1 and bwd(sq=32) == -1 and bwd(V=200, sv=400) == -6
    need = binding.linear_attn_bwd_workspace_size(16, 1, 1, 2, 64, 64, 0)
    assert bwd(wsb=need - 1) == -4


def test_step_refuses(lib):
    def step(**kw):
        a = dict(q=16, k=16, v=16, sq=64, sk=64, sv=128, g=16, per_token=1, scale=1.0, states=16, idx=16, slots=4, B=2, Hk=1,
                 Hv=2, K=64, V=64, dt=0, out=16, status=None, st=None)
        a.update(kw)
        return lib.varlen_linear_attn_step(*a.values())

    assert step(dt=3) == -2 and step(B=-1) == -1 and step(slots=-1) == -1
    assert step(idx=None, B=5) == -1  # more sequences than slots
    assert step(states=None) == -1 and step(states=8) == -3 and step(K=12) == -6 and step(Hv=3, Hk=2) == -1
    assert step(sq=60) == -1 and step(g=None) == -1 and step(out=None) == -1
    assert step(B=2**60) == -6


def test_layer_norm_refuses(lib):
    def norm(**kw):
        a = dict(x=16, sx=64, res=None, w=None, b=None, T=4, D=64, groups=1, eps=1e-5, dt=0, out=16, sum=None, st=None)
        a.update(kw)
        return lib.varlen_layer_norm_fwd(*a.values())

    assert norm(dt=2) == -2 and norm(T=-1) == -1 and norm(D=0) == -1 and norm(groups=0) == -1 and norm(groups=3) == -1
    assert norm(D=60, sx=60) == -6 and norm(D=8200, sx=8200) == -6 and norm(groups=16) == -6
    assert norm(eps=-1.0) == -1 and norm(eps=float("nan")) == -1
    assert norm(x=None) == -1 and norm(out=None) == -1 and norm(x=8) == -3 and norm(w=4) == -3 and norm(res=8) == -3
    assert norm(sx=63) == -1 and norm(sx=66) == -3 and norm(sum=16) == -1 and norm(res=16, sum=8) == -3

    def bwd(**kw):
        a = dict(x=16, sx=64, x_f32=0, w=None, dout=16, dsum=None, T=4, D=64, groups=1, eps=1e-5, dt=1, dx=16, dres=None,
                 dw=None, db=None, ws=16, wsb=1 << 40, st=None)
        a.update(kw)
        return lib.varlen_layer_norm_bwd(*a.values())

    assert bwd(dout=None) == -1 and bwd(dx=None) == -1 and bwd(dsum=8) == -3 and bwd(dres=4) == -3 and bwd(ws=None) == -4
    assert bwd(sx=68) == -3 and bwd(wsb=100) == -4  # rows of bf16 that are no multiple of 16 bytes apart


def test_sizes(lib):
    small = binding.linear_attn_fwd_workspace_size(16, 4, 1, 2, 64, 64, 0)
    assert 0 < small < binding.linear_attn_bwd_workspace_size(16, 4, 1, 2, 64, 64, 0)
    assert small < binding.linear_attn_fwd_workspace_size(4096, 1, 1, 2, 64, 64, 0)
    assert binding.linear_attn_bwd_workspace_size(0, 0, 1, 2, 64, 64, 1) > 0
    for bad in ((16, 4, 3, 2, 64, 64, 0), (16, 4, 1, 2, 63, 64, 0), (16, 4, 1, 2, 64, 136, 0), (16, 4, 1, 2, 64, 64, 7)):
        assert binding.linear_attn_fwd_workspace_size(*bad) == 0 and binding.linear_attn_bwd_workspace_size(*bad) == 0
        assert binding.linear_attn_segment(*bad) == -1
    for io in (0, 1):
        for T, S in ((1, 1), (500, 1), (5000, 1), (32768, 40), (2**31 - 1, 1)):
            seg = binding.linear_attn_segment(T, S, 4, 8, 128, 128, io)
            assert 256 <= seg <= 4096 and seg % 128 == 0
    assert lib.varlen_layer_norm_bwd_workspace_size(4, 60, 1) == 0
    assert 0 < lib.varlen_layer_norm_bwd_workspace_size(0, 64, 1) <= lib.varlen_layer_norm_bwd_workspace_size(4096, 64, 1)


def test_tensors_of_several_devices_are_refused():
    import torch

    class On(torch.Tensor):  # a tensor that says it is on a GPU
        @staticmethod
        def __new__(cls, device):
            t = torch.Tensor._make_subclass(cls, torch.zeros(1))
            t.at = device
            return t

        is_cuda = True

        def get_device(self):
            return self.at

    binding._together(On(1), None, True, On(1))
    with pytest.raises(ValueError):
        binding._together(On(0), None, On(1))
