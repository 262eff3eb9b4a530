"""Host side of the gated delta rule and the q/k norm: the oracle is pinned by
closed forms and differences, and the calls refuse what they cannot do before
they touch the GPU."""
import numpy as np
import pytest

from oracle import gated_delta as od
from selective_ssm_packed_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def case(seed=0, lens=(3, 0, 5, 1), Hk=1, Hv=2, K=8, V=8):
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    k = r.standard_normal((T, Hk, K))
    return dict(q=r.standard_normal((T, Hk, K)), k=k / np.linalg.norm(k, axis=-1, keepdims=True),
                v=r.standard_normal((T, Hv, V)), g=-r.random((T, Hv)), beta=r.random((T, Hv)), cu=cu, scale=0.3,
                init=r.standard_normal((len(lens), Hv, K, V)))


def test_oracle_delta_rule_recalls_what_it_stored():
    # orthonormal keys, no decay, beta 1: S^T k_i = v_i for every stored pair
    K = V = 8
    v = np.random.default_rng(1).standard_normal((K, 1, V))
    out, final = od.delta_fwd(np.eye(K)[:, None], np.eye(K)[:, None], v, np.zeros((K, 1)), np.ones((K, 1)), [0, K], 1.0)
    np.testing.assert_allclose(final[0, 0], v[:, 0], atol=1e-14)
    np.testing.assert_allclose(out, v, atol=1e-14)


def test_oracle_delta_rule_is_a_decayed_sum_without_the_correction():
    # beta = 0 leaves a decayed initial state; one token of weight beta writes beta v
    c = case(lens=(4,))
    g = c["g"]
    out, final = od.delta_fwd(c["q"], c["k"], c["v"], g, np.zeros_like(g), c["cu"], 1.0, c["init"])
    np.testing.assert_allclose(final[0], c["init"][0] * np.exp(g.sum(0))[:, None, None], rtol=1e-12)


def test_oracle_delta_gradient_against_differences():
    c = case()
    r = np.random.default_rng(5)
    T, Hv, V = c["v"].shape
    dout, dfinal = r.standard_normal((T, Hv, V)), r.standard_normal(c["init"].shape)

    def f(x):
        o, s = od.delta_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], c["cu"], c["scale"], x["init"])
        return (o * dout).sum() + (s * dfinal).sum()

    grads = od.delta_bwd(c["q"], c["k"], c["v"], c["g"], c["beta"], dout, c["cu"], c["scale"], c["init"], dfinal)
    for name in ("q", "k", "v", "g", "beta", "init"):
        d = r.standard_normal(c[name].shape)
        h = 1e-6
        up, down = dict(c, **{name: c[name] + h * d}), dict(c, **{name: c[name] - h * d})
        diff = (f(up) - f(down)) / (2 * h)
        assert abs(diff - (grads["d" + name] * d).sum()) <= 1e-7 * max(1.0, abs(diff)), name


@pytest.mark.parametrize("l2", [False, True])
def test_oracle_norm_gradient_against_differences(l2):
    r = np.random.default_rng(2)
    x, w, dy = r.standard_normal((3, 2, 8)), r.standard_normal(8), r.standard_normal((3, 2, 8))
    ang = r.random((5, 3))
    pos = np.array([4, 0, 2])
    a = (np.cos(ang), np.sin(ang), pos, l2)
    _, dx, dw = od.qk_norm(x, w, *a, dy=dy)
    dX, dW, h = r.standard_normal(x.shape), r.standard_normal(8), 1e-6
    diff = ((od.qk_norm(x + h * dX, w + h * dW, *a) - od.qk_norm(x - h * dX, w - h * dW, *a)) * dy).sum() / (2 * h)
    assert abs(diff - (dx * dX).sum() - (dw * dW).sum()) <= 1e-7 * max(1.0, abs(diff))


def test_oracle_rotation_keeps_lengths_and_depends_on_distance():
    r = np.random.default_rng(3)
    x = r.standard_normal((1, 1, 8))
    ang = np.arange(6)[:, None] * np.array([1.0, 0.1, 0.01, 0.001])
    y = [od.qk_norm(x, None, np.cos(ang), np.sin(ang), np.array([p]), True, 0.0)[0, 0] for p in range(6)]
    assert np.allclose([np.linalg.norm(v) for v in y], 1.0)
    assert np.allclose([y[p] @ y[p + 2] for p in range(4)], y[0] @ y[2])


# ------------------------------------------------------------------ refusals (pointers are never dereferenced)
def fwd(lib, **kw):
    a = dict(q=16, k=16, v=16, sq=64, sk=64, sv=128, g=16, beta=16, scale=1.0, cu=16, S=1, T=16, Hk=1, Hv=2, K=64, V=64,
             dt=0, out=16, init=None, final=None, saved=None, sb=0, ws=16, wsb=1 << 40, st=None)
    a.update(kw)
    return lib.varlen_gated_delta_fwd(*a.values())


def test_forward_refuses(lib):
    assert fwd(lib, dt=5) == -2
    assert fwd(lib, T=-1) == -1
    assert fwd(lib, S=0) == -1
    assert fwd(lib, cu=None) == -1
    assert fwd(lib, Hk=3) == -1 and fwd(lib, Hk=0) == -1
    assert fwd(lib, K=60, sq=64, sk=64) == -6 and fwd(lib, K=136, sq=136, sk=136) == -6 and fwd(lib, K=0) == -6
    assert fwd(lib, V=1032, sv=4096) == -6 and fwd(lib, V=4) == -6
    assert fwd(lib, q=None) == -1 and fwd(lib, out=None) == -1 and fwd(lib, g=None) == -1
    assert fwd(lib, v=8) == -3 and fwd(lib, init=4) == -3 and fwd(lib, final=8) == -3
    assert fwd(lib, sq=63) == -1 and fwd(lib, sk=66) == -3 and fwd(lib, sv=64) == -1
    assert fwd(lib, wsb=255) == -4 and fwd(lib, ws=None) == -4 and fwd(lib, ws=8) == -3
    assert fwd(lib, saved=16, sb=100) == -4 and "saved" in binding.last_error()
    assert fwd(lib, T=2**31 - 1, S=2**31 - 1, Hv=4, Hk=1, sv=256) == -6


def test_backward_refuses(lib):
    need = binding.gated_delta_saved_size(16, 1, 1, 2, 64, 64, 0)

    def bwd(**kw):
        a = dict(dout=16, scale=1.0, cu=16, S=1, T=16, Hk=1, Hv=2, K=64, V=64, dt=0, saved=16, sb=need, df=None, di=None,
                 dq=16, dk=16, dv=16, dg=16, db=16, ws=16, wsb=1 << 40, st=None)
        a.update(kw)
        return lib.varlen_gated_delta_bwd(*a.values())

    assert bwd(saved=None) == -4 and bwd(sb=need - 1) == -4
    assert bwd(dout=None) == -1 and bwd(dq=None) == -1 and bwd(dg=None) == -1 and bwd(dk=4) == -3
    assert bwd(df=8) == -3 and bwd(di=8) == -3 and bwd(wsb=0) == -4 and bwd(K=7) == -6 and bwd(dt=9) == -2


def test_step_refuses(lib):
    def step(**kw):
        a = dict(q=16, k=16, v=16, sq=64, sk=64, sv=128, g=16, beta=16, scale=1.0, states=16, idx=16, slots=4, B=2, Hk=1,
                 Hv=2, K=64, V=64, dt=0, out=16, status=None, st=None)
        a.update(kw)
        return lib.varlen_gated_delta_step(*a.values())

    assert step(dt=3) == -2 and step(B=-1) == -1 and step(slots=-1) == -1
    assert step(idx=None, B=5) == -1  # more sequences than slots
    assert step(states=None) == -1 and step(states=8) == -3 and step(K=12) == -6 and step(Hv=3, Hk=2) == -1
    assert step(sq=60) == -1 and step(beta=None) == -1 and step(out=None) == -1


def test_norm_refuses(lib):
    def norm(**kw):
        a = dict(q=16, k=16, sq=128, sk=64, qw=None, kw=None, cos=16, sin=16, pos=16, rows=8, T=4, Hq=2, Hk=1, K=64, rot=32,
                 l2=0, eps=1e-6, dt=0, qo=16, ko=16, status=None, st=None)
        a.update(kw)
        return lib.varlen_qk_norm_rope_fwd(*a.values())

    assert norm(dt=2) == -2 and norm(T=-1) == -1 and norm(K=12) == -6 and norm(K=264, sq=528, sk=264) == -6
    assert norm(rot=33) == -1 and norm(rot=66) == -1 and norm(eps=-1.0) == -1 and norm(eps=float("nan")) == -1
    assert norm(cos=None) == -1 and norm(pos=None) == -1 and norm(q=None) == -1 and norm(ko=None) == -1
    assert norm(q=4) == -3 and norm(sq=127) == -1 and norm(sk=65) == -3 and norm(Hq=0, Hk=0) == -1
    assert lib.varlen_qk_norm_rope_bwd_workspace_size(12) == 0
    assert lib.varlen_qk_norm_rope_bwd(16, 16, 128, 64, None, None, None, None, None, 0, 16, 16, 4, 2, 1, 64, 0, 0, 1e-6, 0,
                                       16, 16, None, None, None, 0, None) == -4


def test_sizes(lib):
    small = binding.gated_delta_saved_size(16, 4, 1, 2, 64, 64, 0)
    assert 0 < binding.gated_delta_fwd_workspace_size(16, 4, 1, 2, 64, 64, 0) < small
    assert small < binding.gated_delta_saved_size(4096, 4, 1, 2, 64, 64, 0)
    assert binding.gated_delta_bwd_workspace_size(0, 0, 1, 2, 64, 64, 1) > 0
    assert binding.gated_delta_saved_size(16, 4, 3, 2, 64, 64, 0) == 0
    assert binding.gated_delta_saved_size(16, 4, 1, 2, 63, 64, 0) == 0
    assert binding.strerror(-20) and binding.status_code(32) == -20
    assert binding.strerror(-21) and binding.status_code(64) == -21


def test_sizes_past_64_bits_are_refused(lib):
    # products of these wrap around to small ones
    assert fwd(lib, T=0, S=2**30, Hk=2**30, Hv=2**30, V=1024, K=8, sq=2**33, sk=2**33, sv=2**40) == -6
    assert binding.gated_delta_saved_size(0, 2**30, 2**30, 2**30, 8, 1024, 0) == 0
    assert fwd(lib, sq=2**62 + 1) == -3 and fwd(lib, sq=2**62 + 4, wsb=0) == -4  # in bytes 2^64 + 4 and 2^64 + 16
    assert lib.varlen_gated_delta_step(16, 16, 16, 64, 64, 128, 16, 16, 1.0, 16, 16, 4, 2**60, 1, 16, 64, 64, 0, 16, None,
                                       None) != 0
    assert "too large" in binding.last_error()
