"""Linear attention with a decay for each head on the GPU against the oracle.

Tolerances, from the arithmetic (errors and references as 2-norms over a
tensor).  An FP32 operand of a product carries 24 bits with FP32 I/O and at
least 16 with bf16 I/O (relative rounding up to 2^-16); a value passes through
at most three such operands (the weighted rows, the state, P), each of them
once a chunk, and the decays are at most 1: 8 * 2^-16 = 1.2e-4 on FP32
outputs of bf16 calls.  FP32 calls are bounded by FP32 sums of up to 128
products in the matrix unit (128 * 2^-24 = 8e-6) over the same steps: 4e-5.
bf16 outputs add one rounding, 2^-9 of each value at least and 2^-8 at most.
dg sums rho - sigma over the rest of a segment, of at most 256 tokens here,
each with an error of its own: sqrt(256) times the bound on one, 2^-16 and
8e-6, is 2.5e-4 and 1.3e-4 of the size of rho, which is no larger than dg's (of
all pairs of tokens across t, rho has those that end at t); sigma doubles the
variance: 3.5e-4 and 1.9e-4.  With one decay a head these are added up: an error
of rho or sigma counts once for every token before it in its segment of n, so
the sum is off by sqrt(2 sum of i^2 over i < n) = 0.82 n^1.5 of them a segment, 0.82 n
sqrt(T) in all, that is 0.82 n * 2^-16 (bf16, n <= 256: 3.2e-3) or 0.82 n * 8e-6
(f32, n <= 128: 8.4e-4) of the 2-norm of the tokens' dg, against which it is held.
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
DG = {"f32": 1.9e-4, "bf16": 3.5e-4}
DG_HEAD = {"f32": 8.4e-4, "bf16": 3.2e-3}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from selective_ssm_packed_gb300 import build
    build.build()
    binding.lib()


def close(name, got, ref, dtype, size=None):
    tol = {"dg": DG, "dg_head": DG_HEAD}.get(name, NET)[dtype] + (2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0)
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
