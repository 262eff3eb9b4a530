"""Plain double-precision oracle of the gated delta rule and of the q/k norm
with rotation: token by token, head by head, numpy, no code shared with the
CUDA path.

  S_t = a_t S_{t-1} + k_t u_t^T,  u_t = beta_t (v_t - a_t S_{t-1}^T k_t),  out_t = scale S_t^T q_t,  a_t = exp(g_t)

The backward is the adjoint of these lines in reverse order.
"""
import numpy as np


def _wide(x, rep):
    return np.repeat(np.asarray(x, dtype=np.float64), rep, axis=1)


def delta_fwd(q, k, v, g, beta, cu, scale, init=None, keep=None):
    """out (T, Hv, V), final (S, Hv, K, V).  keep: a list to receive, for every
    token, the decayed state it meets and its error v - S^T k."""
    v = np.asarray(v, dtype=np.float64)
    T, Hv, V = v.shape
    rep = Hv // q.shape[1]
    q, k = _wide(q, rep), _wide(k, rep)
    a, beta = np.exp(np.asarray(g, dtype=np.float64)), np.asarray(beta, dtype=np.float64)
    S_count = len(cu) - 1
    final = np.zeros((S_count, Hv, k.shape[2], V))
    out = np.zeros((T, Hv, V))
    for s in range(S_count):
        S = np.zeros_like(final[s]) if init is None else np.array(init[s], dtype=np.float64)
        for t in range(cu[s], cu[s + 1]):
            S = S * a[t][:, None, None]
            e = v[t] - np.einsum("hkv,hk->hv", S, k[t])
            if keep is not None:
                keep.append((S, e))
            S = S + k[t][:, :, None] * (beta[t][:, None] * e)[:, None, :]
            out[t] = scale * np.einsum("hkv,hk->hv", S, q[t])
        final[s] = S
    return out, final


def delta_bwd(q, k, v, g, beta, dout, cu, scale, init=None, dfinal=None):
    """dict dq, dk, dv, dg, dbeta, dinit."""
    keep = []
    delta_fwd(q, k, v, g, beta, cu, scale, init, keep)
    T, Hv, V = np.shape(v)
    Hk = q.shape[1]
    rep = Hv // Hk
    q, k = _wide(q, rep), _wide(k, rep)
    a, beta = np.exp(np.asarray(g, dtype=np.float64)), np.asarray(beta, dtype=np.float64)
    dout = np.asarray(dout, dtype=np.float64)
    d = dict(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros((T, Hv, V)), dg=np.zeros((T, Hv)),
             dbeta=np.zeros((T, Hv)), dinit=np.zeros((len(cu) - 1, Hv, q.shape[2], V)))
    for s in range(len(cu) - 1):
        D = np.zeros_like(d["dinit"][s]) if dfinal is None else np.array(dfinal[s], dtype=np.float64)
        for t in range(cu[s + 1] - 1, cu[s] - 1, -1):
            P, e = keep[t]
            u = beta[t][:, None] * e
            do = scale * dout[t]
            d["dq"][t] = np.einsum("hkv,hv->hk", P + k[t][:, :, None] * u[:, None, :], do)
            D = D + q[t][:, :, None] * do[:, None, :]
            du = np.einsum("hkv,hk->hv", D, k[t])
            de = beta[t][:, None] * du
            d["dbeta"][t] = (du * e).sum(-1)
            d["dv"][t] = de
            d["dk"][t] = np.einsum("hkv,hv->hk", D, u) - np.einsum("hkv,hv->hk", P, de)
            D = D - k[t][:, :, None] * de[:, None, :]
            d["dg"][t] = (D * P).sum((-2, -1))
            D = D * a[t][:, None, None]
        d["dinit"][s] = D
    for n in ("dq", "dk"):
        d[n] = d[n].reshape(T, Hk, rep, -1).sum(2)
    return d


def qk_norm(x, w=None, cos=None, sin=None, pos=None, l2=False, eps=1e-6, dy=None):
    """out, or (out, dx, dw) with the gradient dy of out; x (T, H, K)."""
    x = np.asarray(x, dtype=np.float64)
    K = x.shape[2]
    count = 1 if l2 else K
    length = np.sqrt((x * x).sum(-1, keepdims=True) / count + eps)
    n = x / length
    w = np.ones(K) if w is None else np.asarray(w, dtype=np.float64)
    y = n * w

    def turn(z, sign):
        if cos is None:
            return z
        h = cos.shape[1]
        c, s = np.asarray(cos, np.float64)[pos][:, None], sign * np.asarray(sin, np.float64)[pos][:, None]
        a, b = z[..., :h], z[..., h:2 * h]
        return np.concatenate([a * c - b * s, b * c + a * s, z[..., 2 * h:]], -1)

    out = turn(y, 1.0)
    if dy is None:
        return out
    d = turn(np.asarray(dy, dtype=np.float64), -1.0)
    dn = d * w
    dx = dn / length - x * (dn * x).sum(-1, keepdims=True) / (count * length ** 3)
    return out, dx, (d * n).sum((0, 1))
