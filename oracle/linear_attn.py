"""Plain double-precision oracle of linear attention with a decay for each head
and of layer norm: token by token, head by head, numpy, no code shared with
the CUDA path.

  S_t = a_t S_{t-1} + k_t v_t^T,  out_t = scale S_t^T q_t,  a_t = exp(g_t)

The backward is the adjoint of these lines in reverse order.
"""
import numpy as np


def _wide(x, rep):
    return np.repeat(np.asarray(x, dtype=np.float64), rep, axis=1)


def _decays(g, T):
    a = np.exp(np.asarray(g, dtype=np.float64))
    return np.broadcast_to(a, (T, a.shape[-1]))


def linear_fwd(q, k, v, g, cu, scale, init=None, keep=None):
    """out (T, Hv, V), final (S, Hv, K, V); g (T, Hv) or (Hv,).  keep: a list to
    receive, for every token, the state before it and the state after it."""
    v = np.asarray(v, dtype=np.float64)
    T, Hv, V = v.shape
    rep = Hv // q.shape[1]
    q, k, a = _wide(q, rep), _wide(k, rep), _decays(g, T)
    final = np.zeros((len(cu) - 1, Hv, k.shape[2], V))
    out = np.zeros((T, Hv, V))
    for s in range(len(cu) - 1):
        S = np.zeros_like(final[s]) if init is None else np.array(init[s], dtype=np.float64)
        for t in range(cu[s], cu[s + 1]):
            before = S
            S = S * a[t][:, None, None] + k[t][:, :, None] * v[t][:, None, :]
            if keep is not None:
                keep.append((before, S))
            out[t] = scale * np.einsum("hkv,hk->hv", S, q[t])
        final[s] = S
    return out, final


def linear_bwd(q, k, v, g, dout, cu, scale, init=None, dfinal=None):
    """dict dq, dk, dv, dg (shaped as g), dinit."""
    keep = []
    linear_fwd(q, k, v, g, cu, scale, init, keep)
    v = np.asarray(v, dtype=np.float64)
    T, Hv, V = v.shape
    Hk = q.shape[1]
    rep = Hv // Hk
    q, k, a = _wide(q, rep), _wide(k, rep), _decays(g, T)
    dout = np.asarray(dout, dtype=np.float64)
    d = dict(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v), dg=np.zeros((T, Hv)),
             dinit=np.zeros((len(cu) - 1, Hv, q.shape[2], V)))
    for s in range(len(cu) - 1):
        D = np.zeros_like(d["dinit"][s]) if dfinal is None else np.array(dfinal[s], dtype=np.float64)
        for t in range(cu[s + 1] - 1, cu[s] - 1, -1):
            before, after = keep[t]
            do = scale * dout[t]
            d["dq"][t] = np.einsum("hkv,hv->hk", after, do)
            D = D + q[t][:, :, None] * do[:, None, :]
            d["dk"][t] = np.einsum("hkv,hv->hk", D, v[t])
            d["dv"][t] = np.einsum("hkv,hk->hv", D, k[t])
            D = D * a[t][:, None, None]
            d["dg"][t] = (D * before).sum((-2, -1))
        d["dinit"][s] = D
    for n in ("dq", "dk"):
        d[n] = d[n].reshape(T, Hk, rep, q.shape[2]).sum(2)
    if np.ndim(g) == 1:
        d["dg"] = d["dg"].sum(0)
    return d


def layer_norm(x, w=None, b=None, groups=1, eps=1e-5, dy=None):
    """out, or (out, dx, dw, db) with the gradient dy of out; x (T, D)."""
    x = np.asarray(x, dtype=np.float64)
    T, D = x.shape
    w = np.ones(D) if w is None else np.asarray(w, dtype=np.float64)
    rows = x.reshape(T, groups, D // groups)
    c = rows - rows.mean(-1, keepdims=True)
    std = np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    n = c / std
    out = n.reshape(T, D) * w + (0.0 if b is None else np.asarray(b, dtype=np.float64))
    if dy is None:
        return out
    dy = np.asarray(dy, dtype=np.float64)
    u = (dy * w).reshape(n.shape)
    dx = (u - u.mean(-1, keepdims=True) - n * (u * n).mean(-1, keepdims=True)) / std
    return out, dx.reshape(T, D), (dy * n.reshape(T, D)).sum(0), dy.sum(0)
