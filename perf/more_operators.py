"""Linear attention with a decay for each head, and the layer norm around it, on real work: cases, inputs, plain
forms and 64-bit values.

Two operators next to the gated delta rule and the q/k norm, on the same packed layout ((total_tokens, heads, width)
tensors plus int32 cu_seqlens):

  linear  S_t = a_t S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t,  a_t = exp(g_t), the state reset at every sequence
          start; g for each token and head, or one decay for each head: forward (training and prefill), forward +
          backward, and one token for each of many sequences against a pool of states (serving)
  norm    y = (h - mean(h)) / sqrt(var(h) + eps) * weight + bias over a token's channels or each group of them, h = x,
          or x added to the float32 residual stream, which is returned too: forward, and forward + backward with the
          gradients of weight and bias

With `own` false, run() computes them from elementary torch operations in 32 bits: linear attention in chunks of 64
tokens, batched over chunks, heads and sequences.  With `own` true it calls the framework.
"""
import math

import numpy as np
import torch

own = False

CHUNK = 64  # tokens the plain form takes at a time
EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token of one user, added to the residual stream: a call's latency
        dict(name="norm_decode_1", op="norm", train=False, T=1, D=2048, groups=1, residual=True, affine=True,
             dtype="bf16"),
        # the 2048-channel model's training step: 8 packs of 4096 tokens, residual stream in float32
        dict(name="norm_train_2048_bf16", op="norm", train=True, T=32768, D=2048, groups=1, residual=True, affine=True,
             dtype="bf16"),
        # the 4096 inner channels, each of 32 heads on its own, behind the attention
        dict(name="norm_heads_train_bf16", op="norm", train=True, T=32768, D=4096, groups=32, residual=False,
             affine=True, dtype="bf16"),
        # odd sizes in fp32
        dict(name="norm_train_odd_f32", op="norm", train=True, T=3001, D=1000, groups=1, residual=False, affine=True,
             dtype="f32"),
        # the 16-token, 4-sequence pack: the smallest call
        dict(name="linear_tiny_f32", op="linear", train=False, T=16, Hk=2, Hv=4, K=64, V=64, decay="token",
             dtype="f32", pack="tiny", states=False),
        # the 4096-channel layer: 8 packs of 4096 tokens, bf16, two value heads to a key head
        dict(name="linear_4096_bf16", op="linear", train=False, T=32768, Hk=16, Hv=32, K=128, V=128, decay="token",
             dtype="bf16", pack="median800", states=False),
        # one 32768-token sequence (the long tail's longest), continued from a state; fixed decays
        dict(name="linear_long_bf16", op="linear", train=False, T=32768, Hk=32, Hv=32, K=128, V=128, decay="head",
             dtype="bf16", pack="one", states=True),
        # odd sizes in fp32 with states and their gradients: sequences cut across packs
        dict(name="linear_train_odd_f32", op="linear", train=True, T=3001, Hk=3, Hv=6, K=96, V=80, decay="token",
             dtype="f32", pack="median300", states=True),
        # the 4096-channel layer's training step
        dict(name="linear_train_4096_bf16", op="linear", train=True, T=32768, Hk=32, Hv=32, K=128, V=128,
             decay="token", dtype="bf16", pack="median800", states=False),
        # the same channels in 64 heads of 64, keys and queries shared by 8 heads each
        dict(name="linear_train_shared_bf16", op="linear", train=True, T=16384, Hk=8, Hv=64, K=128, V=64,
             decay="token", dtype="bf16", pack="median800", states=False),
        # one user's next token
        dict(name="step_1_bf16", op="step", B=1, slots=1, Hk=16, Hv=32, K=128, V=128, decay="token", dtype="bf16"),
        # a serving batch's next tokens: 256 sequences in a pool of 320 states
        dict(name="step_256_bf16", op="step", B=256, slots=320, Hk=32, Hv=32, K=128, V=128, decay="head",
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_train", "norm_train", "linear", "linear", "linear_train", "linear_train", "step"])
    dtype = rng.choice(["bf16", "f32"])
    if op.startswith("norm"):
        if rng.random() < 0.5:
            groups, D = 1, 8 * _log_int(rng, 8, 1024)
        else:
            groups = rng.randint(2, 48)
            D = groups * 8 * rng.randint(2, 32)
        T = _log_int(rng, 1, max(1, min(32768, 32768 * 2048 // (D * (2 if dtype == "f32" else 1)))))
        return dict(op="norm", train=op == "norm_train", T=T, D=D, groups=groups, residual=rng.random() < 0.5,
                    affine=rng.random() < 0.75, dtype=dtype)
    Hk = rng.randint(1, 12)
    Hv = Hk * rng.choice([1, 2, 4])
    K, V = 8 * rng.randint(2, 16), 8 * rng.randint(2, 16)
    decay = rng.choice(["token", "head"])
    if op == "step":
        B = _log_int(rng, 1, 256)
        return dict(op="step", B=B, slots=B + rng.randint(0, 64), Hk=Hk, Hv=Hv, K=K, V=V, decay=decay, dtype=dtype)
    # at most a quarter of the largest listed case's heads times tokens
    T = _log_int(rng, 7, 32768 * 8 // Hv)
    return dict(op="linear", train=op == "linear_train", T=T, Hk=Hk, Hv=Hv, K=K, V=V, decay=decay, dtype=dtype,
                pack=rng.choice(["median300", "median800", "one"]) if T < 8192 else "median800",
                states=rng.random() < 0.5)


def lengths_of(case):
    """The sequence lengths of a case's pack, summing to T: the case's own, whatever the seed of its values."""
    T, pack = case["T"], case["pack"]
    if pack == "tiny":
        return [4, 2, 3, 7]
    if pack == "one":
        return [T]
    rng = np.random.default_rng(T)
    median, lo, hi, per = {"median300": (300, 16, 2048, T), "median800": (800, 32, 4096, 4096)}[pack]
    out, left = [], T
    while left:
        room = min(left, per)
        left -= room
        while room:
            n = min(max(int(round(math.exp(rng.normal(math.log(median), 1.0)))), lo), hi, room)
            out.append(n)
            room -= n
    return out


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(shape, generator=gen, device=dev)

    s = dict(case)
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        # channels of unlike scale and mean, a residual stream of a few layers' outputs
        s["x"] = (normal(T, D) * torch.exp(0.5 * normal(D)) + 0.3 * normal(D)).to(dt)
        s["res"] = 2 * normal(T, D) * torch.exp(0.5 * normal(D)) + normal(D) if case["residual"] else None
        s["w"] = 1 + 0.1 * normal(D) if case["affine"] else None
        s["b"] = 0.1 * normal(D) if case["affine"] else None
        if case["train"]:
            s["dy"] = normal(T, D).to(dt)
            s["dsum"] = normal(T, D) if case["residual"] else None
        return s

    Hk, Hv, K, V = case["Hk"], case["Hv"], case["K"], case["V"]
    n = case["B"] if case["op"] == "step" else case["T"]

    def unit(x):
        return (x / x.square().sum(-1, keepdim=True).sqrt()).to(dt)

    # keys and queries leave a SiLU convolution (values mostly above zero) and a unit-length norm
    s["q"] = unit(normal(n, Hk, K) + 0.3)
    s["k"] = unit(normal(n, Hk, K) + 0.3)
    s["v"] = normal(n, Hv, V).to(dt)
    if case["decay"] == "token":
        # g = -A softplus(a + dt_bias) with A in [1, 16] and steps of 1e-3 to 1e-1
        step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), Hv))
        bias = step + torch.log(-torch.expm1(-step))
        s["g"] = -uniform(1.0, 16.0, Hv) * torch.nn.functional.softplus(0.5 * normal(n, Hv) + bias)
    else:
        # decays of 1 - 2^-5 .. 1 - 2^-12 over the heads, each off by a little
        e = 5 + 7 * torch.arange(Hv, device=dev) / max(Hv - 1, 1)
        s["g"] = torch.log1p(-torch.exp2(-e - 0.1 * torch.rand(Hv, generator=gen, device=dev)))
    s["scale"] = K ** -0.5
    if case["op"] == "step":
        s["states"] = 0.3 * normal(case["slots"], Hv, K, V)
        s["slots"] = torch.randperm(case["slots"], generator=gen, device=dev)[:n].to(torch.int32)
        return s
    lens = lengths_of(case)
    s["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=dev)
    s["init"] = 0.3 * normal(len(lens), Hv, K, V) if case["states"] else None
    if case["train"]:
        s["dout"] = normal(n, Hv, V).to(dt)
        s["dfinal"] = 0.1 * normal(len(lens), Hv, K, V) if case["states"] else None
    s["plan"] = _plan(lens, dev)
    return s


def _plan(lens, dev):
    """Where the chunks of a pack lie: (chunks, CHUNK) token indices and mask, sequences by falling length, the
    chunks of each step over them."""
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    start = np.concatenate([[0], np.cumsum(lens)])
    rows = [(int(start[i]) + c, min(CHUNK, lens[i] - c)) for i in order for c in range(0, lens[i], CHUNK)]
    at = np.array([r[0] for r in rows])[:, None] + np.arange(CHUNK)[None]
    mask = np.arange(CHUNK)[None] < np.array([r[1] for r in rows])[:, None]
    counts = np.array([-(-lens[i] // CHUNK) for i in order])
    first = np.concatenate([[0], np.cumsum(counts)[:-1]])
    steps = [torch.from_numpy(first[:int((counts > c).sum())] + c).to(dev) for c in range(int(counts.max()))]
    return dict(at=torch.from_numpy(np.minimum(at, int(start[-1]) - 1)).to(dev), mask=torch.from_numpy(mask).to(dev),
                steps=steps, order=torch.tensor(order, device=dev),
                place=torch.from_numpy(np.flatnonzero(mask.ravel())[np.argsort(at[mask], kind="stable")]).to(dev))


# ------------------------------------------------------------------ plain forms
def _plain_norm(s):
    x, w = s["x"], s["w"]
    h = x.float() + s["res"] if s["residual"] else x.float()
    g = h.unflatten(1, (s["groups"], -1))
    c = g - g.mean(-1, keepdim=True)
    r = torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS)
    n = (c * r).flatten(1)
    out = {"y": (n * w + s["b"] if s["affine"] else n).to(x.dtype)}
    if s["residual"]:
        out["sum"] = h
    if s["train"]:
        dy = s["dy"].float()
        dn = (dy * w if s["affine"] else dy).unflatten(1, (s["groups"], -1))
        n3 = n.unflatten(1, (s["groups"], -1))
        dh = (r * (dn - dn.mean(-1, keepdim=True) - n3 * (dn * n3).mean(-1, keepdim=True))).flatten(1)
        if s["residual"]:
            dh = dh + s["dsum"]
            out["dres"] = dh
        out["dx"] = dh.to(x.dtype)
        if s["affine"]:
            out["dw"], out["db"] = (dy * n).sum(0), dy.sum(0)
    return out


def _plain_linear(q, k, v, g, init, scale, plan):
    """out (T, Hv, V) and final states, all float32, in chunks."""
    at, mask = plan["at"], plan["mask"]
    T, Hv, V = v.shape
    rep = Hv // k.shape[1]
    if g.dim() == 1:
        g = g.expand(T, Hv)

    def chunks(x):  # (T, H, ...) -> (H, chunks, CHUNK, ...), zero past a sequence's end
        x = torch.where(mask.reshape(mask.shape + (1,) * (x.dim() - 1)), x[at], 0.0)
        return x.movedim(2, 0)

    q, k, v = chunks(q).repeat_interleave(rep, 0), chunks(k).repeat_interleave(rep, 0), chunks(v)
    G = torch.cumsum(chunks(g), -1)
    i = torch.arange(CHUNK, device=v.device)
    low = i[:, None] >= i[None, :]
    decay = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -torch.inf))
    within = ((q @ k.mT) * decay) @ v
    gam, dec = torch.exp(G)[..., None], torch.exp(G[..., -1:] - G)[..., None]
    qs, kv = gam * q, (dec * k).mT @ v
    S = init[plan["order"]].movedim(1, 0) if init is not None else v.new_zeros(Hv, len(plan["order"]), k.shape[-1], V)
    before, final = [], []
    for ids in plan["steps"]:
        final.append(S[:, len(ids):])
        S = S[:, :len(ids)]
        before.append(S)
        S = gam[:, ids, -1:] * S + kv[:, ids]
    final = torch.cat([S] + final[::-1], 1).movedim(0, 1)
    final = torch.empty_like(final).index_copy(0, plan["order"], final)
    ids = torch.cat(plan["steps"])
    before = torch.cat(before, 1)
    before = torch.empty_like(before).index_copy(1, ids, before)
    o = scale * (within + qs @ before)
    return o.movedim(0, 2).reshape(-1, Hv, V)[plan["place"]], final


def _plain_step(s):
    rep = s["v"].shape[1] // s["k"].shape[1]
    q, k = (x.float().repeat_interleave(rep, 1) for x in (s["q"], s["k"]))
    at = s["slots"].long()
    S = s["states"][at] * torch.exp(s["g"])[..., None, None] + k[..., None] * s["v"].float()[..., None, :]
    s["states"][at] = S
    return {"out": (s["scale"] * (S * q[..., None]).sum(-2)).to(s["v"].dtype), "states": s["states"]}


def _plain(s):
    if s["op"] == "norm":
        return _plain_norm(s)
    if s["op"] == "step":
        return _plain_step(s)
    dt = s["v"].dtype
    names = ["q", "k", "v", "g"] + (["init"] if s["init"] is not None else [])
    x = {n: s[n].float() for n in names}
    if s["train"]:
        x = {n: t.detach().requires_grad_() for n, t in x.items()}
    o, final = _plain_linear(x["q"], x["k"], x["v"], x["g"], x.get("init"), s["scale"], s["plan"])
    out = {"out": o.detach().to(dt)}
    if s["states"]:
        out["final"] = final.detach()
    if s["train"]:
        ys, dys = [o], [s["dout"].float()]
        if s["states"]:
            ys, dys = ys + [final], dys + [s["dfinal"]]
        grads = torch.autograd.grad(ys, [x[n] for n in names], dys)
        for n, d in zip(names, grads):
            out["d" + n] = d.to(dt) if n in ("q", "k", "v") else d
    return out


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import selective_ssm_packed_gb300 as vs
    if s["op"] == "norm":
        res = vs.varlen_layer_norm_fwd(s["x"], s["w"], s["b"], groups=s["groups"], eps=EPS, residual=s["res"])
        y, h = res if s["residual"] else (res, s["x"])
        out = {"y": y}
        if s["residual"]:
            out["sum"] = h
        if s["train"]:
            g = vs.varlen_layer_norm_bwd(h, s["w"], s["b"], s["dy"], groups=s["groups"], eps=EPS,
                                         residual=s["residual"], dsum=s["dsum"])
            out["dx"] = g["dx"]
            if s["residual"]:
                out["dres"] = g["dresidual"]
            if s["affine"]:
                out["dw"], out["db"] = g["dweight"], g["dbias"]
        return out
    if s["op"] == "step":
        out = vs.varlen_linear_attn_step(s["q"], s["k"], s["v"], s["g"], s["states"], state_indices=s["slots"],
                                         scale=s["scale"])
        return {"out": out, "states": s["states"]}
    args = (s["q"], s["k"], s["v"], s["g"])
    res = vs.varlen_linear_attn_fwd(*args, s["cu"], scale=s["scale"], initial_states=s["init"],
                                    final_states=s["states"])
    out = {"out": res[0], "final": res[1]} if s["states"] else {"out": res}
    if s["train"]:
        g = vs.varlen_linear_attn_bwd(*args, s["dout"], s["cu"], scale=s["scale"], initial_states=s["init"],
                                      d_final_states=s["dfinal"], d_initial_states=s["states"])
        out.update(dq=g["dq"], dk=g["dk"], dv=g["dv"], dg=g["dg"])
        if s["states"]:
            out["dinit"] = g["d_initial_states"]
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the work a pass cannot do without
def work(case):
    io = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        rows = case["T"] * case["D"]
        res = 4 if case["residual"] else 0
        per = 2 * io + 2 * res  # x, y, the stream read and written
        if case["train"]:  # h, dy, dx, the stream's gradient read and written; h is read by both passes
            per += (res or io) + 2 * io + 2 * res
        return {"bytes": rows * per, "flops": rows * (22 if case["train"] else 8)}
    Hk, Hv, K, V = case["Hk"], case["Hv"], case["K"], case["V"]
    state = Hv * K * V
    if case["op"] == "step":
        B = case["B"]
        return {"bytes": 8 * B * state + B * (2 * Hk * K + 2 * Hv * V) * io + 4 * Hv, "flops": 5 * B * state}
    T = case["T"]
    seqs = len(lengths_of(case))
    read = T * (2 * Hk * K + Hv * V) * io + (4 * T * Hv if case["decay"] == "token" else 4 * Hv)
    nbytes = read + T * Hv * V * io + (8 * seqs * state if case["states"] else 0)
    if case["train"]:  # inputs again, dout, and the gradients
        nbytes += 2 * read + T * Hv * V * io + (12 * seqs * state if case["states"] else 0)
    return {"bytes": nbytes, "flops": (16 if case["train"] else 5) * T * state}


# ------------------------------------------------------------------ 64-bit values, token by token
def _exact_norm(s):
    T, D, G = s["T"], s["D"], s["groups"]
    out = {}
    h = s["x"].double()
    if s["residual"]:
        h = h + s["res"].double()
        out["sum"] = h
    w = s["w"].double() if s["affine"] else torch.ones(D, dtype=torch.float64, device=h.device)
    hg = h.reshape(T, G, D // G)
    var, mean = torch.var_mean(hg, dim=2, correction=0, keepdim=True)
    std = torch.sqrt(var + EPS)
    n = (hg - mean) / std
    out["y"] = n.reshape(T, D) * w + (s["b"].double() if s["affine"] else 0.0)
    if s["train"]:
        dy = s["dy"].double()
        u = (dy * w).reshape(T, G, D // G)
        # the centred direction's own part, then the part along n, leave the gradient
        u0 = u - u.sum(2, keepdim=True) / (D // G)
        dh = ((u0 - n * ((u * n).sum(2, keepdim=True) / (D // G))) / std).reshape(T, D)
        if s["residual"]:
            dh = dh + s["dsum"].double()
            out["dres"] = dh
        out["dx"] = dh
        if s["affine"]:
            out["dw"] = torch.einsum("td,td->d", dy, n.reshape(T, D))
            out["db"] = torch.einsum("td->d", dy)
    return out


def _exact_linear(s):
    """Token by token; the sequences of a pack step together, longest first, and the ones that are through drop out.
    The backward walks from the end, over states made again from one kept every CHUNK tokens."""
    lens = lengths_of(s)
    idx = sorted(range(len(lens)), key=lambda i: -lens[i])
    dev = s["v"].device
    order = torch.tensor(idx, device=dev)
    start = s["cu"][:-1].long()[order]
    lens = [lens[i] for i in idx]
    alive = [sum(n > t for n in lens) for t in range(lens[0])]
    T, Hv, V = s["v"].shape
    K = s["k"].shape[2]
    rep = Hv // s["k"].shape[1]
    wide = {n: s[n].double().repeat_interleave(rep, 1) for n in ("q", "k")}
    v, a = s["v"].double(), s["g"].double().exp()
    if a.dim() == 1:
        a = a.expand(T, Hv)
    S = s["init"].double()[order] if s["states"] else torch.zeros(len(lens), Hv, K, V, dtype=torch.float64, device=dev)

    def step(X, t, n):  # X[:n] one token on; the rows of that token
        r = start[:n] + t
        X[:n] *= a[r][..., None, None]
        X[:n] += wide["k"][r][..., :, None] * v[r][..., None, :]
        return r

    out = torch.empty(T, Hv, V, dtype=torch.float64, device=dev)
    kept = []
    for t in range(lens[0]):
        n = alive[t]
        if s["train"] and t % CHUNK == 0:
            kept.append(S[:n].clone())
        r = step(S, t, n)
        out[r] = s["scale"] * torch.matmul(wide["q"][r][..., None, :], S[:n])[..., 0, :]
    res = {"out": out}
    if s["states"]:
        res["final"] = torch.empty_like(S).index_copy(0, order, S)
    if not s["train"]:
        return res
    d = {"q": torch.empty_like(wide["q"]), "k": torch.empty_like(wide["k"]), "v": torch.empty_like(v),
         "g": torch.empty(T, Hv, dtype=torch.float64, device=dev)}
    Z = s["dfinal"].double()[order] if s["states"] else torch.zeros_like(S)
    for c in reversed(range(len(kept))):
        X = kept.pop()
        ts = list(range(c * CHUNK, min((c + 1) * CHUNK, lens[0])))
        told = []
        for t in ts:
            before = X[:alive[t]].clone()
            told.append((step(X, t, alive[t]), before, X[:alive[t]].clone()))
        for t in reversed(ts):
            r, P, after = told.pop()
            n = len(r)
            do = s["scale"] * s["dout"][r].double()
            d["q"][r] = torch.matmul(after, do[..., None])[..., 0]
            Z[:n] += wide["q"][r][..., :, None] * do[..., None, :]
            d["k"][r] = torch.matmul(Z[:n], v[r][..., None])[..., 0]
            d["v"][r] = torch.matmul(wide["k"][r][..., None, :], Z[:n])[..., 0, :]
            Z[:n] *= a[r][..., None, None]
            d["g"][r] = (P * Z[:n]).sum((-2, -1))
    for n in ("q", "k"):
        d[n] = d[n].unflatten(1, (-1, rep)).sum(2)
    if s["decay"] == "head":
        d["g"] = d["g"].sum(0)
    res.update({"d" + n: x for n, x in d.items()})
    if s["states"]:
        res["dinit"] = torch.empty_like(Z).index_copy(0, order, Z)
    return res


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "linear":
        return _exact_linear(s)
    rep = case["Hv"] // case["Hk"]
    out = torch.empty(s["v"].shape, dtype=torch.float64, device=s["v"].device)
    states = s["states"].double()
    a = s["g"].double().exp()
    for i, slot in enumerate(s["slots"].tolist()):
        S = states[slot]
        S *= (a[i] if a.dim() == 2 else a)[:, None, None]
        k, q = (s[n][i].double().repeat_interleave(rep, 0) for n in ("k", "q"))
        S += torch.einsum("hk,hv->hkv", k, s["v"][i].double())
        out[i] = s["scale"] * torch.einsum("hk,hkv->hv", q, S)
    return {"out": out, "states": states}
