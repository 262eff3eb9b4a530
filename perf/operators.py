"""The gated-delta-rule operators on real work: cases, inputs, plain forms and 64-bit values.

Two operators next to the packed conv1d and the selective scan, on the same packed layout ((total_tokens, heads,
width) tensors plus int32 cu_seqlens):

  norm    queries and keys normalised for each head, with the position rotation in the same pass; forward, and
          forward + backward
  delta   the gated delta rule  S_t = a_t S_{t-1} + k_t (beta_t (v_t - a_t S_{t-1}^T k_t))^T,  o_t = scale S_t^T q_t,
          a_t = exp(g_t), with the state reset at every sequence start: forward (training and prefill), forward +
          backward, and one token for each of many sequences against a pool of states (serving)

With `own` false, run() computes them from elementary torch operations in 32 bits: the delta rule in chunks of 64
tokens, batched over chunks, heads and sequences.  With `own` true it calls the framework.
"""
import math

import numpy as np
import torch

own = False

CHUNK = 64  # tokens the plain form takes at a time


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token of one user: a call's latency
        dict(name="norm_decode_1", op="norm", train=False, T=1, Hq=16, Hk=16, K=128, rot=128, mode="rms", dtype="bf16",
             pack="decode", max_pos=8192),
        # the 1536-channel layer's 4096-token pack, fp32: the delta rule's unit-length keys, no rotation
        dict(name="norm_l2_1536_f32", op="norm", train=False, T=4096, Hq=12, Hk=12, K=128, rot=0, mode="l2",
             dtype="f32", pack="median300", max_pos=4096),
        # the 4096-channel layer's 32768 packed tokens, q and k as slices of one fused projection, 2:1 shared keys
        dict(name="norm_rope_4096_bf16", op="norm", train=False, T=32768, Hq=32, Hk=16, K=128, rot=128, mode="rms",
             dtype="bf16", pack="median800", max_pos=4096),
        # the same layer's training step, half of each head rotated
        dict(name="norm_rope_train_bf16", op="norm", train=True, T=32768, Hq=32, Hk=16, K=128, rot=64, mode="rms",
             dtype="bf16", pack="median800", max_pos=4096),
        # the 16-token, 4-sequence pack: the smallest forward call
        dict(name="delta_tiny_f32", op="delta", train=False, T=16, Hk=2, Hv=4, K=64, V=64, dtype="f32", pack="tiny",
             states=False),
        # the 1536-channel layer: one 4096-token pack of log-normal lengths, fp32
        dict(name="delta_1536_f32", op="delta", train=False, T=4096, Hk=12, Hv=12, K=128, V=128, dtype="f32",
             pack="median300", states=False),
        # the 4096-channel layer: 8 packs of 4096 tokens, bf16, two value heads to a key head
        dict(name="delta_4096_bf16", op="delta", train=False, T=32768, Hk=16, Hv=32, K=128, V=128, dtype="bf16",
             pack="median800", states=False),
        # one 32768-token sequence (the long tail's longest), continued from a state: prefill of a long prompt's part
        dict(name="delta_long_bf16", op="delta", train=False, T=32768, Hk=16, Hv=32, K=128, V=128, dtype="bf16",
             pack="one", states=True),
        # odd sizes in fp32 with states and their gradients: sequences cut across packs
        dict(name="delta_train_odd_f32", op="delta", train=True, T=3001, Hk=3, Hv=6, K=96, V=80, dtype="f32",
             pack="median300", states=True),
        # the 4096-channel layer's training step
        dict(name="delta_train_4096_bf16", op="delta", train=True, T=32768, Hk=16, Hv=32, K=128, V=128, dtype="bf16",
             pack="median800", states=False),
        # one user's next token
        dict(name="step_1_bf16", op="step", B=1, slots=1, Hk=16, Hv=32, K=128, V=128, dtype="bf16"),
        # a serving batch's next tokens: 256 sequences in a pool of 320 states
        dict(name="step_256_bf16", op="step", B=256, slots=320, Hk=16, Hv=32, K=128, V=128, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_train", "delta", "delta", "delta_train", "delta_train", "step"])
    dtype = rng.choice(["bf16", "f32"])
    if op.startswith("norm"):
        K = 8 * _log_int(rng, 2, 32)
        Hk = rng.randint(1, 16)
        Hq = Hk * rng.choice([1, 2, 3])
        T = _log_int(rng, 1, max(1, min(32768, 32768 * 48 * 128 // ((Hq + Hk) * K * (2 if dtype == "f32" else 1)))))
        rot = rng.choice([0, K, 8 * rng.randint(1, K // 8)])
        return dict(op="norm", train=op == "norm_train", T=T, Hq=Hq, Hk=Hk, K=K, rot=rot,
                    mode=rng.choice(["rms", "l2"]), dtype=dtype, pack=rng.choice(["median300", "decode"]),
                    max_pos=4096)
    Hk = rng.randint(1, 12)
    Hv = Hk * rng.choice([1, 2, 4])
    K, V = 8 * rng.randint(2, 16), 8 * rng.randint(2, 20)
    if op == "step":
        B = _log_int(rng, 1, 256)
        return dict(op="step", B=B, slots=B + rng.randint(0, 64), Hk=Hk, Hv=Hv, K=K, V=V, dtype=dtype)
    # at most a quarter of the largest listed case's heads times tokens
    T = _log_int(rng, 7, 32768 * 8 // Hv)
    return dict(op="delta", train=op == "delta_train", T=T, Hk=Hk, Hv=Hv, K=K, V=V, dtype=dtype,
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
    K = case["K"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(shape, generator=gen, device=dev)

    s = dict(case)
    if case["op"] == "norm":
        T, Hq, Hk = case["T"], case["Hq"], case["Hk"]
        # q, k and v leave one projection: q and k are slices of its rows, channels of unlike scale
        fused = (normal(T, (Hq + 2 * Hk) * K) * torch.exp(0.5 * normal((Hq + 2 * Hk) * K))).to(dt)
        s["q"] = fused[:, :Hq * K].unflatten(1, (Hq, K))
        s["k"] = fused[:, Hq * K:(Hq + Hk) * K].unflatten(1, (Hk, K))
        rms = case["mode"] == "rms"
        s["qw"] = 1 + 0.1 * normal(K) if rms else None
        s["kw"] = 1 + 0.1 * normal(K) if rms else None
        s["cos"] = s["sin"] = s["pos"] = None
        if case["rot"]:
            half = case["rot"] // 2
            freq = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
            angle = torch.arange(case["max_pos"], device=dev, dtype=torch.float64)[:, None] * freq
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
            if case["pack"] == "decode":  # each token of another sequence, at its own position
                s["pos"] = torch.randint(0, case["max_pos"], (T,), generator=gen, device=dev, dtype=torch.int32)
            else:
                s["pos"] = torch.cat([torch.arange(n, dtype=torch.int32) for n in lengths_of(case)]).to(dev)
        if case["train"]:
            s["dq"], s["dk"] = normal(T, Hq, K).to(dt), normal(T, Hk, K).to(dt)
        return s

    Hk, Hv, V = case["Hk"], case["Hv"], case["V"]
    n = case["B"] if case["op"] == "step" else case["T"]

    def unit(x):
        return (x / x.square().sum(-1, keepdim=True).sqrt()).to(dt)

    # keys and queries leave a SiLU convolution (values mostly above zero) and a unit-length norm
    s["q"] = unit(normal(n, Hk, K) + 0.3)
    s["k"] = unit(normal(n, Hk, K) + 0.3)
    s["v"] = normal(n, Hv, V).to(dt)
    # g = -A softplus(a + dt_bias) with A in [1, 16] and steps of 1e-3 to 1e-1; beta in (0, 1)
    step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), Hv))
    bias = step + torch.log(-torch.expm1(-step))
    s["g"] = -uniform(1.0, 16.0, Hv) * torch.nn.functional.softplus(0.5 * normal(n, Hv) + bias)
    s["beta"] = torch.sigmoid(normal(n, Hv))
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
def _norm_rows(x, w, mode):
    x = x.float()
    sq = x.square()
    r = torch.rsqrt((sq.mean(-1, keepdim=True) if mode == "rms" else sq.sum(-1, keepdim=True)) + 1e-6)
    n = x * r
    return n, r, (n * w if w is not None else n)


def _rotate(x, cos, sin, back=False):
    if cos is None:
        return x
    half = cos.shape[1]
    a, b, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
    c, s = cos[:, None], (-sin if back else sin)[:, None]
    return torch.cat([a * c - b * s, b * c + a * s, rest], -1)


def _plain_norm(s):
    cos, sin = (s["cos"][s["pos"].long()], s["sin"][s["pos"].long()]) if s["cos"] is not None else (None, None)
    out = {}
    for x, w, dy, name in ((s["q"], s["qw"], s.get("dq"), "q"), (s["k"], s["kw"], s.get("dk"), "k")):
        n, r, y = _norm_rows(x, w, s["mode"])
        out[name] = _rotate(y, cos, sin).to(x.dtype)
        if dy is not None:
            dy = _rotate(dy.float(), cos, sin, back=True)
            dn = dy * w if w is not None else dy
            dot = (dn * n).sum(-1, keepdim=True)
            out["d" + name] = (r * (dn - n * (dot / n.shape[-1] if s["mode"] == "rms" else dot))).to(x.dtype)
            if w is not None:
                out["d" + name + "w"] = (dy * n).sum((0, 1))
    return out


def _unit_lower_inverse(N):
    """(I + N)^-1 for strictly lower N (..., n, n), n a power of two: halves inverted, then joined."""
    n, block = N.shape[-1], 1
    inv = torch.eye(n, device=N.device).expand_as(N)
    while block < n:
        idx = torch.arange(n, device=N.device) // block
        low = (idx[:, None] == idx[None, :] + 1) & (idx[:, None] % 2 == 1)
        inv = inv - inv @ torch.where(low, N, 0.0) @ inv
        block *= 2
    return inv


def _plain_delta(q, k, v, g, beta, init, scale, plan):
    """out (T, Hv, V) and final states, all float32, in chunks."""
    at, mask = plan["at"], plan["mask"]
    T, Hv, V = v.shape
    rep = Hv // k.shape[1]

    def chunks(x):  # (T, H, ...) -> (H, chunks, CHUNK, ...), zero past a sequence's end
        x = torch.where(mask.reshape(mask.shape + (1,) * (x.dim() - 1)), x[at], 0.0)
        return x.movedim(2, 0)

    q, k, v = chunks(q).repeat_interleave(rep, 0), chunks(k).repeat_interleave(rep, 0), chunks(v)
    G, b = torch.cumsum(chunks(g), -1), chunks(beta)
    i = torch.arange(CHUNK, device=v.device)
    low = i[:, None] >= i[None, :]
    decay = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -torch.inf))
    N = torch.where(i[:, None] > i[None, :], (k @ k.mT) * decay, 0.0) * b[..., None, :]
    inv = _unit_lower_inverse(N)
    P = scale * (q @ k.mT) * decay
    gam, dec = torch.exp(G)[..., None], torch.exp(G[..., -1:] - G)[..., None]
    b = b[..., None]
    ve, ke = inv @ v, inv @ (gam * k)
    qs, kd = scale * gam * q, dec * b * k
    S = init[plan["order"]].movedim(1, 0) if init is not None else v.new_zeros(Hv, len(plan["order"]), k.shape[-1], V)
    out, final = [], []
    for ids in plan["steps"]:
        final.append(S[:, len(ids):])
        S = S[:, :len(ids)]
        e = ve[:, ids] - ke[:, ids] @ S
        out.append(qs[:, ids] @ S + P[:, ids] @ (b[:, ids] * e))
        S = gam[:, ids, -1:] * S + kd[:, ids].mT @ e
    final = torch.cat([S] + final[::-1], 1).movedim(0, 1)
    final = torch.empty_like(final).index_copy(0, plan["order"], final)
    o = torch.empty_like(v).index_copy(1, torch.cat(plan["steps"]), torch.cat(out, 1))
    return o.movedim(0, 2).reshape(-1, Hv, V)[plan["place"]], final


def _plain_step(s):
    rep = s["v"].shape[1] // s["k"].shape[1]
    q, k = (x.float().repeat_interleave(rep, 1) for x in (s["q"], s["k"]))
    at = s["slots"].long()
    S = s["states"][at] * torch.exp(s["g"])[..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    s["states"][at] = S
    return {"out": (s["scale"] * (S * q[..., None]).sum(-2)).to(s["v"].dtype), "states": s["states"]}


def _plain(s):
    if s["op"] == "norm":
        return _plain_norm(s)
    if s["op"] == "step":
        return _plain_step(s)
    dt = s["v"].dtype
    names = ["q", "k", "v", "g", "beta"] + (["init"] if s["init"] is not None else [])
    x = {n: s[n].float() for n in names}
    if s["train"]:
        x = {n: t.detach().requires_grad_() for n, t in x.items()}
    o, final = _plain_delta(x["q"], x["k"], x["v"], x["g"], x["beta"], x.get("init"), s["scale"], s["plan"])
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
        args = (s["q"], s["k"], s["qw"], s["kw"], s["cos"], s["sin"], s["pos"])
        q, k = vs.varlen_qk_norm_rope_fwd(*args, mode=s["mode"])
        out = {"q": q, "k": k}
        if s["train"]:
            g = vs.varlen_qk_norm_rope_bwd(*args, s["dq"], s["dk"], mode=s["mode"])
            out.update(dq=g["dq"], dk=g["dk"])
            if s["qw"] is not None:
                out.update(dqw=g["dq_weight"], dkw=g["dk_weight"])
        return out
    if s["op"] == "step":
        out = vs.varlen_gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"],
                                         state_indices=s["slots"], scale=s["scale"])
        return {"out": out, "states": s["states"]}
    args = (s["q"], s["k"], s["v"], s["g"], s["beta"])
    res = vs.varlen_gated_delta_fwd(*args, s["cu"], scale=s["scale"], saved=s["train"], initial_states=s["init"],
                                    final_states=s["states"])
    out = {"out": res[0]}
    if s["states"]:
        out["final"] = res[2]
    if s["train"]:
        g = vs.varlen_gated_delta_bwd(*args, s["dout"], s["cu"], res[1], scale=s["scale"],
                                      d_final_states=s["dfinal"], d_initial_states=s["states"])
        out.update(dq=g["dq"], dk=g["dk"], dv=g["dv"], dg=g["dg"], dbeta=g["dbeta"])
        if s["states"]:
            out["dinit"] = g["d_initial_states"]
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the work a pass cannot do without
def work(case):
    io = 2 if case["dtype"] == "bf16" else 4
    K = case["K"]
    if case["op"] == "norm":
        T, H = case["T"], case["Hq"] + case["Hk"]
        rows = T * H * K
        table = min(T, case["max_pos"]) * case["rot"] * 4
        passes = 5 if case["train"] else 2  # x and dy read, y and dx written; x is read by both passes
        return {"bytes": passes * rows * io + table, "flops": rows * (20 if case["train"] else 7)}
    Hk, Hv, V = case["Hk"], case["Hv"], case["V"]
    state = Hv * K * V
    if case["op"] == "step":
        B = case["B"]
        return {"bytes": 8 * B * state + B * (2 * Hk * K + 2 * Hv * V) * io + 8 * B * Hv, "flops": 7 * B * state}
    T = case["T"]
    seqs = len(lengths_of(case))
    read = T * (2 * Hk * K + Hv * V) * io + 8 * T * Hv
    nbytes = read + T * Hv * V * io + (8 * seqs * state if case["states"] else 0)
    if case["train"]:  # inputs again, dout, and the gradients
        nbytes += 2 * read + T * Hv * V * io + (8 * seqs * state if case["states"] else 0)
    return {"bytes": nbytes, "flops": (21 if case["train"] else 7) * T * state}


# ------------------------------------------------------------------ 64-bit values, token by token
def _exact_norm(s):
    out = {}
    turn = None
    if s["cos"] is not None:
        p = s["pos"].long()
        turn = torch.complex(s["cos"].double()[p], s["sin"].double()[p])[:, None]

    def turned(y, z):
        if z is None:
            return y
        h = z.shape[-1]
        c = torch.complex(y[..., :h], y[..., h:2 * h]) * z
        return torch.cat([c.real, c.imag, y[..., 2 * h:]], -1)

    for name, wn in (("q", "qw"), ("k", "kw")):
        x = s[name].double()
        w = s[wn].double() if s[wn] is not None else torch.ones(x.shape[-1], device=x.device, dtype=torch.float64)
        count = x.shape[-1] if s["mode"] == "rms" else 1
        length = ((x * x).sum(-1, keepdim=True) / count + 1e-6).sqrt()
        out[name] = turned(w * x / length, turn)
        if "d" + name in s:
            d = turned(s["d" + name].double(), turn.conj() if turn is not None else None)
            dw = d * w
            out["d" + name] = dw / length - x * (dw * x).sum(-1, keepdim=True) / (count * length ** 3)
            if s[wn] is not None:
                out["d" + name + "w"] = (d * x / length).sum((0, 1))
    return out


def _exact_delta(s):
    """Forward token by token; backward by the adjoint recurrence, the states of 64 tokens at a time recomputed."""
    rep = s["v"].shape[1] // s["k"].shape[1]
    cu = s["cu"].tolist()
    seqs = [i for i in np.argsort([-(cu[i + 1] - cu[i]) for i in range(len(cu) - 1)], kind="stable")]
    lens = [cu[i + 1] - cu[i] for i in seqs]
    first = torch.tensor([cu[i] for i in seqs], device=s["v"].device)
    order = torch.tensor([int(i) for i in seqs], device=s["v"].device)
    T, Hv, V = s["v"].shape
    K = s["k"].shape[2]
    S = torch.zeros(len(seqs), Hv, K, V, dtype=torch.float64, device=s["v"].device)
    if s["init"] is not None:
        S += s["init"][order].double()
    alive = np.array([sum(n > t for n in lens) for t in range(lens[0])])

    def tokens(t, n):
        r = first[:n] + t
        wide = lambda x: x[r].double().repeat_interleave(rep, 1)  # noqa: E731
        return r, wide(s["q"]), wide(s["k"]), s["v"][r].double(), s["g"][r].double().exp(), s["beta"][r].double()

    def step(S, t, n):  # advances S[:n] in place; returns what the adjoint needs
        r, q, k, v, a, b = tokens(t, n)
        S[:n] *= a[..., None, None]
        e = v - torch.einsum("shkv,shk->shv", S[:n], k)
        S[:n] += k[..., None] * (b[..., None] * e)[..., None, :]
        return r, q, k, a, b, e

    out = torch.empty(T, Hv, V, dtype=torch.float64, device=S.device)
    kept = []
    for t in range(lens[0]):
        n = int(alive[t])
        if s["train"] and t % CHUNK == 0:
            kept.append(S[:n].clone())
        r, q, *_ = step(S, t, n)
        out[r] = s["scale"] * torch.einsum("shkv,shk->shv", S[:n], q)
    res = {"out": out}
    if s["states"]:
        res["final"] = torch.empty_like(S).index_copy(0, order, S)
    if not s["train"]:
        return res
    d = {n: torch.empty(s[n].shape[0], Hv, *s[n].shape[2:], dtype=torch.float64, device=S.device)
         for n in ("q", "k", "v", "g", "beta")}
    dS = s["dfinal"][order].double() if s["states"] else torch.zeros_like(S)
    for c in reversed(range(len(kept))):
        X = kept.pop()
        ts = list(range(c * CHUNK, min((c + 1) * CHUNK, lens[0])))
        before, told = [], []
        for t in ts:
            n = int(alive[t])
            before.append(X[:n].clone())
            told.append(step(X, t, n))
        for t in reversed(ts):
            n = int(alive[t])
            (r, q, k, a, b, e), P = told.pop(), before.pop()
            D = dS[:n]
            do = s["scale"] * s["dout"][r].double()
            P *= a[..., None, None]                       # the decayed state the token meets
            u = b[..., None] * e
            d["q"][r] = torch.einsum("shkv,shv->shk", P, do) + k * (u * do).sum(-1, keepdim=True)
            D += q[..., None] * do[..., None, :]
            du = torch.einsum("shkv,shk->shv", D, k)
            d["k"][r] = torch.einsum("shkv,shv->shk", D, u) - torch.einsum("shkv,shv->shk", P, b[..., None] * du)
            d["v"][r] = b[..., None] * du
            d["beta"][r] = (du * e).sum(-1)
            D -= k[..., None] * (b[..., None] * du)[..., None, :]
            d["g"][r] = (D * P).sum((-2, -1))
            D *= a[..., None, None]
    for n in ("q", "k"):
        d[n] = d[n].unflatten(1, (-1, rep)).sum(2)
    res.update({"d" + n: x for n, x in d.items()})
    if s["states"]:
        res["dinit"] = torch.empty_like(dS).index_copy(0, order, dS)
    return res


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "delta":
        return _exact_delta(s)
    rep = case["Hv"] // case["Hk"]
    out = torch.empty(s["v"].shape, dtype=torch.float64, device=s["v"].device)
    states = s["states"].double()
    for i, slot in enumerate(s["slots"].tolist()):
        S = states[slot]
        for h in range(case["Hv"]):
            k, q = s["k"][i, h // rep].double(), s["q"][i, h // rep].double()
            S[h] *= s["g"][i, h].double().exp()
            S[h] += torch.outer(k, s["beta"][i, h].double() * (s["v"][i, h].double() - k @ S[h]))
            out[i, h] = s["scale"] * (q @ S[h])
    return {"out": out, "states": states}
