"""A gated-delta-rule layer on packed sequences, trained and then served.

  projections -> varlen_conv1d (SiLU) -> varlen_qk_norm_rope (unit length) -> varlen_gated_delta -> gate -> projection

The toy task is associative recall: a sequence lists (key, value) token pairs
and then asks for some keys again; the model has to answer with their values.
After training, the prompt of each sequence is run once with its final states
kept (prefill), and the remaining tokens one at a time against the state pool
(varlen_gated_delta_step); both ways give the same answers.

    python examples/gated_delta_layer.py [--steps 400]
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import selective_ssm_packed_gb300 as vs  # noqa: E402


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b, cu, pos):
        ctx.save_for_backward(x, w, b, cu, pos)
        return vs.varlen_conv1d_fwd(x, w, b, cu, pos)

    @staticmethod
    def backward(ctx, du):
        x, w, b, cu, pos = ctx.saved_tensors
        return (*vs.varlen_conv1d_bwd(x, w, b, du.contiguous(), cu, pos), None, None)


class UnitQK(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k):
        ctx.save_for_backward(q, k)
        return vs.varlen_qk_norm_rope_fwd(q, k, mode="l2")

    @staticmethod
    def backward(ctx, dq, dk):
        q, k = ctx.saved_tensors
        g = vs.varlen_qk_norm_rope_bwd(q, k, None, None, None, None, None, dq.contiguous(), dk.contiguous(), mode="l2")
        return g["dq"], g["dk"]


class GatedDelta(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, cu):
        out, saved = vs.varlen_gated_delta_fwd(q, k, v, g, beta, cu)
        ctx.save_for_backward(q, k, v, g, beta, cu, saved)
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, g, beta, cu, saved = ctx.saved_tensors
        r = vs.varlen_gated_delta_bwd(q, k, v, g, beta, dout.contiguous(), cu, saved)
        return r["dq"], r["dk"], r["dv"], r["dg"], r["dbeta"], None


class GatedDeltaLayer(torch.nn.Module):
    def __init__(self, d_model, Hk=1, Hv=2, K=64, V=64, W=4):
        super().__init__()
        self.Hk, self.Hv, self.K, self.V, self.W = Hk, Hv, K, V, W
        self.widths = (Hk * K, Hk * K, Hv * V)
        self.proj = torch.nn.Linear(d_model, sum(self.widths) + Hv * V + 2 * Hv, bias=False)
        bound = W ** -0.5
        self.conv_w = torch.nn.Parameter(torch.empty(sum(self.widths), W).uniform_(-bound, bound))
        self.conv_b = torch.nn.Parameter(torch.zeros(sum(self.widths)))
        self.a_log = torch.nn.Parameter(torch.empty(Hv).uniform_(1, 16).log())
        self.dt_bias = torch.nn.Parameter(torch.full((Hv,), -4.0))
        self.out = torch.nn.Linear(Hv * V, d_model, bias=False)

    def split(self, x):
        n = sum(self.widths)
        p = self.proj(x)
        gate, a, b = p[:, n:].split([self.Hv * self.V, self.Hv, self.Hv], 1)
        g = -torch.exp(self.a_log) * torch.nn.functional.softplus(a + self.dt_bias)
        return p[:, :n].contiguous(), gate, g.contiguous(), torch.sigmoid(b).contiguous()

    def heads(self, u):
        q, k, v = u.split(self.widths, 1)
        return q.unflatten(1, (self.Hk, self.K)), k.unflatten(1, (self.Hk, self.K)), v.unflatten(1, (self.Hv, self.V))

    def finish(self, o, gate):
        o = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + 1e-6)
        return self.out(o.flatten(1) * torch.nn.functional.silu(gate))

    def forward(self, x, cu, pos):
        mixed, gate, g, beta = self.split(x)
        q, k, v = self.heads(Conv.apply(mixed, self.conv_w, self.conv_b, cu, pos))
        q, k = UnitQK.apply(q, k)
        return self.finish(GatedDelta.apply(q, k, v, g, beta, cu), gate)

    @torch.no_grad()
    def prefill(self, x, cu):
        """(output, conv tails, states) of whole prompts."""
        mixed, gate, g, beta = self.split(x)
        u, tails = vs.varlen_conv1d_fwd(mixed, self.conv_w, self.conv_b, cu, x_last=True)
        q, k, v = self.heads(u)
        q, k = vs.varlen_qk_norm_rope_fwd(q, k, mode="l2")
        o, _, states = vs.varlen_gated_delta_fwd(q, k, v, g, beta, cu, saved=False, final_states=True)
        return self.finish(o, gate), tails, states

    @torch.no_grad()
    def step(self, x, tails, states):
        """One token of each sequence; the states are updated in place.  Returns (output, tails)."""
        mixed, gate, g, beta = self.split(x)
        cu = torch.arange(x.shape[0] + 1, dtype=torch.int32, device=x.device)
        u, tails = vs.varlen_conv1d_fwd(mixed, self.conv_w, self.conv_b, cu, x_init=tails, x_last=True)
        q, k, v = self.heads(u)
        q, k = vs.varlen_qk_norm_rope_fwd(q, k, mode="l2")
        return self.finish(vs.varlen_gated_delta_step(q, k, v, g, beta, states), gate), tails


class Model(torch.nn.Module):
    def __init__(self, vocab, d_model=128, layers=2):
        super().__init__()
        self.embed = torch.nn.Embedding(vocab, d_model)
        self.layers = torch.nn.ModuleList(GatedDeltaLayer(d_model) for _ in range(layers))
        self.norms = torch.nn.ModuleList(torch.nn.LayerNorm(d_model) for _ in range(layers))
        self.head = torch.nn.Sequential(torch.nn.LayerNorm(d_model), torch.nn.Linear(d_model, vocab))

    def forward(self, tokens, cu, pos):
        x = self.embed(tokens)
        for norm, m in zip(self.norms, self.layers):
            x = x + m(norm(x), cu, pos)
        return self.head(x)


def recall_batch(gen, sequences, keys=32, max_pairs=12, asked=4):
    """Packed tokens, targets (-1 where nothing is asked) and lengths."""
    tokens, targets, lens = [], [], []
    for _ in range(sequences):
        n = int(torch.randint(asked, max_pairs + 1, (1,), generator=gen))
        k = torch.randperm(keys, generator=gen)[:n]
        v = torch.randint(keys, 2 * keys, (n,), generator=gen)
        at = torch.randperm(n, generator=gen)[:asked]
        tokens.append(torch.cat([torch.stack([k, v], 1).flatten(), k[at]]))
        targets.append(torch.cat([torch.full((2 * n,), -1), v[at]]))
        lens.append(2 * n + asked)
    return torch.cat(tokens), torch.cat(targets), lens


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=400)
    args = ap.parse_args()
    torch.manual_seed(0)
    gen = torch.Generator().manual_seed(0)
    dev, asked = torch.device("cuda"), 4
    model = Model(vocab=64).to(dev)
    opt = torch.optim.AdamW(model.parameters(), lr=2e-3)
    first = loss = None
    for i in range(args.steps):
        tokens, targets, lens = recall_batch(gen, 256, asked=asked)
        cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device=dev)
        pos = vs.varlen_position_indices(cu, len(tokens))
        loss = torch.nn.functional.cross_entropy(model(tokens.to(dev), cu, pos), targets.to(dev), ignore_index=-1)
        opt.zero_grad()
        loss.backward()
        opt.step()
        first = first if first is not None else loss.item()
        if i % 20 == 0 or i + 1 == args.steps:
            print(f"step {i:4d}  loss {loss.item():.4f}")
    assert loss.item() < first, "the loss did not fall"

    # serving: the pairs as a prompt, then the questions one token at a time
    tokens, targets, lens = recall_batch(gen, 16, asked=asked)
    tokens, targets = tokens.to(dev), targets.to(dev)
    starts = [0, *torch.tensor(lens).cumsum(0).tolist()]
    cu = torch.tensor(starts, dtype=torch.int32, device=dev)
    with torch.no_grad():
        whole = model(tokens, cu, vs.varlen_position_indices(cu, len(tokens)))
    prompts = torch.cat([tokens[a:b - asked] for a, b in zip(starts, starts[1:])])
    pcu = torch.tensor([0, *torch.tensor([n - asked for n in lens]).cumsum(0).tolist()], dtype=torch.int32, device=dev)
    with torch.no_grad():
        x, kept = model.embed(prompts), []
        for norm, m in zip(model.norms, model.layers):
            y, tails, states = m.prefill(norm(x), pcu)
            kept.append([tails, states])
            x = x + y
        right = worst = 0
        for j in range(asked):
            at = torch.tensor([b - asked + j for b in starts[1:]], device=dev)
            x = model.embed(tokens[at])
            for norm, m, state in zip(model.norms, model.layers, kept):
                y, state[0] = m.step(norm(x), *state)
                x = x + y
            logits = model.head(x)
            worst = max(worst, (logits - whole[at]).abs().max().item() / whole.abs().max().item())
            right += (logits.argmax(-1) == targets[at]).sum().item()
    print(f"served token by token: {right} of {16 * asked} answers right; logits within {worst:.1e} of the packed forward")
    assert worst < 1e-3


if __name__ == "__main__":
    main()
