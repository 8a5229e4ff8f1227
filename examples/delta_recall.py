"""A small language model on the gated delta rule: training and answering.

    python examples/delta_recall.py [--steps 200] [--blocks 2] [--pairs 96]

The task is recall by key: the model reads `pairs` positions that each carry a
key and a value, then is asked for the values of the keys in another order.
Each block is

    u = layernorm(x);  q, k, v, g, beta = projections of u
    o = delta rule(q, k, v, g, beta);  x = x + W layernorm_per_head(o)

Training runs cssd.layernorm / delta_forward and their gradients through two
torch.autograd functions.  Answering reads the prompt with one delta_forward a
block, which leaves the block's state, and then takes the questions one token
at a time with delta_step; its logits must be the ones that a forward over the
whole sequence gives.  Parameters are float32, activations bfloat16; the
projections are torch's matrix products.
"""

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from complex_valued_state_gb300 import cssd  # noqa: E402


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        y, mean, rstd = cssd.layernorm(x, weight, bias)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        g = cssd.layernorm_backward(dy.contiguous(), x, weight, mean, rstd)
        return g["gx"], g["gweight"], g["gbias"]


class DeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta):
        ctx.save_for_backward(q, k, v, g, beta)
        return cssd.delta_forward(q, k, v, g, beta, want_state=False)[0]

    @staticmethod
    def backward(ctx, do):
        r = cssd.delta_backward(*ctx.saved_tensors, do.contiguous())
        return r["gq"], r["gk"], r["gv"], r["gg"], r["gbeta"]


class Block(torch.nn.Module):
    """`heads` value heads of P columns over `kheads` key heads of N rows."""

    def __init__(self, width, heads, kheads, N, P):
        super().__init__()
        self.shape = (heads, kheads, N, P)
        self.sizes = [kheads * N, kheads * N, heads * P, heads, heads]
        self.inp = torch.nn.Parameter(torch.randn(sum(self.sizes), width) * width ** -0.5)
        with torch.no_grad():  # a question starts out looking for its own key
            self.inp[:kheads * N] = self.inp[kheads * N:2 * kheads * N]
        self.out = torch.nn.Parameter(torch.randn(width, heads * P) * (heads * P) ** -0.5)
        self.rate = torch.nn.Parameter(torch.linspace(-6, -3, heads))
        self.norm_w, self.norm_b = (torch.nn.Parameter(f(width)) for f in (torch.ones, torch.zeros))
        self.head_w, self.head_b = (torch.nn.Parameter(f(P)) for f in (torch.ones, torch.zeros))

    def project(self, x, norm):
        """x [..., width] -> q, k of unit length, v, the log decay and the write strength."""
        heads, kheads, N, P = self.shape
        z = norm(x, self.norm_w, self.norm_b) @ self.inp.to(x.dtype).T
        q, k, v, g, beta = z.split(self.sizes, -1)
        q, k = (F.normalize(t.unflatten(-1, (kheads, N)).float(), dim=-1).to(x.dtype) for t in (q, k))
        return q, k, v.unflatten(-1, (heads, P)).contiguous(), -F.softplus(g.float() + self.rate), beta.float().sigmoid()

    def finish(self, x, o, norm):
        return x + norm(o, self.head_w, self.head_b).flatten(-2) @ self.out.to(x.dtype).T

    def forward(self, x):
        return self.finish(x, DeltaRule.apply(*self.project(x, LayerNorm.apply)), LayerNorm.apply)

    def prompt(self, x):
        """The forward of a prompt; also returns the state after it."""
        o, state = cssd.delta_forward(*self.project(x, plain_norm))
        return self.finish(x, o, plain_norm), state

    def step(self, x, state):
        """One token x [batch, width]; `state` is updated in place."""
        return self.finish(x, cssd.delta_step(state, *self.project(x, plain_norm)), plain_norm)


def plain_norm(x, weight, bias):
    return cssd.layernorm(x, weight, bias)[0]


class Model(torch.nn.Module):
    def __init__(self, vocab, width=256, blocks=2, heads=4, kheads=2, N=64, P=64):
        super().__init__()
        self.key = torch.nn.Parameter(torch.randn(vocab, width))
        self.value = torch.nn.Parameter(torch.randn(vocab + 1, width))  # the last: a question
        self.blocks = torch.nn.ModuleList(Block(width, heads, kheads, N, P) for _ in range(blocks))
        self.norm_w, self.norm_b = (torch.nn.Parameter(f(width)) for f in (torch.ones, torch.zeros))
        self.head = torch.nn.Parameter(torch.randn(vocab, width) * width ** -0.5)

    def embed(self, keys, values):
        return (self.key[keys] + self.value[values]).to(torch.bfloat16)

    def logits(self, x, norm):
        return (norm(x, self.norm_w, self.norm_b) @ self.head.to(x.dtype).T).float()

    def forward(self, keys, values):
        x = self.embed(keys, values)
        for b in self.blocks:
            x = b(x)
        return self.logits(x, LayerNorm.apply)

    @torch.no_grad()
    def answer(self, keys, values, asked):
        """Logits of the questions `asked` [batch, n] after the prompt, token by token."""
        x = self.embed(keys, values)
        states = []
        for b in self.blocks:
            x, s = b.prompt(x)
            states.append(s)
        out = []
        for t in range(asked.shape[1]):
            x = self.embed(asked[:, t], torch.full_like(asked[:, t], self.value.shape[0] - 1))
            for b, s in zip(self.blocks, states):
                x = b.step(x, s)
            out.append(self.logits(x, plain_norm))
        return torch.stack(out, 1)


def batch(gen, n, pairs, vocab, device):
    """Distinct keys with random values, and as many questions in another order."""
    keys = torch.rand(n, vocab, generator=gen).argsort(1)[:, :pairs]
    values = torch.randint(vocab, (n, pairs), generator=gen)
    order = torch.rand(n, pairs, generator=gen).argsort(1)
    return tuple(t.to(device) for t in (keys, values, keys.gather(1, order), values.gather(1, order)))


def run(steps=200, blocks=2, pairs=96, vocab=256, rows=32, seed=0, report=print):
    torch.manual_seed(seed)
    gen = torch.Generator().manual_seed(seed)
    model = Model(vocab, blocks=blocks).cuda()
    opt = torch.optim.AdamW(model.parameters(), lr=2e-3, weight_decay=0.0)
    losses = []
    for i in range(steps):
        keys, values, asked, want = batch(gen, rows, pairs, vocab, "cuda")
        blank = torch.full_like(asked, vocab)
        logits = model(torch.cat([keys, asked], 1), torch.cat([values, blank], 1))[:, pairs:]
        loss = F.cross_entropy(logits.flatten(0, 1), want.flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        if i % 20 == 0 or i == steps - 1:
            losses.append(loss.item())
            report(f"step {i:4d}  loss {losses[-1]:.4f}")
    keys, values, asked, want = batch(gen, rows, pairs, vocab, "cuda")
    blank = torch.full_like(asked, vocab)
    with torch.no_grad():
        whole = model(torch.cat([keys, asked], 1), torch.cat([values, blank], 1))[:, pairs:]
    token = model.answer(keys, values, asked)
    right = (token.argmax(-1) == want).float().mean().item()
    apart = ((token - whole).abs().max() / whole.abs().max()).item()
    report(f"answered token by token: {100 * right:.1f} % right; logits within {apart:.1e} of the whole forward's")
    return {"losses": losses, "right": right, "apart": apart}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--pairs", type=int, default=96)
    a = ap.parse_args()
    run(a.steps, a.blocks, a.pairs)
