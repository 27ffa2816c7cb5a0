"""A gated delta rule layer as a model uses it: trained, then prefilled with packed
prompts and decoded token by token.

    h, n = norm(residual + scale * x)              blocknorm.add_*
    q, k, v, z, a, b = n W_in                      (a plain matrix product)
    g = -rate softplus(a + bias), beta = sigmoid(b)
    o = gated delta rule(q, k, v, g, beta)         gdr.forward / backward / step
    x' = (norm(o) * silu(z)) W_out                 blocknorm.gated_*

Run it on a GPU: python examples/gated_delta_layer.py [--steps 20] [--dtype bf16]
It trains two layers to copy a token seen some steps before, then checks that
prefill and decoding give what the whole sequence gives.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from linear_rnn_state_gb300 import blocknorm, gdr  # noqa: E402


class AddNorm(torch.autograd.Function):
    """(residual + scale x, its norm)."""

    @staticmethod
    def forward(ctx, x, residual, weight, scale):
        h, n, rstd = blocknorm.add_forward(x, residual, weight, scale)
        ctx.save_for_backward(x, residual, weight, scale, rstd)
        return h, n

    @staticmethod
    def backward(ctx, dh, dn):
        x, residual, weight, scale, rstd = ctx.saved_tensors
        g = blocknorm.add_backward(x, residual, weight, rstd, dn.contiguous(), dh.contiguous(), scale)
        return g["dx"], g["dresidual"], g["dweight"], g["dscale"]


class GatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, o, z, weight):
        y, rstd = blocknorm.gated_forward(o, z, weight)
        ctx.save_for_backward(o, z, weight, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        o, z, weight, rstd = ctx.saved_tensors
        g = blocknorm.gated_backward(o, z, weight, rstd, dy.contiguous())
        return g["do"], g["dz"], g["dweight"]


class Delta(torch.autograd.Function):
    """(o, s_final) of the gated delta rule with q and k normalised."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, state, starts):
        o, s, saved = gdr.forward(q, k, v, g, beta, state, qk_l2norm=True, seq_starts=starts)
        ctx.save_for_backward(q, k, v, g, beta, saved)
        ctx.starts, ctx.carry = starts, state is not None
        return o, s

    @staticmethod
    def backward(ctx, do, ds):
        q, k, v, g, beta, saved = ctx.saved_tensors
        d = gdr.backward(q, k, v, g, beta, do.contiguous(), saved, dS_final=ds.contiguous(), want_dS_init=ctx.carry,
                         qk_l2norm=True, seq_starts=ctx.starts)
        return d["dq"], d["dk"], d["dv"], d["dg"], d["dbeta"], d["dS_init"], None


class Layer(torch.nn.Module):
    def __init__(self, width, key_heads, heads, key, value, dtype):
        super().__init__()
        self.sizes = [key_heads * key, key_heads * key, heads * value, heads * value, heads, heads]
        self.shape = key_heads, heads, key, value
        self.weight, self.scale = (torch.nn.Parameter(torch.ones(width)) for _ in range(2))
        self.norm = torch.nn.Parameter(torch.ones(value))
        self.w_in = torch.nn.Parameter(torch.randn(width, sum(self.sizes), dtype=dtype) * width ** -0.5)
        self.w_out = torch.nn.Parameter(torch.randn(heads * value, width, dtype=dtype) * (heads * value) ** -0.5)
        self.rate = torch.nn.Parameter(torch.linspace(0.0, 1.0, heads))
        self.bias = torch.nn.Parameter(torch.full((heads,), -4.0))

    def project(self, n):
        """The layer's parts of the projection, q, k, v and z as slices of it."""
        Hk, H, K, V = self.shape
        q, k, v, z, a, b = (n @ self.w_in).split(self.sizes, -1)
        g = -self.rate.exp() * F.softplus(a.float() + self.bias)
        return (q.unflatten(-1, (Hk, K)), k.unflatten(-1, (Hk, K)), v.unflatten(-1, (H, V)), g, torch.sigmoid(b.float()),
                z.unflatten(-1, (H, V)))

    def forward(self, x, residual, state=None, starts=None):
        """x, residual [B][T][width] -> (the layer's output, the residual stream, the final states)."""
        h, n = AddNorm.apply(x, residual, self.weight, self.scale)
        q, k, v, g, beta, z = self.project(n)
        o, s = Delta.apply(q, k, v, g, beta, state, starts)
        return GatedNorm.apply(o, z, self.norm).flatten(-2) @ self.w_out, h, s

    @torch.no_grad()
    def step(self, x, residual, pool, slots):
        """One token of each request: x, residual [R][1][width]; pool's states are updated."""
        h, n, _ = blocknorm.add_forward(x, residual, self.weight, self.scale)
        q, k, v, g, beta, z = self.project(n)
        o = gdr.step(q, k, v, g, beta, pool, slots=slots, qk_l2norm=True)
        return blocknorm.gated_forward(o, z, self.norm)[0].flatten(-2) @ self.w_out, h


class Model(torch.nn.Module):
    def __init__(self, vocab=32, width=128, layers=2, key_heads=2, heads=4, key=32, value=64, dtype=torch.bfloat16):
        super().__init__()
        self.dtype = dtype
        self.embed = torch.nn.Parameter(torch.randn(vocab, width))
        self.layers = torch.nn.ModuleList(Layer(width, key_heads, heads, key, value, dtype) for _ in range(layers))
        self.weight = torch.nn.Parameter(torch.ones(width))
        self.head = torch.nn.Parameter(torch.randn(width, vocab, dtype=dtype) * width ** -0.5)

    def forward(self, tokens, states=None, starts=None):
        """tokens [B][T] -> (logits, the layers' final states). The residual stream is fp32."""
        h = self.embed[tokens]
        x = torch.zeros_like(h, dtype=self.dtype)
        out = []
        for i, layer in enumerate(self.layers):
            x, h, s = layer(x, h, None if states is None else states[i], starts)
            out.append(s)
        _, n = AddNorm.apply(x, h, self.weight, torch.ones_like(self.weight))
        return (n @ self.head).float(), out

    @torch.no_grad()
    def step(self, tokens, pools, slots):
        """The next token of each request, tokens [R]; logits [R][vocab]."""
        h = self.embed[tokens][:, None]
        x = torch.zeros_like(h, dtype=self.dtype)
        for layer, pool in zip(self.layers, pools):
            x, h = layer.step(x, h, pool, slots)
        _, n, _ = blocknorm.add_forward(x, h, self.weight)
        return (n @ self.head).float()[:, 0]


def train(model, steps, batch=16, length=96, back=3):
    """Learn to say the token of `back` steps before; the losses."""
    opt = torch.optim.Adam(model.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        tokens = torch.randint(0, model.embed.shape[0], (batch, length), device="cuda")
        logits, _ = model(tokens)
        loss = F.cross_entropy(logits[:, back:].flatten(0, 1), tokens[:, :-back].flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


@torch.no_grad()
def serve(model, lengths=(37, 1, 90), extra=8):
    """Prefill packed prompts, keep their states in a pool and decode; the largest
    difference of the logits from those of each whole sequence."""
    texts = [torch.randint(0, model.embed.shape[0], (n + extra,), device="cuda") for n in lengths]
    starts = torch.tensor([0, *torch.tensor(lengths).cumsum(0)], dtype=torch.int32, device="cuda")
    _, states = model(torch.cat([t[:n] for t, n in zip(texts, lengths)])[None], starts=starts)
    slots = torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")[: len(lengths)]
    pools = [torch.zeros(6, *s.shape[1:], device="cuda") for s in states]
    for pool, s in zip(pools, states):
        pool[slots.long()] = s
    worst = 0.0
    for i in range(extra):
        logits = model.step(torch.stack([t[n + i] for t, n in zip(texts, lengths)]), pools, slots)
        for r, (t, n) in enumerate(zip(texts, lengths)):
            worst = max(worst, float((model(t[None, : n + i + 1])[0][0, -1] - logits[r]).abs().max()))
    return worst


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    a = ap.parse_args()
    torch.manual_seed(0)
    model = Model(dtype=torch.bfloat16 if a.dtype == "bf16" else torch.float32).cuda()
    losses = train(model, a.steps)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {a.steps} steps")
    print(f"decoding against the whole sequence: largest logit difference {serve(model):.2e}")


if __name__ == "__main__":
    main()
