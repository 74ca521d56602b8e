"""A small language model of pre-norm recurrent blocks, trained on packed
sequences and then run token by token.

    s = s + mixer(norm(s)),   mixer(y) = (recurrence(y Wx, gates) * silu(y Wz)) Wo

Every norm takes the residual add in front of it (``kla.layernorm_fwd`` with
``residual``), the mixer's recurrence is ``kla.glr_fwd`` over packed sequences
of different lengths, the loss comes from ``kla.logprob_fwd``, all with their
backward passes; decoding carries one state per block with ``kla.glr_step``.
The projections are plain matrix products.  The task: repeat, in every position, the token seen `lag` positions
before, which takes memory.

    python examples/recurrent_lm.py [--steps 200]
"""
from __future__ import annotations

import argparse
import functools
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from linear_attention_delta_gb300 import kla  # noqa: E402


def first_order(backward):
    """For a backward pass that is not differentiable itself: an error where a
    graph of it is asked for (create_graph), as what autograd would record of
    it is not its derivative."""
    @functools.wraps(backward)
    def wrapped(ctx, *grads):
        if torch.is_grad_enabled():
            raise RuntimeError("there is no second derivative of this "
                               "operator (create_graph)")
        return backward(ctx, *grads)
    return wrapped


class AddNorm(torch.autograd.Function):
    """(norm(x + r), x + r); r may be None."""

    @staticmethod
    def forward(ctx, x, r, w, b):
        y, s, mean, rstd = kla.layernorm_fwd(x, w, b, residual=r)
        s = x if s is None else s
        ctx.save_for_backward(s, w, mean, rstd)
        ctx.add = r is not None
        return y, s.view_as(s)

    @staticmethod
    @first_order
    def backward(ctx, dy, ds):
        s, w, mean, rstd = ctx.saved_tensors
        g = kla.layernorm_bwd(dy.contiguous(), s, w, mean, rstd,
                              sum_grad=ds.contiguous())
        dx = g["x_grad"]
        return dx, dx if ctx.add else None, g["weight_grad"], g["bias_grad"]


class Recurrence(torch.autograd.Function):
    """h_t = exp(log_alpha_t) h_{t-1} + x_t over packed sequences."""

    @staticmethod
    def forward(ctx, x, log_alpha, cu):
        o, hT = kla.glr_fwd(x, log_alpha, cu_seqlens=cu)
        ctx.save_for_backward(o, log_alpha, cu)
        return o, hT

    @staticmethod
    @first_order
    def backward(ctx, do, dhT):
        o, log_alpha, cu = ctx.saved_tensors
        g = kla.glr_bwd(o, log_alpha, do.contiguous(), dhT, cu_seqlens=cu,
                        want_h0_grad=False)
        return g["x_grad"], g["log_alpha_grad"], None


class TokenLoss(torch.autograd.Function):
    """Minus the mean log probability of the targets that are there (a target
    below 0 is none)."""

    @staticmethod
    def forward(ctx, logits, target):
        logp, _, lse, _, _ = kla.logprob_fwd(logits, target)
        count = (target >= 0).sum().clamp(min=1)
        ctx.save_for_backward(logits, target, lse, count)
        return -logp.sum() / count

    @staticmethod
    @first_order
    def backward(ctx, g):
        logits, target, lse, count = ctx.saved_tensors
        weight = (-g / count).expand(target.shape).contiguous()
        return kla.logprob_bwd(logits, target, lse, logp_grad=weight), None


class Model(torch.nn.Module):
    def __init__(self, vocab=32, dim=256, inner=512, blocks=2,
                 dtype=torch.bfloat16):
        super().__init__()
        p = lambda *s: torch.nn.Parameter(  # noqa: E731
            torch.randn(*s, device="cuda", dtype=dtype) * s[0] ** -0.5)
        one = lambda n, v: torch.nn.Parameter(  # noqa: E731
            torch.full((n,), v, device="cuda", dtype=dtype))
        self.embed = torch.nn.Parameter(
            torch.randn(vocab, dim, device="cuda", dtype=dtype))
        self.blocks = torch.nn.ModuleList()
        for _ in range(blocks):
            b = torch.nn.Module()
            b.w, b.b = one(dim, 1.0), one(dim, 0.0)
            # x, gate and output gate from one product
            b.win, b.out = p(dim, 3 * inner), p(inner, dim)
            # decays from a few to some hundred tokens
            b.rate = torch.nn.Parameter(torch.linspace(
                -5.0, 0.0, inner, device="cuda"))
            self.blocks.append(b)
        self.w, self.b = one(dim, 1.0), one(dim, 0.0)
        self.head = p(dim, vocab)
        self.inner = inner

    def gates(self, b, y):
        """(x, log_alpha, z) of a block; log_alpha <= 0 in fp32."""
        x, u, z = (y @ b.win).split(self.inner, -1)
        return x, -torch.exp(b.rate) * torch.sigmoid(u.float()), z

    def forward(self, tokens, cu):
        """Logits [T, vocab] and the last states of packed sequences."""
        s, add, states = F.embedding(tokens, self.embed), None, []
        for b in self.blocks:
            y, s = AddNorm.apply(s, add, b.w, b.b)
            x, log_alpha, z = self.gates(b, y)
            o, hT = Recurrence.apply(x, log_alpha, cu)
            states.append(hT)
            add = (o * F.silu(z)) @ b.out
        y, _ = AddNorm.apply(s, add, self.w, self.b)
        return y @ self.head, states

    @torch.no_grad()
    def step(self, tokens, states):
        """Logits of one more token of each sequence; states in place."""
        s, add = F.embedding(tokens, self.embed), None
        for b, S in zip(self.blocks, states):
            y, r, _, _ = kla.layernorm_fwd(s, b.w, b.b, residual=add,
                                           want_stats=False)
            s = s if r is None else r
            x, log_alpha, z = self.gates(b, y)
            o = kla.glr_step(x, log_alpha, S)
            add = (o * F.silu(z)) @ b.out
        y, _, _, _ = kla.layernorm_fwd(s, self.w, self.b, residual=add,
                                       want_stats=False)
        return y @ self.head


def batch(lens, vocab, lag, gen):
    """Packed tokens, the tokens `lag` before them (-1: none) and offsets."""
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
    tokens = torch.randint(0, vocab, (int(cu[-1]),), device="cuda",
                           generator=gen)
    target = torch.full_like(tokens, -1)
    for a, n in zip(cu.tolist(), lens):
        target[a + lag:a + n] = tokens[a:max(a, a + n - lag)]
    return tokens, target, cu


def main(steps=200, lag=2, vocab=32, seed=0):
    torch.manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    model = Model(vocab)
    opt = torch.optim.Adam(model.parameters(), lr=2e-3)
    lens = [257, 1, 640, 33, 0, 900, 217]
    losses = []
    for i in range(steps):
        tokens, target, cu = batch(lens, vocab, lag, gen)
        logits, _ = model(tokens, cu)
        loss = TokenLoss.apply(logits, target)
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if i % 20 == 0 or i == steps - 1:
            print(f"step {i:4d}  loss {loss.item():.4f}")

    # prompts of different lengths at once, then token by token
    prompt, new = [5, 64, 129], 8
    tokens, _, _ = batch([n + new for n in prompt], vocab, lag, gen)
    seqs = tokens.split([n + new for n in prompt])
    with torch.no_grad():
        whole, _ = model(tokens, torch.tensor(
            [0] + [n + new for n in prompt], device="cuda").cumsum(0).int())
        packed = torch.cat([s[:n] for s, n in zip(seqs, prompt)])
        _, states = model(packed, torch.tensor(
            [0] + prompt, device="cuda").cumsum(0).int())
        worst = 0.0
        for k in range(new):
            logits = model.step(torch.stack([s[n + k] for s, n in
                                             zip(seqs, prompt)]), states)
            rows, a = [], 0
            for n in prompt:
                rows.append(whole[a + n + k])
                a += n + new
            diff = (logits.float() - torch.stack(rows).float()).abs().max()
            worst = max(worst, diff.item())
    scale = whole.float().abs().max().item()
    print(f"decoding against the whole prompts: largest difference "
          f"{worst:.4f} of logits up to {scale:.2f}")
    return [x.item() for x in losses], worst, scale


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=200)
    main(ap.parse_args().steps)
