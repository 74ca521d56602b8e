"""A small language model of pre-norm linear-attention blocks with a fixed decay
for each head, trained on batches and then run token by token.

    s = s + mixer(norm(s)),   mixer(y) = (attention(y Wq, y Wk, y Wv) * silu(y Wz)) Wo

Every norm takes the residual add in front of it (``kla.layernorm_fwd`` with
``residual``), the mixer is ``kla.linattn_fwd`` on slices of one projection's
output, the loss comes from ``kla.logprob_fwd`` (positions without a target have
the token -1), all with their backward passes.  Decoding carries one state a
block with ``kla.linattn_step`` and scores each next token, with the likeliest
alternatives.  The projections are plain matrix products.  The task: repeat, in
every position, the token seen `lag` positions before, which takes memory.

    python examples/linattn_lm.py [--steps 200]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from examples.recurrent_lm import AddNorm, TokenLoss, first_order  # noqa: E402
from linear_attention_delta_gb300 import kla  # noqa: E402


class Attention(torch.autograd.Function):
    """Linear attention with a decay for each head: (o, last states)."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay):
        o, hT = kla.linattn_fwd(q, k, v, log_decay)
        ctx.save_for_backward(q, k, v, log_decay)
        return o, hT

    @staticmethod
    @first_order
    def backward(ctx, do, dhT):
        q, k, v, log_decay = ctx.saved_tensors
        g = kla.linattn_bwd(q, k, v, log_decay, do.contiguous(), hT_grad=dhT,
                            want_h0_grad=False)
        return g["q_grad"], g["k_grad"], g["v_grad"], None


class Model(torch.nn.Module):
    def __init__(self, vocab=32, dim=256, heads=4, width=64, blocks=2,
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
            # queries, keys, values and output gate from one product
            b.win = p(dim, 4 * heads * width)
            b.out = p(heads * width, dim)
            self.blocks.append(b)
        self.w, self.b = one(dim, 1.0), one(dim, 0.0)
        self.head = p(dim, vocab)
        self.shape = (4, heads, width)
        # memories from two tokens to some hundred, a head each
        self.register_buffer("log_decay", -torch.exp2(
            -torch.linspace(1.0, 8.0, heads, device="cuda")))

    def inputs(self, b, y):
        """(q, k, v, z) of a block, slices of one tensor."""
        x = (y @ b.win).unflatten(-1, self.shape)
        q, k, v, z = x.unbind(-3)
        # unit-sized scores: a factor on the queries
        return q * self.shape[2] ** -0.5, k, v, z

    def forward(self, tokens):
        """Logits [B, T, vocab] and the last states."""
        s, add, states = F.embedding(tokens, self.embed), None, []
        for b in self.blocks:
            y, s = AddNorm.apply(s, add, b.w, b.b)
            q, k, v, z = self.inputs(b, y)
            o, hT = Attention.apply(q, k, v, self.log_decay)
            states.append(hT)
            add = (o * F.silu(z)).flatten(-2) @ b.out
        y, _ = AddNorm.apply(s, add, self.w, self.b)
        return y @ self.head, states

    @torch.no_grad()
    def step(self, tokens, states):
        """Logits [B, vocab] of one more token; states in place."""
        s, add = F.embedding(tokens, self.embed), None
        for b, S in zip(self.blocks, states):
            y, r, _, _ = kla.layernorm_fwd(s, b.w, b.b, residual=add,
                                           want_stats=False)
            s = s if r is None else r
            q, k, v, z = self.inputs(b, y)
            o = kla.linattn_step(q, k, v, self.log_decay, S)
            add = (o * F.silu(z)).flatten(-2) @ b.out
        y, _, _, _ = kla.layernorm_fwd(s, self.w, self.b, residual=add,
                                       want_stats=False)
        return y @ self.head


def batch(B, T, vocab, lag, gen):
    """Tokens and the tokens `lag` before them (-1: none)."""
    tokens = torch.randint(0, vocab, (B, T), device="cuda", generator=gen)
    target = torch.full_like(tokens, -1)
    target[:, lag:] = tokens[:, :T - lag]
    return tokens, target


def main(steps=200, lag=2, vocab=32, seed=0):
    torch.manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    model = Model(vocab)
    opt = torch.optim.Adam(model.parameters(), lr=2e-3)
    losses = []
    for i in range(steps):
        tokens, target = batch(4, 300, vocab, lag, gen)
        logits, _ = model(tokens)
        loss = TokenLoss.apply(logits, target)
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if i % 20 == 0 or i == steps - 1:
            print(f"step {i:4d}  loss {loss.item():.4f}")

    # a prompt at once, then token by token, each scored before it is taken
    prompt, new = 130, 8
    tokens, target = batch(3, prompt + new, vocab, lag, gen)
    with torch.no_grad():
        whole, _ = model(tokens)
        _, states = model(tokens[:, :prompt])
        worst = 0.0
        for t in range(prompt, prompt + new):
            logits = model.step(tokens[:, t], states)
            diff = (logits.float() - whole[:, t].float()).abs().max()
            worst = max(worst, diff.item())
            logp, entropy, _, top, ids = kla.logprob_fwd(
                logits, target[:, t].contiguous(), top=3)
        print(f"last token: log probability {logp[0].item():.3f}, entropy "
              f"{entropy[0].item():.3f}, likeliest "
              + ", ".join(f"{i} ({p:.3f})" for i, p in
                          zip(ids[0].tolist(), top[0].tolist())))
    scale = whole.float().abs().max().item()
    print(f"decoding against the whole prompts: largest difference "
          f"{worst:.4f} of logits up to {scale:.2f}")
    return [x.item() for x in losses], worst, scale


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=200)
    main(ap.parse_args().steps)
