#!/usr/bin/env python3
"""A small language model on the gated delta rule: trained, then served from a prompt token by token.

    python examples/delta_lm.py [--steps 60]

token ids -> embedding -> two blocks -> norm -> logits -> drawn tokens.  A block adds what the block
before it gave to the residual and normalises the sum (one kernel), projects it to queries, keys,
values and gates, and mixes along time with the gated delta rule, two value heads on every key head.
Projections and the loss are torch.  The text is synthetic: every token follows from the one before
the last by a fixed table, so a model predicts it only if it carries tokens along time.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import chunked_ssd_scan_gb300 as pkg  # noqa: E402

VOCAB, WIDTH, KEY_HEADS, HEADS, KEY, VALUE, BLOCKS = 64, 128, 1, 2, 32, 64, 2
CUT = (KEY_HEADS * KEY, KEY_HEADS * KEY, HEADS * VALUE, HEADS, HEADS)   # q, k, v, g, beta


class Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table, scale):
        ctx.save_for_backward(ids)
        ctx.rows, ctx.scale = table.shape[0], scale
        return pkg.embedding_forward(ids, table, scale=scale)

    @staticmethod
    def backward(ctx, dout):
        (ids,) = ctx.saved_tensors
        return None, pkg.embedding_backward(ids, dout.contiguous(), ctx.rows, scale=ctx.scale), None


class AddNorm(torch.autograd.Function):
    """(y, h): the norm of h = x + residual, and h itself for the next block."""

    @staticmethod
    def forward(ctx, x, residual, weight):
        y, h, rstd, _ = pkg.rms_norm_forward(x, weight, residual=residual)
        ctx.save_for_backward(h, rstd, weight)
        return y, h

    @staticmethod
    def backward(ctx, dy, dh):
        h, rstd, weight = ctx.saved_tensors
        g = pkg.rms_norm_backward(h, dy.contiguous(), rstd, weight, dresidual=dh.contiguous())
        return g["dx"], g["dx"], g["dweight"]


class DeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta):
        y, _, states = pkg.gated_delta_rule_forward(q, k, v, g, beta, return_final_state=False,
                                                    return_states=True)
        ctx.save_for_backward(q, k, v, g, beta, states)
        return y

    @staticmethod
    def backward(ctx, dy):
        *qkv, states = ctx.saved_tensors
        d = pkg.gated_delta_rule_backward(*qkv, dy.contiguous(), states=states, return_dinit=False)
        return d["dq"], d["dk"], d["dv"], d["dg"], d["dbeta"]


def make_params(seed=0):
    g = torch.Generator().manual_seed(seed)

    def mat(rows, cols, by=1.0):
        return (by * torch.randn(rows, cols, generator=g) / math.sqrt(rows)).cuda().requires_grad_()

    p = {"table": mat(VOCAB, WIDTH, math.sqrt(VOCAB / WIDTH)), "out": mat(WIDTH, VOCAB),
         "norm": torch.ones(WIDTH).cuda().requires_grad_()}
    for i in range(BLOCKS):
        p.update({f"norm{i}": torch.ones(WIDTH).cuda().requires_grad_(),
                  f"in{i}": mat(WIDTH, sum(CUT)), f"out{i}": mat(HEADS * VALUE, WIDTH, 0.5)})
    return p


def rule_inputs(p, i, y):
    """q and k of unit length, v, the logarithm of the decay and beta."""
    q, k, v, g, beta = (y @ p[f"in{i}"]).split(CUT, -1)
    q, k = (F.normalize(t.unflatten(-1, (KEY_HEADS, KEY)), dim=-1) for t in (q, k))
    return q, k, v.unflatten(-1, (HEADS, VALUE)), -F.softplus(g - 3).contiguous(), torch.sigmoid(beta).contiguous()


def forward(p, ids):
    x = Embed.apply(ids, p["table"], math.sqrt(WIDTH))
    h = torch.zeros_like(x)
    for i in range(BLOCKS):
        y, h = AddNorm.apply(x, h, p[f"norm{i}"])
        x = DeltaRule.apply(*rule_inputs(p, i, y)).flatten(2) @ p[f"out{i}"]
    return AddNorm.apply(x, h, p["norm"])[0] @ p["out"]


def batch(seed, size=16, length=128):
    follows = torch.randperm(VOCAB, generator=torch.Generator().manual_seed(99))
    g = torch.Generator().manual_seed(seed)
    text = [torch.randint(0, VOCAB, (size,), generator=g) for _ in range(2)]
    while len(text) <= length:
        text.append(follows[text[-2]])
    return torch.stack(text, 1).cuda()


def train(steps, seed=0, log=print):
    """Trains with Adam; returns the parameters and the losses."""
    p = make_params(seed)
    opt = torch.optim.Adam(p.values(), lr=3e-3)
    losses = []
    for step in range(steps):
        text = batch(1000 + step)
        logits = forward(p, text[:, :-1].contiguous())
        loss = F.cross_entropy(logits.reshape(-1, VOCAB), text[:, 1:].reshape(-1))
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step:4d}  loss {losses[-1]:.4f}")
    return p, losses


@torch.no_grad()
def serve(p, ids, states=None):
    """Logits of the last of ids [b,T], and the blocks' states behind it: a prompt in one call, or one token."""
    x = pkg.embedding_forward(ids, p["table"], scale=math.sqrt(WIDTH))
    h, after = torch.zeros_like(x), []
    for i in range(BLOCKS):
        y, h, _, _ = pkg.rms_norm_forward(x, p[f"norm{i}"], residual=h)
        rule = rule_inputs(p, i, y)
        if states is not None and ids.shape[1] == 1:
            o, state = pkg.gated_delta_rule_step(*(t[:, 0] for t in rule), states[i])   # in place
            o = o.unsqueeze(1)
        else:
            o, state, _ = pkg.gated_delta_rule_forward(*rule, init_state=None if states is None else states[i])
        after.append(state)
        x = o.flatten(2) @ p[f"out{i}"]
    return pkg.rms_norm_forward(x, p["norm"], residual=h)[0][:, -1] @ p["out"], after


@torch.no_grad()
def generate(p, prompt, tokens, seed=0, **settings):
    """Draws `tokens` tokens behind the prompt [b,T]: their ids and log probabilities."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits, states = serve(p, prompt)
    ids, logprobs = [], []
    for _ in range(tokens):
        u = torch.rand(prompt.shape[0], generator=g, device="cuda")
        new, logprob = pkg.token_sample(logits, u, **settings)
        ids.append(new)
        logprobs.append(logprob)
        logits, states = serve(p, new.unsqueeze(1), states)
    return torch.stack(ids, 1), torch.stack(logprobs, 1)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    p, _ = train(a.steps)
    text = batch(7, size=8, length=48)
    ids, logprob = generate(p, text[:, :24].contiguous(), 24, temperature=0.7, top_p=0.95)
    hits = float((ids == text[:, 24:48]).float().mean())
    print(f"drawn behind a prompt of 24 tokens: {100 * hits:.1f} % as the text goes on, "
          f"mean log probability {float(logprob.mean()):.3f}")


if __name__ == "__main__":
    main()
