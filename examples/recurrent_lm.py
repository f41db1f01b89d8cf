#!/usr/bin/env python3
"""A small recurrent language model on the library's kernels: trained, then served token by token.

    python examples/recurrent_lm.py [--steps 60]

token ids -> embedding -> two mixer blocks -> norm -> logits.  One block mixes along time with the
chunked SSD scan, the other with the gated linear recurrence; both normalise each head of the
mixer's output with the channels-last group norm and its SiLU.  Projections and the loss are torch.
The text is synthetic: every token follows from the one before the last by a fixed table, so a model
predicts it only if it carries tokens along time.
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

VOCAB, WIDTH, HEADS, STATE = 64, 128, 2, 64   # heads of 64 channels


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


class Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate_a, gate_x, decay):
        y, _, states = pkg.gated_recurrence_forward(x, gate_a, gate_x, decay, return_states=True)
        ctx.save_for_backward(x, gate_a, gate_x, decay, states)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, gate_a, gate_x, decay, states = ctx.saved_tensors
        g = pkg.gated_recurrence_backward(x, gate_a, gate_x, decay, dy.contiguous(), states=states,
                                          return_dinit=False)
        return g["dx"], g["dgate_a"], g["dgate_x"], g["ddecay"]


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, groups, weight, bias, activation):
        y, mean, rstd = pkg.group_norm_forward(x, groups, weight, bias, activation=activation)
        ctx.save_for_backward(x, mean, rstd, weight, bias)
        ctx.groups, ctx.activation = groups, activation
        return y

    @staticmethod
    def backward(ctx, dy):
        x, mean, rstd, weight, bias = ctx.saved_tensors
        g = pkg.group_norm_backward(x, dy.contiguous(), ctx.groups, mean, rstd, weight, bias,
                                    activation=ctx.activation)
        return g["dx"], None, g["dweight"], g["dbias"], None


class Scan(torch.autograd.Function):
    """Chunked SSD scan, x [b,T,1,H,P], dA [b,T,H], B and C [b,T,1,1,N]."""

    @staticmethod
    def forward(ctx, x, dA, B, C):
        ctx.save_for_backward(x, dA, B, C)
        return pkg.ssd_chunked_forward(x, dA, B, C, chunk_len=64, return_final_state=False)[0]

    @staticmethod
    def backward(ctx, dy):
        g = pkg.ssd_chunked_backward(*ctx.saved_tensors, dy.contiguous(), return_dinit=False)
        return g["dx"], g["ddA"], g["dB"], g["dC"]


def make_params(seed=0):
    g = torch.Generator().manual_seed(seed)

    def mat(rows, cols):
        return (torch.randn(rows, cols, generator=g) / math.sqrt(rows)).cuda().requires_grad_()

    def vec(value):
        return value.float().cuda().requires_grad_()

    p = {"table": (torch.randn(VOCAB, WIDTH, generator=g) / math.sqrt(WIDTH)).cuda().requires_grad_(),
         "out": mat(WIDTH, VOCAB), "nw": vec(torch.ones(WIDTH)), "nb": vec(torch.zeros(WIDTH))}
    for k in ("s", "r"):   # the SSD block and the recurrent block
        p.update({k + "nw": vec(torch.ones(WIDTH)), k + "nb": vec(torch.zeros(WIDTH)),
                  k + "hw": vec(torch.ones(WIDTH)), k + "hb": vec(torch.zeros(WIDTH)),
                  k + "out": mat(WIDTH, WIDTH)})
    p["sin"] = mat(WIDTH, WIDTH + HEADS + 2 * STATE)
    p["rin"] = mat(WIDTH, 3 * WIDTH)
    # channels that forget between a few steps and a few hundred
    keep = torch.linspace(0.5, 0.995, WIDTH)
    p["decay"] = vec(torch.log(torch.expm1(-torch.log(keep) / 8.0)))
    return p


def token_norm(x, groups, w, b, act):
    return Norm.apply(x.reshape(-1, WIDTH), groups, w, b, act).view(x.shape)


def ssd_inputs(p, h):
    z = token_norm(h, 1, p["snw"], p["snb"], None) @ p["sin"]
    b, T = z.shape[:2]
    x, dt, B, C = (v.contiguous() for v in z.split((WIDTH, HEADS, STATE, STATE), -1))
    return (x.reshape(b, T, 1, HEADS, WIDTH // HEADS), -F.softplus(dt - 2),
            (B / math.sqrt(STATE)).reshape(b, T, 1, 1, STATE),
            C.reshape(b, T, 1, 1, STATE))


def recurrence_inputs(p, h):
    return (token_norm(h, 1, p["rnw"], p["rnb"], None) @ p["rin"]).split(WIDTH, -1)   # no copies


def mix(p, k, h, y):
    """The block's end: norm of each head and SiLU, projection, residual."""
    return h + token_norm(y.reshape(h.shape), HEADS, p[k + "hw"], p[k + "hb"], "silu") @ p[k + "out"]


def logits_of(p, h):
    return token_norm(h, 1, p["nw"], p["nb"], None) @ p["out"]


def forward(p, ids):
    h = Embed.apply(ids, p["table"], math.sqrt(WIDTH))
    h = mix(p, "s", h, Scan.apply(*ssd_inputs(p, h)))
    h = mix(p, "r", h, Recurrence.apply(*recurrence_inputs(p, h), p["decay"]))
    return logits_of(p, h)


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
    """Logits of ids [b,T] one token at a time, from the states that an earlier call returned."""
    b, T = ids.shape
    if states is None:
        states = {"ssd": torch.zeros(b, HEADS, WIDTH // HEADS, STATE, device="cuda"),
                  "rec": torch.zeros(b, WIDTH, device="cuda")}
    out = []
    for t in range(T):
        h = pkg.embedding_forward(ids[:, t:t + 1].contiguous(), p["table"], scale=math.sqrt(WIDTH))
        y, states["ssd"] = pkg.ssd_chunked_forward(*ssd_inputs(p, h), chunk_len=64,
                                                   init_state=states["ssd"])
        h = mix(p, "s", h, y)
        x, ga, gx = (v[:, 0] for v in recurrence_inputs(p, h))
        y, _ = pkg.gated_recurrence_step(x, ga, gx, p["decay"], states["rec"])   # in place
        h = mix(p, "r", h, y)
        out.append(logits_of(p, h))
    return torch.cat(out, 1), states


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    p, losses = train(a.steps)
    text = batch(7, size=4)
    whole = forward(p, text[:, :-1].contiguous()).detach()
    served, _ = serve(p, text[:, :-1])
    off = float((whole - served).abs().max())
    hits = float((served[:, 1:].argmax(-1) == text[:, 2:]).float().mean())
    print(f"served token by token: logits off by at most {off:.2e}, {100 * hits:.1f} % of the tokens "
          "predicted")


if __name__ == "__main__":
    main()
