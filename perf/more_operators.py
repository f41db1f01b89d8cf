"""Cases of further operators of a recurrent language model: the gated delta rule, the
root-mean-square norm with a residual and an 8-bit output, and the drawing of tokens, each in its
plain form and through the library.

``listed()`` names the cases, ``draw(rng)`` makes more of the same ranges, ``prepare`` builds the
inputs on the GPU, ``run`` makes one pass (the plain form in 32 bits with elementary torch
operations, in 64 where a choice hangs on it, or with ``own`` the library's calls), ``work`` counts
what a pass cannot do without and ``exact`` evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

CHUNK = 64          # the delta rule's state is kept every CHUNK steps for its gradient
EPS = 1e-6          # the norm's epsilon
E4M3_MOST = 448.0   # the largest value of 8 bits with a sign, 4 of exponent and 3 of mantissa
BLOCK = 128         # channels that share a scale in blocks
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one new token for each of 16 requests: latency of the serving loop
        {"name": "delta_step_b16", "op": "delta_step", "dtype": "bf16", "b": 16, "Hk": 8, "H": 16,
         "K": 128, "V": 128},
        # a wide batch of requests, fp32 activations
        {"name": "delta_step_b256_f32", "op": "delta_step", "dtype": "f32", "b": 256, "Hk": 16,
         "H": 16, "K": 64, "V": 128},
        # a short ragged prompt, odd head widths, shared keys, fp32
        {"name": "delta_ragged_f32", "op": "delta", "dtype": "f32", "b": 3, "T": 777, "Hk": 2,
         "H": 6, "K": 60, "V": 100, "train": False},
        # training forward: keeps the chunk states for the gradient
        {"name": "delta_train_bf16", "op": "delta", "dtype": "bf16", "b": 8, "T": 4096, "Hk": 16,
         "H": 16, "K": 128, "V": 128, "train": True},
        # a long prompt of one request: few sequences for the machine's width
        {"name": "delta_long_bf16", "op": "delta", "dtype": "bf16", "b": 1, "T": 32768, "Hk": 8,
         "H": 16, "K": 128, "V": 128, "train": False},
        # training backward, two value heads on every key head
        {"name": "delta_grad_bf16", "op": "delta_grad", "dtype": "bf16", "b": 4, "T": 4096,
         "Hk": 8, "H": 16, "K": 128, "V": 128},
        # residual and norm of a training batch
        {"name": "norm_residual_bf16", "op": "norm", "dtype": "bf16", "N": 16384, "C": 2048,
         "residual": True, "quant": "none"},
        # the same of one token for each of 16 requests, written in 8 bits for the next product
        {"name": "norm_8bit_b16", "op": "norm", "dtype": "bf16", "N": 16, "C": 5120,
         "residual": True, "quant": "token"},
        # a prompt's norm in 8 bits with a scale for every 128 channels, odd number of tokens
        {"name": "norm_8bit_blocks", "op": "norm", "dtype": "bf16", "N": 10007, "C": 2560,
         "residual": True, "quant": "block"},
        # gradient of the norm, with the gradient that the residual brings
        {"name": "norm_grad_bf16", "op": "norm_grad", "dtype": "bf16", "N": 16384, "C": 2048,
         "residual": True},
        # one token for each of 16 requests, every request with settings of its own
        {"name": "sample_b16", "op": "sample", "dtype": "bf16", "n": 16, "V": 50000, "kind": "all"},
        # a wide batch, plain temperature: the whole vocabulary takes part
        {"name": "sample_b512_f32", "op": "sample", "dtype": "f32", "n": 512, "V": 50000,
         "kind": "plain"},
    ]


def _log_int(rng, lo, hi):
    return min(max(int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))), lo), hi)


def _head(rng):
    """Channels of a head: the usual widths, other multiples of 8, or any number."""
    return rng.choice((64, 128, 128, 8 * rng.randint(2, 16), rng.randint(16, 128)))


def draw(rng):
    op = rng.choice(("delta_step", "delta", "delta", "delta_grad", "delta_grad", "norm", "norm",
                     "norm_grad", "sample", "sample"))
    c = {"op": op, "dtype": rng.choice(("f32", "bf16"))}
    if op.startswith("delta"):
        Hk = rng.choice((1, 2, 4, 5, 8, 16))
        H = Hk * rng.choice((1, 1, 2, 3))
        K, V = _head(rng), _head(rng)
        c.update(Hk=Hk, H=H, K=K, V=V)
        if op == "delta_step":
            c["b"] = _log_int(rng, 1, max(1, 60_000_000 // (H * K * V)))
        else:   # tokens times heads
            most = (1 << 18 if op == "delta_grad" else 1 << 19) // H
            if c["dtype"] == "f32":
                most //= 2
            T = _log_int(rng, 1, min(most, 60000))
            c.update(T=T, b=_log_int(rng, 1, max(1, min(16, most // T))))
            if op == "delta":
                c["train"] = rng.random() < 0.5
    elif op in ("norm", "norm_grad"):
        C = _log_int(rng, 64, 9000)
        C = max(8, C // 8 * 8) if rng.random() < 0.7 else C
        c.update(N=_log_int(rng, 1, 30_000_000 // C), C=C, residual=rng.random() < 0.7)
        if op == "norm":
            c["quant"] = rng.choice(("none", "token", "block"))
    else:
        V = _log_int(rng, 300, 200000)
        c.update(V=V, n=_log_int(rng, 1, max(1, min(1000, 25_000_000 // V))),
                 kind=rng.choice(("all", "plain", "top_k", "top_p", "min_p")))
    return c


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, op = DTYPES[case["dtype"]], case["op"]
    s = {"op": op, "dt": dt}
    if op.startswith("delta"):
        b, Hk, H, K, V = (case[k] for k in ("b", "Hk", "H", "K", "V"))
        lead = (b,) if op == "delta_step" else (b, case["T"])
        # q and k of unit length; a head forgets over about 2 to 500 steps, some tokens more
        unit = torch.nn.functional.normalize
        slow = torch.exp(_rand(g, H) * math.log(250.0)) * 2
        s.update(q=unit(_randn(g, *lead, Hk, K), dim=-1).to(dt),
                 k=unit(_randn(g, *lead, Hk, K) + 0.5 * _randn(g, Hk, K), dim=-1).to(dt),
                 v=_randn(g, *lead, H, V, dtype=dt),
                 g=-torch.nn.functional.softplus(_randn(g, *lead, H) * 1.5) / slow,
                 beta=torch.sigmoid(_randn(g, *lead, H) * 1.5), scale=K ** -0.5)
        s["state"] = _randn(g, b, H, V, K) * 0.3
        if op != "delta_step":
            s["train"] = case.get("train", False)
        if op == "delta_grad":
            s.update(dy=_randn(g, *lead, H, V, dtype=dt), dfinal=_randn(g, b, H, V, K) * 0.3)
            s["states"] = _delta(s | {"train": True})[2]   # what the forward pass kept
    elif op in ("norm", "norm_grad"):
        N, C = case["N"], case["C"]
        s.update(x=_randn(g, N, C, dtype=dt), w=1 + 0.2 * _randn(g, C))
        s["res"] = (_randn(g, N, C) * 2 * _rand(g, N, 1)).to(dt) if case["residual"] else None
        if op == "norm":
            s["quant"] = case["quant"]
        else:
            # the sum and its statistic as the forward pass kept them, the output's gradient and
            # the one that the residual brings
            h = s["x"].float() + (s["res"].float() if case["residual"] else 0)
            s.update(h=h.to(dt), rstd=1 / torch.sqrt((h * h).mean(1) + EPS),
                     dy=_randn(g, N, C, dtype=dt))
            s["dres"] = _randn(g, N, C, dtype=dt) if case["residual"] else None
            del s["x"], s["res"]
    else:
        n, V, kind = case["n"], case["V"], case["kind"]
        # logits: a wide body and a few dozen likely tokens
        x = _randn(g, n, V) * 2.5
        likely = torch.randint(0, V, (n, 40), generator=g, device="cuda")
        x.scatter_add_(1, likely, _rand(g, n, 40) * 12)
        s.update(logits=x.to(dt), u=_rand(g, n))
        every = kind == "all"
        s["temperature"] = 0.3 + 1.2 * _rand(g, n)
        if every:   # some requests take the likeliest token
            s["temperature"][torch.arange(n, device="cuda") % 5 == 4] = 0.0
        s["top_k"] = (torch.randint(1, 200, (n,), generator=g, device="cuda", dtype=torch.int32)
                      if every or kind == "top_k" else None)
        if every:   # 0: no limit
            s["top_k"][torch.arange(n, device="cuda") % 3 == 1] = 0
        s["top_p"] = 0.5 + 0.49 * _rand(g, n) if every or kind == "top_p" else None
        s["min_p"] = 0.1 * _rand(g, n) if every or kind == "min_p" else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        s["plan"] = _plan(s)
    return s


def _plan(s):
    """The plan that a program keeps for repeated calls on its buffers: arguments checked, outputs
    and workspace allocated; calling it computes everything anew."""
    import chunked_ssd_scan_gb300 as pkg
    op = s["op"]
    if op.startswith("delta"):
        qkv = [s[k] for k in ("q", "k", "v", "g", "beta")]
    if op == "delta_step":
        return pkg.GatedDeltaRuleStepPlan(*qkv, s["state"], scale=s["scale"],
                                          state_out=torch.empty_like(s["state"]))
    if op == "delta":
        return pkg.GatedDeltaRulePlan(*qkv, scale=s["scale"], init_state=s["state"],
                                      return_states=s["train"])
    if op == "delta_grad":
        return pkg.GatedDeltaRuleBackwardPlan(*qkv, s["dy"], scale=s["scale"],
                                              init_state=s["state"], states=s["states"],
                                              dfinal=s["dfinal"])
    if op == "norm":
        quant = None if s["quant"] == "none" else s["quant"]
        return pkg.RMSNormPlan(s["x"], s["w"], residual=s["res"], eps=EPS, quantize=quant)
    if op == "norm_grad":
        return pkg.RMSNormBackwardPlan(s["h"], s["dy"], s["rstd"], s["w"], dresidual=s["dres"])
    return pkg.TokenSamplePlan(s["logits"], s["u"], temperature=s["temperature"],
                               top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])


# ------------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------------
def _heads(t, H):
    """[b,T,h,D] in 32 bits as [b,H,chunks,CHUNK,D]: heads repeated, steps padded by zeros."""
    t = t.float()
    b, T, h, D = t.shape
    pad = -T % CHUNK
    t = torch.cat((t, t.new_zeros(b, pad, h, D)), 1) if pad else t
    t = t.permute(0, 2, 1, 3).repeat_interleave(H // h, 1)
    return t.reshape(b, H, (T + pad) // CHUNK, CHUNK, D)


def _after(M, N):
    """S_c = M_c S_{c-1} + N_c along axis 2 from S = 0: after k doublings every element holds the
    composition of the last 2^k maps."""
    k = 1
    while k < M.shape[2]:
        N = torch.cat((N[:, :, :k], N[:, :, k:] + M[:, :, k:] @ N[:, :, :-k]), 2)
        M = torch.cat((M[:, :, :k], M[:, :, k:] @ M[:, :, :-k]), 2)
        k *= 2
    return N


def _delta_32(q, k, v, g, beta, init, scale):
    """Output, final state and states before every chunk, in 32 bits.  Within a chunk every step's
    write u solves a unit lower triangular system; between chunks the state is an affine map."""
    b, T, H, V = v.shape
    q, k, v = _heads(q, H), _heads(k, H), _heads(v, H)
    g, beta = _heads(g.unsqueeze(3), H).squeeze(-1), _heads(beta.unsqueeze(3), H)
    cum = g.cumsum(-1)
    at = torch.arange(CHUNK, device=v.device)
    earlier, own_too = at[:, None] > at, at[:, None] >= at
    decay = torch.exp(torch.where(own_too, cum[..., :, None] - cum[..., None, :], 0.0))
    A = beta * decay * (k @ k.transpose(-1, -2)) * earlier
    grow = torch.exp(cum).unsqueeze(-1)
    K = k.shape[-1]
    solved = torch.linalg.solve_triangular(A, torch.cat((beta * grow * k, beta * v), -1),
                                           upper=False, unitriangular=True)
    W, U = solved[..., :K], solved[..., K:]
    last = cum[..., -1:]
    kd = (k * torch.exp(last - cum).unsqueeze(-1)).transpose(-1, -2)
    M = torch.exp(last).unsqueeze(-1) * torch.eye(K, device=v.device) - kd @ W
    N = kd @ U
    first = init.transpose(-1, -2).unsqueeze(2)
    N = torch.cat((N[:, :, :1] + M[:, :, :1] @ first, N[:, :, 1:]), 2)
    S = _after(M, N)
    before = torch.cat((first, S[:, :, :-1]), 2)
    U = U - W @ before
    o = grow * (q @ before) + (decay * (q @ k.transpose(-1, -2)) * own_too) @ U
    o = (o * scale).reshape(b, H, -1, V)[:, :, :T].transpose(1, 2)
    return o, S[:, :, -1].transpose(-1, -2), before.permute(0, 2, 1, 4, 3)


def _delta(s):
    o, final, states = _delta_32(*(s[k] for k in ("q", "k", "v", "g", "beta", "state", "scale")))
    out = o.to(s["dt"]).contiguous(), final.contiguous()
    return (*out, states.contiguous()) if s["train"] else out


def _delta_grad(s):
    names = ("q", "k", "v", "g", "beta", "state")
    leaves = [s[k].to(torch.float32, copy=True).requires_grad_() for k in names]
    o, final, _ = _delta_32(*leaves, s["scale"])
    dq, dk, dv, dg, dbeta, dinit = torch.autograd.grad((o, final), leaves,
                                                       (s["dy"].float(), s["dfinal"]))
    dt = s["dt"]
    return {"dq": dq.to(dt), "dk": dk.to(dt), "dv": dv.to(dt), "dg": dg, "dbeta": dbeta,
            "dinit": dinit}


def _delta_step(s):
    H = s["v"].shape[1]
    q, k = (s[n].float().repeat_interleave(H // s[n].shape[1], 1).unsqueeze(-2) for n in "qk")
    S = s["state"] * torch.exp(s["g"])[..., None, None]
    u = s["beta"].unsqueeze(-1) * (s["v"].float() - (S * k).sum(-1))
    S = S + u.unsqueeze(-1) * k
    return ((S * q).sum(-1) * s["scale"]).to(s["dt"]), S


def _norm(s):
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    rstd = 1 / torch.sqrt((h * h).mean(1) + EPS)
    y = h * rstd[:, None] * s["w"]
    out = {"rstd": rstd}
    if s["res"] is not None:
        out["h"] = h.to(s["dt"])
    if s["quant"] == "none":
        return out | {"y": y.to(s["dt"])}
    N, C = y.shape
    wide = C if s["quant"] == "token" else BLOCK
    y = torch.cat((y, y.new_zeros(N, -C % wide)), 1).view(N, -1, wide)
    scale = y.abs().amax(2) / E4M3_MOST
    scale = torch.where(scale > 0, scale, 1.0)
    q = (y / scale.unsqueeze(2)).to(torch.float8_e4m3fn)
    return out | _values(q.view(N, -1)[:, :C], scale, wide)


def _values(q, scale, wide):
    """What the 8 bits stand for, and their scales."""
    each = scale.repeat_interleave(wide, 1)[:, :q.shape[1]]
    return {"y": (q.float() * each).to(torch.bfloat16), "scale": scale}


def _norm_grad(s):
    h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"].unsqueeze(1)
    xh, q = h * rstd, dy * s["w"]
    dx = rstd * (q - xh * (q * xh).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["dt"]), "dweight": (dy * xh).sum(0)}


def _sample(s):
    """In 64 bits: a choice hangs on sums over the vocabulary."""
    f8 = torch.float64
    x, t = s["logits"].to(f8), s["temperature"].to(f8).unsqueeze(1)
    z, order = torch.sort(x, dim=1, descending=True, stable=True)   # equal ones: lowest index first
    greedy = t == 0
    w = torch.exp((z - z[:, :1]) / torch.where(greedy, 1.0, t))
    place = torch.arange(x.shape[1], device=x.device)
    keep = ~greedy | (place == 0)
    if s["top_k"] is not None:
        k = s["top_k"].unsqueeze(1)
        keep = keep & ((place < k) | (k <= 0))
    if s["min_p"] is not None:
        keep = keep & (w >= s["min_p"].to(f8).unsqueeze(1))
    w = w * keep
    if s["top_p"] is not None:   # the fewest tokens that hold top_p of what the others left
        before = w.cumsum(1) - w
        w = w * (before < s["top_p"].to(f8).unsqueeze(1) * w.sum(1, keepdim=True))
    w = torch.zeros_like(w).scatter_(1, order, w)
    upto = w.cumsum(1)
    total = upto[:, -1:]
    ids = (upto > s["u"].to(f8).unsqueeze(1) * total).to(torch.int8).argmax(1, keepdim=True)
    return ids.squeeze(1), torch.log(w.gather(1, ids) / total).squeeze(1).float()


PLAIN = {"delta": _delta, "delta_grad": _delta_grad, "delta_step": _delta_step, "norm": _norm,
         "norm_grad": _norm_grad, "sample": _sample}


def run(state):
    if not own:
        return PLAIN[state["op"]](state)
    out = state["plan"]()
    if state["op"] == "delta" and not state["train"]:
        return out[:2]
    if state["op"] == "norm":
        y, h, rstd, scale = out
        named = {"rstd": rstd}
        if h is not None:
            named["h"] = h
        if scale is None:
            return named | {"y": y}
        return named | _values(y, scale, y.shape[1] if state["quant"] == "token" else BLOCK)
    return out


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def work(case):
    e, op = (4 if case["dtype"] == "f32" else 2), case["op"]
    if op.startswith("delta"):
        b, Hk, H, K, V = (case[k] for k in ("b", "Hk", "H", "K", "V"))
        n, T = b * case.get("T", 1), case.get("T", 1)
        qk, v, gates, state = 2 * n * Hk * K * e, n * H * V * e, 8 * n * H, 4 * b * H * K * V
        # S k, the write, S q: three products with the state a step
        if op != "delta_grad":
            kept = state * -(-T // CHUNK) if case.get("train") else 0
            return {"bytes": qk + 2 * v + gates + 2 * state + kept, "flops": 6 * n * H * K * V}
        return {"bytes": 2 * qk + 3 * v + 2 * gates + 2 * state + state * -(-T // CHUNK),
                "flops": 16 * n * H * K * V}
    if op == "norm":
        n = case["N"] * case["C"]
        y = e if case["quant"] == "none" else 1
        scales = {"none": 0, "token": 1, "block": -(-case["C"] // BLOCK)}[case["quant"]]
        return {"bytes": n * ((3 if case["residual"] else 1) * e + y) + 4 * case["C"]
                + 4 * case["N"] * (1 + scales), "flops": 5 * n}
    if op == "norm_grad":
        n = case["N"] * case["C"]
        return {"bytes": n * (4 if case["residual"] else 3) * e + 4 * case["N"] + 8 * case["C"],
                "flops": 9 * n}
    n, V = case["n"], case["V"]
    return {"bytes": n * V * e + 28 * n, "flops": 6 * n * V}


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def _exact_delta(case, s):
    """The recurrence, one step at a time, and its reverse mode."""
    f8, T, H = torch.float64, case["T"], case["H"]
    q, k, v = (s[n].to(f8).transpose(0, 1) for n in "qkv")
    r = H // case["Hk"]
    a, beta = torch.exp(s["g"].to(f8)).transpose(0, 1), s["beta"].to(f8).transpose(0, 1)
    grad = case["op"] == "delta_grad"

    def rows(t, i):   # a key head's row for each of its value heads
        return t[i].repeat_interleave(r, 1)

    def step(S, i):
        ki = rows(k, i)
        S = S * a[i][..., None, None]
        e = v[i] - torch.einsum("bhvk,bhk->bhv", S, ki)
        return S + torch.einsum("bhv,bhk->bhvk", beta[i].unsqueeze(-1) * e, ki), S, e, ki

    S, o, kept = s["state"].to(f8), torch.empty_like(v), []
    for i in range(T):
        if i % CHUNK == 0:
            kept.append(S)
        S = step(S, i)[0]
        if not grad:
            o[i] = torch.einsum("bhvk,bhk->bhv", S, rows(q, i)) * s["scale"]
    if not grad:
        out = o.transpose(0, 1), S
        return (*out, torch.stack(kept, 1)) if case["train"] else out
    dy = s["dy"].to(f8).transpose(0, 1)
    G = s["dfinal"].to(f8)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.empty_like(v)
    dg, dbeta = torch.empty_like(a), torch.empty_like(a)

    def shared(t):
        return t.view(t.shape[0], case["Hk"], r, t.shape[-1]).sum(2)

    for c in reversed(range(len(kept))):
        chain, S = [], kept[c]
        for i in range(c * CHUNK, min(T, (c + 1) * CHUNK)):
            S, decayed, e, ki = step(S, i)
            chain.append((S, decayed, e, ki))
        for i in reversed(range(c * CHUNK, min(T, (c + 1) * CHUNK))):
            S, decayed, e, ki = chain.pop()
            di, qi, bi = dy[i] * s["scale"], rows(q, i), beta[i].unsqueeze(-1)
            dq[i] = shared(torch.einsum("bhvk,bhv->bhk", S, di))
            G = G + torch.einsum("bhv,bhk->bhvk", di, qi)
            du = torch.einsum("bhvk,bhk->bhv", G, ki)
            dv[i] = bi * du
            dbeta[i] = (du * e).sum(-1)
            dk[i] = shared(torch.einsum("bhvk,bhv->bhk", G, bi * e)
                           - torch.einsum("bhvk,bhv->bhk", decayed, dv[i]))
            G = G - torch.einsum("bhv,bhk->bhvk", dv[i], ki)
            dg[i] = (G * decayed).sum((-1, -2))
            G = G * a[i][..., None, None]
    return {"dq": dq.transpose(0, 1), "dk": dk.transpose(0, 1), "dv": dv.transpose(0, 1),
            "dg": dg.transpose(0, 1), "dbeta": dbeta.transpose(0, 1), "dinit": G}


def _nearest(v):
    """The nearest of the values that 4 bits of exponent and 3 of mantissa hold, ties to even."""
    step = torch.exp2(torch.frexp(v).exponent.clamp(min=-5).to(v.dtype) - 4)
    return torch.round(v / step) * step


def exact(case, seed):
    s, f8 = _inputs(case, seed), torch.float64
    op = case["op"]
    if op in ("delta", "delta_grad"):
        # steps and the size of what they touch: beyond this it takes too long
        state = case["b"] * case["H"] * case["K"] * case["V"]
        if case["T"] * (3 if op == "delta_grad" else 1) * (8 + state / 2 ** 18) > 900_000:
            return None
        return _exact_delta(case, s)
    if op == "delta_step":
        H, dims = case["H"], (case["b"], case["H"], 1, case["K"])
        q, k = (s[n].to(f8).repeat_interleave(H // case["Hk"], 1).view(dims) for n in "qk")
        old = s["state"].to(f8) * s["g"].to(f8).exp().view(*dims[:2], 1, 1)
        miss = s["v"].to(f8) - torch.matmul(old, k.transpose(2, 3)).squeeze(3)
        new = old + (miss * s["beta"].to(f8).unsqueeze(2)).unsqueeze(3) * k
        return torch.matmul(new, q.transpose(2, 3)).squeeze(3) * s["scale"], new
    if op == "norm":
        h = s["x"].to(f8) if s["res"] is None else s["x"].to(f8) + s["res"].to(f8)
        rstd = torch.rsqrt(h.square().mean(1) + EPS)
        y = torch.einsum("nc,n,c->nc", h, rstd, s["w"].to(f8))
        out = {"rstd": rstd}
        if s["res"] is not None:
            out["h"] = h
        if s["quant"] == "none":
            return out | {"y": y}
        parts = y.split(case["C"] if s["quant"] == "token" else BLOCK, 1)
        most = torch.stack([p.abs().amax(1) for p in parts], 1)
        scale = torch.where(most > 0, most / E4M3_MOST, 1.0)
        out["y"] = torch.cat([_nearest(p / scale[:, i:i + 1]) * scale[:, i:i + 1]
                              for i, p in enumerate(parts)], 1)
        return out | {"scale": scale}
    if op == "norm_grad":
        h, dy, w, r = (s[n].to(f8) for n in ("h", "dy", "w", "rstd"))
        inner = torch.einsum("nc,nc,c->n", h, dy, w) / case["C"]
        dx = torch.einsum("n,nc,c->nc", r, dy, w) - h * (r ** 3 * inner).unsqueeze(1)
        if s["dres"] is not None:
            dx = dx + s["dres"].to(f8)
        return {"dx": dx, "dweight": torch.einsum("nc,nc,n->c", h, dy, r)}
    # the drawn token's number is a choice; its log probability is computed
    return None, _exact_logprob(s)


def _exact_logprob(s):
    """By a running walk through every row's sorted probabilities on the host's terms: softmax
    first, then the cuts, then the first token in vocabulary order whose running sum passes u."""
    f8 = torch.float64
    found = []
    for r in range(s["logits"].shape[0]):
        x, t = s["logits"][r].to(f8), s["temperature"][r].to(f8)
        if t == 0:
            found.append(torch.zeros((), dtype=f8, device=x.device))
            continue
        p, order = torch.softmax(x / t, 0).sort(descending=True, stable=True)
        m = x.numel()
        if s["top_k"] is not None and int(s["top_k"][r]) > 0:
            m = min(m, int(s["top_k"][r]))
        if s["min_p"] is not None:
            m = min(m, int((p >= s["min_p"][r].to(f8) * p[0]).sum()))
        p = p[:m] / p[:m].sum()
        if s["top_p"] is not None:
            m = min(m, 1 + int((p.cumsum(0) < s["top_p"][r].to(f8)).sum()))
            p = p[:m] / p[:m].sum()
        by_index = order[:m].sort().indices
        upto = p[by_index].cumsum(0)
        at = min(int((upto <= s["u"][r].to(f8)).sum()), m - 1)
        found.append(p[by_index[at]].log())
    return torch.stack(found)
