"""Cases of the operators around a scan: the gated linear recurrence, the group norm with an
activation and the embedding, each in its plain form and through the library.

``listed()`` names the cases, ``draw(rng)`` makes more of the same ranges, ``prepare`` builds the
inputs on the GPU, ``run`` makes one pass (the plain form in 32 bits with elementary torch
operations, or with ``own`` the library's calls), ``work`` counts what a pass cannot do without and
``exact`` evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

CHUNK = 64          # the recurrence's state is kept every CHUNK steps for its gradient
C_DECAY = 8.0       # the recurrence's decay exponent scale
EPS = 1e-5          # the norm's epsilon
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one new token for each of 16 requests: latency of the serving loop
        {"name": "step_b16", "op": "step", "dtype": "bf16", "b": 16, "D": 2048},
        # a wide batch of requests, fp32 activations
        {"name": "step_b512_f32", "op": "step", "dtype": "f32", "b": 512, "D": 2560},
        # a short ragged prompt of odd width, gates cut from one projection, fp32
        {"name": "scan_ragged_f32", "op": "scan", "dtype": "f32", "b": 3, "T": 777, "D": 500,
         "fused": True, "train": False},
        # training forward: keeps the chunk states for the gradient, gates cut from one projection
        {"name": "scan_train_bf16", "op": "scan", "dtype": "bf16", "b": 8, "T": 4096, "D": 2048,
         "fused": True, "train": True},
        # one very long sequence, few channels for the machine's width
        {"name": "scan_long_f32", "op": "scan", "dtype": "f32", "b": 1, "T": 131072, "D": 1024,
         "fused": False, "train": True},
        # training backward of the ordinary shape
        {"name": "scan_grad_bf16", "op": "scan_grad", "dtype": "bf16", "b": 8, "T": 4096,
         "D": 2048, "fused": True},
        # norm of every token's heads (64 channels each) after a scan, training forward
        {"name": "norm_tokens_bf16", "op": "norm", "dtype": "bf16", "N": 16384, "S": 1, "C": 2048,
         "G": 32, "act": True},
        # norm over a feature map of a convolutional stem, fp32, odd sizes
        {"name": "norm_map_f32", "op": "norm", "dtype": "f32", "N": 6, "S": 3969, "C": 320,
         "G": 32, "act": True},
        # gradient of the per-token norm
        {"name": "norm_tokens_grad_bf16", "op": "norm_grad", "dtype": "bf16", "N": 16384, "S": 1,
         "C": 2048, "G": 32, "act": True},
        # gradient over a feature map
        {"name": "norm_map_grad_bf16", "op": "norm_grad", "dtype": "bf16", "N": 8, "S": 4096,
         "C": 512, "G": 32, "act": True},
        # lookup of a training batch
        {"name": "embed_bf16", "op": "embed", "dtype": "bf16", "n": 32768, "V": 50000, "D": 2048},
        # its gradient: tokens of a natural (Zipf) frequency, some of them padding
        {"name": "embed_grad_bf16", "op": "embed_grad", "dtype": "bf16", "n": 32768, "V": 50000,
         "D": 2048},
    ]


MOST = 1_000_000_000   # bytes that a drawn case moves, about


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(max(v, lo), hi)
    return v if v % 1024 else v + 1   # no draw is a multiple of the usual power of two


def _width(rng, lo, hi):
    """Channels: a multiple of 64, of 8, or any number."""
    m = rng.choice((64, 8, 1))
    v = max(1, _log_int(rng, lo, hi) // m) * m
    return v + m if v in (1024, 3 * 1024) else v


def draw(rng):
    op = rng.choice(("step", "scan", "scan", "scan_grad", "norm", "norm", "norm_grad", "embed",
                     "embed_grad"))
    c = {"op": op, "dtype": rng.choice(("f32", "bf16"))}
    e = 4 if c["dtype"] == "f32" else 2
    if op == "step":
        c.update(b=_log_int(rng, 1, 1000), D=_width(rng, 128, 5000))
    elif op in ("scan", "scan_grad"):
        most = MOST // (e * (7 if op == "scan_grad" else 4))   # elements
        D, T = _width(rng, 96, 4000), _log_int(rng, 1, 130000)
        while D * T > most:
            T = T // 2 + 1
        c.update(b=max(1, min(_log_int(rng, 1, 32), most // (D * T))), T=T, D=D,
                 fused=rng.random() < 0.5)
        if op == "scan":
            c["train"] = rng.random() < 0.5
    elif op in ("norm", "norm_grad"):
        most = MOST // (e * 3)
        G = rng.choice((1, 4, 8, 16, 32, 40))
        cg = _log_int(rng, 8, 128) if G > 1 else _log_int(rng, 64, 5000)
        S = 1 if rng.random() < 0.5 else _log_int(rng, 16, 20000)
        C = G * cg if G * cg != 3 * 1024 else G * (cg + 1)
        while S * C > most:
            S = S // 2 + 1
        N = max(1, min(_log_int(rng, 1, 40000), most // (S * C)))
        c.update(N=N, S=S, C=C, G=G, act=rng.random() < 0.7)
    else:
        D, V = _width(rng, 96, 4000), _log_int(rng, 300, 200000)
        n = _log_int(rng, 1, 100000)
        while D * n * e > MOST // 3:
            n = n // 2 + 1
        while D * V * 4 > MOST // 2:
            V = V // 2 + 1
        c.update(n=n, V=V, D=D)
    return c


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _decay(g, D):
    """Channels whose decay at an open gate lies between 0.9 and 0.999."""
    u = torch.rand(D, generator=g, device="cuda") * 0.099 + 0.9
    return torch.log(torch.expm1(-torch.log(u) / C_DECAY))


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, op = DTYPES[case["dtype"]], case["op"]
    s = {"op": op, "dt": dt}
    if op == "step":
        b, D = case["b"], case["D"]
        p = _randn(g, b, 3 * D, dtype=dt)   # one projection of the token, cut in three
        s.update(x=p[:, :D], ga=p[:, D:2 * D], gx=p[:, 2 * D:], decay=_decay(g, D),
                 state=_randn(g, b, D))
    elif op in ("scan", "scan_grad"):
        b, T, D = case["b"], case["T"], case["D"]
        if case["fused"]:
            p = _randn(g, b, T, 3 * D, dtype=dt)
            s.update(x=p[:, :, :D], ga=p[:, :, D:2 * D], gx=p[:, :, 2 * D:])
        else:
            s.update(x=_randn(g, b, T, D, dtype=dt), ga=_randn(g, b, T, D, dtype=dt),
                     gx=_randn(g, b, T, D, dtype=dt))
        s.update(decay=_decay(g, D), init=_randn(g, b, D), train=case.get("train", False))
        if op == "scan_grad":
            s.update(dy=_randn(g, b, T, D, dtype=dt), dfinal=_randn(g, b, D))
            # what the forward pass kept: the state before steps 0, CHUNK, 2 CHUNK, ...
            s["states"] = _scan(s)[2]
    elif op in ("norm", "norm_grad"):
        N, S, C, G = case["N"], case["S"], case["C"], case["G"]
        s.update(x=(_randn(g, N, S, C) * 1.5 + _randn(g, C) * 0.5).to(dt), G=G,
                 w=1 + 0.2 * _randn(g, C), bias=0.2 * _randn(g, C), act=case["act"])
        if op == "norm_grad":
            s["dy"] = _randn(g, N, S, C, dtype=dt)
            _, s["mean"], s["rstd"] = _norm(s)   # what the forward pass kept
    else:
        n, V, D = case["n"], case["V"], case["D"]
        # token frequencies fall as 1/rank; every rank has an id of its own; 2 % are padding
        rank = torch.exp(torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
                         * math.log(V)).long().clamp_(1, V) - 1
        ids = torch.randperm(V, generator=g, device="cuda")[rank]
        ids[torch.rand(n, generator=g, device="cuda") < 0.02] = -1
        s.update(ids=ids, V=V, scale=math.sqrt(D))
        if op == "embed":
            s["table"] = (_randn(g, V, D) / math.sqrt(D)).to(dt)
        else:
            s["dout"] = _randn(g, n, D, dtype=dt)
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
    if op == "step":
        return pkg.GatedRecurrenceStepPlan(s["x"], s["ga"], s["gx"], s["decay"], s["state"],
                                           c=C_DECAY, state_out=torch.empty_like(s["state"]))
    if op == "scan":
        return pkg.GatedRecurrencePlan(s["x"], s["ga"], s["gx"], s["decay"], c=C_DECAY,
                                       init_state=s["init"], return_states=s["train"])
    if op == "scan_grad":
        return pkg.GatedRecurrenceBackwardPlan(s["x"], s["ga"], s["gx"], s["decay"], s["dy"],
                                               c=C_DECAY, init_state=s["init"],
                                               states=s["states"], dfinal=s["dfinal"])
    act = "silu" if s.get("act") else None
    if op == "norm":
        return pkg.GroupNormPlan(s["x"], s["G"], s["w"], s["bias"], eps=EPS, activation=act)
    if op == "norm_grad":
        return pkg.GroupNormBackwardPlan(s["x"], s["dy"], s["G"], s["mean"], s["rstd"], s["w"],
                                         s["bias"], activation=act)
    if op == "embed":
        return pkg.EmbeddingPlan(s["ids"], s["table"], scale=s["scale"])
    return pkg.EmbeddingBackwardPlan(s["ids"], s["dout"], s["V"], scale=s["scale"])


# ------------------------------------------------------------------------------------------------
# plain forms, 32 bits
# ------------------------------------------------------------------------------------------------
def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _coefficients(s):
    """log a, a, m, i, r and x of every step, in 32 bits."""
    x, ga, gx, d = s["x"].float(), s["ga"].float(), s["gx"].float(), s["decay"]
    rate = torch.clamp(d, min=0) + torch.log1p(torch.exp(-d.abs()))   # softplus
    r, i = _sigmoid(ga), _sigmoid(gx)
    la = -C_DECAY * rate * r
    return la, torch.exp(la), torch.sqrt(-torch.expm1(2 * la)), i, r, x


def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h = 0: after k doublings every element holds the
    composition of the last 2^k steps."""
    k = 1
    while k < a.shape[1]:
        b = torch.cat((b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]), 1)
        a = torch.cat((a[:, :k], a[:, k:] * a[:, :-k]), 1)
        k *= 2
    return b


def _scan(s):
    la, a, m, i, r, x = _coefficients(s)
    b = m * i * x
    b[:, 0] += a[:, 0] * s["init"]
    h = _doubling(a, b)
    states = torch.cat((s["init"].unsqueeze(1), h[:, CHUNK - 1:-1:CHUNK]), 1)
    return h.to(s["dt"]), h[:, -1].clone(), states


def _scan_grad(s):
    la, a, m, i, r, x = _coefficients(s)
    b = m * i * x
    b[:, 0] += a[:, 0] * s["init"]
    h = _doubling(a, b)
    prev = torch.cat((s["init"].unsqueeze(1), h[:, :-1]), 1)
    dy = s["dy"].to(torch.float32, copy=True)
    dy[:, -1] += s["dfinal"]
    later = torch.cat((a[:, 1:], torch.zeros_like(a[:, :1])), 1)   # the decay of the step after
    G = _doubling(later.flip(1), dy.flip(1)).flip(1)
    dl = G * (a * prev - a * a * i * x / m)
    ddecay = (dl * r).sum((0, 1)) * -C_DECAY * _sigmoid(s["decay"])
    dt = s["dt"]
    return {"dx": (G * m * i).to(dt), "dgate_a": (dl * la * (1 - r)).to(dt),
            "dgate_x": (G * m * x * i * (1 - i)).to(dt), "ddecay": ddecay,
            "dinit": a[:, 0] * G[:, 0]}


def _step(s):
    la, a, m, i, r, x = _coefficients(s)
    h = a * s["state"] + m * i * x
    return h.to(s["dt"]), h


def _norm(s):
    x = s["x"].float()
    N, S, C = x.shape
    x = x.view(N, S, s["G"], C // s["G"])
    mean = x.mean((1, 3))
    x = x - mean[:, None, :, None]
    rstd = 1 / torch.sqrt((x * x).mean((1, 3)) + EPS)
    z = (x * rstd[:, None, :, None]).view(N, S, C) * s["w"] + s["bias"]
    if s["act"]:
        z = z * _sigmoid(z)
    return z.to(s["dt"]), mean, rstd


def _norm_grad(s):
    x, dz = s["x"].float(), s["dy"].float()
    N, S, C = x.shape
    grouped = (N, S, s["G"], C // s["G"])
    rstd = s["rstd"][:, None, :, None]
    xh = ((x.view(grouped) - s["mean"][:, None, :, None]) * rstd).view(N, S, C)
    if s["act"]:
        z = xh * s["w"] + s["bias"]
        sg = _sigmoid(z)
        dz = dz * sg * (1 + z * (1 - sg))
    q, xg = (dz * s["w"]).view(grouped), xh.view(grouped)
    dx = rstd * (q - q.mean((1, 3), keepdim=True) - xg * (q * xg).mean((1, 3), keepdim=True))
    return {"dx": dx.view(N, S, C).to(s["dt"]), "dweight": (dz * xh).sum((0, 1)),
            "dbias": dz.sum((0, 1))}


def _embed(s):
    ok = (s["ids"] >= 0) & (s["ids"] < s["V"])
    rows = s["table"][torch.where(ok, s["ids"], 0)].float() * s["scale"]
    return (rows * ok[:, None]).to(s["dt"])


def _embed_grad(s):
    ok = (s["ids"] >= 0) & (s["ids"] < s["V"])
    d = s["dout"].float() * (ok[:, None] * s["scale"])
    table = torch.zeros(s["V"], d.shape[1], device=d.device)
    return table.index_add_(0, torch.where(ok, s["ids"], 0), d)


PLAIN = {"step": _step, "scan_grad": _scan_grad, "norm": _norm, "norm_grad": _norm_grad,
         "embed": _embed, "embed_grad": _embed_grad}


def run(state):
    if own:
        out = state["plan"]()
        if state["op"] == "scan" and not state["train"]:
            return out[:2]
        return out
    if state["op"] == "scan":
        return _scan(state) if state["train"] else _scan(state)[:2]
    return PLAIN[state["op"]](state)


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def work(case):
    e, op = (4 if case["dtype"] == "f32" else 2), case["op"]
    if op == "step":
        n = case["b"] * case["D"]
        return {"bytes": n * (4 * e + 8) + 4 * case["D"], "flops": 24 * n}
    if op in ("scan", "scan_grad"):
        b, T, D = case["b"], case["T"], case["D"]
        n, states = b * T * D, b * -(-T // CHUNK) * D * 4
        if op == "scan":   # x, gates in, y out; initial and final state; the states that are kept
            return {"bytes": 4 * e * n + 8 * b * D + 4 * D + (states if case["train"] else 0),
                    "flops": 24 * n}
        return {"bytes": 7 * e * n + states + 12 * b * D + 8 * D, "flops": 44 * n}
    if op == "norm":
        n = case["N"] * case["S"] * case["C"]
        return {"bytes": 2 * e * n + 8 * case["N"] * case["G"] + 8 * case["C"], "flops": 14 * n}
    if op == "norm_grad":
        n = case["N"] * case["S"] * case["C"]
        return {"bytes": 3 * e * n + 8 * case["N"] * case["G"] + 16 * case["C"], "flops": 28 * n}
    n, V, D = case["n"], case["V"], case["D"]
    if op == "embed_grad":
        return {"bytes": 8 * n + n * D * e + 4 * V * D, "flops": 2 * n * D}
    v = torch.arange(1, V + 1, dtype=torch.float64)
    p = 0.98 * torch.log((v + 1) / v) / math.log(V)
    distinct = float((-torch.expm1(n * torch.log1p(-p.clamp(max=1 - 1e-12)))).sum())
    return {"bytes": 8 * n + (distinct + n) * D * e, "flops": n * D}


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    s, f8 = _inputs(case, seed), torch.float64
    op = case["op"]
    if op in ("step", "scan", "scan_grad"):
        x, d = s["x"].to(f8), s["decay"].to(f8)
        r, i = torch.sigmoid(s["ga"].to(f8)), torch.sigmoid(s["gx"].to(f8))
        la = torch.nn.functional.softplus(d, threshold=700.0).mul(-C_DECAY) * r
        a = la.exp()
        m = torch.expm1(2 * la).neg_().sqrt_()
        if op == "step":
            h = torch.addcmul(m * i * x, a, s["state"].to(f8))
            return h, h
        b, T, D = x.shape
        h = torch.empty_like(x)
        u = m * i * x
        now = s["init"].to(f8)
        for t in range(T):   # the recurrence, one step at a time
            now = torch.addcmul(u[:, t], a[:, t], now, out=h[:, t])
        if op == "scan":
            keep = torch.cat((s["init"].to(f8).unsqueeze(1), h[:, CHUNK - 1:T - 1:CHUNK]), 1)
            return (h, h[:, -1], keep) if case["train"] else (h, h[:, -1])
        del u
        g = s["dy"].to(f8)
        g[:, -1] += s["dfinal"].to(f8)
        for t in range(T - 2, -1, -1):
            g[:, t].addcmul_(a[:, t + 1], g[:, t + 1])
        out = {"dinit": a[:, 0] * g[:, 0]}
        out["dx"] = g * m * i
        out["dgate_x"] = out["dx"] * x * (1 - i)
        dl = -a * a * i * x / m
        dl[:, 0] += a[:, 0] * s["init"].to(f8)
        dl[:, 1:] += a[:, 1:] * h[:, :-1]
        dl *= g
        out["ddecay"] = (dl * la).sum((0, 1)) * torch.sigmoid(d) / torch.nn.functional.softplus(
            d, threshold=700.0)
        out["dgate_a"] = dl * la * (1 - r)
        return out
    if op in ("norm", "norm_grad"):
        grad = op == "norm_grad"
        N, S, C, G = case["N"], case["S"], case["C"], case["G"]
        x, w, bias = (s[k].to(f8).requires_grad_(grad) for k in ("x", "w", "bias"))
        xg = x.view(N, S, G, C // G)
        var, mean = torch.var_mean(xg, (1, 3), correction=0)
        z = (xg - mean[:, None, :, None]) * torch.rsqrt(var + EPS)[:, None, :, None]
        z = z.view(N, S, C) * w + bias
        y = torch.nn.functional.silu(z) if case["act"] else z
        if not grad:
            return y, mean, torch.rsqrt(var + EPS)
        dx, dw, db = torch.autograd.grad(y, (x, w, bias), s["dy"].to(f8))
        return {"dx": dx, "dweight": dw, "dbias": db}
    ids, V = s["ids"], case["V"]
    ok = (ids >= 0) & (ids < V)
    if op == "embed":
        out = torch.zeros(case["n"], case["D"], dtype=f8, device="cuda")
        out[ok] = s["table"][ids[ok]].to(f8) * s["scale"]
        return out
    out = torch.zeros(V, case["D"], dtype=f8, device="cuda")
    out.index_put_((ids[ok],), s["dout"][ok].to(f8) * s["scale"], accumulate=True)
    return out
