"""Plain fp64 forms (numpy) of the gated delta rule, the root-mean-square norm and the drawing of tokens, straight from
their definitions, and the gate that the GPU tests compare with."""
from __future__ import annotations

import numpy as np

# A rounding to bf16 is off by at most half a step, 2^-8 of the value (bf16 has eps 2^-7).
BF16_REL = 2.0 ** -8

# What the arithmetic itself may add, relative to the larger of the value and the output's root mean square.
# f32: one operation is off by 2^-24; a step of the delta rule does up to 2 * 256 of them a value, which add up like
# their square root (23), over a memory of up to 500 steps whose errors are independent (another 23), at least 3e-5.
# bf16: on the tensor cores what is computed on the way is two bf16 terms, off by at most 2^-17 (the first term's half
# step 2^-8, times the second's 2^-8, and the products of second terms that are left out, 2^-16 at most but of
# alternating sign).  About eight such roundings lie between an input and an output: 8 * 2^-17 = 6e-5, and a largest
# error of a sum of 64 to 128 of them is no more than twice that.
UNIT = {"f32": 3e-5, "bf16": 1.2e-4}


def check(got, ref, dtype, what, rounded=False, scale=None):
    """|got - ref| <= (a rounding to bf16) |ref| + UNIT max(rms, |ref|), rms of ref or of `scale` (where a value is a
    sum of larger terms)."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, f"{what}: shape {got.shape} != {ref.shape}"
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN elsewhere"
    if not ref.size:
        return
    base = np.asarray(ref if scale is None else scale, np.float64)
    rms = np.sqrt(np.nanmean(np.where(np.isfinite(base), base, np.nan) ** 2))
    rel = BF16_REL if rounded and dtype == "bf16" else 0.0
    bound = rel * np.abs(ref) + UNIT[dtype] * np.maximum(rms, np.abs(ref))
    with np.errstate(invalid="ignore"):
        bad = ~((got == ref) | np.isnan(ref) | (np.abs(got - ref) <= bound))
    if bad.any():
        k = np.unravel_index(np.argmax(np.where(bad, np.abs(got - ref) / bound, -np.inf)), ref.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} values off, worst at {k}: got {got[k]:.8g} "
                             f"ref {ref[k]:.8g} bound {np.broadcast_to(bound, ref.shape)[k]:.3g}")


def _inputs(q, k, v, g, beta, init, scale):
    b, T, H, V = v.shape
    r = H // q.shape[2]
    a = np.ones((b, T, H)) if g is None else np.exp(g)
    S = np.zeros((b, H, V, q.shape[3])) if init is None else init.copy()
    return q.repeat(r, 2), k.repeat(r, 2), a, S, q.shape[3] ** -0.5 if scale is None else scale


def delta(q, k, v, g, beta, init=None, scale=None, chunk=64):
    """(y, final_state, states before steps 0, chunk, ...)."""
    q, k, a, S, scale = _inputs(q, k, v, g, beta, init, scale)
    T = v.shape[1]
    y, states = np.empty_like(v), []
    for t in range(T):
        if t % chunk == 0:
            states.append(S)
        S = S * a[:, t, :, None, None]
        u = beta[:, t, :, None] * (v[:, t] - np.einsum("bhvk,bhk->bhv", S, k[:, t]))
        S = S + u[..., None] * k[:, t, :, None, :]
        y[:, t] = scale * np.einsum("bhvk,bhk->bhv", S, q[:, t])
    states = np.stack(states, 1) if states else np.zeros((v.shape[0], 0, *S.shape[1:]))
    return y, S, states


def delta_grad(q, k, v, g, beta, dy, init=None, scale=None, dfinal=None):
    """Gradients of <dy, y> + <dfinal, final_state>."""
    b, T, Hk, K = q.shape
    H = v.shape[2]
    q, k, a, S, scale = _inputs(q, k, v, g, beta, init, scale)
    before, errs = [], []
    for t in range(T):
        S = S * a[:, t, :, None, None]
        before.append(S)
        errs.append(v[:, t] - np.einsum("bhvk,bhk->bhv", S, k[:, t]))
        S = S + (beta[:, t, :, None] * errs[-1])[..., None] * k[:, t, :, None, :]
    G = np.zeros_like(S) if dfinal is None else dfinal.copy()
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dg, dbeta = np.zeros((b, T, H)), np.zeros((b, T, H))
    for t in reversed(range(T)):
        S, u = before[t], beta[:, t, :, None] * errs[t]
        after = S + u[..., None] * k[:, t, :, None, :]
        dq[:, t] = scale * np.einsum("bhvk,bhv->bhk", after, dy[:, t])
        G = G + scale * dy[:, t][..., None] * q[:, t, :, None, :]
        du = np.einsum("bhvk,bhk->bhv", G, k[:, t])
        dv[:, t] = beta[:, t, :, None] * du
        dbeta[:, t] = (du * errs[t]).sum(-1)
        dk[:, t] = np.einsum("bhvk,bhv->bhk", G, u) - np.einsum("bhvk,bhv->bhk", S, dv[:, t])
        G = G - dv[:, t][..., None] * k[:, t, :, None, :]
        dg[:, t] = (G * S).sum((-1, -2))
        G = G * a[:, t, :, None, None]
    share = lambda d: d.reshape(b, T, Hk, H // Hk, K).sum(3)   # noqa: E731
    return {"dq": share(dq), "dk": share(dk), "dv": dv, "dg": dg, "dbeta": dbeta, "dinit": G}


def rms_norm(x, w=None, res=None, eps=1e-6):
    """(y, h, rstd)."""
    h = x if res is None else x + res
    rstd = 1 / np.sqrt((h * h).mean(-1) + eps)
    y = h * rstd[..., None]
    return (y if w is None else y * w), h, rstd


def rms_norm_grad(h, dy, rstd, w=None, dres=None):
    xh, q = h * rstd[..., None], dy if w is None else dy * w
    dx = rstd[..., None] * (q - xh * (q * xh).mean(-1, keepdims=True))
    return {"dx": dx if dres is None else dx + dres,
            "dweight": (dy * xh).reshape(-1, h.shape[-1]).sum(0)}


def e4m3(v):
    """The nearest value with 4 bits of exponent and 3 of mantissa, ties to even, at most 448."""
    v = np.clip(v, -448.0, 448.0)
    step = np.exp2(np.maximum(np.frexp(v)[1], -5) - 4.0)
    return np.round(v / step) * step


def kept(logits, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The weights of one row (fp64, zero where a token is not kept), by a walk down the sorted logits."""
    x = np.where(np.isnan(logits), -np.inf, logits)
    most = x.max()
    out = np.zeros_like(x)
    if most == -np.inf:
        return out
    order = np.argsort(-x, kind="stable")
    if temperature == 0:
        out[order[0]] = 1.0
        return out
    with np.errstate(invalid="ignore"):
        w = np.where(x == most, 1.0, np.exp((x - most) / temperature))
    m = len(x) if top_k <= 0 else min(top_k, len(x))
    ws = w[order]
    if min_p > 0:
        m = max(1, min(m, int((ws >= min_p).sum())))
    if top_p < 1:
        upto = ws[:m].cumsum()
        m = 1 + int((upto[:m - 1] < top_p * upto[-1]).sum())
    out[order[:m]] = ws[:m]
    return out


def sample(logits, u, **settings):
    """(id, logprob) of one row."""
    w = kept(logits, **settings)
    total = w.sum()
    if total == 0:
        return -1, np.nan
    at = int(np.argmax(w.cumsum() > u * total))
    return at, np.log(w[at] / total)
