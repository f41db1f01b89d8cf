"""Plain fp64 forms (numpy) of the gated recurrence, the channels-last group norm and the embedding,
straight from their formulas, and the gates that the GPU tests compare with."""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def softplus(v):
    return np.logaddexp(0.0, v)


def recurrence_coefficients(ga, gx, decay, c):
    r, i = sigmoid(ga), sigmoid(gx)
    la = -c * softplus(decay) * r
    return la, np.exp(la), np.sqrt(-np.expm1(2 * la)), i, r


def recurrence(x, ga, gx, decay, c=8.0, init=None, chunk=64):
    """(y, final_state, states before steps 0, chunk, ...)."""
    b, T, D = x.shape
    _, a, m, i, _ = recurrence_coefficients(ga, gx, decay, c)
    h = np.zeros((b, D)) if init is None else init.copy()
    y, states = np.zeros((b, T, D)), np.zeros((b, -(-T // chunk), D))
    for t in range(T):
        if t % chunk == 0:
            states[:, t // chunk] = h
        h = a[:, t] * h + m[:, t] * i[:, t] * x[:, t]
        y[:, t] = h
    return y, h, states


def recurrence_grad(x, ga, gx, decay, dy, c=8.0, init=None, dfinal=None):
    b, T, D = x.shape
    la, a, m, i, r = recurrence_coefficients(ga, gx, decay, c)
    y, _, _ = recurrence(x, ga, gx, decay, c, init)
    h0 = np.zeros((b, D)) if init is None else init
    carry = np.zeros((b, D)) if dfinal is None else dfinal.copy()
    g = {"dx": np.zeros_like(x), "dgate_a": np.zeros_like(x), "dgate_x": np.zeros_like(x)}
    dl_r = np.zeros(D)
    for t in range(T - 1, -1, -1):
        G = dy[:, t] + carry
        prev = y[:, t - 1] if t else h0
        mt, at = m[:, t], a[:, t]
        over_m = np.divide(1.0, mt, out=np.zeros_like(mt), where=mt > 0)   # limit: l / m -> 0
        dl = G * at * (prev - at * i[:, t] * x[:, t] * over_m)
        g["dx"][:, t] = G * mt * i[:, t]
        g["dgate_x"][:, t] = G * mt * x[:, t] * i[:, t] * (1 - i[:, t])
        g["dgate_a"][:, t] = dl * la[:, t] * (1 - r[:, t])
        dl_r += (dl * r[:, t]).sum(0)
        carry = at * G
    g["ddecay"] = -c * dl_r * sigmoid(decay)
    g["dinit"] = carry
    return g


def group_norm(x, groups, w=None, bias=None, eps=1e-5, act="silu"):
    """x [N,S,C] -> (y, mean, rstd)."""
    N, S, C = x.shape
    xg = x.reshape(N, S, groups, C // groups)
    mean = xg.mean((1, 3))
    d = xg - mean[:, None, :, None]
    rstd = 1.0 / np.sqrt((d * d).mean((1, 3)) + eps)
    z = (d * rstd[:, None, :, None]).reshape(N, S, C)
    z = z * (1.0 if w is None else w) + (0.0 if bias is None else bias)
    return (z * sigmoid(z) if act == "silu" else z), mean, rstd


def group_norm_grad(x, dy, groups, w=None, bias=None, eps=1e-5, act="silu"):
    N, S, C = x.shape
    shape = (N, S, groups, C // groups)
    _, mean, rstd = group_norm(x, groups, w, bias, eps, act)
    rs = rstd[:, None, :, None]
    xh = (x.reshape(shape) - mean[:, None, :, None]) * rs
    wv = np.ones(C) if w is None else w
    dz = dy
    if act == "silu":
        z = xh.reshape(N, S, C) * wv + (0.0 if bias is None else bias)
        s = sigmoid(z)
        dz = dy * s * (1 + z * (1 - s))
    q = (dz * wv).reshape(shape)
    dx = rs * (q - q.mean((1, 3), keepdims=True) - xh * (q * xh).mean((1, 3), keepdims=True))
    return {"dx": dx.reshape(N, S, C), "dweight": (dz * xh.reshape(N, S, C)).sum((0, 1)),
            "dbias": dz.sum((0, 1))}


def embedding(ids, table, scale):
    ok = (ids >= 0) & (ids < table.shape[0])
    return scale * table[np.where(ok, ids, 0)] * ok[..., None]


def embedding_grad(ids, dout, rows, scale):
    ids, dout = ids.reshape(-1), dout.reshape(-1, dout.shape[-1])
    ok = (ids >= 0) & (ids < rows)
    out = np.zeros((rows, dout.shape[-1]))
    np.add.at(out, ids[ok], scale * dout[ok])
    return out


# Gates.  An output rounded to bf16 is off by at most half a unit in its last place, 2^-9 of its value;
# twice that leaves room for a value that the fp32 error moves across a rounding boundary.  In fp32
# one operation is off by 2^-24 = 6e-8 and the special functions by a few of those.
BF16_REL = 2.0 ** -8


def check(got, ref, rel, what, scale=None, axis=None):
    """|got - ref| <= rel |ref| + fp32 term, the fp32 term being 2e-5 of the root mean square of ref (over
    `axis`, or of `scale` where the value is a sum of larger terms).  2e-5 is some 170 fp32 units:
    a step's coefficients carry about 10 of them and a channel with memory 1 / (1 - a) <= 1000
    steps adds independent ones up to sqrt(1000 / 2) times."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, f"{what}: shape {got.shape} != {ref.shape}"
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaNs elsewhere"
    if not ref.size:
        return
    base = ref if scale is None else np.broadcast_to(np.asarray(scale, np.float64), ref.shape)
    rms = np.sqrt(np.nanmean(np.where(np.isfinite(base), base, np.nan) ** 2, axis=axis, keepdims=True))
    bound = rel * np.abs(ref) + 2e-5 * np.maximum(rms, np.abs(ref))
    with np.errstate(invalid="ignore"):
        err = np.abs(got - ref)
    same = (got == ref) | np.isnan(ref)
    bad = ~(same | (err <= bound))
    if bad.any():
        k = np.unravel_index(np.argmax(np.where(bad, err - bound, -np.inf)), ref.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} values off, worst at {k}: "
                             f"got {got[k]:.8g} ref {ref[k]:.8g} bound {np.broadcast_to(bound, ref.shape)[k]:.3g}")
