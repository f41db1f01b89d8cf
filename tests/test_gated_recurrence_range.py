"""The gated recurrence where states are large against what follows them, where decays are strong, and where
infinities come in.  Bounds are of single values: errors are carried along the recurrence step by step
(`Errors`), so that a state that a gate has closed may not leak into what comes after it."""
import numpy as np
import pytest
import torch

import chunked_ssd_scan_gb300 as pkg
from tests import lm_reference as ref
from tests.parity_util import to_np

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
C = 8.0
ULP = 2.0 ** -24   # half a unit in the last place


class Errors:
    """First-order error bounds of the fp32 evaluation, value by value.

    r and i: 2^x is good to 2^-22 and its argument, |g| log2 e rounded twice, to |g| 2^-23 of the
    result; that counts with 1 - r; the sum and the reciprocal add 2^-22.  The rate -c softplus: 2^-21.
    l is their product: `l`, relative.  A decay below e^-1/4 is 2^(l log2 e): its error is that of l times |l|,
    the argument's rounding |l| 2^-23 and 2^-22.  One above is carried as a - 1, good to 1.2 `l` + 2^-21
    of itself.  b = m i x: half of 1 - a^2's error, i's, and a few units: `b`.  A step rounds its
    result and, for a decay near one, w h + b.  The states that spans of steps start from go through
    composed maps instead: 2^-22 of a h a step covers their roundings."""

    def __init__(self, x, ga, gx, decay, init):
        self.la, self.a, self.m, self.i, self.r = ref.recurrence_coefficients(ga, gx, decay, C)
        l = 2.0 ** -20 + np.abs(ga) * 2.0 ** -23
        far = self.la < -0.25
        w = -np.expm1(self.la)
        self.da = np.where(far, self.a * (np.abs(self.la) * (l + 2.0 ** -23) + 2.0 ** -22), w * (1.2 * l + 2.0 ** -21))
        self.da += np.where(self.a < 2.0 ** -126, 2.0 ** -126, 0.0)   # fp32 has no such number to its full precision
        self.db = 2.0 ** -19 + (np.abs(ga) + np.abs(gx)) * 2.0 ** -23
        self.x, self.w, self.far = x, w, far
        bx = self.m * self.i * x
        h, e = init.copy(), np.zeros_like(init)
        self.prev, self.eprev = np.empty_like(x), np.empty_like(x)
        self.h, self.eh = np.empty_like(x), np.empty_like(x)
        for t in range(x.shape[1]):
            self.prev[:, t], self.eprev[:, t] = h, e
            h, e = self.step(t, h, e, bx[:, t], self.db[:, t] * np.abs(bx[:, t]))
            self.h[:, t], self.eh[:, t] = h, e

    def step(self, t, h, e, b, eb):
        a, ah = self.a[:, t], np.abs(self.a[:, t] * h)
        new = a * h + b
        e = (a + self.da[:, t]) * e + self.da[:, t] * np.abs(h) + eb + ULP * np.abs(new) + 4 * ULP * ah
        return new, e + np.where(self.far[:, t], 0.0, ULP * (self.w[:, t] * np.abs(h) + np.abs(b)))

    def gradient(self, dy, dfinal, decay):
        """Bounds of dx, dgate_a, dgate_x, ddecay and dinit."""
        la, a, m, i, r, x = self.la, self.a, self.m, self.i, self.r, self.x
        k0 = a * i * np.divide(x, m, out=np.zeros_like(x), where=m > 0)
        k = self.prev - k0
        ek = self.eprev + self.db * np.abs(k0) + 4 * ULP * (np.abs(self.prev) + np.abs(k0))
        out = {n: np.empty_like(x) for n in ("dx", "dgate_a", "dgate_x")}
        terms = np.empty_like(x)
        G, e = dfinal.copy(), np.zeros_like(dfinal)
        for t in range(x.shape[1] - 1, -1, -1):
            e = e + ULP * np.abs(G + dy[:, t])
            G = G + dy[:, t]
            aG, db = np.abs(G), self.db[:, t]
            mi = m[:, t] * i[:, t]
            out["dx"][:, t] = mi * (e + 2 * db * aG)
            gx = np.abs(mi * x[:, t])
            # 1 - i, rounded: 2^-22 absolute
            out["dgate_x"][:, t] = gx * (1 - i[:, t]) * (e + 2 * db * aG) + gx * aG * 2.0 ** -22
            dl = a[:, t] * np.abs(k[:, t])
            edl = a[:, t] * ek[:, t] + self.da[:, t] * np.abs(k[:, t])
            term = np.abs(la[:, t])
            out["dgate_a"][:, t] = term * ((1 - r[:, t]) * (edl * aG + dl * (e + 2 * db * aG)) + dl * aG * 2.0 ** -22)
            terms[:, t] = r[:, t] * (edl * aG + dl * (e + (2 * db + 2.0 ** -20) * aG))
            G, e = self.step(t, G, e, np.zeros_like(G), 0.0)
        out["dinit"] = e
        out["ddecay"] = C * ref.sigmoid(decay) * terms.sum((0, 1))
        return out


def within(got, want, bound, dtype, what):
    """`bound`, and for bf16 the rounding of the result (2^-8 of it: see lm_reference)."""
    bound = 2 * bound + (ref.BF16_REL * np.abs(want) if dtype == "bf16" else 0) + 1e-36   # 2: higher orders
    err = np.abs(got - want)
    if not np.all(err <= bound):
        k = np.unravel_index(np.argmax(err / bound), want.shape)
        raise AssertionError(f"{what}: {int((err > bound).sum())} of {err.size} off, worst at {k}: got {got[k]:.8g}, "
                             f"want {want[k]:.8g}, bound {bound[k]:.3g}")


def mixed(b, T, D, dtype, seed):
    """Gates from closed to open, rates from -1e-3 to -400, and x of 1e5 beside 1e-3: states of 1e5 that a
    step closes by e^-0.3 to e^-400 and that are followed by values of size 1e-3."""
    g = torch.Generator().manual_seed(seed)
    pick = lambda v, *s: torch.tensor(v)[torch.randint(0, len(v), s, generator=g)]   # noqa: E731
    rate = pick([1e-3, 0.1, 0.3, 1.0, 5.0, 24.0, 400.0], D).double() / C
    d = {"decay": torch.where(rate > 30, rate, torch.log(torch.expm1(rate))).float(),
         "x": torch.randn(b, T, D, generator=g) * pick([1e-3, 1e-3, 1.0, 1e5], b, T, D),
         "ga": pick([-20.0, -6.0, -1.0, 2.0, 12.0], b, T, D) + torch.randn(b, T, D, generator=g) * 0.1,
         "gx": torch.randn(b, T, D, generator=g) * 2,
         "init": torch.randn(b, D, generator=g) * 1e5, "dfinal": torch.randn(b, D, generator=g) * 1e4,
         "dy": torch.randn(b, T, D, generator=g) * pick([1e-3, 1e-3, 1.0, 1e4], b, T, D)}
    return {k: (v.to(DT[dtype]) if k in ("x", "ga", "gx", "dy") else v).cuda() for k, v in d.items()}


def forward(d, **kw):
    plan = pkg.GatedRecurrencePlan(d["x"], d["ga"], d["gx"], d["decay"], c=C, init_state=d["init"],
                                   return_states=True, **kw)
    out = plan()
    assert pkg.workspace_status(plan.workspace) == ("SSD_OK", 0)
    return out


def backward(d, states):
    return pkg.gated_recurrence_backward(d["x"], d["ga"], d["gx"], d["decay"], d["dy"], c=C, init_state=d["init"],
                                         states=states, dfinal=d["dfinal"])


SHAPES = [(2, 1, 40), (2, 17, 96), (1, 64, 64), (2, 300, 70), (1, 1000, 192), (3, 130, 31)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_large_states_behind_strong_decays(shape, dtype):
    d = mixed(*shape, dtype, seed=41)
    y, fin, states = forward(d)
    n = {k: to_np(v) for k, v in d.items()}
    e = Errors(n["x"], n["ga"], n["gx"], n["decay"], n["init"])
    within(to_np(y), e.h, e.eh, dtype, "y")
    within(to_np(fin), e.h[:, -1], e.eh[:, -1], "f32", "final_state")
    within(to_np(states), e.prev[:, ::64], e.eprev[:, ::64], "f32", "states")
    g = backward(d, states)
    want = ref.recurrence_grad(n["x"], n["ga"], n["gx"], n["decay"], n["dy"], c=C, init=n["init"], dfinal=n["dfinal"])
    bound = e.gradient(n["dy"], n["dfinal"], n["decay"])
    for k in ("dx", "dgate_x", "dgate_a"):
        within(to_np(g[k]), want[k], bound[k], dtype, k)
    for k in ("dinit", "ddecay"):
        within(to_np(g[k]), want[k], bound[k], "f32", k)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bD", [(2, 40), (3, 31), (64, 10240)], ids=str)
def test_large_states_closed_by_one_step(bD, dtype):
    d = mixed(bD[0], 1, bD[1], dtype, seed=42)
    n = {k: to_np(v) for k, v in d.items()}
    e = Errors(n["x"], n["ga"], n["gx"], n["decay"], n["init"])
    y, state = pkg.gated_recurrence_step(d["x"][:, 0], d["ga"][:, 0], d["gx"][:, 0], d["decay"], d["init"], c=C)
    within(to_np(y), e.h[:, 0], e.eh[:, 0], dtype, "y")
    within(to_np(state), e.h[:, 0], e.eh[:, 0], "f32", "state")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_closed_input_gate_on_large_values(dtype):
    """i far below 2^-64, but not too small for fp32, times an x that makes up for it."""
    d = mixed(2, 150, 72, dtype, seed=43)
    g = torch.Generator().manual_seed(44)
    at = torch.randint(0, 5, (2, 150, 72), generator=g).cuda()
    gx, x = (d[k].float() for k in ("gx", "x"))
    for k, (gate, size) in enumerate(((-43.0, 1e15), (-46.0, 1e20), (-60.0, 1e25), (-80.0, 1e33))):
        gx = torch.where(at == k, gate, gx)
        x = torch.where(at == k, torch.randn(x.shape, generator=g).cuda() * size, x)
    d["gx"], d["x"] = gx.to(DT[dtype]), x.to(DT[dtype])
    n = {k: to_np(v) for k, v in d.items()}
    e = Errors(n["x"], n["ga"], n["gx"], n["decay"], n["init"])
    y, fin, _ = forward(d)
    within(to_np(y), e.h, e.eh, dtype, "y")
    within(to_np(fin), e.h[:, -1], e.eh[:, -1], "f32", "final_state")
    y, _ = pkg.gated_recurrence_step(*(d[k][:, 0] for k in ("x", "ga", "gx")), d["decay"], d["init"].clone(), c=C)
    within(to_np(y), e.h[:, 0], e.eh[:, 0], dtype, "y of one step")


def ordinary(b, T, D, dtype, seed, strong):
    """Decays of 0.9 to 0.999 at an open gate, or of e^-0.1 to e^-12."""
    g = torch.Generator().manual_seed(seed)
    rate = -torch.log(torch.rand(D, generator=g) * 0.099 + 0.9) / C
    if strong:
        rate = torch.linspace(0.1, 12.0, D) / C
    d = {k: torch.randn(b, T, D, generator=g).to(DT[dtype]).cuda() for k in ("x", "ga", "gx", "dy")}
    d.update(decay=torch.log(torch.expm1(rate)).cuda(), init=torch.randn(b, D, generator=g).cuda(),
             dfinal=torch.randn(b, D, generator=g).cuda())
    return d


def same_kind(got, want, what):
    """NaN, +inf and -inf at the same places."""
    for name, is_ in (("NaN", np.isnan), ("inf", np.isposinf), ("-inf", np.isneginf)):
        assert np.array_equal(is_(got), is_(want)), f"{what}: {name} elsewhere"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("strong", [False, True], ids=["slow", "strong"])
@pytest.mark.parametrize("T", [1, 64, 256, 300])
def test_infinities(T, strong, dtype):
    """An infinite x or initial state stays what the formula makes of it (its decays are not zero), in its channel
    alone, and so do an infinite dy and dfinal on their way back."""
    b, D = 2, 70
    inf, last = float("inf"), T - 1
    d = ordinary(b, T, D, dtype, 45, strong)
    clean = {k: v.clone() for k, v in d.items()}
    d["x"][0, T // 3, 5], d["x"][1, 0, 33], d["x"][1, last, 34] = inf, -inf, inf
    d["x"][0, 0, 40], d["x"][0, last, 40] = inf, -inf if T > 1 else inf     # meet: NaN
    d["init"][0, 69], d["init"][1, 2] = -inf, inf
    d["dy"][0, last, 10], d["dy"][1, T // 2, 64], d["dfinal"][1, 20] = inf, -inf, inf
    n = {k: to_np(v) for k, v in d.items()}
    with np.errstate(invalid="ignore"):
        wy, wf, ws = ref.recurrence(n["x"], n["ga"], n["gx"], n["decay"], C, n["init"])
        wg = ref.recurrence_grad(n["x"], n["ga"], n["gx"], n["decay"], n["dy"], c=C, init=n["init"], dfinal=n["dfinal"])
    y, fin, states = forward(d)
    g = backward(d, states)
    same_kind(to_np(y), wy, "y")
    same_kind(to_np(fin), wf, "final_state")
    same_kind(to_np(states), ws, "states")
    for k in ("dx", "dgate_a", "dgate_x", "dinit", "ddecay"):
        same_kind(to_np(g[k]), wg[k], k)
    ok = np.isfinite(wy)
    ref.check(np.where(ok, to_np(y), 0), np.where(ok, wy, 0), ref.BF16_REL if dtype == "bf16" else 0.0, "y")
    # channels that no infinity touches have the bits that they have without
    touched = torch.zeros(D, dtype=torch.bool)
    touched[[5, 33, 34, 40, 69, 2, 10, 64, 20]] = True
    cy, cf, cs = forward(clean)
    cg = backward(clean, cs)
    for got, was in ((y, cy), (fin, cf), (states, cs), (g["dx"], cg["dx"]), (g["dgate_a"], cg["dgate_a"])):
        assert torch.equal(got[..., ~touched], was[..., ~touched])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinities_in_one_step(dtype):
    b, D = 3, 72
    inf = float("inf")
    for strong in (False, True):
        d = ordinary(b, 1, D, dtype, 46, strong)
        d["x"][0, 0, 3], d["x"][1, 0, 3], d["init"][1, 3], d["init"][2, 71], d["init"][0, 9] = inf, inf, -inf, -inf, inf
        n = {k: to_np(v) for k, v in d.items()}
        with np.errstate(invalid="ignore"):
            wy, wf, _ = ref.recurrence(n["x"], n["ga"], n["gx"], n["decay"], C, n["init"])
        y, state = pkg.gated_recurrence_step(*(d[k][:, 0] for k in ("x", "ga", "gx")), d["decay"], d["init"], c=C)
        same_kind(to_np(y), wy[:, 0], "y")
        same_kind(to_np(state), wf, "state")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_lowest_value_of_the_type(dtype):
    """A mask of the type's lowest value in x: a finite state of that size, and what follows from it."""
    d = ordinary(2, 200, 70, dtype, 47, True)
    lowest = torch.finfo(DT[dtype]).min
    d["x"][0, 70, 7], d["x"][1, 0, 69], d["x"][1, 199, 11] = lowest, lowest, lowest
    n = {k: to_np(v) for k, v in d.items()}
    e = Errors(n["x"], n["ga"], n["gx"], n["decay"], n["init"])
    y, fin, _ = forward(d)
    within(to_np(y), e.h, e.eh, dtype, "y")
    within(to_np(fin), e.h[:, -1], e.eh[:, -1], "f32", "final_state")
