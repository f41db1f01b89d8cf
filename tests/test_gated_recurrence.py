"""Gated linear recurrence: the fp64 form against differences (CPU), the kernels against the fp64
form (GPU), and the refusals."""
import ctypes

import numpy as np
import pytest
import torch

import chunked_ssd_scan_gb300 as pkg
from chunked_ssd_scan_gb300 import _build
from tests import lm_reference as ref
from tests.parity_util import GUARD_FILL, Guarded, to_np

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
REL = {"f32": 0.0, "bf16": ref.BF16_REL}
C = 8.0


def inputs(b, T, D, dtype="f32", seed=0, layout="plain", dev="cpu", slow=False):
    """x, gates [b,T,D] (separate, slices of one projection, or slices that start at an odd element),
    decay, init, dy, dfinal."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    u = torch.rand(D, generator=g) * 0.099 + 0.9
    if slow:
        u = 1 - 10 ** (-2 - 3 * torch.rand(D, generator=g))
    d = {"decay": torch.log(torch.expm1(-torch.log(u) / C)), "init": rnd(b, D),
         "dfinal": rnd(b, D)}
    if layout == "plain":
        d.update({k: rnd(b, T, D) for k in ("x", "ga", "gx", "dy")})
    else:
        off = 1 if layout == "odd" else 0
        p = rnd(b, T, 4 * D + off).to(DT[dtype]).to(dev)[..., off:]
        d.update(x=p[..., :D], ga=p[..., D:2 * D], gx=p[..., 2 * D:3 * D], dy=p[..., 3 * D:])
    for k in ("x", "ga", "gx", "dy"):
        d[k] = d[k].to(DT[dtype]).to(dev)
    for k in ("decay", "init", "dfinal"):
        d[k] = d[k].to(dev)
    return d


def reference(d, init=True):
    return ref.recurrence(*(to_np(d[k]) for k in ("x", "ga", "gx", "decay")), c=C,
                          init=to_np(d["init"]) if init else None)


def reference_grad(d, init=True, dfinal=True):
    return ref.recurrence_grad(*(to_np(d[k]) for k in ("x", "ga", "gx", "decay", "dy")), c=C,
                               init=to_np(d["init"]) if init else None,
                               dfinal=to_np(d["dfinal"]) if dfinal else None)


def test_reference_gradient_against_differences():
    d = {k: to_np(v) for k, v in inputs(2, 9, 5, seed=3).items()}
    keys = ("x", "ga", "gx", "decay", "init")
    loss = lambda e: sum((a * w).sum() for a, w in zip(   # noqa: E731
        ref.recurrence(*(e[k] for k in keys[:4]), c=C, init=e["init"])[:2], (d["dy"], d["dfinal"])))
    g = ref.recurrence_grad(*(d[k] for k in keys[:4]), d["dy"], c=C, init=d["init"],
                            dfinal=d["dfinal"])
    rng = np.random.default_rng(0)
    for k, gk in zip(keys, ("dx", "dgate_a", "dgate_x", "ddecay", "dinit")):
        v = rng.standard_normal(d[k].shape)
        eps = 1e-5
        num = (loss({**d, k: d[k] + eps * v}) - loss({**d, k: d[k] - eps * v})) / (2 * eps)
        # central differences: the third derivative's term eps^2 and the rounding 1e-16 / eps
        assert abs(num - (g[gk] * v).sum()) <= 1e-7 * (1 + abs(num)), k


# b, T, D: one step, around the 64-step chunk and the 64-channel column, long, odd
SHAPES = [(1, 1, 1), (2, 1, 64), (3, 2, 7), (1, 63, 130), (3, 64, 64), (2, 65, 66), (2, 128, 40),
          (2, 129, 31), (1, 1000, 96), (2, 777, 500), (5, 300, 257), (1, 9001, 72)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["plain", "fused", "odd"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dtype, layout):
    b, T, D = shape
    d = inputs(b, T, D, dtype, seed=1, layout=layout, dev="cuda")
    e = 2 if dtype == "bf16" else 4
    bands = {"y": Guarded(b * T * D * e, "cuda", GUARD_FILL), "final": Guarded(b * D * 4, "cuda"),
             "states": Guarded(b * -(-T // 64) * D * 4, "cuda", GUARD_FILL)}
    plan = pkg.GatedRecurrencePlan(
        d["x"], d["ga"], d["gx"], d["decay"], c=C, init_state=d["init"],
        y=bands["y"].view(DT[dtype], (b, T, D)), final_state=bands["final"].view(torch.float32, (b, D)),
        states=bands["states"].view(torch.float32, (b, -(-T // 64), D)))
    y, fin, st = plan()
    assert pkg.workspace_status(plan.workspace) == ("SSD_OK", 0)
    for k, v in bands.items():
        v.check(k)
    ry, rf, rs = reference(d)
    ref.check(to_np(y), ry, REL[dtype], "y")
    ref.check(to_np(fin), rf, 0.0, "final_state", scale=ry[:, -1])
    ref.check(to_np(st), rs, 0.0, "states")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["plain", "fused", "odd"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, dtype, layout):
    b, T, D = shape
    d = inputs(b, T, D, dtype, seed=2, layout=layout, dev="cuda")
    e = 2 if dtype == "bf16" else 4
    out = {k: Guarded(b * T * D * e, "cuda", GUARD_FILL) for k in ("dx", "dgate_a", "dgate_x")}
    out["ddecay"], out["dinit"] = Guarded(D * 4, "cuda"), Guarded(b * D * 4, "cuda")
    grads = {k: v.view(DT[dtype], (b, T, D)) for k, v in out.items() if k[1] in "xg"}
    grads["ddecay"] = out["ddecay"].view(torch.float32, (D,))
    grads["dinit"] = out["dinit"].view(torch.float32, (b, D))
    args = (d["x"], d["ga"], d["gx"], d["decay"], d["dy"])
    kw = dict(c=C, init_state=d["init"], dfinal=d["dfinal"])
    _, _, states = pkg.gated_recurrence_forward(*args[:4], c=C, init_state=d["init"], return_states=True)
    plan = pkg.GatedRecurrenceBackwardPlan(*args, states=states, grads=grads, **kw)
    g = {k: to_np(v) for k, v in plan().items()}
    assert pkg.workspace_status(plan.workspace) == ("SSD_OK", 0)
    for k, v in out.items():
        v.check(k)
    r = reference_grad(d)
    for k in ("dx", "dgate_x", "dgate_a"):
        ref.check(g[k], r[k], REL[dtype], k)
    # dl is a difference of two terms: its error goes with their size, and the sum's with its terms'
    ref.check(g["ddecay"], r["ddecay"], 0.0, "ddecay", scale=np.sqrt(b * T) * 4 + np.abs(r["ddecay"]))
    ref.check(g["dinit"], r["dinit"], 0.0, "dinit")
    # recomputed states: the same values, so the same bits
    again = pkg.gated_recurrence_backward(*args, **kw)
    for k in g:
        assert np.array_equal(to_np(again[k]), g[k]), k


@pytest.mark.gpu
def test_without_optional_arguments():
    d = inputs(2, 200, 96, seed=4, dev="cuda")
    y, fin, st = pkg.gated_recurrence_forward(d["x"], d["ga"], d["gx"], d["decay"], c=C,
                                              return_final_state=False)
    assert fin is None and st is None
    ref.check(to_np(y), reference(d, init=False)[0], 0.0, "y")
    g = pkg.gated_recurrence_backward(d["x"], d["ga"], d["gx"], d["decay"], d["dy"], c=C,
                                      return_dinit=False)
    assert g["dinit"] is None
    r = reference_grad(d, init=False, dfinal=False)
    for k in ("dx", "dgate_a", "dgate_x"):
        ref.check(to_np(g[k]), r[k], 0.0, k)


@pytest.mark.gpu
def test_slow_channels_keep_their_precision():
    """1 - a^2 from 1e-2 down to 1e-5: a difference of rounded numbers would lose three digits."""
    d = inputs(2, 500, 128, seed=5, dev="cuda", slow=True)
    y, _, _ = pkg.gated_recurrence_forward(d["x"], d["ga"], d["gx"], d["decay"], c=C)
    r = ref.recurrence(*(to_np(d[k]) for k in ("x", "ga", "gx", "decay")), c=C)[0]
    ref.check(to_np(y), r, 0.0, "y", axis=1)   # each channel by its own size


EXTREME = [float("-inf"), -1e30, -200.0, -104.0, -89.0, -40.0, 0.0, 40.0, 89.0, 200.0, float("inf")]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_extreme_gates_and_decays(dtype):
    """Gates from closed to open beyond what exp holds, decays from 1e-26 to 50: finite everywhere,
    and the limits are met."""
    n = len(EXTREME)
    g = torch.Generator().manual_seed(6)
    T, D = 70, n * n
    ga = torch.tensor(EXTREME).repeat_interleave(n).expand(1, T, D)
    gx = torch.tensor(EXTREME).repeat(n).expand(1, T, D)
    decay = torch.tensor([-60.0, -3.0, 0.0, 50.0, 1.0])[torch.arange(D) % 5]
    d = {"x": torch.randn(1, T, D, generator=g), "ga": ga, "gx": gx, "decay": decay,
         "init": torch.randn(1, D, generator=g), "dy": torch.randn(1, T, D, generator=g),
         "dfinal": torch.randn(1, D, generator=g)}
    d = {k: (v.to(DT[dtype]) if k in ("x", "ga", "gx", "dy") else v).cuda() for k, v in d.items()}
    y, fin, _ = pkg.gated_recurrence_forward(d["x"], d["ga"], d["gx"], d["decay"], c=C, init_state=d["init"])
    gr = pkg.gated_recurrence_backward(d["x"], d["ga"], d["gx"], d["decay"], d["dy"], c=C,
                                       init_state=d["init"], dfinal=d["dfinal"])
    ry, rf, _ = reference(d)
    ref.check(to_np(y), ry, REL[dtype], "y")
    ref.check(to_np(fin), rf, 0.0, "final_state")
    r = reference_grad(d)
    for k in ("dx", "dgate_a", "dgate_x", "dinit"):
        ref.check(to_np(gr[k]), r[k], REL[dtype], k)
    assert torch.isfinite(gr["ddecay"]).all()


@pytest.mark.gpu
def test_nan_stays_in_its_channel_and_after_its_step():
    d = inputs(2, 300, 70, seed=7, dev="cuda")
    for k, (b, t, c) in {"x": (0, 130, 5), "ga": (1, 64, 33), "gx": (1, 299, 69)}.items():
        d[k][b, t, c] = float("nan")
    y = to_np(pkg.gated_recurrence_forward(d["x"], d["ga"], d["gx"], d["decay"], c=C)[0])
    bad = np.zeros(y.shape, bool)
    bad[0, 130:, 5] = bad[1, 64:, 33] = bad[1, 299:, 69] = True
    assert np.array_equal(np.isnan(y), bad)


@pytest.mark.gpu
def test_continuation_through_final_state():
    d = inputs(2, 333, 100, seed=8, dev="cuda")
    whole, fin, _ = pkg.gated_recurrence_forward(d["x"], d["ga"], d["gx"], d["decay"], c=C)
    state = None
    for lo, hi in ((0, 1), (1, 130), (130, 333)):
        part, state, _ = pkg.gated_recurrence_forward(*(d[k][:, lo:hi] for k in ("x", "ga", "gx")),
                                                      d["decay"], c=C, init_state=state)
        ref.check(to_np(part), to_np(whole[:, lo:hi]), 0.0, f"steps {lo} to {hi}")
    ref.check(to_np(state), to_np(fin), 0.0, "final_state")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bD", [(1, 1), (3, 70), (16, 2048), (7, 333), (129, 1000)], ids=str)
@pytest.mark.parametrize("layout", ["plain", "fused", "odd"])
def test_step(bD, dtype, layout):
    b, D = bD
    d = inputs(b, 1, D, dtype, seed=9, layout=layout, dev="cuda")
    ry, rf, _ = reference(d)
    state = d["init"].clone()
    args = (d["x"][:, 0], d["ga"][:, 0], d["gx"][:, 0], d["decay"])
    out = torch.full_like(state, float("nan"))
    y, new = pkg.gated_recurrence_step(*args, state, c=C, state_out=out)
    assert new.data_ptr() == out.data_ptr() and torch.equal(state, d["init"])
    y2, same = pkg.gated_recurrence_step(*args, state, c=C)
    assert same.data_ptr() == state.data_ptr()
    assert torch.equal(new, same) and torch.equal(y, y2)
    ref.check(to_np(y), ry[:, 0], REL[dtype], "y")
    ref.check(to_np(new), rf, 0.0, "state")


@pytest.mark.gpu
def test_steps_follow_the_scan():
    d = inputs(3, 40, 96, seed=10, dev="cuda")
    y, fin, _ = pkg.gated_recurrence_forward(d["x"], d["ga"], d["gx"], d["decay"], c=C, init_state=d["init"])
    state = d["init"].clone()
    for t in range(40):
        yt, _ = pkg.gated_recurrence_step(d["x"][:, t], d["ga"][:, t], d["gx"][:, t], d["decay"], state, c=C)
        ref.check(to_np(yt), to_np(y[:, t]), 0.0, f"step {t}")
    ref.check(to_np(state), to_np(fin), 0.0, "final_state")


@pytest.mark.gpu
def test_same_bits_every_run_and_on_another_stream():
    d = inputs(3, 3000, 200, "bf16", seed=11, dev="cuda")
    args = (d["x"], d["ga"], d["gx"], d["decay"])
    f0 = pkg.gated_recurrence_forward(*args, c=C, init_state=d["init"], return_states=True)
    g0 = pkg.gated_recurrence_backward(*args, d["dy"], c=C, init_state=d["init"], states=f0[2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, None):
        f = pkg.gated_recurrence_forward(*args, c=C, init_state=d["init"], return_states=True, stream=stream)
        g = pkg.gated_recurrence_backward(*args, d["dy"], c=C, init_state=d["init"], states=f[2],
                                          stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(f, f0))
        assert all(torch.equal(g[k], g0[k]) for k in g0)


@pytest.mark.gpu
def test_replays_in_a_graph():
    """A captured call computes anew at every replay (nothing that the workspace holds from the replay
    before passes for this one's)."""
    d = inputs(1, 2000, 64, seed=12, dev="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan = pkg.GatedRecurrencePlan(d["x"], d["ga"], d["gx"], d["decay"], c=C, init_state=d["init"],
                                   return_states=True, stream=side)
    states = plan.states
    back = pkg.GatedRecurrenceBackwardPlan(d["x"], d["ga"], d["gx"], d["decay"], d["dy"], c=C,
                                           init_state=d["init"], states=states, stream=side)
    with torch.cuda.stream(side):
        plan(), back()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        plan(), back()
    for seed in (13, 14):
        e = inputs(1, 2000, 64, seed=seed, dev="cuda")
        for k in d:
            d[k].copy_(e[k])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref.check(to_np(plan.y), reference(d)[0], 0.0, "y")
        r = reference_grad(d, dfinal=False)
        ref.check(to_np(back.grads["dgate_a"]), r["dgate_a"], 0.0, "dgate_a")


@pytest.mark.gpu
def test_gradient_against_differences_of_the_kernel():
    """Central differences of the fp32 forward.  With steps of 2^-5 the cubic term is 1e-3 of the
    derivative's scale and the fp32 rounding of the loss, a sum of n terms of size one, about
    sqrt(n) 1e-6 / 2^-5."""
    d = inputs(2, 150, 40, seed=15, dev="cuda")
    names = {"x": "dx", "ga": "dgate_a", "gx": "dgate_x", "decay": "ddecay", "init": "dinit"}

    def loss(e):
        y, fin, _ = pkg.gated_recurrence_forward(e["x"], e["ga"], e["gx"], e["decay"], c=C,
                                                 init_state=e["init"])
        return float((y.double() * e["dy"]).sum() + (fin.double() * e["dfinal"]).sum())

    g = pkg.gated_recurrence_backward(d["x"], d["ga"], d["gx"], d["decay"], d["dy"], c=C,
                                      init_state=d["init"], dfinal=d["dfinal"])
    gen = torch.Generator().manual_seed(1)
    for k, gk in names.items():
        v = torch.randn(d[k].shape, generator=gen).cuda()
        eps = 2.0 ** -5
        num = (loss({**d, k: d[k] + eps * v}) - loss({**d, k: d[k] - eps * v})) / (2 * eps)
        size = float((g[gk].double() ** 2).sum().sqrt())   # of the derivative along a random direction
        assert abs(num - float((g[gk].double() * v).sum())) <= 5e-3 * size + 1e-2, k


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """2.2e9 elements (inputs broadcast along the steps): with constant gates h approaches
    m i x / (1 - a), reached within fp32 long before step 2^20 at a <= 0.9999."""
    T, D = 1_100_000, 2048
    d = inputs(1, 1, D, "bf16", seed=16, dev="cuda")
    x, ga, gx = (d[k].expand(1, T, D) for k in ("x", "ga", "gx"))
    y, fin, st = pkg.gated_recurrence_forward(x, ga, gx, d["decay"], c=C, return_states=True)
    torch.cuda.synchronize()
    _, a, m, i, _ = ref.recurrence_coefficients(*(to_np(d[k])[:, 0] for k in ("ga", "gx")),
                                                to_np(d["decay"]), C)
    # the fixed point's relative error is that of a against 1 - a, and h stops moving where a step's
    # change is below half a unit of h: together 2^-24 / (1 - a), doubled
    limit = m * i * to_np(d["x"])[:, 0] / (1 - a)
    near = 2 ** -23 / (1 - a) + 1e-5
    for t in (2 ** 20, T - 1):   # element 2^31 lies at step 2^20
        assert np.all(np.abs(to_np(y[:, t]) - limit) <= (2 ** -8 + near) * np.abs(limit)), t
    assert np.all(np.abs(to_np(fin) - limit) <= near * np.abs(limit))
    assert np.all(np.abs(to_np(st[:, -1]) - limit) <= near * np.abs(limit))


@pytest.mark.gpu
@pytest.mark.parametrize("b,T", [(0, 5), (2, 0)])
def test_empty(b, T):
    D = 6
    z = torch.zeros(b, T, D, device="cuda")
    decay, init = torch.zeros(D, device="cuda"), torch.randn(b, D, device="cuda")
    y, fin, st = pkg.gated_recurrence_forward(z, z, z, decay, init_state=init, return_states=True)
    assert y.shape == (b, T, D) and torch.equal(fin, init) and st.numel() == 0
    assert torch.equal(pkg.gated_recurrence_forward(z, z, z, decay)[1], torch.zeros_like(init))
    g = pkg.gated_recurrence_backward(z, z, z, decay, z, init_state=init, dfinal=init)
    assert torch.equal(g["dinit"], init) and torch.equal(g["ddecay"], torch.zeros_like(decay))


# ------------------------------------------------------------------------------------------------
# refusals
# ------------------------------------------------------------------------------------------------
A16 = 0x100000
_VP = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkg.load_library()


def _shape(**kw):
    d = dict(batch=2, seqlen=10, d_model=8, x_stride=(80, 8), gate_a_stride=(80, 8),
             gate_x_stride=(80, 8), dy_stride=(80, 8), c=8.0, io_dtype=0)
    d.update(kw)
    for k in d:
        if k.endswith("stride"):
            d[k] = (ctypes.c_int64 * 2)(*d[k])
    return pkg.lm_ops.gated_recurrence_shape(**d)


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(seqlen=-1), dict(d_model=0), dict(c=0.0),
                                dict(c=float("inf")), dict(c=float("nan")), dict(io_dtype=2),
                                dict(x_stride=(-1, 8)), dict(gate_x_stride=(8, -8)),
                                dict(batch=1 << 30, seqlen=1 << 30)], ids=str)
def test_invalid_shapes(lib, kw):
    s = _shape(**kw)
    assert lib.gated_recurrence_workspace_bytes(ctypes.byref(s), 0) == 0
    f = lib.gated_recurrence_forward
    assert f(ctypes.byref(s), *[_VP(A16)] * 9, ctypes.c_size_t(1 << 40), None) in (1, 2)


def test_invalid_pointers(lib):
    """Rejected on the host before any launch: none of these pointers is read."""
    s = _shape()
    need = lib.gated_recurrence_workspace_bytes(ctypes.byref(s), 0)
    call = lambda p, n=need: lib.gated_recurrence_forward(   # noqa: E731
        ctypes.byref(s), *(_VP(v) for v in p), ctypes.c_size_t(n), None)
    good = [A16] * 9
    for k in (0, 1, 2, 3):
        assert call([None if j == k else v for j, v in enumerate(good)]) == 1
        assert call([A16 + 2 if j == k else v for j, v in enumerate(good)]) == 1
    assert call(good[:-1] + [None]) == 4
    assert call(good[:-1] + [A16 + 16]) == 4
    assert call(good, need - 1) == 4
    needb = lib.gated_recurrence_workspace_bytes(ctypes.byref(s), 1)
    callb = lambda p, n=needb: lib.gated_recurrence_backward(   # noqa: E731
        ctypes.byref(s), *(_VP(v) for v in p), ctypes.c_size_t(n), None)
    goodb = [A16] * 14
    for k in (0, 3, 6, 8, 9, 10, 11):
        assert callb([None if j == k else v for j, v in enumerate(goodb)]) == 1, k
    assert callb(goodb, needb - 1) == 4
    one = _shape(seqlen=2)
    assert lib.gated_recurrence_step(ctypes.byref(one), *[_VP(A16)] * 7, None) == 1


@pytest.mark.gpu
def test_binding_refuses():
    d = inputs(2, 5, 8, dev="cuda")
    x, ga, gx, decay, dy = (d[k] for k in ("x", "ga", "gx", "decay", "dy"))
    f = pkg.gated_recurrence_forward
    for bad in (lambda: f(x[0], ga, gx, decay), lambda: f(x, ga[:, :4], gx, decay),
                lambda: f(x, ga.bfloat16(), gx, decay), lambda: f(x.half(), ga.half(), gx.half(), decay),
                lambda: f(x, ga, gx, decay.double()), lambda: f(x, ga, gx, decay, c=0.0),
                lambda: f(x, ga, gx, decay, c=float("nan")),
                lambda: f(x.transpose(1, 2).contiguous().transpose(1, 2), ga, gx, decay),
                lambda: f(x, ga, gx, decay, init_state=d["init"][:1]),
                lambda: f(x.cpu(), ga, gx, decay),
                lambda: f(x, ga, gx, decay, y=torch.empty(2, 5, 9, device="cuda")),
                lambda: pkg.gated_recurrence_backward(x, ga, gx, decay, dy[:, :4]),
                lambda: pkg.gated_recurrence_backward(x, ga, gx, decay, dy, states=d["init"]),
                lambda: pkg.gated_recurrence_step(x, ga, gx, decay, d["init"]),
                lambda: pkg.gated_recurrence_step(x[:, 0], ga[:, 0], gx[:, 0], decay, None)):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks host tensors on CPU hosts")
def test_refuses_host_tensors():
    d = inputs(1, 4, 8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pkg.gated_recurrence_forward(d["x"], d["ga"], d["gx"], d["decay"])
    with pytest.raises(ValueError, match="CUDA tensor"):
        pkg.gated_recurrence_backward(d["x"], d["ga"], d["gx"], d["decay"], d["dy"])
    with pytest.raises(ValueError, match="CUDA tensor"):
        pkg.gated_recurrence_step(d["x"][:, 0], d["ga"][:, 0], d["gx"][:, 0], d["decay"], d["init"])
