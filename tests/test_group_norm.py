"""Channels-last group norm with an activation: the fp64 form against differences (CPU), the kernels
against the fp64 form (GPU), and the refusals."""
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


def inputs(N, S, C, dtype="f32", seed=0, layout="plain", dev="cpu", mean=0.5):
    """x, dy [N,S,C] (separate, slices of one wider buffer, or slices that start at an odd element),
    weight, bias."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    d = {"w": 1 + 0.2 * rnd(C), "bias": 0.2 * rnd(C)}
    x, dy = 1.5 * rnd(N, S, C) + mean * rnd(C), rnd(N, S, C)
    if layout == "plain":
        d.update(x=x.to(DT[dtype]).to(dev), dy=dy.to(DT[dtype]).to(dev))
    else:
        off = 1 if layout == "odd" else 0
        p = torch.cat((torch.zeros(N, S, off), x, dy), 2).to(DT[dtype]).to(dev)
        d.update(x=p[..., off:off + C], dy=p[..., off + C:])
    d["w"], d["bias"] = d["w"].to(dev), d["bias"].to(dev)
    return d


def test_reference_gradient_against_differences():
    d = {k: to_np(v) for k, v in inputs(2, 3, 12, seed=1).items()}
    g = ref.group_norm_grad(d["x"], d["dy"], 4, d["w"], d["bias"])
    loss = lambda x, w, b: (ref.group_norm(x, 4, w, b)[0] * d["dy"]).sum()   # noqa: E731
    rng = np.random.default_rng(0)
    for j, (k, gk) in enumerate((("x", "dx"), ("w", "dweight"), ("bias", "dbias"))):
        v = rng.standard_normal(d[k].shape)
        at = lambda s: loss(*(d[n] + (s * v if m == j else 0) for m, n in enumerate(("x", "w", "bias"))))  # noqa: E731
        num = (at(1e-5) - at(-1e-5)) / 2e-5
        assert abs(num - (g[gk] * v).sum()) <= 1e-7 * (1 + abs(num)), k


# N, S, C, G: tokens (S = 1) and maps, one value a group, odd group widths, groups wider than a block,
# one channel a group over many positions
SHAPES = [(1, 1, 1, 1), (5, 1, 64, 1), (7, 1, 96, 12), (300, 1, 2048, 32), (3, 1, 2560, 1),
          (2, 1, 5000, 1), (9, 1, 130, 13), (4, 1, 300, 10), (3, 1, 40, 40), (2, 1, 20000, 1),
          (1, 7, 8, 2), (2, 100, 48, 4), (2, 1000, 320, 32), (1, 4097, 24, 3), (3, 64, 66, 11),
          (1, 30000, 16, 2), (2, 3, 20000, 1), (40, 16, 64, 8), (1, 2, 1, 1), (2, 333, 7, 7),
          (1, 9000, 512, 4)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["plain", "fused", "odd"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dtype, layout):
    N, S, C, G = shape
    act = "silu" if (N + S) % 2 else None
    d = inputs(N, S, C, dtype, seed=2, layout=layout, dev="cuda")
    out = {"y": Guarded(N * S * C * d["x"].element_size(), "cuda", GUARD_FILL),
           "mean": Guarded(N * G * 4, "cuda", GUARD_FILL), "rstd": Guarded(N * G * 4, "cuda", GUARD_FILL)}
    plan = pkg.GroupNormPlan(d["x"], G, d["w"], d["bias"], activation=act,
                             y=out["y"].view(DT[dtype], (N, S, C)),
                             mean=out["mean"].view(torch.float32, (N, G)),
                             rstd=out["rstd"].view(torch.float32, (N, G)))
    y, mean, rstd = plan()
    assert pkg.workspace_status(plan.workspace) == ("SSD_OK", 0)
    for k, v in out.items():
        v.check(k)
    ry, rm, rr = ref.group_norm(to_np(d["x"]), G, to_np(d["w"]), to_np(d["bias"]), act=act)
    ref.check(to_np(mean), rm, 0.0, "mean", scale=1.0)
    ref.check(to_np(rstd), rr, 0.0, "rstd")
    ref.check(to_np(y), ry, REL[dtype], "y")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["plain", "fused", "odd"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, dtype, layout):
    N, S, C, G = shape
    act = None if (N + S) % 2 else "silu"
    d = inputs(N, S, C, dtype, seed=3, layout=layout, dev="cuda")
    out = {"dx": Guarded(N * S * C * d["x"].element_size(), "cuda", GUARD_FILL),
           "dweight": Guarded(C * 4, "cuda", GUARD_FILL), "dbias": Guarded(C * 4, "cuda", GUARD_FILL)}
    grads = {"dx": out["dx"].view(DT[dtype], (N, S, C)), "dweight": out["dweight"].view(torch.float32, (C,)),
             "dbias": out["dbias"].view(torch.float32, (C,))}
    _, mean, rstd = pkg.group_norm_forward(d["x"], G, d["w"], d["bias"], activation=act)
    plan = pkg.GroupNormBackwardPlan(d["x"], d["dy"], G, mean, rstd, d["w"], d["bias"], activation=act,
                                     grads=grads)
    g = plan()
    assert pkg.workspace_status(plan.workspace) == ("SSD_OK", 0)
    for k, v in out.items():
        v.check(k)
    r = ref.group_norm_grad(to_np(d["x"]), to_np(d["dy"]), G, to_np(d["w"]), to_np(d["bias"]), act=act)
    # dx is a difference of terms of the size rstd |dy w| (a group of one value: exactly zero)
    size = np.abs(to_np(rstd)).mean() * 1.5
    ref.check(to_np(g["dx"]), r["dx"], REL[dtype], "dx", scale=np.maximum(np.abs(r["dx"]), size))
    for k in ("dweight", "dbias"):   # a sum of N S terms of about size one
        ref.check(to_np(g[k]), r[k], 0.0, k, scale=np.abs(r[k]) + np.sqrt(N * S))


@pytest.mark.gpu
def test_without_weight_and_bias_and_in_more_axes():
    g = torch.Generator().manual_seed(4)
    x, dy = (torch.randn(2, 5, 6, 24, generator=g).cuda() for _ in range(2))
    y, mean, rstd = pkg.group_norm_forward(x, 3)
    xr, dyr = (to_np(t).reshape(2, 30, 24) for t in (x, dy))
    ref.check(to_np(y).reshape(2, 30, 24), ref.group_norm(xr, 3)[0], 0.0, "y")
    gr = pkg.group_norm_backward(x, dy, 3, mean, rstd)
    r = ref.group_norm_grad(xr, dyr, 3)
    ref.check(to_np(gr["dx"]).reshape(2, 30, 24), r["dx"], 0.0, "dx")
    ref.check(to_np(gr["dweight"]), r["dweight"], 0.0, "dweight")
    gr = pkg.group_norm_backward(x, dy, 3, mean, rstd, param_grads=False)
    assert gr["dweight"] is None and gr["dbias"] is None
    ref.check(to_np(gr["dx"]).reshape(2, 30, 24), r["dx"], 0.0, "dx")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(4, 1, 512, 8), (2, 700, 64, 8), (1, 40000, 32, 2)], ids=str)
def test_variance_around_a_large_mean(shape):
    """mean 1000, deviation 1: E[x^2] - mean^2 would lose 6 of fp32's 7 digits.  Around the mean, what
    remains is the mean's own rounding, 1000 * 2^-24 = 6e-5 of a deviation."""
    N, S, C, G = shape
    g = torch.Generator().manual_seed(5)
    x = (1000 + torch.randn(N, S, C, generator=g)).cuda()
    y, mean, rstd = pkg.group_norm_forward(x, G, activation=None)
    ry, rm, rr = ref.group_norm(to_np(x), G, act=None)
    ref.check(to_np(rstd), rr, 0.0, "rstd")
    assert np.abs(to_np(y) - ry).max() <= 2.5e-4   # four of the mean's rounding units, and z's own


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(4, 1, 512, 8), (2, 300, 64, 8)], ids=str)
def test_constant_groups_and_zero_variance(shape):
    N, S, C, G = shape
    x = torch.full((N, S, C), 3.0, device="cuda")
    bias = torch.randn(C, generator=torch.Generator().manual_seed(6)).cuda()
    y, mean, rstd = pkg.group_norm_forward(x, G, None, bias, eps=1e-4)
    assert torch.equal(mean, torch.full_like(mean, 3.0))
    assert torch.allclose(rstd, torch.full_like(rstd, 100.0), rtol=1e-6)
    ref.check(to_np(y), np.broadcast_to(to_np(torch.nn.functional.silu(bias.double())), y.shape), 0.0, "y")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(4, 1, 512, 8), (2, 300, 64, 8), (3, 5000, 24, 3)], ids=str)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_bad_values_stay_in_their_group(shape, value):
    N, S, C, G = shape
    d = inputs(N, S, C, seed=7, dev="cuda")
    x = d["x"].clone()
    x[1, S // 2, C // G + 1] = value   # sample 1, group 1
    y, mean, rstd = pkg.group_norm_forward(x, G, d["w"], d["bias"])
    bad = torch.zeros(N, S, C, dtype=torch.bool, device="cuda")
    bad[1, :, C // G:2 * C // G] = True
    assert bool(torch.isnan(y[bad]).any()) and bool(torch.isfinite(y[~bad]).all())
    clean = pkg.group_norm_forward(d["x"], G, d["w"], d["bias"])
    assert torch.equal(y[~bad], clean[0][~bad])
    g = pkg.group_norm_backward(x, d["dy"], G, mean, rstd, d["w"], d["bias"])
    assert bool(torch.isfinite(g["dx"][~bad]).all())
    ch = torch.zeros(C, dtype=torch.bool, device="cuda")
    ch[C // G:2 * C // G] = True
    assert bool(torch.isfinite(g["dweight"][~ch]).all()) and bool(torch.isfinite(g["dbias"][~ch]).all())


@pytest.mark.gpu
def test_saturated_activation():
    """silu far from zero: z on the right, 0 on the left, and gradients 1 and 0, no NaN."""
    x = torch.randn(6, 64, generator=torch.Generator().manual_seed(8)).cuda()
    for b in (300.0, -300.0):
        bias = torch.full((64,), b, device="cuda")
        y, mean, rstd = pkg.group_norm_forward(x, 4, None, bias)
        ry = ref.group_norm(to_np(x)[:, None], 4, None, to_np(bias))[0][:, 0]
        ref.check(to_np(y), ry, 0.0, "y", scale=1.0)
        g = pkg.group_norm_backward(x, torch.ones_like(x), 4, mean, rstd, None, bias)
        r = ref.group_norm_grad(to_np(x)[:, None], np.ones((6, 1, 64)), 4, None, to_np(bias))
        ref.check(to_np(g["dbias"]), r["dbias"], 0.0, "dbias", scale=1.0)
        assert torch.isfinite(g["dx"]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(700, 1, 512, 8), (3, 900, 96, 8), (2, 30000, 64, 4)], ids=str)
def test_same_bits_every_run_and_on_another_stream(shape):
    N, S, C, G = shape
    d = inputs(N, S, C, "bf16", seed=9, dev="cuda")
    f0 = pkg.group_norm_forward(d["x"], G, d["w"], d["bias"])
    g0 = pkg.group_norm_backward(d["x"], d["dy"], G, *f0[1:], d["w"], d["bias"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, None):
        f = pkg.group_norm_forward(d["x"], G, d["w"], d["bias"], stream=stream)
        g = pkg.group_norm_backward(d["x"], d["dy"], G, *f[1:], d["w"], d["bias"], stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(f, f0))
        assert all(torch.equal(g[k], g0[k]) for k in g0)


@pytest.mark.gpu
def test_replays_in_a_graph():
    d = inputs(2, 5000, 64, seed=10, dev="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan = pkg.GroupNormPlan(d["x"], 8, d["w"], d["bias"], stream=side)
    back = pkg.GroupNormBackwardPlan(d["x"], d["dy"], 8, plan.mean, plan.rstd, d["w"], d["bias"], stream=side)
    with torch.cuda.stream(side):
        plan(), back()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        plan(), back()
    for seed in (11, 12):
        e = inputs(2, 5000, 64, seed=seed, dev="cuda")
        for k in d:
            d[k].copy_(e[k])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        x, dy, w, b = (to_np(d[k]) for k in ("x", "dy", "w", "bias"))
        ref.check(to_np(plan.y), ref.group_norm(x, 8, w, b)[0], 0.0, "y")
        r = ref.group_norm_grad(x, dy, 8, w, b)
        ref.check(to_np(back.grads["dx"]), r["dx"], 0.0, "dx")
        ref.check(to_np(back.grads["dweight"]), r["dweight"], 0.0, "dweight", scale=100.0)


@pytest.mark.gpu
def test_gradient_against_differences_of_the_kernel():
    """Central differences of the fp32 forward, steps of 2^-6: the cubic term is some 1e-3 of the
    derivative, the rounding of the loss some 1e-5 / 2^-6."""
    d = inputs(3, 20, 48, seed=13, dev="cuda")
    loss = lambda e: float((pkg.group_norm_forward(e["x"], 6, e["w"], e["bias"])[0].double()  # noqa: E731
                            * d["dy"]).sum())
    _, mean, rstd = pkg.group_norm_forward(d["x"], 6, d["w"], d["bias"])
    g = pkg.group_norm_backward(d["x"], d["dy"], 6, mean, rstd, d["w"], d["bias"])
    gen = torch.Generator().manual_seed(2)
    for k, gk in (("x", "dx"), ("w", "dweight"), ("bias", "dbias")):
        v, eps = torch.randn(d[k].shape, generator=gen).cuda(), 2.0 ** -6
        num = (loss({**d, k: d[k] + eps * v}) - loss({**d, k: d[k] - eps * v})) / (2 * eps)
        size = float((g[gk].double() ** 2).sum().sqrt())
        assert abs(num - float((g[gk].double() * v).sum())) <= 5e-3 * size + 1e-2, k


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2_200_000, 1, 1024, 16), (1, 34_000_000, 64, 8)], ids=str)
def test_offsets_beyond_32_bits(shape):
    """2.2e9 elements, the input broadcast along samples or positions: every row of y is the first."""
    N, S, C, G = shape
    row = torch.randn(1, 1, C, generator=torch.Generator().manual_seed(14)).bfloat16().cuda()
    y, mean, rstd = pkg.group_norm_forward(row.expand(N, S, C), G)
    ry = ref.group_norm(to_np(row), G)[0][0, 0]
    flat = y.view(-1, C)
    for at in (0, 2 ** 31 // C, flat.shape[0] - 1):
        ref.check(to_np(flat[at]), ry, REL["bf16"], f"row {at}")


@pytest.mark.gpu
def test_empty():
    w = torch.ones(8, device="cuda")
    for N, S in ((0, 3), (2, 0)):
        x = torch.zeros(N, S, 8, device="cuda")
        y, mean, rstd = pkg.group_norm_forward(x, 2, w)
        assert y.shape == x.shape
        g = pkg.group_norm_backward(x, x, 2, mean, rstd, w)
        assert torch.equal(g["dweight"], torch.zeros_like(w)) and torch.equal(g["dbias"], torch.zeros_like(w))


# tokens in groups that no wide vector divides, rows that start on 16 bytes: one row and many, a tile that is
# not full, several tiles, groups of a vector and of a block's width, two values past a vector
ODD = [(300, 520, 40), (1, 24, 3), (7, 104, 8), (1300, 104, 8), (1000, 1000, 8), (5, 4040, 40), (60, 4040, 40),
       (9, 2040, 8), (100, 2040, 8), (80, 2080, 32), (2000, 72, 4), (901, 160, 16), (4000, 1560, 40)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", None])
@pytest.mark.parametrize("shape", ODD, ids=str)
def test_tokens_in_groups_of_odd_width(shape, act, dtype):
    N, C, G = shape
    d = inputs(N, 1, C, dtype, seed=15, layout="fused", dev="cuda")
    out = {"y": Guarded(N * C * d["x"].element_size(), "cuda", GUARD_FILL),
           "dx": Guarded(N * C * d["x"].element_size(), "cuda", GUARD_FILL)}
    y, mean, rstd = pkg.group_norm_forward(d["x"], G, d["w"], d["bias"], activation=act,
                                           y=out["y"].view(DT[dtype], (N, 1, C)))
    plan = pkg.GroupNormBackwardPlan(d["x"], d["dy"], G, mean, rstd, d["w"], d["bias"], activation=act,
                                     grads={"dx": out["dx"].view(DT[dtype], (N, 1, C))})
    g = plan()
    assert pkg.workspace_status(plan.workspace) == ("SSD_OK", 0)
    for k, v in out.items():
        v.check(k)
    x, dy, w, b = (to_np(d[k]) for k in ("x", "dy", "w", "bias"))
    ry, rm, rr = ref.group_norm(x, G, w, b, act=act)
    ref.check(to_np(mean), rm, 0.0, "mean", scale=1.0)
    ref.check(to_np(rstd), rr, 0.0, "rstd")
    ref.check(to_np(y), ry, REL[dtype], "y")
    r = ref.group_norm_grad(x, dy, G, w, b, act=act)
    size = np.abs(to_np(rstd)).mean() * 1.5
    ref.check(to_np(g["dx"]), r["dx"], REL[dtype], "dx", scale=np.maximum(np.abs(r["dx"]), size))
    for k in ("dweight", "dbias"):
        ref.check(to_np(g[k]), r[k], 0.0, k, scale=np.abs(r[k]) + np.sqrt(N))
    again = pkg.group_norm_backward(d["x"], d["dy"], G, mean, rstd, d["w"], d["bias"], activation=act)
    assert all(torch.equal(again[k], g[k]) for k in g)


@pytest.mark.gpu
def test_bad_values_stay_in_their_odd_group():
    """Neighbouring groups share a thread's vector: a NaN of one must not reach the other."""
    d = inputs(300, 1, 520, seed=16, dev="cuda")
    x = d["x"].clone()
    x[2, 0, 13] = float("nan")   # the first value of group 1, in a vector with the last of group 0
    x[4, 0, 25] = float("inf")   # its last
    y, mean, rstd = pkg.group_norm_forward(x, 40, d["w"], d["bias"])
    g = pkg.group_norm_backward(x, d["dy"], 40, mean, rstd, d["w"], d["bias"])
    clean = pkg.group_norm_forward(d["x"], 40, d["w"], d["bias"])
    bad = torch.zeros(300, 1, 520, dtype=torch.bool, device="cuda")
    bad[2, 0, 13:26] = bad[4, 0, 13:26] = True
    assert torch.equal(y[~bad], clean[0][~bad]) and bool(torch.isnan(y[2, 0, 13:26]).all())
    assert bool(torch.isfinite(g["dx"][~bad]).all())
    ch = torch.zeros(520, dtype=torch.bool, device="cuda")
    ch[13:26] = True
    assert bool(torch.isfinite(g["dweight"][~ch]).all()) and bool(torch.isfinite(g["dbias"][~ch]).all())


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
    d = dict(batch=2, rows=3, channels=8, groups=2, x_stride=(24, 8), dy_stride=(24, 8), eps=1e-5,
             activation=1, io_dtype=0)
    d.update(kw)
    for k in ("x_stride", "dy_stride"):
        d[k] = (ctypes.c_int64 * 2)(*d[k])
    return pkg.lm_ops.group_norm_shape(**d)


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(rows=-1), dict(channels=0), dict(groups=0),
                                dict(groups=3), dict(eps=-1.0), dict(eps=float("nan")),
                                dict(activation=2), dict(io_dtype=5), dict(x_stride=(24, -8)),
                                dict(batch=1 << 31), dict(rows=1 << 40)], ids=str)
def test_invalid_shapes(lib, kw):
    s = _shape(**kw)
    assert lib.group_norm_workspace_bytes(ctypes.byref(s), 0) == 0
    assert lib.group_norm_forward(ctypes.byref(s), *[_VP(A16)] * 7, ctypes.c_size_t(1 << 40), None) in (1, 2)
    assert lib.group_norm_backward(ctypes.byref(s), *[_VP(A16)] * 10, ctypes.c_size_t(1 << 40), None) in (1, 2)


def test_invalid_pointers(lib):
    """Rejected on the host before any launch: none of these pointers is read."""
    s = _shape()
    need, needb = (lib.group_norm_workspace_bytes(ctypes.byref(s), k) for k in (0, 1))
    call = lambda p, n=need: lib.group_norm_forward(   # noqa: E731
        ctypes.byref(s), *(_VP(v) for v in p), ctypes.c_size_t(n), None)
    good = [A16] * 7
    for k in (0, 3, 4, 5):   # x, y, and one of mean and rstd without the other
        assert call([None if j == k else v for j, v in enumerate(good)]) == 1
    for k in range(6):
        assert call([A16 + 2 if j == k else v for j, v in enumerate(good)]) == 1
    assert call(good[:-1] + [None]) == 4 and call(good[:-1] + [A16 + 8]) == 4 and call(good, need - 1) == 4
    callb = lambda p, n=needb: lib.group_norm_backward(   # noqa: E731
        ctypes.byref(s), *(_VP(v) for v in p), ctypes.c_size_t(n), None)
    goodb = [A16] * 10
    for k in (0, 1, 2, 3, 6):
        assert callb([None if j == k else v for j, v in enumerate(goodb)]) == 1
    assert callb(goodb, needb - 1) == 4


@pytest.mark.gpu
def test_binding_refuses():
    x, w = torch.randn(2, 3, 8, device="cuda"), torch.ones(8, device="cuda")
    f = pkg.group_norm_forward
    st = torch.zeros(2, 2, device="cuda")
    for bad in (lambda: f(x, 3), lambda: f(x, 0), lambda: f(x.half(), 2), lambda: f(x, 2, w[:4]),
                lambda: f(x, 2, w.bfloat16()), lambda: f(x, 2, activation="tanh"),
                lambda: f(x, 2, eps=-1.0), lambda: f(x[0, 0], 2), lambda: f(x.transpose(1, 2), 3),
                lambda: f(x.cpu(), 2), lambda: f(x[:, :, None].expand(2, 3, 4, 8), 2),
                lambda: pkg.group_norm_backward(x, x[:, :2], 2, st, st),
                lambda: pkg.group_norm_backward(x, x.bfloat16(), 2, st, st),
                lambda: pkg.group_norm_backward(x, x, 2, st, st[:1])):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks host tensors on CPU hosts")
def test_refuses_host_tensors():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pkg.group_norm_forward(x, 2)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pkg.group_norm_backward(x, x, 2, torch.zeros(2, 2), torch.zeros(2, 2))
