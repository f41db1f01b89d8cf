"""Root-mean-square norm with the residual's addition and an 8-bit output: the fp64 form against differences (CPU), the
kernels against the fp64 form (GPU), and the refusals."""
import ctypes

import numpy as np
import pytest
import torch

import chunked_ssd_scan_gb300 as pkg
from chunked_ssd_scan_gb300 import _build
from tests import delta_reference as ref
from tests.parity_util import GUARD_FILL, Guarded, to_np

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
# A row's sum of C squares is off by some C 2^-24 at the very most, a few 2^-24 in practice, an output by three more
# operations: 64 of them.
UNIT = 64 * 2.0 ** -24


def check(got, want, rel, what, scale=None):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, what
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    size = np.abs(want) if scale is None else np.maximum(np.abs(want), scale)
    bad = ~(np.isnan(want) | (got == want) | (np.abs(got - want) <= rel * np.abs(want) + UNIT * size))
    assert not bad.any(), (what, int(bad.sum()), got[bad][:3], want[bad][:3])


def inputs(N, C, dtype="f32", seed=0, layout="plain", dev="cpu"):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    d = {k: rnd(N, C) * (2.0 if k == "res" else 1.0) for k in ("x", "res", "dy", "dres")}
    d = {k: v.to(DT[dtype]).to(dev) for k, v in d.items()}
    if layout != "plain":
        off = 1 if layout == "odd" else 0
        flat = torch.cat([torch.zeros(N, off, dtype=DT[dtype], device=dev), *d.values()], 1)
        d = {k: flat[:, off + i * C:off + (i + 1) * C] for i, k in enumerate(d)}
    return d | {"w": (1 + 0.2 * rnd(C)).to(dev)}


def test_reference_gradient_against_differences():
    d = {k: to_np(v) for k, v in inputs(3, 7, seed=1).items()}

    def loss(x, w):
        y, h, _ = ref.rms_norm(x, w, d["res"], 1e-3)
        return (y * d["dy"]).sum() + (h * d["dres"]).sum()

    _, h, rstd = ref.rms_norm(d["x"], d["w"], d["res"], 1e-3)
    g = ref.rms_norm_grad(h, d["dy"], rstd, d["w"], d["dres"])
    rng = np.random.default_rng(0)
    for j, (n, k) in enumerate((("x", "dx"), ("w", "dweight"))):
        way = rng.standard_normal(d[n].shape)
        at = lambda s: loss(*(d[m] + (s * way if i == j else 0) for i, m in enumerate(("x", "w"))))   # noqa: E731
        num = (at(1e-5) - at(-1e-5)) / 2e-5
        assert abs(num - (g[k] * way).sum()) <= 1e-7 * (1 + abs(num)), n


def test_reference_rounds_to_8_bits_as_torch_does():
    v = torch.linspace(-460, 460, 20001).clamp(-448, 448)
    small = torch.linspace(-0.05, 0.05, 20001)
    for t in (v, small):
        assert np.array_equal(ref.e4m3(to_np(t)), to_np(t.to(torch.float8_e4m3fn).float()))


# one channel, odd widths, the widths at which vectors and threads change, wider than the registers hold
SHAPES = [(1, 1), (3, 7), (5, 64), (2, 127), (9, 128), (300, 130), (4, 257), (17, 1000), (1000, 2048), (2, 4096), (3, 5120),
          (2, 8200), (5, 9001), (2, 16384), (1, 40000), (70000, 8), (2500, 520), (2, 33001)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["plain", "fused", "odd"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, layout, dtype):
    N, C = shape
    d = inputs(N, C, dtype, seed=2, layout=layout, dev="cuda")
    e = d["x"].element_size()
    for res in (None, d["res"]):
        out = {"y": Guarded(N * C * e, "cuda", GUARD_FILL), "h": Guarded(N * C * e, "cuda", GUARD_FILL),
               "rstd": Guarded(N * 4, "cuda", GUARD_FILL)}
        y, h, rstd, scale = pkg.rms_norm_forward(
            d["x"], d["w"], residual=res, y=out["y"].view(DT[dtype], (N, C)),
            h=None if res is None else out["h"].view(DT[dtype], (N, C)), rstd=out["rstd"].view(torch.float32, (N,)))
        torch.cuda.synchronize()
        for k, v in out.items():
            v.check(k)
        assert scale is None and (h is None) == (res is None)
        ry, rh, rr = ref.rms_norm(to_np(d["x"]), to_np(d["w"]), None if res is None else to_np(res))
        check(to_np(rstd), rr, 0, "rstd")
        check(to_np(y), ry, ref.BF16_REL if dtype == "bf16" else 0, "y")
        if res is not None:
            assert torch.equal(h, (d["x"].float() + res.float()).to(DT[dtype]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("quantize", ["token", "block"])
@pytest.mark.parametrize("layout", ["plain", "odd"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_8_bits(shape, layout, quantize, dtype):
    N, C = shape
    d = inputs(N, C, dtype, seed=3, layout=layout, dev="cuda")
    d["x"][0] *= 1000
    wide = C if quantize == "token" else 128
    blocks = -(-C // wide)
    out = {"y": Guarded(N * C, "cuda", GUARD_FILL), "scale": Guarded(N * blocks * 4, "cuda", GUARD_FILL)}
    y, h, rstd, scale = pkg.rms_norm_forward(
        d["x"], d["w"], residual=d["res"], quantize=quantize, y=out["y"].view(torch.float8_e4m3fn, (N, C)),
        scale=out["scale"].view(torch.float32, (N, blocks)))
    torch.cuda.synchronize()
    for k, v in out.items():
        v.check(k)
    assert torch.equal(h, (d["x"].float() + d["res"].float()).to(DT[dtype]))
    ry, _, _ = ref.rms_norm(to_np(d["x"]), to_np(d["w"]), to_np(d["res"]))
    padded = np.pad(ry, ((0, 0), (0, blocks * wide - C))).reshape(N, blocks, wide)
    most = np.abs(padded).max(2)
    check(to_np(scale), np.where(most > 0, most / 448, 1.0), 0, "scale")
    # against the kernel's own scale: within half a step of 8 bits (2^-4 of a value, 2^-10 where they are subnormal)
    each = np.repeat(to_np(scale), wide, 1)[:, :C]
    got = to_np(y.float()) * each
    assert (np.abs(got - ry) <= (2.0 ** -4 * np.abs(ry) + 2.0 ** -10 * each) * (1 + 1e-4)).all()
    # and the nearest value but where the quotient lies within fp32's error of a border between two
    same = got == ref.e4m3(ry / each) * each
    assert same.mean() >= 1 - 1e-4 - 2.0 / same.size, same.mean()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["plain", "fused", "odd"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, layout, dtype):
    N, C = shape
    d = inputs(N, C, dtype, seed=4, layout=layout, dev="cuda")
    e = d["x"].element_size()
    rstd = pkg.rms_norm_forward(d["x"], d["w"])[2]
    for dres in (None, d["dres"]):
        out = {"dx": Guarded(N * C * e, "cuda", GUARD_FILL), "dweight": Guarded(C * 4, "cuda", GUARD_FILL)}
        plan = pkg.RMSNormBackwardPlan(d["x"], d["dy"], rstd, d["w"], dresidual=dres,
                                       grads={"dx": out["dx"].view(DT[dtype], (N, C)),
                                              "dweight": out["dweight"].view(torch.float32, (C,))})
        g = plan()
        assert pkg.workspace_status(plan.workspace) == ("SSD_OK", 0)
        for k, v in out.items():
            v.check(k)
        want = ref.rms_norm_grad(to_np(d["x"]), to_np(d["dy"]), to_np(rstd), to_np(d["w"]),
                                 None if dres is None else to_np(dres))
        # differences of terms of the size rstd |w dy|, and sums of N terms of size one
        size = to_np(rstd)[:, None] * (1 + np.abs(to_np(d["dy"]) * to_np(d["w"])))
        check(to_np(g["dx"]), want["dx"], ref.BF16_REL if dtype == "bf16" else 0, "dx", size)
        check(to_np(g["dweight"]), want["dweight"], 0, "dweight", np.sqrt(N))
        again = pkg.rms_norm_backward(d["x"], d["dy"], rstd, d["w"], dresidual=dres)
        assert all(torch.equal(again[k], g[k]) for k in g)
    assert pkg.rms_norm_backward(d["x"], d["dy"], rstd, param_grads=False)["dweight"] is None


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_axes_without_weight_and_in_place(dtype):
    d = inputs(24, 40, dtype, seed=5, dev="cuda")
    x, res = (d[k].view(2, 3, 4, 40) for k in ("x", "res"))
    want = ref.rms_norm(to_np(x), None, to_np(res))
    kept = res.clone()
    y, h, rstd, _ = pkg.rms_norm_forward(x, residual=res, h=res)   # the sum takes the residual's place
    assert h is res and rstd.shape == (2, 3, 4)
    assert torch.equal(res, (x.float() + kept.float()).to(DT[dtype]))
    check(to_np(y), want[0], ref.BF16_REL if dtype == "bf16" else 0, "y")
    q, _, _, scale = pkg.rms_norm_forward(x, quantize="block")
    assert q.dtype == torch.float8_e4m3fn and scale.shape == (2, 3, 4, 1)
    g = pkg.rms_norm_backward(x, y, rstd)
    assert g["dx"].shape == x.shape and g["dweight"].shape == (40,)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [64, 130, 2048, 33001])
def test_rows_of_zeros_and_bad_values(C, dtype):
    d = inputs(6, C, dtype, seed=6, dev="cuda")
    x = d["x"]
    x[1] = 0
    x[3, C // 2] = float("nan")
    x[4, 0] = float("inf")
    clean = [0, 2, 5]
    for quantize in (None, "token", "block"):
        y, _, rstd, scale = pkg.rms_norm_forward(x, d["w"], quantize=quantize)
        y = y.float()
        assert bool((y[1] == 0).all()) and bool(torch.isfinite(y[clean]).all())
        assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(rstd[3]))
        if scale is not None:
            assert bool((scale[1] == 1).all()) and bool(torch.isfinite(scale[clean]).all())
        alone = pkg.rms_norm_forward(x[5:], d["w"], quantize=quantize)
        assert torch.equal(alone[0].float()[0], y[5])


@pytest.mark.gpu
def test_another_stream_a_graph_and_no_rows():
    d = inputs(500, 1032, "bf16", seed=7, dev="cuda")
    want = pkg.rms_norm_forward(d["x"], d["w"], residual=d["res"], quantize="token")
    gw = pkg.rms_norm_backward(want[1], d["dy"], want[2], d["w"], dresidual=d["dres"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    f = pkg.RMSNormPlan(d["x"], d["w"], residual=d["res"], quantize="token", stream=side)
    b = pkg.RMSNormBackwardPlan(f.h, d["dy"], f.rstd, d["w"], dresidual=d["dres"], stream=side)
    with torch.cuda.stream(side):
        f(), b()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        f(), b()
    b.grads["dweight"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(f.y.float(), want[0].float()) and all(torch.equal(b.grads[k], gw[k]) for k in gw)
    x = torch.zeros(0, 16, device="cuda")
    y, h, rstd, scale = pkg.rms_norm_forward(x, quantize="block")
    assert y.shape == (0, 16) and rstd.shape == (0,) and scale.shape == (0, 1)
    assert torch.equal(pkg.rms_norm_backward(x, x, rstd)["dweight"], torch.zeros(16, device="cuda"))


@pytest.mark.gpu
def test_offsets_past_31_bits():
    N, C = (1 << 31) // 2048 + 3, 2048
    row = torch.randn(1, C, generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    y, _, rstd, _ = pkg.rms_norm_forward(row.expand(N, C))
    one = pkg.rms_norm_forward(row)
    for at in (0, N // 2, N - 1):
        assert torch.equal(y[at], one[0][0])
    assert bool((rstd == rstd[0]).all())


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkg.load_library()


A16 = 0x100000
_VP = ctypes.c_void_p


def shape_of(N=4, C=64, io=0, quantize=0, **kw):
    s = pkg.lm_ops.rms_norm_shape(N, C, C, C, C, 1e-6, quantize, io)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


@pytest.mark.parametrize("change", [dict(rows=-1), dict(channels=0), dict(x_stride=-1), dict(res_stride=-1),
                                    dict(eps=-1.0), dict(eps=float("nan")), dict(io_dtype=5), dict(quantize=3)], ids=str)
def test_bad_shapes(lib, change):
    s = shape_of(**change)
    assert lib.rms_norm_forward(ctypes.byref(s), *[_VP(A16)] * 7, None) == 1
    if "quantize" not in change:
        assert lib.rms_norm_workspace_bytes(ctypes.byref(s)) == 0


def test_bad_pointers_and_workspaces(lib):
    s, good = shape_of(quantize=1), [_VP(A16)] * 7
    for i in (0, 3, 6):   # x, y, scale
        assert lib.rms_norm_forward(ctypes.byref(s), *good[:i], None, *good[i + 1:], None) == 1
    for i in (0, 1, 2, 4, 5, 6):
        assert lib.rms_norm_forward(ctypes.byref(s), *good[:i], _VP(A16 + 1), *good[i + 1:], None) == 1
    s, back = shape_of(), lib.rms_norm_backward
    for i in (0, 1, 2, 5):   # h, dy, rstd, dx
        assert back(ctypes.byref(s), *good[:i], None, *good[i + 1:], _VP(A16), 1 << 40, None) == 1
    for i in range(7):
        assert back(ctypes.byref(s), *good[:i], _VP(A16 + 1), *good[i + 1:], _VP(A16), 1 << 40, None) == 1
    need = lib.rms_norm_workspace_bytes(ctypes.byref(s))
    assert back(ctypes.byref(s), *good, _VP(A16), need - 1, None) == 4
    assert back(ctypes.byref(s), *good, None, need, None) == 4


@pytest.mark.gpu
def test_refusals_of_the_binding():
    d = inputs(4, 16, dev="cuda")
    for bad in (dict(quantize="row"), dict(eps=-1.0), dict(residual=d["res"][:3]), dict(residual=d["res"].bfloat16()),
                dict(scale=torch.zeros(4, 1, device="cuda"))):
        with pytest.raises(ValueError):
            pkg.rms_norm_forward(d["x"], d["w"], **bad)
    with pytest.raises(ValueError):
        pkg.rms_norm_forward(d["x"].half(), d["w"])
    with pytest.raises(ValueError):
        pkg.rms_norm_forward(d["x"], d["w"][:8])
    with pytest.raises(ValueError):
        pkg.rms_norm_forward(d["x"].t())
    with pytest.raises(ValueError):
        pkg.rms_norm_backward(d["x"], d["dy"][:2], torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        pkg.rms_norm_backward(d["x"], d["dy"], torch.ones(3, device="cuda"))
