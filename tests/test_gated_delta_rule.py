"""Gated delta rule: the fp64 form against differences (CPU), the kernels against the fp64 form (GPU), and the
refusals."""
import ctypes

import numpy as np
import pytest
import torch

import chunked_ssd_scan_gb300 as pkg
from chunked_ssd_scan_gb300 import _build
from tests import delta_reference as ref
from tests.parity_util import GUARD_FILL, Guarded, to_np

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(b, T, Hk, H, K, V, dtype="f32", seed=0, layout="plain", dev="cpu", slow=20.0):
    """q, k of about unit length, v, dy; one projection's slices (layout "fused"), such that start at an odd element
    ("odd"), or the steps before the batch ("time")."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)   # noqa: E731
    q, k = (torch.nn.functional.normalize(rnd(b, T, Hk, K) + 0.3 * rnd(Hk, K), dim=-1) for _ in range(2))
    v, dy = rnd(b, T, H, V), rnd(b, T, H, V)
    q, k, v, dy = (t.to(DT[dtype]).to(dev) for t in (q, k, v, dy))
    if layout in ("fused", "odd"):
        off = 1 if layout == "odd" else 0
        flat = torch.cat([torch.zeros(b, T, off, dtype=DT[dtype], device=dev)]
                         + [t.reshape(b, T, -1) for t in (q, k, v, dy)], 2)
        at, out = off, []
        for t in (q, k, v, dy):
            n = t.shape[2] * t.shape[3]
            out.append(flat[..., at:at + n].unflatten(2, t.shape[2:]))
            at += n
        q, k, v, dy = out
    elif layout == "time":
        q, k, v, dy = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v, dy))
    d = {"q": q, "k": k, "v": v, "dy": dy,
         "g": (-torch.nn.functional.softplus(rnd(b, T, H)) / slow).to(dev), "beta": torch.sigmoid(rnd(b, T, H)).to(dev),
         "init": (0.3 * rnd(b, H, V, K)).to(dev), "dfinal": (0.3 * rnd(b, H, V, K)).to(dev)}
    return d


def args(d):
    return tuple(d[k] for k in ("q", "k", "v", "g", "beta"))


def host(d):
    return {k: None if v is None else to_np(v) for k, v in d.items()}


def test_reference_gradient_against_differences():
    d = host(inputs(2, 7, 2, 4, 5, 3, seed=1))
    g = ref.delta_grad(*(d[k] for k in ("q", "k", "v", "g", "beta", "dy", "init")), dfinal=d["dfinal"])
    names = ("q", "k", "v", "g", "beta", "init")

    def loss(*a):
        y, final, _ = ref.delta(*a)
        return (y * d["dy"]).sum() + (final * d["dfinal"]).sum()

    rng = np.random.default_rng(0)
    for j, n in enumerate(names):
        way = rng.standard_normal(d[n].shape)
        at = lambda s: loss(*(d[m] + (s * way if i == j else 0) for i, m in enumerate(names)))   # noqa: E731
        num = (at(1e-5) - at(-1e-5)) / 2e-5
        assert abs(num - (g["d" + n] * way).sum()) <= 1e-7 * (1 + abs(num)), n


# b, T, Hk, H, K, V: one step, around a chunk's end, heads that share keys, odd widths, the widest, long ones
SHAPES = [(1, 1, 1, 1, 1, 1), (2, 3, 1, 2, 8, 8), (1, 63, 2, 2, 64, 64), (2, 64, 1, 3, 64, 40), (1, 65, 2, 2, 128, 128),
          (3, 130, 2, 6, 60, 100), (1, 200, 1, 1, 200, 48), (2, 129, 1, 2, 256, 130), (1, 777, 2, 4, 96, 120),
          (2, 321, 1, 1, 40, 128), (1, 1500, 1, 2, 128, 128), (1, 191, 3, 3, 33, 257), (2, 256, 2, 2, 72, 136),
          (5, 17, 1, 2, 128, 24), (1, 640, 4, 4, 64, 128)]


def run_forward(d, dtype, states=True, **kw):
    b, T, H, V = d["v"].shape
    K = d["q"].shape[-1]
    out = {"y": Guarded(b * T * H * V * d["q"].element_size(), "cuda", GUARD_FILL),
           "final_state": Guarded(b * H * V * K * 4, "cuda", GUARD_FILL)}
    made = {"y": out["y"].view(DT[dtype], (b, T, H, V)),
            "final_state": out["final_state"].view(torch.float32, (b, H, V, K))}
    if states:
        nch = -(-T // 64)
        out["states"] = Guarded(b * nch * H * V * K * 4, "cuda", GUARD_FILL)
        made["states"] = out["states"].view(torch.float32, (b, nch, H, V, K))
    plan = pkg.GatedDeltaRulePlan(*args(d), init_state=d["init"], **made, **kw)
    r = plan()
    assert pkg.workspace_status(plan.workspace) == ("SSD_OK", 0)
    for k, v in out.items():
        v.check(k)
    return r


def run_backward(d, dtype, states, **kw):
    b, T, H, V = d["v"].shape
    Hk, K = d["q"].shape[2:]
    e = d["q"].element_size()
    sizes = {"dq": ((b, T, Hk, K), DT[dtype], e), "dk": ((b, T, Hk, K), DT[dtype], e),
             "dv": ((b, T, H, V), DT[dtype], e), "dg": ((b, T, H), torch.float32, 4),
             "dbeta": ((b, T, H), torch.float32, 4), "dinit": ((b, H, V, K), torch.float32, 4)}
    out = {k: Guarded(int(np.prod(s)) * n, "cuda", GUARD_FILL) for k, (s, _, n) in sizes.items()}
    plan = pkg.GatedDeltaRuleBackwardPlan(*args(d), d["dy"], init_state=d["init"], states=states, dfinal=d["dfinal"],
                                          grads={k: out[k].view(t, s) for k, (s, t, _) in sizes.items()}, **kw)
    g = plan()
    assert pkg.workspace_status(plan.workspace) == ("SSD_OK", 0)
    for k, v in out.items():
        v.check(k)
    return g


def check_forward(r, d, dtype, scale=None):
    h = host(d)
    want = ref.delta(h["q"], h["k"], h["v"], h["g"], h["beta"], h["init"], scale)
    ref.check(to_np(r[0]), want[0], dtype, "y", rounded=True)
    ref.check(to_np(r[1]), want[1], dtype, "final_state")
    if r[2] is not None:
        ref.check(to_np(r[2]), want[2], dtype, "states")


def check_backward(g, d, dtype, scale=None):
    h = host(d)
    want = ref.delta_grad(h["q"], h["k"], h["v"], h["g"], h["beta"], h["dy"], h["init"], scale, h["dfinal"])
    for k, w in want.items():
        if g[k] is not None:
            # dbeta and dg are inner products over a head's values and its state: terms of the size of the output's rms
            # times the root of their number at most
            ref.check(to_np(g[k]), w, dtype, k, rounded=k in ("dq", "dk", "dv"))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["plain", "fused", "odd", "time"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, layout, dtype):
    d = inputs(*shape, dtype, seed=2, layout=layout, dev="cuda")
    check_forward(run_forward(d, dtype), d, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["plain", "fused", "odd", "time"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, layout, dtype):
    d = inputs(*shape, dtype, seed=3, layout=layout, dev="cuda")
    given = shape[1] % 2 == 0
    states = pkg.gated_delta_rule_forward(*args(d), init_state=d["init"], return_states=True)[2] if given else None
    check_backward(run_backward(d, dtype, states), d, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 100, 1, 2, 64, 64), (1, 200, 2, 2, 128, 128), (2, 70, 1, 1, 30, 20)], ids=str)
def test_nothing_given(shape, dtype):
    """No g, no initial state, no dfinal, another scale; what is not asked for is not there."""
    d = inputs(*shape, dtype, seed=4, dev="cuda") | {"g": None, "init": None, "dfinal": None}
    r = pkg.gated_delta_rule_forward(*args(d), scale=0.7)
    assert r[2] is None
    check_forward(r, d, dtype, 0.7)
    assert pkg.gated_delta_rule_forward(*args(d), return_final_state=False)[1] is None
    g = pkg.gated_delta_rule_backward(*args(d), d["dy"], scale=0.7)
    assert g["dg"] is None
    check_backward(g, d, dtype, 0.7)
    assert pkg.gated_delta_rule_backward(*args(d), d["dy"], return_dinit=False)["dinit"] is None


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["resets", "strong", "still", "grow", "shut", "twice"])
@pytest.mark.parametrize("shape", [(1, 150, 1, 2, 64, 64), (1, 200, 1, 1, 128, 128), (1, 90, 1, 1, 20, 12)], ids=str)
def test_extreme_gates(shape, kind, dtype):
    """Decays of zero within a chunk, strong ones, none, a little growth; betas of zero, and of two with unit keys (a
    reflection: the largest that does not grow)."""
    d = inputs(*shape, dtype, seed=5, dev="cuda")
    g = d["g"]
    if kind == "resets":
        g[:, ::29] = -float("inf")
        g[:, 7::31] = -250.0
    elif kind == "strong":
        g.mul_(-1).add_(1e-3).reciprocal_().neg_()   # -3 to -60 a step
    elif kind == "still":
        g.zero_()
    elif kind == "grow":
        g.copy_(0.01 * torch.rand(g.shape, generator=torch.Generator().manual_seed(6)).cuda())
    elif kind == "shut":
        d["beta"][:, ::2] = 0.0
    else:
        d["beta"].fill_(2.0)
        d["k"].copy_(torch.nn.functional.normalize(d["k"].float(), dim=-1) * 0.99)
    r = run_forward(d, dtype)
    check_forward(r, d, dtype)
    h = host(d)
    with np.errstate(invalid="ignore"):
        want = ref.delta_grad(h["q"], h["k"], h["v"], h["g"], h["beta"], h["dy"], h["init"], None, h["dfinal"])
    got = run_backward(d, dtype, r[2])
    for k, w in want.items():
        # dg where decays are zero is zero; what is left of the sums it is formed from is of the size of q . dq
        size = np.abs(w) + (np.sqrt((h["q"] ** 2).sum(-1).mean()) * np.abs(want["dq"]).max() if k == "dg" else 0)
        ref.check(to_np(got[k]), w, dtype, k, rounded=k in ("dq", "dk", "dv"), scale=size)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_keys_all_alike(dtype):
    """Every key the same and beta one: the triangular system of a chunk is the worst that unit keys make (powers of its
    strict part grow like binomial coefficients), the result harmless."""
    d = inputs(1, 192, 1, 1, 64, 64, dtype, seed=7, dev="cuda")
    d["k"].copy_(d["k"][:, :1].expand_as(d["k"]))
    d["beta"].fill_(1.0)
    d["g"].zero_()
    h = host(d)
    # bf16: the inverse's entries are then the same numbers in every row of a chunk, and so are their roundings to two
    # terms, 2^-18 each (half a step of the second term): the 64 writes of a chunk, which cancel all but the last, leave
    # an error of up to 64 * 2^-18 = 2.4e-4 of the largest |v| = 4, in a state whose entries are v's times k's.
    size = 4.0 * 64 * 2.0 ** -18 / ref.UNIT["bf16"] if dtype == "bf16" else 1.0
    r = run_forward(d, dtype)
    want = ref.delta(h["q"], h["k"], h["v"], h["g"], h["beta"], h["init"])
    for got, w, what in zip(r, want, ("y", "final_state", "states")):
        ref.check(to_np(got), w, dtype, what, rounded=what == "y", scale=size * np.maximum(1.0, np.abs(w)))
    # the walk backwards is of the same form, with dR for the writes
    got = run_backward(d, dtype, None)
    want = ref.delta_grad(h["q"], h["k"], h["v"], h["g"], h["beta"], h["dy"], h["init"], None, h["dfinal"])
    for k, w in want.items():
        ref.check(to_np(got[k]), w, dtype, k, rounded=k in ("dq", "dk", "dv"), scale=size * np.maximum(1.0, np.abs(w)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cut", [1, 64, 100, 255])
def test_a_sequence_in_two_calls(cut, dtype):
    d = inputs(2, 256, 1, 2, 64, 128, dtype, seed=8, dev="cuda")
    first = pkg.gated_delta_rule_forward(*(t[:, :cut] for t in args(d)), init_state=d["init"])
    second = pkg.gated_delta_rule_forward(*(t[:, cut:] for t in args(d)), init_state=first[1])
    check_forward((torch.cat((first[0], second[0]), 1), second[1], None), d, dtype)


STEPS = [(1, 1, 1, 1, 1), (3, 2, 4, 64, 64), (16, 8, 16, 128, 128), (5, 1, 3, 60, 100), (2, 1, 1, 256, 33),
         (7, 2, 2, 30, 17), (200, 1, 2, 64, 40)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", STEPS, ids=str)
def test_step(shape, dtype):
    b, Hk, H, K, V = shape
    d = inputs(b, 1, Hk, H, K, V, dtype, seed=9, layout="fused", dev="cuda")
    want = ref.delta(*(to_np(t) for t in args(d)), to_np(d["init"]))
    one = tuple(t[:, 0] for t in args(d))
    kept = d["init"].clone()
    out = Guarded(b * H * V * K * 4, "cuda", GUARD_FILL)
    y, state = pkg.gated_delta_rule_step(*one, d["init"], state_out=out.view(torch.float32, (b, H, V, K)))
    out.check("state")
    ref.check(to_np(y), want[0][:, 0], "f32", "y") if dtype == "f32" else ref.check(to_np(y), want[0][:, 0], dtype, "y", True)
    ref.check(to_np(state), want[1], "f32", "state")
    assert torch.equal(d["init"], kept)
    again = pkg.gated_delta_rule_step(*one, d["init"])   # in place
    assert again[1] is d["init"] and torch.equal(d["init"], state) and torch.equal(again[0], y)


@pytest.mark.gpu
def test_steps_of_a_state_that_is_not_on_a_16_byte_border():
    d = inputs(2, 1, 1, 2, 64, 16, seed=10, dev="cuda")
    big = torch.zeros(2 * 2 * 16 * 64 + 1, device="cuda")
    off = big[1:].view(2, 2, 16, 64)
    off.copy_(d["init"])
    one = tuple(t[:, 0] for t in args(d))
    y, state = pkg.gated_delta_rule_step(*one, off, state_out=torch.empty_like(d["init"]))
    y2, state2 = pkg.gated_delta_rule_step(*one, d["init"])
    assert torch.equal(y, y2) and torch.equal(state, state2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bad_values_stay_in_their_head_and_sequence(dtype):
    d = inputs(2, 200, 2, 4, 64, 64, dtype, seed=11, dev="cuda")
    clean = pkg.gated_delta_rule_forward(*args(d), init_state=d["init"])
    cg = pkg.gated_delta_rule_backward(*args(d), d["dy"], init_state=d["init"])
    v = d["v"].clone()
    v[0, 100, 1] = float("nan")
    bad = d | {"v": v}
    r = pkg.gated_delta_rule_forward(*args(bad), init_state=d["init"])
    gr = pkg.gated_delta_rule_backward(*args(bad), d["dy"], init_state=d["init"])
    assert bool(torch.isnan(r[0][0, 100:, 1].float()).all()) and bool(torch.isnan(r[1][0, 1]).all())
    assert torch.equal(r[0][1], clean[0][1]) and torch.equal(r[0][0, :, 2:], clean[0][0, :, 2:])
    assert torch.equal(r[0][0, :, 0], clean[0][0, :, 0]) and torch.equal(r[0][0, :64, 1], clean[0][0, :64, 1])
    for k in ("dq", "dk", "dv", "dg", "dbeta", "dinit"):
        assert torch.equal(gr[k][1], cg[k][1]), k
    assert torch.equal(gr["dq"][0, :, 1], cg["dq"][0, :, 1])   # the other key head


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_every_run_on_another_stream_and_in_a_graph(dtype):
    d = inputs(2, 300, 1, 2, 128, 64, dtype, seed=12, dev="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    runs = []
    for stream in (None, side, None):
        f = pkg.gated_delta_rule_forward(*args(d), init_state=d["init"], return_states=True, stream=stream)
        g = pkg.gated_delta_rule_backward(*args(d), d["dy"], init_state=d["init"], states=f[2], dfinal=d["dfinal"],
                                          stream=stream)
        torch.cuda.synchronize()
        runs.append([*f, *g.values()])
    for other in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(runs[0], other))
    plan = pkg.GatedDeltaRulePlan(*args(d), init_state=d["init"], return_states=True, stream=side)
    back = pkg.GatedDeltaRuleBackwardPlan(*args(d), d["dy"], init_state=d["init"], states=plan.states,
                                          dfinal=d["dfinal"], stream=side)
    with torch.cuda.stream(side):
        plan(), back()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        plan(), back()
    for shift in (0.0, 0.25):
        d["v"].add_(shift)
        for t in (plan.y, back.grads["dk"]):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check_forward((plan.y, plan.final_state, plan.states), d, dtype)
        check_backward(back.grads, d, dtype)


@pytest.mark.gpu
def test_offsets_past_31_bits():
    """The last of two sequences lies 2^31 elements behind the first."""
    d = inputs(2, 70, 1, 1, 64, 64, "bf16", seed=13, dev="cuda")
    far = {}
    for k in ("q", "k", "v", "dy"):
        t = d[k]
        base = torch.empty((1 << 31) + t[0].numel() + 64, dtype=t.dtype, device="cuda")
        far[k] = base.as_strided(t.shape, ((1 << 31) + 64, *t.stride()[1:]))
        far[k].copy_(t)
    e = d | far
    near = pkg.gated_delta_rule_forward(*args(d), init_state=d["init"])
    f = pkg.gated_delta_rule_forward(*args(e), init_state=d["init"])
    assert torch.equal(f[0], near[0]) and torch.equal(f[1], near[1])
    gn = pkg.gated_delta_rule_backward(*args(d), d["dy"])
    gf = pkg.gated_delta_rule_backward(*args(e), e["dy"])
    assert all(torch.equal(gn[k], gf[k]) for k in gn)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty(dtype):
    for b, T in ((0, 5), (3, 0)):
        d = inputs(b, T, 1, 2, 8, 8, dtype, seed=14, dev="cuda")
        y, final, states = pkg.gated_delta_rule_forward(*args(d), init_state=d["init"], return_states=True)
        assert y.shape == (b, T, 2, 8) and torch.equal(final, d["init"]) and states.shape[1] == 0 or b == 0
        g = pkg.gated_delta_rule_backward(*args(d), d["dy"], dfinal=d["dfinal"])
        assert torch.equal(g["dinit"], d["dfinal"])
    d = inputs(0, 1, 1, 2, 8, 8, dtype, seed=14, dev="cuda")
    assert pkg.gated_delta_rule_step(*(t[:, 0] for t in args(d)), d["init"])[0].shape == (0, 2, 8)


# ------------------------------------------------------------------------------------------------
# refusals
# ------------------------------------------------------------------------------------------------
A16 = 0x100000
_VP = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkg.load_library()


def shape_of(b=2, T=100, Hk=1, H=2, K=64, V=64, io=0, **kw):
    s3 = (ctypes.c_int64 * 3)
    qk, v, g = s3(T * Hk * K, Hk * K, K), s3(T * H * V, H * V, V), (ctypes.c_int64 * 2)(T * H, H)
    s = pkg.lm_ops.gated_delta_rule_shape(b, T, Hk, H, K, V, qk, qk, v, v, g, g, 0.125, io)
    for k, x in kw.items():
        setattr(s, k, x)
    return s


BAD = [dict(batch=-1), dict(seqlen=-1), dict(key_heads=0), dict(heads=3, key_heads=2), dict(key_dim=0), dict(value_dim=0),
       dict(scale=float("inf")), dict(scale=float("nan")), dict(io_dtype=2), dict(q_stride=(ctypes.c_int64 * 3)(-1, 0, 0)),
       dict(v_stride=(ctypes.c_int64 * 3)(0, 0, -5)), dict(beta_stride=(ctypes.c_int64 * 2)(0, -1))]


@pytest.mark.parametrize("change", BAD, ids=str)
def test_bad_shapes(lib, change):
    s = shape_of(**change)
    for back in (0, 1):
        assert lib.gated_delta_rule_workspace_bytes(ctypes.byref(s), back) == 0
    p = [_VP(A16)] * 9
    assert lib.gated_delta_rule_forward(ctypes.byref(s), *p, _VP(A16), 1 << 40, None) == 1


@pytest.mark.parametrize("change", [dict(key_dim=257), dict(batch=1 << 40), dict(seqlen=1 << 50)], ids=str)
def test_unsupported_shapes(lib, change):
    s = shape_of(**change)
    assert lib.gated_delta_rule_workspace_bytes(ctypes.byref(s), 1) == 0
    assert lib.gated_delta_rule_forward(ctypes.byref(s), *[_VP(A16)] * 9, _VP(A16), 1 << 62, None) == 2


@pytest.mark.parametrize("final,states", [(0, None), (4, None), (-4, None), (None, 0), (None, -4)], ids=str)
def test_states_over_the_initial_state(lib, final, states):
    # written by one segment's block while another one still reads the state
    s, far = shape_of(), 1 << 40
    size = 4 * 2 * 2 * 64 * 64
    at = lambda off, n: None if off is None else _VP(far + (off if off >= 0 else off - n + 8))   # noqa: E731
    p = [_VP(A16 * (i + 1)) for i in range(5)]
    assert lib.gated_delta_rule_forward(ctypes.byref(s), *p, _VP(far), _VP(A16 * 9), at(final, size), at(states, 2 * size),
                                        _VP(A16), 1 << 40, None) == 1


def test_bad_pointers_and_workspaces(lib):
    s = shape_of()
    fwd = lambda p, ws=A16, n=1 << 40: lib.gated_delta_rule_forward(ctypes.byref(s), *p, _VP(ws), n, None)   # noqa: E731
    good = [_VP(A16)] * 9
    for i in (0, 1, 2, 4):   # q, k, v, beta
        assert fwd(good[:i] + [None] + good[i + 1:]) == 1
    for i in range(9):
        assert fwd(good[:i] + [_VP(A16 + 1)] + good[i + 1:]) == 1
    need = lib.gated_delta_rule_workspace_bytes(ctypes.byref(s), 0)
    assert fwd(good, n=need - 1) == 4 and fwd(good, ws=0) == 4 and fwd(good, ws=A16 + 16) == 4
    bwd = lambda p, ws=A16, n=1 << 40: lib.gated_delta_rule_backward(ctypes.byref(s), *p, _VP(ws), n, None)   # noqa: E731
    good = [_VP(A16)] * 15
    for i in (0, 1, 2, 4, 7, 9, 10, 11, 13):
        assert bwd(good[:i] + [None] + good[i + 1:]) == 1
    for i in range(15):
        assert bwd(good[:i] + [_VP(A16 + 1)] + good[i + 1:]) == 1
    need = lib.gated_delta_rule_workspace_bytes(ctypes.byref(s), 1)
    assert bwd(good, n=need - 1) == 4
    step = lambda p, sh: lib.gated_delta_rule_step(ctypes.byref(sh), *p, None)   # noqa: E731
    good = [_VP(A16)] * 8
    assert step(good, s) == 1   # more than one step
    one = shape_of(T=1)
    for i in (0, 1, 2, 4, 6, 7):
        assert step(good[:i] + [None] + good[i + 1:], one) == 1
    for i in range(8):
        assert step(good[:i] + [_VP(A16 + 1)] + good[i + 1:], one) == 1


@pytest.mark.gpu
def test_refusals_of_the_binding():
    d = inputs(2, 10, 1, 2, 8, 8, dev="cuda")
    a = args(d)
    with pytest.raises(ValueError):
        pkg.gated_delta_rule_forward(a[0].double(), *a[1:])
    with pytest.raises(ValueError):
        pkg.gated_delta_rule_forward(a[0], a[1].bfloat16(), *a[2:])
    with pytest.raises(ValueError):
        pkg.gated_delta_rule_forward(a[0], a[1][..., :7], *a[2:])
    with pytest.raises(ValueError):
        pkg.gated_delta_rule_forward(a[0], a[1], a[2][:, :9], *a[3:])
    with pytest.raises(ValueError):
        pkg.gated_delta_rule_forward(*a[:3], a[3].bfloat16(), a[4])
    with pytest.raises(ValueError):
        pkg.gated_delta_rule_forward(*a, scale=float("nan"))
    with pytest.raises(ValueError):
        pkg.gated_delta_rule_forward(a[0].transpose(2, 3), *a[1:])
    with pytest.raises(ValueError):
        pkg.gated_delta_rule_forward(a[0].cpu(), *a[1:])
    with pytest.raises(ValueError):
        pkg.gated_delta_rule_forward(*a, init_state=d["init"].transpose(2, 3))
    with pytest.raises(ValueError):
        pkg.gated_delta_rule_forward(a[0].repeat(1, 1, 3, 1), a[1].repeat(1, 1, 3, 1), *a[2:])   # 3 does not divide 2
    with pytest.raises(ValueError):
        pkg.gated_delta_rule_backward(*a, d["dy"].bfloat16())
    with pytest.raises(ValueError):
        pkg.gated_delta_rule_step(*(t[:, 0] for t in a), None)
    with pytest.raises(pkg.SSDError):
        pkg.gated_delta_rule_backward(*a, d["dy"], workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
