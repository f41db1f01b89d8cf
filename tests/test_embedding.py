"""Token embedding and the gradient of its table: the kernels against the plain form (GPU) and the
refusals."""
import ctypes
import math

import numpy as np
import pytest
import torch

import chunked_ssd_scan_gb300 as pkg
from chunked_ssd_scan_gb300 import _build
from tests import lm_reference as ref
from tests.parity_util import GUARD_FILL, Guarded, to_np

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
REL = {"f32": 0.0, "bf16": ref.BF16_REL}


def make_ids(kind, n, V, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "zipf":      # frequencies fall as 1/rank
        ids = (torch.exp(torch.rand(n, generator=g, dtype=torch.float64) * math.log(V)).long() - 1).clamp_(0, V - 1)
        ids = torch.randperm(V, generator=g)[ids]
    elif kind == "one":
        ids = torch.full((n,), V // 2)
    elif kind == "ends":    # the first and the last row, and ids just outside and far outside
        ids = torch.tensor([0, V - 1, -1, V, 1 << 30, -(1 << 31)]).repeat(n // 6 + 1)[:n]
    else:
        ids = torch.randint(0, V, (n,), generator=g)
    if kind == "zipf" and n > 3:
        ids[torch.rand(n, generator=g) < 0.05] = -1
    return ids


# ids, n, V, D
CASES = [("uniform", 1, 1, 1), ("uniform", 1, 300, 64), ("uniform", 7, 5, 33), ("zipf", 1000, 777, 96),
         ("zipf", 4097, 50000, 64), ("one", 5000, 300, 40), ("ends", 900, 129, 200),
         ("uniform", 3000, 3, 500), ("uniform", 64, 100001, 16), ("zipf", 20001, 2048, 130),
         ("uniform", 65, 2049, 2048), ("one", 33, 1, 2500), ("zipf", 9000, 70000, 8),
         ("uniform", 100003, 40, 24), ("zipf", 3000, 5_000_000, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("idt", [torch.int32, torch.int64], ids=["i32", "i64"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case, dtype, idt):
    kind, n, V, D = case
    ids = make_ids(kind, n, V).to(idt).cuda()
    table = torch.randn(V, D, generator=torch.Generator().manual_seed(1)).to(DT[dtype]).cuda()
    band = Guarded(n * D * table.element_size(), "cuda", GUARD_FILL)
    out = pkg.embedding_forward(ids, table, scale=3.7, out=band.view(DT[dtype], (n, D)))
    torch.cuda.synchronize()
    band.check("out")
    r = ref.embedding(ids.cpu().numpy().astype(np.int64), to_np(table), np.float64(np.float32(3.7)))
    ref.check(to_np(out), r, REL[dtype], "out")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("idt", [torch.int32, torch.int64], ids=["i32", "i64"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case, dtype, idt):
    kind, n, V, D = case
    ids = make_ids(kind, n, V, seed=2).to(idt).cuda()
    dout = torch.randn(n, D, generator=torch.Generator().manual_seed(3)).to(DT[dtype]).cuda()
    band = Guarded(V * D * 4, "cuda", GUARD_FILL)
    plan = pkg.EmbeddingBackwardPlan(ids, dout, V, scale=0.3, dtable=band.view(torch.float32, (V, D)))
    g = plan()
    assert pkg.workspace_status(plan.workspace) == ("SSD_OK", 0)
    band.check("dtable")
    npids = ids.cpu().numpy().astype(np.int64)
    r = ref.embedding_grad(npids, to_np(dout), V, np.float64(np.float32(0.3)))
    # a row is a sum of `count` terms of size 0.3: its fp32 error goes with sqrt(count)
    count = np.bincount(npids[(npids >= 0) & (npids < V)], minlength=V)[:, None]
    got = to_np(g)
    assert np.all(np.abs(got - r) <= 2e-5 * 0.3 * np.sqrt(count) * (1 + np.abs(r)))
    assert np.all(got[count[:, 0] == 0] == 0)
    assert torch.equal(pkg.embedding_backward(ids, dout, V, scale=0.3), g)   # the same bits


@pytest.mark.gpu
def test_shapes_of_ids_and_odd_alignment():
    ids = make_ids("zipf", 60, 100, seed=4).view(3, 4, 5).cuda()
    flat = torch.randn(1 + 100 * 48, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    table = flat[1:].view(100, 48)   # starts two bytes past a 16-byte boundary
    out = pkg.embedding_forward(ids, table, scale=2.0)
    assert out.shape == (3, 4, 5, 48)
    ref.check(to_np(out), ref.embedding(ids.cpu().numpy(), to_np(table), 2.0), REL["bf16"], "out")
    buf = torch.empty(1 + 60 * 48, device="cuda", dtype=torch.bfloat16)
    dout = buf[1:].view(3, 4, 5, 48)
    dout.copy_(out)
    g = pkg.embedding_backward(ids, dout, 100)
    ref.check(to_np(g), ref.embedding_grad(ids.cpu().numpy(), to_np(dout), 100, 1.0), 0.0, "dtable")
    gbuf = torch.empty(1 + 100 * 48, device="cuda")
    g2 = pkg.embedding_backward(ids, dout, 100, dtable=gbuf[1:].view(100, 48))
    assert torch.equal(g, g2)


@pytest.mark.gpu
def test_bad_values_stay_in_their_rows():
    ids = torch.tensor([3, 3, 7, 2, -1, 9], device="cuda")
    dout = torch.ones(6, 40, device="cuda")
    dout[2, 5], dout[4] = float("inf"), float("nan")   # the padding's gradient is never used
    g = pkg.embedding_backward(ids, dout, 10)
    want = torch.zeros(10, 40, device="cuda")
    want[3], want[7], want[2], want[9] = 2, 1, 1, 1
    want[7, 5] = float("inf")
    assert torch.equal(g, want)
    table = torch.ones(10, 40, device="cuda")
    table[0] = float("nan")   # padding never reads a row
    out = pkg.embedding_forward(ids, table)
    assert torch.equal(out[4], torch.zeros(40, device="cuda")) and torch.isfinite(out).all()


@pytest.mark.gpu
def test_gradient_against_differences():
    """The lookup is linear: differences of any step size are exact up to rounding."""
    ids = make_ids("zipf", 300, 50, seed=6).cuda()
    gen = torch.Generator().manual_seed(7)
    table, v = (torch.randn(50, 16, generator=gen).cuda() for _ in range(2))
    dout = torch.randn(300, 16, generator=gen).cuda()
    loss = lambda t: float((pkg.embedding_forward(ids, t, scale=1.5).double() * dout).sum())   # noqa: E731
    num = (loss(table + v) - loss(table - v)) / 2
    g = pkg.embedding_backward(ids, dout, 50, scale=1.5)
    # 4800 terms of size about 3, each rounded in fp32
    assert abs(num - float((g.double() * v).sum())) <= math.sqrt(4800) * 3 * 1e-6


@pytest.mark.gpu
def test_replays_in_a_graph_and_on_another_stream():
    ids = make_ids("zipf", 6000, 900, seed=8).cuda()
    dout = torch.randn(6000, 72, generator=torch.Generator().manual_seed(9)).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan = pkg.EmbeddingBackwardPlan(ids, dout, 900, stream=side)
    with torch.cuda.stream(side):
        plan()
    side.synchronize()
    assert torch.equal(plan.dtable, pkg.embedding_backward(ids, dout, 900))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        plan()
    for seed in (10, 11):
        ids.copy_(make_ids("zipf", 6000, 900, seed=seed))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(plan.dtable, pkg.embedding_backward(ids, dout, 900))


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    V, D = 1_100_000, 2048   # 2.25e9 elements
    table = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    table[V - 1], table[V - 2] = 3.0, 5.0
    ids = torch.tensor([V - 1, 0, V - 2, V], device="cuda")
    out = pkg.embedding_forward(ids, table, scale=0.5)
    assert out[:, 0].tolist() == [1.5, 0.0, 2.5, 0.0] and out[0].eq(1.5).all()
    del table
    g = pkg.embedding_backward(ids, out, V)
    assert g[V - 1].eq(1.5).all() and g[V - 2].eq(2.5).all() and int((g != 0).sum()) == 2 * D


@pytest.mark.gpu
def test_empty():
    table = torch.randn(5, 8, device="cuda")
    ids = torch.zeros(0, 3, dtype=torch.int64, device="cuda")
    out = pkg.embedding_forward(ids, table)
    assert out.shape == (0, 3, 8)
    assert torch.equal(pkg.embedding_backward(ids, out, 5), torch.zeros(5, 8, device="cuda"))


# ------------------------------------------------------------------------------------------------
# refusals
# ------------------------------------------------------------------------------------------------
A16 = 0x100000
_VP = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkg.load_library()


def test_invalid_arguments(lib):
    """Rejected on the host before any launch: none of these pointers is read."""
    def fwd(ids=A16, bits=64, n=4, table=A16, V=10, D=8, io=0, out=A16):
        return lib.embedding_forward(_VP(ids), bits, n, _VP(table), V, D, io, 1.0, _VP(out), None)

    def bwd(ids=A16, bits=64, n=4, dout=A16, V=10, D=8, io=0, dtable=A16, ws=A16, size=1 << 40):
        return lib.embedding_backward(_VP(ids), bits, n, _VP(dout), V, D, io, 1.0, _VP(dtable), _VP(ws),
                                      ctypes.c_size_t(size), None)

    for kw in (dict(ids=None), dict(bits=16), dict(n=-1), dict(table=None), dict(V=0), dict(D=0),
               dict(io=2), dict(out=None), dict(ids=A16 + 4), dict(table=A16 + 2), dict(out=A16 + 1)):
        assert fwd(**kw) == 1, kw
    assert fwd(n=1 << 40) == 2 and fwd(V=1 << 40) == 2
    for kw in (dict(ids=None), dict(bits=8), dict(n=-1), dict(dout=None), dict(V=-1), dict(D=0),
               dict(io=7), dict(dtable=None), dict(dtable=A16 + 2)):
        assert bwd(**kw) == 1, kw
    need = lib.embedding_backward_workspace_bytes(4, 10, 8)
    assert need > 0 and lib.embedding_backward_workspace_bytes(4, 0, 8) == 0
    assert bwd(ws=None) == 4 and bwd(size=need - 1) == 4 and bwd(ws=A16 + 64) == 4


@pytest.mark.gpu
def test_binding_refuses():
    ids, table = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(5, 8, device="cuda")
    f, b = pkg.embedding_forward, pkg.embedding_backward
    for bad in (lambda: f(ids.float(), table), lambda: f(ids, table.half()), lambda: f(ids, table[0]),
                lambda: f(ids.cpu(), table), lambda: f(ids, table.t()),
                lambda: f(ids, table, out=torch.empty(4, 9, device="cuda")),
                lambda: b(ids, table, 5), lambda: b(ids, torch.zeros(4, 8, device="cuda"), 0),
                lambda: b(ids[::2], torch.zeros(2, 8, device="cuda"), 5)):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks host tensors on CPU hosts")
def test_refuses_host_tensors():
    with pytest.raises(ValueError, match="CUDA tensor"):
        pkg.embedding_forward(torch.zeros(3, dtype=torch.int64), torch.zeros(5, 8))
    with pytest.raises(ValueError, match="CUDA tensor"):
        pkg.embedding_backward(torch.zeros(3, dtype=torch.int64), torch.zeros(3, 8), 5)
