"""Sizes of nothing, workspaces, streams and extreme arguments of the recurrence, the norm and the embedding."""
import ctypes

import pytest
import torch

import chunked_ssd_scan_gb300 as pkg


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(2, 0, 8), (5, 0, 12), (0, 3, 8), (3, 0, 2, 8)], ids=str)
def test_statistics_of_no_positions(shape, dtype):
    """Every value of mean and rstd is written: the mean of nothing is NaN."""
    x = torch.zeros(shape, dtype=dtype, device="cuda")
    mean, rstd = (torch.full((shape[0], 4), 3.0, device="cuda") for _ in range(2))
    y, m, r = pkg.group_norm_forward(x, 4, mean=mean, rstd=rstd)
    assert y.shape == x.shape and m.data_ptr() == mean.data_ptr()
    assert bool(torch.isnan(m).all()) and bool(torch.isnan(r).all()) and m.shape == r.shape == (shape[0], 4)


def _norm_shape(N, S, C, G, io):
    st = (ctypes.c_int64 * 2)(S * C, C)
    return pkg.lm_ops.group_norm_shape(N, S, C, G, st, st, 1e-5, 1, io)


@pytest.fixture(scope="module")
def lib():
    from chunked_ssd_scan_gb300 import _build
    _build.build()
    return pkg.load_library()


# tokens in wide groups that some vectors take into registers, and some that none does; maps of few positions
@pytest.mark.parametrize("io", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(131072, 1, 4096, 1), (131072, 1, 8192, 1), (100000, 1, 4999, 1), (70000, 1, 2048, 2),
                                   (40000, 16, 64, 8), (20000, 2, 20000, 1)], ids=str)
def test_norm_backward_workspace_does_not_grow_with_the_activation(lib, shape, io):
    """Two floats a sample's group and chunk and two for the join, and partial rows of parameter gradients whose
    number is bounded whatever N is: at most 912, twice C floats each."""
    N, S, C, G = shape
    need = lambda n: lib.group_norm_workspace_bytes(ctypes.byref(_norm_shape(n, S, C, G, io)), 1)   # noqa: E731
    assert 0 < need(N) <= 16 * N * G + 2 * 912 * 4 * C + 5 * 256
    assert need(2 * N) - need(N) <= 16 * N * G + 5 * 256


@pytest.mark.gpu
def test_a_workspace_made_here_is_zero_in_its_header_only():
    """The header alone has to be: nothing else of a workspace is read before it is written.  What is handed out is
    filled with 0xff before, and the results stay."""
    g = torch.Generator().manual_seed(51)
    x, dy = (torch.randn(3000, 96, generator=g).cuda() for _ in range(2))
    _, mean, rstd = pkg.group_norm_forward(x, 6)
    want = pkg.group_norm_backward(x, dy, 6, mean, rstd)
    ids = torch.randint(0, 500, (3000,), generator=g).cuda()
    wemb = pkg.embedding_backward(ids, dy, 500)
    r = [torch.randn(2, 300, 96, generator=g).cuda() for _ in range(4)]
    decay = torch.randn(96, generator=g).cuda() - 4
    wrec = pkg.gated_recurrence_backward(*r[:3], decay, r[3])
    torch.cuda.synchronize()
    junk = torch.full((64 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    del junk   # the allocator gives it out again
    plan = pkg.GroupNormBackwardPlan(x, dy, 6, mean, rstd)
    assert not bool(plan.workspace[:256].any())
    assert all(torch.equal(v, want[k]) for k, v in plan().items())
    plan = pkg.EmbeddingBackwardPlan(ids, dy, 500)
    assert not bool(plan.workspace[:256].any())
    assert torch.equal(plan(), wemb)
    plan = pkg.GatedRecurrenceBackwardPlan(*r[:3], decay, r[3])
    assert not bool(plan.workspace[:256].any())
    assert all(torch.equal(v, wrec[k]) for k, v in plan().items())


@pytest.mark.gpu
def test_what_the_caller_passes_is_kept_for_the_stream(monkeypatch):
    """Inputs, outputs and a workspace that the caller passes are recorded on the plan's stream, so that their memory
    is not given out again while the work on it goes on."""
    seen = set()
    real = torch.Tensor.record_stream
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: (seen.add((t.data_ptr(), s.cuda_stream)), real(t, s))[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    new = lambda *s: torch.zeros(*s, device="cuda")   # noqa: E731
    ws = lambda: torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")   # noqa: E731
    x, ga, gx, dy = (new(2, 70, 8) for _ in range(4))
    decay, init = new(8), new(2, 8)
    ids, table = torch.zeros(5, dtype=torch.int64, device="cuda"), new(6, 8)
    calls = [
        (pkg.GatedRecurrencePlan, (x, ga, gx, decay), dict(init_state=init, y=new(2, 70, 8), final_state=new(2, 8),
                                                           states=new(2, 2, 8), workspace=ws())),
        (pkg.GatedRecurrenceBackwardPlan, (x, ga, gx, decay, dy), dict(
            states=new(2, 2, 8), dfinal=new(2, 8), workspace=ws(),
            grads={"dx": new(2, 70, 8), "dgate_a": new(2, 70, 8), "dgate_x": new(2, 70, 8), "ddecay": new(8),
                   "dinit": new(2, 8)})),
        (pkg.GatedRecurrenceStepPlan, (x[:, 0], ga[:, 0], gx[:, 0], decay, init), dict(y=new(2, 8), state_out=new(2, 8))),
        (pkg.GroupNormPlan, (x, 2, decay), dict(bias=new(8), y=new(2, 70, 8), mean=new(2, 2), rstd=new(2, 2),
                                                workspace=ws())),
        (pkg.GroupNormBackwardPlan, (x, dy, 2, new(2, 2), new(2, 2)), dict(
            workspace=ws(), grads={"dx": new(2, 70, 8), "dweight": new(8), "dbias": new(8)})),
        (pkg.EmbeddingPlan, (ids, table), dict(out=new(5, 8))),
        (pkg.EmbeddingBackwardPlan, (ids, new(5, 8), 6), dict(dtable=new(6, 8), workspace=ws()))]
    for plan, args, kw in calls:
        seen.clear()
        plan(*args, stream=side, **kw)()
        grads = kw.pop("grads", {})
        for t in (*args, *kw.values(), *grads.values()):
            if isinstance(t, torch.Tensor):
                assert (t.data_ptr(), side.cuda_stream) in seen, (plan.__name__, tuple(t.shape))
    side.synchronize()


@pytest.mark.gpu
def test_a_workspace_elsewhere_is_refused():
    x = torch.zeros(2, 5, 8, device="cuda")
    for bad in (torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(1 << 20, device="cuda"),
                torch.zeros(1 << 21, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            pkg.group_norm_forward(x, 2, workspace=bad)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [40, 41])
@pytest.mark.parametrize("scale", [float("inf"), float("nan"), 0.0, -2.0])
def test_padding_is_zeros_whatever_the_scale(scale, D, dtype):
    ids = torch.tensor([1, -1, 2, 99, 0, -7, 1], device="cuda")
    table = torch.ones(3, D, dtype=dtype, device="cuda")
    out = pkg.embedding_forward(ids, table, scale=scale).float()
    pad = torch.tensor([False, True, False, True, False, True, False], device="cuda")
    assert torch.equal(out[pad], torch.zeros(3, D, device="cuda"))
    assert torch.equal(out[~pad].nan_to_num(7.0, 8.0), torch.full((4, D), scale, device="cuda").nan_to_num(7.0, 8.0))
    g = pkg.embedding_backward(ids, torch.ones(7, D, dtype=dtype, device="cuda"), 5, scale=scale)
    assert torch.equal(g[3:], torch.zeros(2, D, device="cuda"))   # rows without tokens


def test_rows_too_wide_are_refused_as_unsupported(lib):
    """Rows of more vectors than a grid has blocks for: refused on the host, none of these pointers is read."""
    A = 0x100000
    vp = ctypes.c_void_p

    def fwd(D, io, table=A):
        return lib.embedding_forward(vp(A), 64, 1, vp(table), 1, D, io, 1.0, vp(A), None)

    def bwd(D, io, dout=A):
        return lib.embedding_backward(vp(A), 64, 1, vp(dout), 1, D, io, 1.0, vp(A), vp(A), ctypes.c_size_t(1 << 45), None)

    most = 65535 * 256
    assert fwd(most + 1, 0) == 2 and fwd(most + 1, 1) == 2            # an odd width: one value a vector
    assert fwd(8 * most + 8, 1) == 2 and fwd(4 * most + 4, 0) == 2    # the widest vectors
    assert fwd(2 * most, 1, table=A + 2) == 2                         # rows that start on 2 bytes
    assert bwd(most + 1, 0) == 2 and bwd(4 * most + 4, 0) == 2 and bwd(2 * most, 1, dout=A + 2) == 2


@pytest.mark.gpu
def test_wide_rows():
    """34 million values a row, in vectors of four: within the limit."""
    D = 1 << 25
    table = torch.arange(D, dtype=torch.float32, device="cuda").repeat(2, 1)
    table[1].neg_()
    ids = torch.tensor([1, 5, 0], device="cuda")
    out = pkg.embedding_forward(ids, table)
    assert torch.equal(out[0], table[1]) and torch.equal(out[2], table[0]) and not bool(out[1].any())
    g = pkg.embedding_backward(ids, out, 2)
    assert torch.equal(g, table)


def test_step_strides_are_ignored_by_the_single_step(lib):
    """A shape without sequences launches nothing and reads none of these pointers."""
    two = lambda *v: (ctypes.c_int64 * 2)(*v)   # noqa: E731
    vp = ctypes.c_void_p
    s = pkg.lm_ops.gated_recurrence_shape(0, 1, 8, two(8, -3), two(8, -3), two(8, -3), two(0, 0), 8.0, 0)
    assert lib.gated_recurrence_step(ctypes.byref(s), *[vp(0x100000)] * 7, None) == 0
    s.x_stride[0] = -8
    assert lib.gated_recurrence_step(ctypes.byref(s), *[vp(0x100000)] * 7, None) == 1
