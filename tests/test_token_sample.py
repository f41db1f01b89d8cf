"""Drawing of tokens: the kernel against a walk down the sorted weights in fp64, ties, extremes, and the refusals."""
import ctypes

import numpy as np
import pytest
import torch

import chunked_ssd_scan_gb300 as pkg
from chunked_ssd_scan_gb300 import _build
from tests import delta_reference as ref
from tests.parity_util import to_np

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def compare(logits, u, ids, logprob, **settings):
    """Token for token.  Settings are fp32, so that is what they are here: a top_p of 0.4 is 0.400000006, which of 2000
    equal tokens keeps 801.  A draw at most 1e-9 of the sum from a border between two tokens (fixed-point weights have 2^-30 of
    their value) may be the other one, which at these sizes is none."""
    x, uu, got, lp = to_np(logits), to_np(u), to_np(ids), to_np(logprob)
    for r in range(len(uu)):
        s = {k: float(np.float32(v)) if not isinstance(v, torch.Tensor) else float(to_np(v)[r]) for k, v in settings.items()}
        if "top_k" in s:
            s["top_k"] = int(s["top_k"])
        at, want = ref.sample(x[r], uu[r], **s)
        assert got[r] == at, (r, got[r], at, s)
        # fp32 of a logarithm of up to 100
        assert np.isnan(want) and np.isnan(lp[r]) or abs(lp[r] - want) <= 1e-6 * (1 + abs(want)), (r, lp[r], want)


def make(n, V, dtype, seed, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, V, generator=g) * spread
    x.scatter_add_(1, torch.randint(0, V, (n, 8), generator=g), 10 * torch.rand(n, 8, generator=g))
    return x.to(DT[dtype]).cuda(), torch.rand(n, generator=g).cuda(), g


def test_the_walk_itself():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    assert [ref.sample(x, u)[0] for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.69, 0.71, 0.99)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert np.allclose(ref.kept(x, top_k=2) / 4, [0, 0.25, 0, 0.1875])
    assert (ref.kept(x, top_p=0.6) > 0).tolist() == [False, True, False, True]   # 0.4 < 0.6 <= 0.7
    assert (ref.kept(x, min_p=0.45) > 0).tolist() == [False, True, True, True]   # of 0.4: at least 0.18
    assert (ref.kept(x, top_k=3, top_p=0.7) > 0).tolist() == [False, True, False, True]   # 0.4 + 0.3 >= 0.63
    assert ref.sample(x, 0.99, temperature=0)[0] == 1 and ref.sample(np.full(3, -np.inf), 0.5)[0] == -1


SIZES = [(1, 1), (5, 2), (7, 31), (3, 33), (4, 1000), (9, 1025), (6, 5001), (3, 50000), (2, 131073), (40, 300)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_every_setting(size, dtype):
    n, V = size
    logits, u, g = make(n, V, dtype, 1)
    rand = lambda lo, hi: (lo + (hi - lo) * torch.rand(n, generator=g)).cuda()   # noqa: E731
    k = torch.randint(0, min(V, 300) + 1, (n,), generator=g, dtype=torch.int32).cuda()
    t = rand(0.2, 1.5)
    t[::4] = 0.0
    for settings in ({}, {"temperature": 0.7}, {"temperature": 0}, {"temperature": t}, {"top_k": 1}, {"top_k": 5},
                     {"top_k": k}, {"top_p": 0.3}, {"top_p": rand(0.0, 1.1)}, {"min_p": rand(0.0, 0.2)}, {"min_p": 1.0},
                     {"top_p": 0.0}, {"top_k": V + 5, "top_p": 1.0, "min_p": 0.0},
                     {"temperature": t, "top_k": k, "top_p": rand(0.5, 1.0), "min_p": rand(0.0, 0.1)}):
        compare(logits, u, *pkg.token_sample(logits, u, **settings), **settings)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_at_odd_places_and_strides(dtype):
    logits, u, _ = make(6, 1037, dtype, 2)
    wide = torch.zeros(6, 1300, dtype=DT[dtype], device="cuda")
    for at in (0, 1, 3, 8):
        view = wide[:, at:at + 1037]
        view.copy_(logits)
        compare(logits, u, *pkg.token_sample(view, u, top_p=0.8), top_p=0.8)
    one = logits[:1].expand(6, 1037)   # one row for all, as for several draws of one prompt
    compare(one, u, *pkg.token_sample(one, u, top_k=50), top_k=50)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [7, 2000, 60000])
def test_ties(V, dtype):
    """Equal logits are kept by rising index: a few values over many tokens, and all alike."""
    g = torch.Generator().manual_seed(3)
    n = 6
    x = (torch.randint(0, 4, (n, V), generator=g) * 0.5).to(DT[dtype]).cuda()
    x[1] = 1.25
    u = torch.rand(n, generator=g).cuda()
    for settings in ({"top_k": 3}, {"top_k": V // 2 + 1}, {"top_p": 0.4}, {"top_p": 0.9, "top_k": V // 3 + 1}, {"min_p": 0.3},
                     {"temperature": 0}):
        compare(x, u, *pkg.token_sample(x, u, **settings), **settings)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [9, 3000])
def test_infinities_nan_and_extremes(V):
    g = torch.Generator().manual_seed(4)
    x = torch.randn(8, V, generator=g).cuda()
    inf = float("inf")
    x[0] = -inf                       # nothing to draw
    x[1, : V - 1] = -inf              # one
    x[2, 3] = float("nan")            # counts as -inf
    x[3, [2, 5]] = inf                # these two alone
    x[4] = float("nan")
    x[5] = torch.finfo(torch.float32).min
    x[6, 4] = torch.finfo(torch.float32).max
    x[7, ::2] = -inf
    u = torch.rand(8, generator=g).cuda()
    for settings in ({}, {"top_k": 3}, {"top_p": 0.5}, {"min_p": 0.5}, {"temperature": 0}, {"temperature": 1e-6},
                     {"temperature": 1e30}, {"top_k": 4, "top_p": 0.9, "temperature": 3.0}):
        compare(x, u, *pkg.token_sample(x, u, **settings), **settings)


@pytest.mark.gpu
def test_the_ends_of_u():
    x = torch.zeros(4, 1000, device="cuda")
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 0.5, 2.0 ** -30], device="cuda")
    ids, logprob = pkg.token_sample(x, u)
    assert ids.tolist() == [0, 999, 500, 0]
    assert torch.allclose(logprob, torch.full_like(logprob, -np.log(1000.0)), rtol=1e-6, atol=0)
    # out of its range: the ends
    assert pkg.token_sample(x, torch.tensor([-1.0, 1.0, 7.0, float("nan")], device="cuda"))[0].tolist() == [0, 999, 999, 0]


@pytest.mark.gpu
def test_settings_out_of_range_act_as_none():
    x, u, _ = make(4, 500, "f32", 5)
    want = pkg.token_sample(x, u)[0]
    bad = torch.tensor([-1.0, float("nan"), -1.0, float("nan")], device="cuda")
    assert torch.equal(pkg.token_sample(x, u, temperature=bad, min_p=bad)[0], want)
    assert torch.equal(pkg.token_sample(x, u, top_p=torch.full((4,), float("nan"), device="cuda"))[0], want)
    assert torch.equal(pkg.token_sample(x, u, top_k=-3, min_p=-1.0, top_p=2.0)[0], want)


@pytest.mark.gpu
def test_shares():
    """Draws over a grid of u hit each token by its share, to one draw."""
    x = torch.log(torch.tensor([0.05, 0.5, 0.15, 0.3], device="cuda"))[None].expand(10000, 4)
    u = (torch.arange(10000, device="cuda") + 0.5) / 10000
    count = torch.bincount(pkg.token_sample(x, u.float())[0], minlength=4)
    assert (count - torch.tensor([500, 5000, 1500, 3000], device="cuda")).abs().max() <= 1


@pytest.mark.gpu
def test_many_rows_another_stream_and_a_graph():
    x, u, _ = make(700, 997, "bf16", 6)
    want = pkg.token_sample(x, u, top_p=0.9, top_k=40)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan = pkg.TokenSamplePlan(x, u, top_p=0.9, top_k=40, stream=side)
    with torch.cuda.stream(side):
        plan()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        plan()
    plan.ids.fill_(-7)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(plan.ids, want[0]) and torch.equal(plan.logprob, want[1])
    compare(x[:40], u[:40], want[0][:40], want[1][:40], top_p=0.9, top_k=40)
    assert pkg.token_sample(x[:0], u[:0])[0].shape == (0,)


@pytest.mark.gpu
def test_offsets_past_31_bits():
    x, u, _ = make(2, 4096, "bf16", 7)
    base = torch.empty((1 << 31) + 8192, dtype=torch.bfloat16, device="cuda")
    far = base.as_strided((2, 4096), ((1 << 31) + 64, 1))
    far.copy_(x)
    assert torch.equal(pkg.token_sample(far, u, top_k=100)[0], pkg.token_sample(x, u, top_k=100)[0])


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkg.load_library()


def test_refusals_of_the_library(lib):
    A, vp = 0x100000, ctypes.c_void_p
    good = [vp(A)] * 8

    def call(p=good, rows=2, vocab=100, stride=100, io=0):
        s = pkg.lm_ops.token_sample_shape(rows, vocab, stride, 1.0, 1.0, 0.0, 0, io)
        return lib.token_sample(ctypes.byref(s), *p, None)

    assert call(rows=-1) == 1 and call(vocab=0) == 1 and call(stride=-1) == 1 and call(io=7) == 1
    assert call(vocab=(1 << 20) + 1) == 2 and call(rows=0) == 0
    for i in (0, 1, 6):   # logits, u, ids
        assert call(good[:i] + [None] + good[i + 1:]) == 1
    for i in range(8):
        assert call(good[:i] + [vp(A + 1)] + good[i + 1:]) == 1


@pytest.mark.gpu
def test_refusals_of_the_binding():
    x, u, _ = make(3, 50, "f32", 8)
    for bad in (dict(temperature=-1.0), dict(temperature=float("nan")), dict(top_p=float("nan")),
                dict(top_k=torch.ones(3, device="cuda")), dict(min_p=torch.ones(2, device="cuda"))):
        with pytest.raises(ValueError):
            pkg.token_sample(x, u, **bad)
    with pytest.raises(ValueError):
        pkg.token_sample(x.half(), u)
    with pytest.raises(ValueError):
        pkg.token_sample(x, u[:2])
    with pytest.raises(ValueError):
        pkg.token_sample(x[0], u)
    with pytest.raises(ValueError):
        pkg.token_sample(x.t(), u)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [40, 3001, 50000])
def test_numbers_at_and_beside_the_borders(V):
    """Random numbers that lie on a border between two tokens, as near as fp32 comes, and flat rows, whose borders lie
    everywhere: the draw is the exact one."""
    g = torch.Generator().manual_seed(9)
    n = 24
    x = torch.randn(n, V, generator=g) * torch.linspace(0, 4, n)[:, None]
    shares = torch.softmax(x.double(), 1).cumsum(1)
    at = torch.randint(0, V, (n,), generator=g)
    u = shares[torch.arange(n), at].float().clamp(max=1 - 2.0 ** -24)
    up = torch.nextafter(u, torch.ones(())).clamp(max=1 - 2.0 ** -24)
    for uu in (u, up, torch.nextafter(u, torch.zeros(()))):
        for rows in (n, 1):   # a block a row, and several
            d = x[:rows].cuda(), uu[:rows].cuda()
            compare(*d, *pkg.token_sample(*d))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [3, 200])   # several blocks a row, and one
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinite_temperature(dtype, n):
    # every logit above -inf weighs the same, however low it is
    V = 1000
    logits, u, _ = make(n, V, dtype, 7)
    logits[:, ::3] = -float("inf")
    logits[:, 1::7] = torch.finfo(DT[dtype]).min
    live = torch.isfinite(logits[0].float()).nonzero().flatten().cpu()
    for t in (float("inf"), torch.full((n,), float("inf"), device="cuda")):
        for settings in ({}, {"min_p": 0.5}, {"min_p": 1.0}):
            ids, lp = pkg.token_sample(logits, u, temperature=t, **settings)
            live_r = [(torch.isfinite(logits[r].float())).nonzero().flatten().cpu() for r in range(n)]
            want = torch.stack([x[int(float(u[r]) * len(x))] for r, x in enumerate(live_r)])
            assert torch.equal(ids.cpu(), want)
            assert torch.allclose(lp.cpu(), torch.full((n,), -float(np.log(len(live)))), rtol=1e-6, atol=0)
        ids, lp = pkg.token_sample(logits, u, temperature=t, top_k=5)
        for r in range(n):
            top = torch.sort(logits[r].float().cpu(), descending=True, stable=True)[1][:5].sort()[0]
            assert int(ids[r]) == int(top[int(float(u[r]) * 5)])
        assert torch.allclose(lp.cpu(), torch.full((n,), -float(np.log(5.0))), rtol=1e-6, atol=0)
