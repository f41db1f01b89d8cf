"""Forms of the recurrence, the norm and the embedding that only some sizes, strides or alignments reach
(GPU), each against the fp64 form."""
import numpy as np
import pytest
import torch

import chunked_ssd_scan_gb300 as pkg
from tests import lm_reference as ref
from tests import test_embedding as te
from tests import test_gated_recurrence as tr
from tests import test_group_norm as tn
from tests.parity_util import to_np

pytestmark = pytest.mark.gpu


def moved(d, how, dtype):
    """The inputs of test_gated_recurrence.inputs with other strides: what the axes of a model's tensors may be."""
    d = dict(d)
    b, T, D = d["x"].shape
    if how == "dy_steps":        # the gradient of a mean over the steps
        d["dy"] = d["dy"][:, :1].expand(b, T, D)
    elif how == "dy_all":
        d["dy"] = d["dy"][:1, :1].expand(b, T, D)
    elif how == "x_batch":       # one sequence under several gates
        d["x"] = d["x"][:1].expand(b, T, D)
    elif how == "gates_steps":   # gates that do not change along time
        for k in ("ga", "gx"):
            d[k] = d[k][:, :1].expand(b, T, D)
    elif how == "time_major":    # [T,b,D] in memory: the batch stride is the smaller one
        for k in ("x", "ga", "gx", "dy"):
            d[k] = d[k].transpose(0, 1).contiguous().transpose(0, 1)
    elif how == "each_its_own":  # contiguous, time-major, a slice of wider rows, a slice that starts one element late
        d["ga"] = d["ga"].transpose(0, 1).contiguous().transpose(0, 1)
        d["gx"] = torch.cat((d["gx"], d["gx"]), 2)[..., D:]
        d["dy"] = torch.cat((d["dy"][..., :1], d["dy"]), 2)[..., 1:]
    return d


# D: a multiple of 8 but not of a tile's width, and one that is odd (2-byte copies for bf16)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(3, 200, 72), (2, 129, 200), (2, 150, 31)], ids=str)
@pytest.mark.parametrize("how", ["dy_steps", "dy_all", "x_batch", "gates_steps", "time_major", "each_its_own"])
def test_recurrence_strides(how, shape, dtype):
    d = moved(tr.inputs(*shape, dtype, seed=31, dev="cuda"), how, dtype)
    args = (d["x"], d["ga"], d["gx"], d["decay"])
    plan = pkg.GatedRecurrencePlan(*args, c=tr.C, init_state=d["init"], return_states=True)
    y, fin, states = plan()
    assert pkg.workspace_status(plan.workspace) == ("SSD_OK", 0)
    ry, rf, rs = tr.reference(d)
    ref.check(to_np(y), ry, tr.REL[dtype], "y")
    ref.check(to_np(fin), rf, 0.0, "final_state", scale=ry[:, -1])
    ref.check(to_np(states), rs, 0.0, "states")
    back = pkg.GatedRecurrenceBackwardPlan(*args, d["dy"], c=tr.C, init_state=d["init"], states=states,
                                           dfinal=d["dfinal"])
    g = {k: to_np(v) for k, v in back().items()}
    assert pkg.workspace_status(back.workspace) == ("SSD_OK", 0)
    r = tr.reference_grad(d)
    for k in ("dx", "dgate_x", "dgate_a"):
        ref.check(g[k], r[k], tr.REL[dtype], k)
    b, T, _ = shape
    # the difference in dl is as in the contiguous form; G along broadcast steps grows to 1 / (1 - a) <= 1000
    # times dy where dy does not change sign, so the sums' scale goes with the terms' own
    size = np.abs(r["ddecay"]) + np.sqrt(b * T) * 4 * max(1.0, np.abs(r["dx"]).max())
    ref.check(g["ddecay"], r["ddecay"], 0.0, "ddecay", scale=size)
    ref.check(g["dinit"], r["dinit"], 0.0, "dinit")


# more samples than the gradient sums take side by side, in maps and in tokens whose groups no token kernel holds
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", None])
@pytest.mark.parametrize("layout", ["plain", "odd"])
@pytest.mark.parametrize("shape", [(1500, 4, 24, 3), (1500, 1, 1031, 1), (913, 2, 40, 5), (3000, 17, 16, 1),
                                   (2100, 3, 600, 2)], ids=str)
def test_norm_backward_of_many_samples(shape, layout, act, dtype):
    N, S, C, G = shape
    d = tn.inputs(N, S, C, dtype, seed=32, layout=layout, dev="cuda")
    y, mean, rstd = pkg.group_norm_forward(d["x"], G, d["w"], d["bias"], activation=act)
    x, dy, w, b = (to_np(d[k]) for k in ("x", "dy", "w", "bias"))
    ref.check(to_np(y), ref.group_norm(x, G, w, b, act=act)[0], tn.REL[dtype], "y")
    plan = pkg.GroupNormBackwardPlan(d["x"], d["dy"], G, mean, rstd, d["w"], d["bias"], activation=act)
    g = plan()
    assert pkg.workspace_status(plan.workspace) == ("SSD_OK", 0)
    r = ref.group_norm_grad(x, dy, G, w, b, act=act)
    size = np.abs(to_np(rstd)).mean() * 1.5
    ref.check(to_np(g["dx"]), r["dx"], tn.REL[dtype], "dx", scale=np.maximum(np.abs(r["dx"]), size))
    for k in ("dweight", "dbias"):
        ref.check(to_np(g[k]), r[k], 0.0, k, scale=np.abs(r[k]) + np.sqrt(N * S))
    again = pkg.group_norm_backward(d["x"], d["dy"], G, mean, rstd, d["w"], d["bias"], activation=act)
    assert all(torch.equal(again[k], g[k]) for k in g)
    only = pkg.group_norm_backward(d["x"], d["dy"], G, mean, rstd, d["w"], d["bias"], activation=act, param_grads=False)
    assert torch.equal(only["dx"], g["dx"])


# tokens in one group that is too wide for a token kernel, with rows that the widest vectors divide
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [3, 950])
def test_norm_of_very_wide_tokens(N, dtype):
    C = 16384
    d = tn.inputs(N, 1, C, dtype, seed=33, dev="cuda")
    y, mean, rstd = pkg.group_norm_forward(d["x"], 1, d["w"], d["bias"])
    x, dy, w, b = (to_np(d[k]) for k in ("x", "dy", "w", "bias"))
    ref.check(to_np(y), ref.group_norm(x, 1, w, b)[0], tn.REL[dtype], "y")
    g = pkg.group_norm_backward(d["x"], d["dy"], 1, mean, rstd, d["w"], d["bias"])
    r = ref.group_norm_grad(x, dy, 1, w, b)
    size = np.abs(to_np(rstd)).mean() * 1.5
    ref.check(to_np(g["dx"]), r["dx"], tn.REL[dtype], "dx", scale=np.maximum(np.abs(r["dx"]), size))
    for k in ("dweight", "dbias"):
        ref.check(to_np(g[k]), r[k], 0.0, k, scale=np.abs(r[k]) + np.sqrt(N))


# sequences enough for two a thread, an odd number of them, and one row that is not aligned for it
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["plain", "fused", "odd"])
@pytest.mark.parametrize("bD", [(257, 2560), (512, 1216), (2049, 305)], ids=str)
def test_step_of_many_sequences(bD, layout, dtype):
    b, D = bD
    d = tr.inputs(b, 1, D, dtype, seed=34, layout=layout, dev="cuda")
    ry, rf, _ = tr.reference(d)
    y, state = pkg.gated_recurrence_step(d["x"][:, 0], d["ga"][:, 0], d["gx"][:, 0], d["decay"], d["init"], c=tr.C)
    ref.check(to_np(y), ry[:, 0], tr.REL[dtype], "y")
    ref.check(to_np(state), rf, 0.0, "state")


# more tokens than 64 tiles of 2048 sorted keys, keys of one, two and three digits
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("idt", [torch.int32, torch.int64], ids=["i32", "i64"])
@pytest.mark.parametrize("case", [("zipf", 131073, 70000, 24), ("zipf", 300001, 90001, 12), ("uniform", 140001, 200, 40),
                                  ("one", 200000, 70000, 8), ("ends", 131072 + 7, 500, 33),
                                  ("uniform", 131072, 300, 20)], ids=str)
def test_embedding_gradient_of_many_tokens(case, idt, dtype):
    kind, n, V, D = case
    ids = te.make_ids(kind, n, V, seed=35).to(idt).cuda()
    dout = torch.randn(n, D, generator=torch.Generator().manual_seed(36)).to(te.DT[dtype]).cuda()
    plan = pkg.EmbeddingBackwardPlan(ids, dout, V, scale=0.3)
    g = plan()
    assert pkg.workspace_status(plan.workspace) == ("SSD_OK", 0)
    npids = ids.cpu().numpy().astype(np.int64)
    r = ref.embedding_grad(npids, to_np(dout), V, np.float64(np.float32(0.3)))
    # as in test_embedding: a row is a sum of `count` terms of size 0.3
    count = np.bincount(npids[(npids >= 0) & (npids < V)], minlength=V)[:, None]
    got = to_np(g)
    assert np.all(np.abs(got - r) <= 2e-5 * 0.3 * np.sqrt(count) * (1 + np.abs(r)))
    assert np.all(got[count[:, 0] == 0] == 0)
    assert torch.equal(pkg.embedding_backward(ids, dout, V, scale=0.3), g)
