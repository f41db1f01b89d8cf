"""The index-checked debug library on the recurrence, the norm and the embedding (GPU): at the sizes whose
edges an out-of-bounds store would hide in, no check may fire and the outputs are the normal
library's, bit for bit."""
import pytest
import torch

import chunked_ssd_scan_gb300 as pkg
from chunked_ssd_scan_gb300 import _build
from tests import test_embedding as te
from tests import test_gated_recurrence as tr
from tests import test_group_norm as tn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def checked():
    return pkg.load_library(_build.build_checked())


def both(checked, plan, outputs):
    """Runs the plan through the normal and the checked library; the workspace's error word stays clean."""
    plan()
    torch.cuda.synchronize()
    want = [o.clone() for o in outputs]
    for o in outputs:
        o.fill_(float("nan"))
    st = getattr(checked, plan._name)(*plan._args)
    assert st == 0, pkg.STATUS.get(st, st)
    assert pkg.workspace_status(plan.workspace) == ("SSD_OK", 0)
    for o, w in zip(outputs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["fused", "odd"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 65, 66), (2, 777, 500), (2, 300, 31)], ids=str)
def test_recurrence(checked, shape, layout, dtype):
    d = tr.inputs(*shape, dtype, seed=21, layout=layout, dev="cuda")
    args = (d["x"], d["ga"], d["gx"], d["decay"])
    plan = pkg.GatedRecurrencePlan(*args, init_state=d["init"], return_states=True)
    both(checked, plan, (plan.y, plan.final_state, plan.states))
    back = pkg.GatedRecurrenceBackwardPlan(*args, d["dy"], init_state=d["init"], states=plan.states,
                                           dfinal=d["dfinal"])
    both(checked, back, tuple(back.grads.values()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["fused", "odd"])
@pytest.mark.parametrize("shape", [(7, 1, 96, 12), (9, 1, 130, 13), (2, 1, 5000, 1), (2, 1000, 320, 32),
                                   (3, 64, 66, 11), (2, 3, 20000, 1), (300, 1, 520, 40)], ids=str)
def test_norm(checked, shape, layout, dtype):
    N, S, C, G = shape
    d = tn.inputs(N, S, C, dtype, seed=22, layout=layout, dev="cuda")
    plan = pkg.GroupNormPlan(d["x"], G, d["w"], d["bias"])
    both(checked, plan, (plan.y, plan.mean, plan.rstd))
    back = pkg.GroupNormBackwardPlan(d["x"], d["dy"], G, plan.mean, plan.rstd, d["w"], d["bias"])
    both(checked, back, tuple(back.grads.values()))


@pytest.mark.parametrize("case", [("zipf", 4097, 5000, 65), ("one", 500, 300, 40), ("ends", 900, 129, 200),
                                  ("zipf", 140001, 70000, 8)], ids=str)
def test_embedding_gradient(checked, case):
    kind, n, V, D = case
    ids = te.make_ids(kind, n, V, seed=23).cuda()
    dout = torch.randn(n, D, generator=torch.Generator().manual_seed(24)).cuda()
    plan = pkg.EmbeddingBackwardPlan(ids, dout, V)
    both(checked, plan, (plan.dtable,))
