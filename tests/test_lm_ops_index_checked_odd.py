"""The index-checked debug library on the recurrence's slower forms (GPU): tiles with huge states and with input
gates that are nearly closed, at the sizes whose edges an out-of-bounds store would hide in."""
import pytest
import torch

import chunked_ssd_scan_gb300 as pkg
from chunked_ssd_scan_gb300 import _build
from tests import test_gated_recurrence as tr
from tests.test_lm_ops_index_checked import both

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def checked():
    return pkg.load_library(_build.build_checked())


# huge x in some steps, a huge initial state, a huge dy, a huge dfinal: each makes other tiles odd, in their maps or
# in what their warps start from; strong decays take the mixed forms
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["plain", "fused", "odd"])
@pytest.mark.parametrize("what", ["gates", "x", "init", "dy", "dfinal", "strong"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 65, 66), (2, 777, 500), (2, 300, 31)], ids=str)
def test_recurrence(checked, shape, what, layout, dtype):
    b, T, D = shape
    d = tr.inputs(*shape, dtype, seed=61, layout=layout, dev="cuda")
    if what == "gates":
        d["gx"][:, ::7] = -50.0
    elif what == "strong":
        d["decay"] = torch.linspace(-2.0, 1.0, D, device="cuda")
    elif what in ("x", "dy"):
        d[what][:, T // 3, ::3] = 2.0 ** 110
    else:
        d[what][:, ::3] = 2.0 ** 110
    args = (d["x"], d["ga"], d["gx"], d["decay"])
    plan = pkg.GatedRecurrencePlan(*args, init_state=d["init"], return_states=True)
    both(checked, plan, (plan.y, plan.final_state, plan.states))
    back = pkg.GatedRecurrenceBackwardPlan(*args, d["dy"], init_state=d["init"], states=plan.states,
                                           dfinal=d["dfinal"])
    both(checked, back, tuple(back.grads.values()))
    assert bool(torch.isfinite(plan.y.float()).all()) and bool(torch.isfinite(back.grads["dx"].float()).all())
