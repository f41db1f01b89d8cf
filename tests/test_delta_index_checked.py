"""The index-checked build on the ways through the delta rule and the norm's gradient that the other tests of it leave out:
no store lies outside its array, and the results are the normal build's."""
import pytest
import torch

import chunked_ssd_scan_gb300 as pkg
from chunked_ssd_scan_gb300 import _build
from tests import test_gated_delta_rule as td
from tests import test_rms_norm as tn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def checked():
    return pkg.load_library(_build.build_checked())


def same(checked, plan, outs):
    plan()
    want = [o.clone() for o in outs()]
    for o in outs():
        o.zero_()
    assert getattr(checked, plan._name)(*plan._args) == 0
    assert pkg.workspace_status(plan.workspace) == ("SSD_OK", 0)
    assert all(torch.equal(a, b) for a, b in zip(outs(), want))


# segments and their carry, two tiles of values, wide heads, shared keys with a tail of one step, values past the gradient's
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1025, 2, 2, 128, 128), (1, 2113, 1, 2, 128, 200), (2, 100, 1, 2, 200, 40),
                                   (2, 193, 1, 3, 72, 24), (1, 70, 1, 1, 64, 264)], ids=str)
def test_delta_rule(checked, shape, dtype):
    d = td.inputs(*shape, dtype, seed=61, dev="cuda")
    f = pkg.GatedDeltaRulePlan(*td.args(d), init_state=d["init"], return_states=True)
    same(checked, f, lambda: (f.y, f.final_state, f.states))
    for states in (None, f.states):
        b = pkg.GatedDeltaRuleBackwardPlan(*td.args(d), d["dy"], init_state=d["init"], states=states, dfinal=d["dfinal"])
        same(checked, b, lambda: tuple(b.grads.values()))


# vectors of eight, four, two and one, rows beyond the registers, more rows than partial sums
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(300, 130), (1000, 2048), (5, 9001), (3000, 64), (2, 33001)], ids=str)
def test_norm_gradient(checked, shape, dtype):
    d = tn.inputs(*shape, dtype, seed=62, dev="cuda")
    rstd = torch.rsqrt(d["x"].float().square().mean(1))
    p = pkg.RMSNormBackwardPlan(d["x"], d["dy"], rstd, d["w"], dresidual=d["dres"])
    same(checked, p, lambda: tuple(p.grads.values()))
