"""Gated delta rule on the tensor cores: waits that run out.  The index-checked build lets a test name a wait's site and the
warps in which it gives up at once; the call then ends by itself, reports the site, and leaves the device as it was for the
next call."""
import pytest
import torch

import chunked_ssd_scan_gb300 as pkg
from chunked_ssd_scan_gb300 import _build
from tests import test_gated_delta_rule as td

pytestmark = pytest.mark.gpu
ALL = -1


@pytest.fixture(scope="module")
def checked():
    return pkg.load_library(_build.build_checked())


@pytest.fixture(scope="module")
def plans():
    """Forward and backward plans of a shape, and their results, made once."""
    made = {}

    def get(shape):
        if shape not in made:
            d = td.inputs(*shape, "bf16", seed=51, dev="cuda")
            f = pkg.GatedDeltaRulePlan(*td.args(d), init_state=d["init"], return_states=True)
            b = pkg.GatedDeltaRuleBackwardPlan(*td.args(d), d["dy"], init_state=d["init"], dfinal=d["dfinal"])
            made[shape] = f, [t.clone() for t in f()], b, {k: v.clone() for k, v in b().items()}
        return made[shape]
    return get


def give_up(checked, plan, site, warps):
    """(status, site) of a call whose wait gives up, and of one after it."""
    header = plan.workspace[:256].view(torch.int32)
    header[6], header[7] = site, warps
    assert getattr(checked, plan._name)(*plan._args) == 0
    first = pkg.workspace_status(plan.workspace)
    header[6] = header[7] = 0
    assert getattr(checked, plan._name)(*plan._args) == 0
    return first, pkg.workspace_status(plan.workspace)


# one block of keys and several heads on it; two blocks of keys
SMALL, WIDE = (1, 200, 1, 2, 64, 64), (1, 330, 2, 2, 128, 128)


def forward(checked, plans, shape, site, warps):
    plan, want = plans(shape)[:2]
    assert give_up(checked, plan, site, warps) == (("SSD_ERR_TIMEOUT", site), ("SSD_OK", 0))
    assert all(torch.equal(a, b) for a, b in zip((plan.y, plan.final_state, plan.states), want))


def backward(checked, plans, shape, site, warps):
    plan, want = plans(shape)[2:]
    assert give_up(checked, plan, site, warps) == (("SSD_ERR_TIMEOUT", site), ("SSD_OK", 0))
    assert all(torch.equal(plan.grads[k], want[k]) for k in want)


@pytest.mark.parametrize("shape", [SMALL, WIDE], ids=str)
@pytest.mark.parametrize("site,warps", [(1, ALL), (2, ALL), (2, 1), (2, 2), (2, 8)], ids=str)
def test_chunks(checked, plans, site, warps, shape):
    forward(checked, plans, shape, site, warps)
    backward(checked, plans, shape, site, warps)


# in segments, too
LONG = (1, 1025, 2, 2, 128, 128)
ONE = [(site, 1 << w) for site in (21, 22, 23, 24) for w in (0, 6, 15)] + [(site, 1 << w) for site in (25, 26, 27) for w in (16, 19)]


@pytest.mark.parametrize("shape", [SMALL, LONG], ids=str)
@pytest.mark.parametrize("site,warps", [(site, ALL) for site in (10, *range(12, 20), *range(21, 28))] + ONE, ids=str)
def test_walk(checked, plans, site, warps, shape):
    """All warps of a role, or one of those that share a barrier: the others of its quarter must not wait for it."""
    forward(checked, plans, shape, site, warps)


ONE_BACK = ([(site, 1 << w) for site in (55, 56, 57, 58) for w in (0, 6, 15)]
            + [(site, 1 << w) for site in (59, 60, 61) for w in (16, 19)])


@pytest.mark.parametrize("shape", [SMALL, WIDE], ids=str)
@pytest.mark.parametrize("site,warps", [(site, ALL) for site in (*range(40, 44), *range(45, 54), *range(55, 62))] + ONE_BACK,
                         ids=str)
def test_walk_back(checked, plans, site, warps, shape):
    backward(checked, plans, shape, site, warps)


@pytest.mark.parametrize("shape", [SMALL, WIDE], ids=str)
@pytest.mark.parametrize("site,warps", [(site, w) for site in range(70, 76) for w in (ALL, 1, 1 << 6, 1 << 15)], ids=str)
def test_gradient(checked, plans, site, warps, shape):
    backward(checked, plans, shape, site, warps)
