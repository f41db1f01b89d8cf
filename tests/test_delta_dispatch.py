"""Forms of the delta rule that sizes, strides and the number of sequences choose: segments of few sequences, several
tiles of values, states formed anew, the walk on the CUDA cores beside the tensor cores, the index-checked build."""
import pytest
import torch

import chunked_ssd_scan_gb300 as pkg
from chunked_ssd_scan_gb300 import _build
from tests import delta_reference as ref
from tests import test_gated_delta_rule as td
from tests.parity_util import to_np

pytestmark = pytest.mark.gpu


# one sequence of many chunks (segments, a last one that is shorter), values in two tiles, a tail of one step
@pytest.mark.parametrize("shape", [(1, 3000, 1, 1, 64, 64), (1, 2113, 1, 2, 128, 200), (2, 1345, 1, 1, 40, 264),
                                   (1, 1025, 2, 2, 128, 128)], ids=str)
def test_segments(shape):
    d = td.inputs(*shape, "bf16", seed=31, dev="cuda", slow=200.0)   # memories across segments
    td.check_forward(td.run_forward(d, "bf16"), d, "bf16")


# many short sequences: half a chunk, around its end, no room for them on the CUDA cores at once
@pytest.mark.parametrize("shape", [(40, 32, 2, 2, 64, 64), (24, 65, 4, 4, 128, 128), (30, 64, 2, 4, 72, 40),
                                   (11, 100, 1, 4, 8, 136), (300, 33, 1, 2, 16, 8), (50, 17, 1, 2, 64, 64)], ids=str)
def test_many_short_sequences(shape):
    d = td.inputs(*shape, "bf16", seed=38, dev="cuda")
    td.check_forward(td.run_forward(d, "bf16"), d, "bf16")
    td.check_backward(td.run_backward(d, "bf16", None), d, "bf16")


@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 8, 8), (2, 5, 1, 3, 128, 128), (1, 31, 2, 2, 64, 40)], ids=str)
def test_gradients_of_a_few_steps(shape):
    d = td.inputs(*shape, "bf16", seed=39, dev="cuda")
    td.check_backward(td.run_backward(d, "bf16", None), d, "bf16")


def test_states_that_are_not_on_a_16_byte_border():
    d = td.inputs(2, 700, 1, 2, 64, 64, "bf16", seed=40, dev="cuda")
    off = {}
    for k in ("init", "dfinal"):
        off[k] = torch.zeros(d[k].numel() + 1, device="cuda")[1:].view(d[k].shape)
        off[k].copy_(d[k])
    a = pkg.gated_delta_rule_forward(*td.args(d), init_state=d["init"])
    b = pkg.gated_delta_rule_forward(*td.args(d), init_state=off["init"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    td.check_backward(pkg.gated_delta_rule_backward(*td.args(d), d["dy"], init_state=off["init"], dfinal=off["dfinal"]), d, "bf16")


@pytest.mark.parametrize("shape", [(1, 1300, 1, 2, 128, 128), (2, 200, 2, 4, 64, 96)], ids=str)
def test_states_known_or_formed_anew_give_the_same_gradients(shape):
    d = td.inputs(*shape, "bf16", seed=32, dev="cuda")
    f = pkg.gated_delta_rule_forward(*td.args(d), init_state=d["init"], return_states=True)
    one = pkg.gated_delta_rule_backward(*td.args(d), d["dy"], init_state=d["init"], states=f[2], dfinal=d["dfinal"])
    two = pkg.gated_delta_rule_backward(*td.args(d), d["dy"], init_state=d["init"], dfinal=d["dfinal"])
    for k in one:
        assert torch.equal(one[k], two[k]), k


@pytest.mark.parametrize("V", [64, 128])
def test_both_cores_agree(V):
    """The same values at a place the tensor-core kernels take, and at an odd element that they do not."""
    d = td.inputs(2, 330, 1, 2, 64, V, "bf16", seed=33, dev="cuda")
    odd = td.inputs(2, 330, 1, 2, 64, V, "bf16", seed=33, layout="odd", dev="cuda")
    a = pkg.gated_delta_rule_forward(*td.args(d), init_state=d["init"])
    b = pkg.gated_delta_rule_forward(*td.args(odd), init_state=odd["init"])
    ref.check(to_np(a[1]), to_np(b[1]), "bf16", "final_state")
    ga = pkg.gated_delta_rule_backward(*td.args(d), d["dy"], init_state=d["init"])
    gb = pkg.gated_delta_rule_backward(*td.args(odd), odd["dy"], init_state=odd["init"])
    for k in ("dg", "dbeta", "dinit"):
        ref.check(to_np(ga[k]), to_np(gb[k]), "bf16", k)


def test_many_chunks_of_a_block():
    """More chunks and key heads than SMs, three heads on each: a block of the gradient's goes through several of them."""
    d = td.inputs(3, 64 * 30 + 5, 2, 6, 64, 64, "bf16", seed=34, dev="cuda")
    td.check_backward(td.run_backward(d, "bf16", None), d, "bf16")


def test_calls_on_two_streams_at_once():
    d = [td.inputs(2, 700, 1, 4, 128, 128, "bf16", seed=35 + i, dev="cuda") for i in range(2)]
    want = [pkg.gated_delta_rule_backward(*td.args(x), x["dy"], init_state=x["init"]) for x in d]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in d]
    plans = [pkg.GatedDeltaRuleBackwardPlan(*td.args(x), x["dy"], init_state=x["init"], stream=s) for x, s in zip(d, streams)]
    torch.cuda.synchronize()
    for _ in range(3):
        for plan in plans:
            plan()
    torch.cuda.synchronize()
    for plan, w in zip(plans, want):
        assert all(torch.equal(plan.grads[k], w[k]) for k in w)


def test_a_workspace_with_anything_in_it_but_its_header():
    d = td.inputs(1, 1200, 1, 2, 64, 64, "bf16", seed=37, dev="cuda")
    plan = pkg.GatedDeltaRulePlan(*td.args(d), return_states=True)
    want = [t.clone() for t in plan()]
    plan.workspace[256:].fill_(0xff)
    for t in plan():
        pass
    assert all(torch.equal(a, b) for a, b in zip((plan.y, plan.final_state, plan.states), want))
    back = pkg.GatedDeltaRuleBackwardPlan(*td.args(d), d["dy"], states=plan.states)
    want = {k: v.clone() for k, v in back().items()}
    back.workspace[256:].fill_(0xff)
    assert all(torch.equal(v, want[k]) for k, v in back().items())


@pytest.fixture(scope="module")
def checked():
    return pkg.load_library(_build.build_checked())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 77, 1, 2, 30, 17), (1, 200, 2, 2, 64, 72)], ids=str)
def test_index_checked_build(checked, shape, dtype):
    d = td.inputs(*shape, dtype, seed=36, dev="cuda")
    plan = pkg.GatedDeltaRulePlan(*td.args(d), init_state=d["init"], return_states=True)
    back = pkg.GatedDeltaRuleBackwardPlan(*td.args(d), d["dy"], init_state=d["init"], dfinal=d["dfinal"])
    for p, outs in ((plan, lambda: (plan.y, plan.final_state, plan.states)), (back, lambda: tuple(back.grads.values()))):
        p()
        want = [o.clone() for o in outs()]
        assert getattr(checked, p._name)(*p._args) == 0
        assert pkg.workspace_status(p.workspace) == ("SSD_OK", 0)
        assert all(torch.equal(a, b) for a, b in zip(outs(), want))
