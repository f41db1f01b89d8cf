"""Gated delta rule on the CUDA cores: infinities in calls whose last tile has steps past the end."""
import numpy as np
import pytest
import torch

import chunked_ssd_scan_gb300 as pkg
from tests import delta_reference as ref
from tests import test_gated_delta_rule as td
from tests.parity_util import to_np


FULL = (64, 128)   # keys that fill the lanes; elsewhere an infinity may be NaN


def same_kind(got, want, what, exact=True):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    if not exact:
        assert np.array_equal(np.isfinite(got), np.isfinite(want)), what
        return
    for kind in (np.isnan, np.isposinf, np.isneginf):
        assert np.array_equal(kind(got), kind(want)), (what, kind.__name__, int(kind(got).sum()), int(kind(want).sum()))


# T: within a tile of 8 or 16 steps, at its end, in the second; K: all lanes full, some keys short, wider
@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 16, 21])
@pytest.mark.parametrize("K", [1, 30, 64, 100, 128, 200])
@pytest.mark.parametrize("both_signs", [False, True])
def test_an_infinite_value_of_the_last_step(both_signs, K, T):
    """Its write makes a row of the state infinite, and that step's output with it; nothing else."""
    d = td.inputs(2, T, 1, 2, K, 20, seed=41, dev="cuda")
    for t in (d["q"], d["k"]):
        t.abs_()   # an output of infinities of one sign
    d["v"][1, T - 1, 1, 7] = float("inf")
    if both_signs:
        d["k"][1, T - 1, 0, K // 2:].neg_()
    h = td.host(d)
    with np.errstate(invalid="ignore"):
        want = ref.delta(h["q"], h["k"], h["v"], h["g"], h["beta"], h["init"])
    y, final, states = td.run_forward(d, "f32")
    same_kind(to_np(y), want[0], "y", K in FULL)
    same_kind(to_np(final), want[1], "final_state")
    same_kind(to_np(states), want[2], "states")
    assert int(torch.isinf(final).sum()) == K
    # the same by the single step, of the state before it
    before = pkg.gated_delta_rule_forward(*(t[:, :T - 1] for t in td.args(d)), init_state=d["init"])[1]
    y1, s1 = pkg.gated_delta_rule_step(*(t[:, T - 1] for t in td.args(d)), before)
    same_kind(to_np(y1), want[0][:, -1], "y of a step", K in FULL)
    same_kind(to_np(s1), want[1], "state of a step")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 16, 21])
@pytest.mark.parametrize("K", [1, 30, 64, 100, 200])
def test_an_infinite_gradient_of_the_last_step(K, T):
    """dy or dfinal of one value infinite: dv of the last step is, and dbeta; the steps before get what the formula gives."""
    for name in ("dy", "dfinal"):
        d = td.inputs(1, T, 1, 2, K, 20, seed=42, dev="cuda")
        for t in (d["q"], d["k"]):
            t.abs_()
        if name == "dy":
            d["dy"][0, T - 1, 1, 7] = float("inf")
        else:
            d["dfinal"][0, 1, 7] = float("inf")
        h = td.host(d)
        with np.errstate(invalid="ignore"):
            want = ref.delta_grad(h["q"], h["k"], h["v"], h["g"], h["beta"], h["dy"], h["init"], None, h["dfinal"])
        got = td.run_backward(d, "f32", None)
        for n in ("dv", "dbeta", "dinit"):
            same_kind(to_np(got[n]), want[n], f"{n} of {name}", K in FULL)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_gradients_of_queries_before_a_bad_value(bad):
    """A query's gradient hangs on the steps up to it alone: a bad value further on in its chunk does not reach it."""
    d = td.inputs(1, 50, 1, 2, 30, 20, seed=43, dev="cuda")
    want = pkg.gated_delta_rule_backward(*td.args(d), d["dy"], init_state=d["init"])["dq"]
    d["v"][0, 33, 1, 4] = bad
    got = pkg.gated_delta_rule_backward(*td.args(d), d["dy"], init_state=d["init"])["dq"]
    assert torch.equal(got[:, :33], want[:, :33])
    assert bool((~torch.isfinite(got[:, 33:])).any())
