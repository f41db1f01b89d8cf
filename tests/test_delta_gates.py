"""Gated delta rule: the gradient of the gates behind a reset of a large state, and decays between steps that lie far down
a chunk's sum of g."""
import math

import numpy as np
import pytest
import torch

import chunked_ssd_scan_gb300 as pkg
from tests import delta_reference as ref
from tests import test_gated_delta_rule as td
from tests.parity_util import to_np


# the CUDA cores (f32, bf16 behind an odd element, wide heads) and the tensor cores
@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 64, 1, 1, 64, 64), (2, 150, 2, 4, 60, 100), (1, 130, 1, 2, 128, 72),
                                   (1, 100, 1, 1, 200, 40), (1, 70, 1, 2, 64, 264)], ids=str)
@pytest.mark.parametrize("dtype,layout", [("f32", "plain"), ("bf16", "odd"), ("bf16", "plain")])
@pytest.mark.parametrize("size", [30.0, 1000.0])
def test_gate_gradient_behind_a_reset(size, dtype, layout, shape):
    """The initial state is large and cut off at step 8 by a decay of e^-30: what g's gradient is behind that does not
    depend on it, and is held to the same bound as without it."""
    d = td.inputs(*shape, dtype, seed=21, layout=layout, dev="cuda")
    d["init"] = torch.randn(d["init"].shape, generator=torch.Generator().manual_seed(22)).cuda() * size
    d["g"][:, 8] = -30.0
    h = td.host(d)
    want = ref.delta_grad(h["q"], h["k"], h["v"], h["g"], h["beta"], h["dy"], h["init"], None, h["dfinal"])
    got = td.run_backward(d, dtype, None)
    # (fp32 of a state that has decayed by e^-30 from 1000: 1e-10)
    ref.check(to_np(got["dg"])[:, 9:], want["dg"][:, 9:], dtype, "dg behind the reset")
    ref.check(to_np(got["dg"])[:, :9], want["dg"][:, :9], dtype, "dg up to the reset")


@pytest.mark.gpu
@pytest.mark.parametrize("H", [32, 96])   # few sequences, and many
def test_decays_between_neighbours_far_down_a_chunk(H):
    """Two steps write the same key, the second one v = 0 with beta 1 behind a decay of a half: what is left is a half of
    the first write less a half of it, nothing.  The sum of g up to there is -20 to -79 (by the chunk's first step, before
    which there is no state), where fp32 is off by up to 3.8e-6: sums as pairs of floats bring that down to the rounding of the
    decays themselves.  Of the half: two exponentials of 2 units of 2^-24 with a product each for the low part (2), two
    products more (2), the decay behind the first step (3), four additions: 15 units, rounded up to 16; the two terms of the
    operands hold a half and what it is off by exactly."""
    b, T, K, V, at = 1, 128, 64, 64, 40
    g = torch.zeros(b, T, H)
    g[:, 0] = -20 - 59.2 * torch.rand(b, H, generator=torch.Generator().manual_seed(23))
    g[:, at + 1] = -math.log(2)
    beta = torch.zeros(b, T, H)
    beta[:, at:at + 2] = 1
    k = torch.zeros(b, T, 1, K)
    k[:, at:at + 2, :, 0] = 1
    v = torch.zeros(b, T, H, V)
    v[:, at] = 1
    a = (torch.zeros(b, T, 1, K).bfloat16(), k.bfloat16(), v.bfloat16(), g, beta)
    y, final, states = pkg.gated_delta_rule_forward(*(t.cuda() for t in a), return_states=True)
    assert float(final.abs().max()) <= 0.5 * 16 * 2.0 ** -24
    assert float(states[:, 1].abs().max()) <= 0.5 * 16 * 2.0 ** -24
    # a write's gradient goes the same way back: of dfinal = 1 for that key, half through the decay, less half of it
    d = pkg.gated_delta_rule_backward(*(t.cuda() for t in a), torch.zeros(b, T, H, V).bfloat16().cuda(), states=states,
                                      dfinal=torch.ones(b, H, V, K, device="cuda"))
    assert float(d["dv"][:, at].float().abs().max()) <= 0.5 * 16 * 2.0 ** -24 * (1 + ref.BF16_REL)
    assert np.allclose(to_np(d["dv"][:, at + 1]), 1.0, rtol=0, atol=2.0 ** -20)
