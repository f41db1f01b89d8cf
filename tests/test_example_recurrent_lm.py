"""The example model on the GPU: it learns, its gradients agree with differences, and the token by token
form gives the logits of the whole sequence."""
import os
import sys

import pytest
import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import recurrent_lm as lm  # noqa: E402

pytestmark = pytest.mark.gpu


def test_training_lowers_the_loss_and_serving_agrees():
    p, losses = lm.train(40, log=lambda s: None)
    # log(64) = 4.16 at the start; 40 steps have to take it well below that of guessing
    assert losses[0] > 3.5 and losses[-1] < 0.75 * losses[0], (losses[0], losses[-1])
    text = lm.batch(5, size=3, length=70)
    whole = lm.forward(p, text[:, :-1].contiguous()).detach()
    served, states = lm.serve(p, text[:, :40])
    rest, _ = lm.serve(p, text[:, 40:-1], states)
    # fp32 through two blocks and three norms, summed in other orders: 1e-4 of the logits' size
    both = torch.cat((served, rest), 1)
    assert float((both - whole).abs().max()) <= 1e-3 * float(whole.abs().max())


def test_gradients_of_the_whole_model_against_differences():
    p = lm.make_params(3)
    text = lm.batch(11, size=2, length=70)

    def loss():
        logits = lm.forward(p, text[:, :-1].contiguous()).double()
        return F.cross_entropy(logits.reshape(-1, lm.VOCAB), text[:, 1:].reshape(-1))

    loss().backward()
    gen = torch.Generator().manual_seed(1)
    for k in ("table", "sin", "rin", "decay", "rhw", "snb", "out"):
        v = torch.randn(p[k].shape, generator=gen).cuda()
        # a step of 1e-2 parameter units along the direction: the cubic term is some 1e-3 of the derivative's
        # scale, the loss's rounding (1e-6) 1e-4 of a unit
        eps = 1e-2 / float(v.norm()) * float(p[k].detach().norm().clamp(min=1.0))
        with torch.no_grad():
            p[k] += eps * v
            up = float(loss())
            p[k] -= 2 * eps * v
            down = float(loss())
            p[k] += eps * v
        num, ana = (up - down) / (2 * eps), float((p[k].grad * v).sum())
        size = float(p[k].grad.norm())
        assert abs(num - ana) <= 2e-2 * max(abs(ana), size) + 1e-4 / eps * 1e-2, k
