"""The example model on the delta rule: it runs, its gradients agree with differences, serving a prompt and token by token
gives the logits of the whole sequence, and what it draws is likely under them."""
import os
import sys

import pytest
import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import delta_lm as lm  # noqa: E402

pytestmark = pytest.mark.gpu


def test_it_trains_and_draws():
    p, losses = lm.train(3, log=lambda s: None)
    assert all(torch.isfinite(torch.tensor(losses)))
    ids, logprob = lm.generate(p, lm.batch(7, size=3, length=20)[:, :20].contiguous(), 6, top_k=10, temperature=0.8)
    assert ids.shape == logprob.shape == (3, 6) and bool((ids >= 0).all()) and bool((logprob <= 0).all())
    again = lm.generate(p, lm.batch(7, size=3, length=20)[:, :20].contiguous(), 6, top_k=10, temperature=0.8)
    assert torch.equal(ids, again[0])


def test_serving_gives_the_logits_of_the_whole_sequence():
    p = lm.make_params(1)
    text = lm.batch(5, size=3, length=75)[:, :75].contiguous()
    whole = lm.forward(p, text).detach()
    logits, states = lm.serve(p, text[:, :70].contiguous())
    # fp32 through three norms and two rules, summed in other orders: 1e-4 of the logits' size
    top = 1e-3 * float(whole.abs().max())
    assert float((logits - whole[:, 69]).abs().max()) <= top
    for t in range(70, 75):
        logits, states = lm.serve(p, text[:, t:t + 1].contiguous(), states)
        assert float((logits - whole[:, t]).abs().max()) <= top
    greedy, _ = lm.generate(p, text, 1, temperature=0.0)
    assert torch.equal(greedy[:, 0], whole[:, -1].argmax(-1))


def test_gradients_of_the_whole_model_against_differences():
    p = lm.make_params(3)
    text = lm.batch(11, size=2, length=70)

    def loss():
        logits = lm.forward(p, text[:, :-1].contiguous()).double()
        return F.cross_entropy(logits.reshape(-1, lm.VOCAB), text[:, 1:].reshape(-1))

    loss().backward()
    gen = torch.Generator().manual_seed(1)
    for k in p:
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
