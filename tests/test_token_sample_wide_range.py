"""Drawing of tokens whose logits lie further apart than the largest fp32 number."""
import numpy as np
import pytest
import torch

import chunked_ssd_scan_gb300 as pkg
from tests import delta_reference as ref
from tests.parity_util import to_np
from tests.test_token_sample import compare


@pytest.mark.gpu
@pytest.mark.parametrize("n", [3, 200])   # several blocks a row, and one
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_distances_past_the_largest_number(dtype, n):
    V = 1000
    g = torch.Generator().manual_seed(11)
    most = float(torch.finfo(dtype).max)
    x = (torch.rand(n, V, generator=g, dtype=torch.float64) * 2 - 1) * most
    x[:, 3], x[:, 5] = most, -most
    x = x.to(dtype).cuda()
    u = torch.rand(n, generator=g).cuda()
    # a temperature of the same size: weights from 1 down to e^-6.8
    for settings in ({}, {"top_p": 0.6}, {"min_p": 0.05}, {"top_k": 100}, {"top_k": 700, "top_p": 0.9}):
        compare(x, u, *pkg.token_sample(x, u, temperature=1e38, **settings), temperature=1e38, **settings)
    # an infinite one: all weigh the same
    live = x.double().cpu().numpy()
    for settings, count in (({}, V), ({"min_p": 1.0}, V), ({"top_k": 40}, 40)):
        ids, logprob = pkg.token_sample(x, u, temperature=float("inf"), **settings)
        for r in range(n):
            kept = np.sort(np.argsort(-live[r], kind="stable")[:count])
            assert int(ids[r]) == kept[int(float(u[r]) * count)]
        assert np.allclose(to_np(logprob), -np.log(count), rtol=1e-6, atol=0)


@pytest.mark.gpu
def test_beside_infinities():
    """Distances that overflow are not distances from or to an infinity."""
    inf, most = float("inf"), float(torch.finfo(torch.float32).max)
    x = torch.tensor([[most, -most, -inf, 0.0], [inf, most, -most, -inf], [-most, -inf, -inf, -inf]], device="cuda")
    u = torch.tensor([0.9, 0.9, 0.9], device="cuda")
    for t in (1e38, 1.0, 1e-3):
        compare(x, u, *pkg.token_sample(x, u, temperature=t), temperature=t)
    ids, logprob = pkg.token_sample(x, u, temperature=inf)
    assert ids.tolist() == [3, 0, 0]
    assert np.allclose(to_np(logprob), [-np.log(3), 0, 0], rtol=1e-6, atol=0)
    assert ref.sample(to_np(x)[0], 0.9, temperature=1e38)[0] in (0, 1, 3)
