"""Sizes of nothing, workspaces, streams and extreme arguments of the recurrence, the norm and the embedding."""
import ctypes

import pytest
import torch

import chunked_ssd_scan_gb300 as pkg


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(2, 0, 8), (5, 0, 12), (0, 3, 8), (3, 0, 2, 8)], ids=str)
def test_statistics_of_no_positions(shape, dtype):
    """Every value of mean and rstd is written: the mean of nothing is NaN."""
    x = torch.zeros(shape, dtype=dtype, device="cuda")
    mean, rstd = (torch.full((shape[0], 4), 3.0, device="cuda") for _ in range(2))
    y, m, r = pkg.group_norm_forward(x, 4, mean=mean, rstd=rstd)
    assert y.shape == x.shape and m.data_ptr() == mean.data_ptr()
    assert bool(torch.isnan(m).all()) and bool(torch.isnan(r).all()) and m.shape == r.shape == (shape[0], 4)
