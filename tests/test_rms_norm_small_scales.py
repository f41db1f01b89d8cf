"""8-bit outputs of the root-mean-square norm whose scales are so small that their reciprocal is no fp32 number: blocks of
channels with next to no weight, rows of subnormal values."""
import numpy as np
import pytest
import torch

import chunked_ssd_scan_gb300 as pkg
from tests import delta_reference as ref
from tests.parity_util import to_np

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
STEP = 2.0 ** -149   # of subnormal fp32
UNIT = 64 * 2.0 ** -24   # a row's sum of squares and an output's three products, as in the tests of ordinary rows


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("quantize", ["token", "block"])
@pytest.mark.parametrize("odd", [False, True])   # rows on 16-byte borders, and behind an odd element
@pytest.mark.parametrize("C", [128, 264, 2048, 33001])
@pytest.mark.parametrize("small", [1e-37, 1e-38, 3e-40, 2e-42, 1e-45])
def test_quotients_of_small_scales(small, C, odd, quantize, dtype):
    g = torch.Generator().manual_seed(1)
    N = 5
    x = torch.randn(N, C, generator=g)
    w = torch.ones(C) if quantize == "block" else torch.full((C,), small)
    w[:128] = small * torch.rand(128, generator=g)
    w[5:60:3] = 0.0                       # exact zeros among them
    x[2] *= small * 1e3                   # and a row of next to nothing
    wide = torch.zeros(N, C + 1, dtype=DT[dtype], device="cuda")
    view = wide[:, 1:] if odd else torch.empty(N, C, dtype=DT[dtype], device="cuda")
    view.copy_(x)
    y, _, rstd, scale = pkg.rms_norm_forward(view, w.cuda(), quantize=quantize)
    ry, _, rr = ref.rms_norm(to_np(view), to_np(w))
    block = C if quantize == "token" else 128
    blocks = -(-C // block)
    most = np.abs(np.pad(ry, ((0, 0), (0, blocks * block - C)))).reshape(N, blocks, block).max(2)
    got, sc = to_np(y.float()), to_np(scale)
    assert np.isfinite(got).all() and (sc > 0).all()
    assert (got[:, 5:60:3] == 0).all()
    # A product of two inputs below the normal range is off by half a step, which 1 / rms of the row may enlarge; with the
    # quotient's own rounding three half steps.
    each_row = STEP * (1 + rr[:, None]) + 2 * UNIT * most
    none = sc == 1.0   # what rounds to zero, or nearly
    assert (np.abs(sc - most / 448)[~none] <= (each_row / 448 + 1.5 * STEP)[~none]).all()
    assert (most[none] <= (each_row + 448 * STEP)[none]).all()
    # half a step of 8 bits from the kernel's own scale, or the largest value where the scale is rounded down
    each = np.repeat(sc, block, 1)[:, :C]
    slack = STEP * (1 + rr[:, None]) + UNIT * np.abs(ry)
    half = np.maximum(2.0 ** -4 * np.abs(ry) + 2.0 ** -10 * each, np.abs(ry) - 448 * each)
    assert (np.abs(got * each - ry) <= half * (1 + 1e-4) + slack).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("quantize", ["token", "block"])
@pytest.mark.parametrize("C", [64, 1280, 33001])
def test_the_quotient_is_rounded_once(C, quantize, dtype):
    """q is the nearest 8-bit value of fp32's y / scale, ties to even: with weights of one a channel's y is h * rstd, one
    product of numbers that are known here."""
    g = torch.Generator().manual_seed(2)
    x = (torch.randn(64, C, generator=g) * 3).to(DT[dtype]).cuda()
    y, _, rstd, scale = pkg.rms_norm_forward(x, quantize=quantize)
    block = C if quantize == "token" else 128
    each = scale.repeat_interleave(block, 1)[:, :C]
    want = ((x.float() * rstd[:, None]) / each).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert torch.equal(y.float(), want.float())
