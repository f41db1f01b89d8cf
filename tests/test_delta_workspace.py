"""Gated delta rule: a workspace holds what the larger of the two ways through a call needs, not both."""
import ctypes

import pytest

import chunked_ssd_scan_gb300 as pkg
from chunked_ssd_scan_gb300 import _build
from tests.test_gated_delta_rule import shape_of


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkg.load_library()


@pytest.mark.parametrize("b,T,Hk,H,K,V", [(4, 4096, 8, 16, 128, 128), (2, 300, 1, 2, 64, 64), (1, 8192, 4, 4, 64, 128)], ids=str)
def test_backward(lib, b, T, Hk, H, K, V):
    f32, bf16 = (lib.gated_delta_rule_workspace_bytes(ctypes.byref(shape_of(b, T, Hk, H, K, V, io)), 1) for io in (0, 1))
    fwd = lib.gated_delta_rule_workspace_bytes(ctypes.byref(shape_of(b, T, Hk, H, K, V, 1)), 0)
    nch = -(-T // 64)
    cells = b * nch * H
    both = 2 * cells * V * K * 4                        # states and their gradients, in either way
    cores = 2 * b * T * H * V * 4                       # errors and their gradients on the CUDA cores,
    cores += -(-K // 64) * cells * 64 * 4               # and dg by blocks of keys
    squares = cells * (6 * 8192 + 4 * 64 * 4 + 4 * 8192)   # squares, decays and writes on the tensor cores
    segments = fwd - 256 - cells * (4 * 8192 + 4 * 64 * 4)   # of the forward walk that recomputes the states
    slack = 8 * 256                                     # every array starts on a border of 256 bytes
    assert both + cores <= f32 <= 256 + both + cores + slack
    assert both + max(cores, squares) <= bf16 <= 256 + both + max(cores, squares + max(segments, 0)) + slack
