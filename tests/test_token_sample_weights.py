"""The polynomial behind token_sample's table of weights, with the constants and the integer steps of its source."""
import os
import re

import numpy as np

import chunked_ssd_scan_gb300 as pkg


def test_powers_of_two_of_a_fraction():
    """2^31 2^-f for fractions f of 32 bits: off by at most 3, as its comment says."""
    path = os.path.join(os.path.dirname(pkg.__file__), "csrc", "token_sample.cu")
    with open(path) as fh:
        body = re.search(r"exp2_fraction\(uint32_t f\) \{(.*?)\n\}", fh.read(), re.S).group(1)
    first, *rest = (int(c, 16) for c in re.findall(r"0x([0-9a-f]+)u", body))
    assert len(rest) == 8 and body.count("__umulhi(f, m)") == 8
    f = np.unique(np.concatenate([np.arange(256, dtype=np.uint64) << np.uint64(24),   # the table's own
                                  np.random.default_rng(0).integers(0, 1 << 32, 200000, dtype=np.uint64),
                                  np.array([0, 1, (1 << 32) - 1], np.uint64)]))
    m = np.full_like(f, first)
    for c in rest:
        m = np.uint64(c) - (f * m >> np.uint64(32))
    want = 2.0 ** (31 - f.astype(np.float64) / 2.0 ** 32)
    assert np.abs(m.astype(np.float64) - want).max() <= 3
