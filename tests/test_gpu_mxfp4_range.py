"""The decode over the 4-bit cache at the ends of its formats' ranges: queries
and block scales that are far apart, and weights that are.

Tolerances as in test_gpu_mxfp4.py.
"""
import numpy as np
import pytest
import torch

import oracle
import synth
from _helpers import dev, host
from oracle import cache_ops
from test_gpu_mxfp4 import check_decode, quantised

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def gqa():
    from kv_cache_02_b200 import gqa as g

    return g


@pytest.mark.parametrize("top", [2.0 ** 119, 2.0 ** 120, 2.0 ** 126, 1.5 * 2.0 ** 127, 3.38e38])
def test_decode_queries_near_the_end_of_bfloat16(gqa, top):
    # keys as small as such queries are large: scores of a few units
    B, H, K, S = 1, 8, 1, 152
    cache = quantised(B, K, S, 0x3901, spread=0.2)
    cache[1] = np.clip(cache[1].astype(int) - int(np.log2(top)) - 2, 0, 254).astype(np.uint8)
    q = oracle.widen(synth.normal((B, H, D), synth.BF16, 0x3901, 1))
    q = np.clip(q, -2.0, 2.0) * top / 2.0
    q[:, ::2, 0] = top
    q = host(torch.from_numpy(q).float().bfloat16())
    assert np.isfinite(oracle.widen(q)).all()
    check_decode(gqa, q, cache, (S,), 0.3, what=f"{top}")
