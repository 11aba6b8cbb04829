"""The norm of float32 rows to its last bits: rows of whole numbers, whose sums
of squares are exact in float32 in any order. What is left is the reciprocal
root, which may be off by what a rounded root and a rounded quotient are (2^-24
each), and the product with the row (2^-24)."""
import numpy as np
import pytest
import torch

import synth
from _helpers import dev, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [3, 3000])
def test_norm_of_whole_numbers(d, T):
    from kv_cache_02_b200 import gqa

    H, K = 4, 2
    x = np.round(synth.normal((1, T, H + K, d), synth.F64, 0x3A01 + d, 1) * 40)
    x *= np.exp2(np.arange(T) % 9 - 4)[None, :, None, None]  # powers of two change nothing
    assert np.abs((x * x).sum(-1)).max() < 2.0 ** 24 * 2.0 ** 8 and (x * x).sum(-1).min() > 0
    q, k = dev(x[:, :, :H].astype(np.float32)), dev(x[:, :, H:].astype(np.float32))
    one = torch.ones(d, device="cuda")
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    gqa.gqa_qk_norm_rope(q_out, q, k, None, None, one, one, eps=0.0, k_out=k_out)
    assert gqa.gqa_get_last_error() == (0, 0)
    want = x / np.sqrt((x * x).mean(-1, keepdims=True))
    got = np.concatenate([host(q_out), host(k_out)], axis=2)
    err = np.abs(got - want) / np.maximum(np.abs(want), 1e-30)
    assert err.max() <= 3 * 2.0 ** -24 * (1 + 2.0 ** -20), err.max() * 2.0 ** 24
