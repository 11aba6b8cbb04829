"""The outputs of gqa_decode_scores where the weights' own rounding shows.

Tolerance: a weight is two bfloat16 terms (2^-18 of it), else as in
test_gpu_scores.py: REL = 2 d 2^-23 A + 2^-20 of sum p |v|, here with A the one
product of a query and a key that is not zero, and 2^-8 of the result.
"""
import numpy as np
import pytest
import torch

import oracle
from _helpers import dev, host
from oracle import cache_ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("splits", [1, 0])
@pytest.mark.parametrize("G,d,mantissa", [(4, 128, 1 + 2.0 ** -8), (8, 64, 1 + 3 * 2.0 ** -8), (12, 128, 1.5 + 2.0 ** -8)])
def test_light_keys_against_heavy_ones(G, d, mantissa, splits):
    # a heavy key in each 16 of the first 64, thousands of light ones of one weight, values that cancel: what the
    # rounding takes off one light key it takes off all, and the result is what is left
    from kv_cache_02_b200 import gqa

    S, w = 4000, mantissa * 2.0 ** -9
    k, v = np.zeros((1, 1, S, d), np.float32), np.ones((1, 1, S, d), np.float32)
    k[0, 0, :64:16, 0] = 4.0
    v[0, 0, :64:16] = -(S - 4) * w / 4
    q = np.zeros((1, G, d), np.float32)
    q[..., 0] = 1.0
    scale = float(np.float32(-np.log(w) / 4))
    tk, tv, tq = (dev(a).bfloat16() for a in (k, v, q))
    out, scores = torch.empty_like(tq), torch.zeros(1, 1, S, device="cuda")
    ws = torch.empty(gqa.gqa_decode_scores_workspace_bytes(1, G, 1, S, d, splits), dtype=torch.uint8, device="cuda")
    gqa.gqa_decode_scores(out, scores, tq, tk, tv, torch.tensor([S], dtype=torch.int32, device="cuda"), scale, splits,
                          workspace=ws)
    assert gqa.gqa_get_last_error() == (0, 0)
    want, _, spread = cache_ops.decode_scores(host(tq), host(tk), host(tv), (S,), scale)
    assert np.abs(want).max() < 2.0 ** -8 * spread.min()
    tol = (2.0 ** -18 + 2 * d * 2.0 ** -23 * 4.0 * scale + 2.0 ** -20) * spread + 2.0 ** -8 * np.abs(want)
    err = np.abs(oracle.widen(host(out)) - want)
    assert np.all(err <= tol), np.max(err / tol)
