"""The outputs of gqa_decode_scores where the weights' own rounding shows.

Tolerance: a weight is two bfloat16 terms (2^-15 of it), else as in
test_gpu_scores.py: REL = 2 d 2^-23 A + 2^-20 of sum p |v|, here with A the one
product of a query and a key that is not zero, and 2^-8 of the result.
"""
import numpy as np
import pytest
import torch

import oracle
import synth
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
    tol = (2.0 ** -15 + 2 * d * 2.0 ** -23 * 4.0 * scale + 2.0 ** -20) * spread + 2.0 ** -8 * np.abs(want)
    err = np.abs(oracle.widen(host(out)) - want)
    assert np.all(err <= tol), np.max(err / tol)


@pytest.mark.parametrize("splits", [1, 0, 3])
@pytest.mark.parametrize("H,K,S,d", [(4, 2, 1, 128), (8, 2, 900, 64), (12, 1, 777, 128)])
def test_infinite_values_stay_infinite(H, K, S, d, splits):
    # values at infinity, weights that one bfloat16 holds exactly (equal scores, a single key) and ones that it does not
    from kv_cache_02_b200 import gqa

    k, v = synth.normal((2, K, S, d), synth.F32, 0x3B01, 2), synth.normal((2, K, S, d), synth.F32, 0x3B01, 3)
    k[0] = 0.0
    v[:, :, S // 2, 3], v[:, :, S // 3, 5], v[:, 0, S - 1, 7] = np.inf, -np.inf, np.nan
    v[:, :, 0, 9], v[:, :, S - 1, 9] = np.inf, -np.inf  # NaN where there are two keys
    q = synth.normal((2, H, d), synth.F32, 0x3B01, 1)
    tk, tv, tq = (dev(a).bfloat16() for a in (k, v, q))
    out, scores = torch.empty_like(tq), torch.zeros(2, K, S, device="cuda")
    ws = torch.empty(gqa.gqa_decode_scores_workspace_bytes(2, H, K, S, d, splits), dtype=torch.uint8, device="cuda")
    gqa.gqa_decode_scores(out, scores, tq, tk, tv, torch.tensor([S, S], dtype=torch.int32, device="cuda"), d ** -0.5,
                          splits, workspace=ws)
    assert gqa.gqa_get_last_error() == (0, 0) and bool(torch.isfinite(scores).all())
    with np.errstate(invalid="ignore"):
        want, _, _ = cache_ops.decode_scores(host(tq), host(tk), host(tv), (S, S), d ** -0.5)
    got = oracle.widen(host(out))
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isinf(want).any()
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)]) and np.isfinite(got[np.isfinite(want)]).all()
