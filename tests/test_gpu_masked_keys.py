"""Caches masked by their keys: a key at -inf weighs nothing, and the keys that
are left weigh what they would without it, however low their scores are.

Tolerances as in test_gpu_scores.py; the queries hold three elements and zeros,
so that A, the bound of scale * sum |q k|, is near the scores themselves.
"""
import numpy as np
import pytest
import torch

import synth
from _helpers import dev, host
from oracle import cache_ops
from test_gpu_scores import assert_scores, largest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gqa():
    from kv_cache_02_b200 import gqa as g

    return g


def low_scores(T, H, S, d, masked, level, seed):
    """(q, k, k with 0 for -inf): the first `masked` keys at -inf, key t's scaled score level(t) natural units and a
    little of its own, scale d^-0.5."""
    q = np.zeros((1, T, H, d), np.float32)
    q[..., 0] = 1.0
    q[..., 1:3] = synth.normal((1, T, H, 2), synth.F32, seed, 1)
    k = synth.normal((1, 1, S, d), synth.F32, seed, 2)
    k[0, 0, :, 0] = level(np.arange(S)) * np.sqrt(d)
    finite = k.copy()
    finite[0, 0, :masked] = 0.0
    k[0, 0, :masked, 0] = -np.inf
    return (dev(a).bfloat16() for a in (q, k, finite))


@pytest.mark.parametrize("level", ["-150", "-2000", "-87 and -89", "+150"])
@pytest.mark.parametrize("T,H,S,d,masked", [(60, 4, 800, 128, 200), (33, 3, 700, 64, 130), (5, 8, 2100, 128, 1100),
                                            (300, 8, 900, 64, 70)])
def test_prompt_scores_of_low_keys_behind_masked_ones(gqa, T, H, S, d, masked, level):
    # no reference score is known while a query has seen keys at -inf alone; those that follow may all lie below 2^-126
    # of any fixed one, or, at -87 and -89, on both sides of that
    at = {"-150": lambda t: -150.0 + 0 * t, "-2000": lambda t: -2000.0 + 0 * t, "+150": lambda t: 150.0 + 0 * t,
          "-87 and -89": lambda t: np.where(t // 128 % 2 == 0, -89.0, -87.0)}[level]
    n = S - 3
    q, k, finite = low_scores(T, H, S, d, masked, at, 0x3701)
    scores = torch.zeros(1, 1, S, device="cuda")
    ws = torch.empty(gqa.gqa_prompt_scores_workspace_bytes(1, T, H, 1, S, d), dtype=torch.uint8, device="cuda")
    gqa.gqa_prompt_scores(scores, q, k, torch.tensor([n], dtype=torch.int32, device="cuda"), d ** -0.5, workspace=ws)
    assert gqa.gqa_get_last_error() == (0, 0)
    added = cache_ops.prompt_scores(host(q), host(k), (n,), d ** -0.5)
    assert not added[0, 0, :masked].any() and np.isfinite(added).all()
    rel = 2 * d * 2.0 ** -23 * largest(host(q), host(finite), d ** -0.5) + 2.0 ** -20
    assert_scores(host(scores), np.zeros((1, 1, S), np.float32), added, (n,), rel, T * H + S, level)
