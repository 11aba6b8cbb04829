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
from test_gpu_scores import assert_out, assert_scores, largest

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


def padded(B, T, H, K, S, d, pads, seed):
    """q [B, T, H, d] and k [B, K, S, d] of which the first pads[b] keys of each sequence are at -inf."""
    q, k = synth.normal((B, T, H, d), synth.F32, seed, 1), synth.normal((B, K, S, d), synth.F32, seed, 2)
    q[..., 0] = 1.0
    k[..., 0] = 0.0
    finite = k.copy()
    for b, n in enumerate(pads):
        k[b, :, :n, 0] = -np.inf
    return (dev(a).bfloat16() for a in (q, k, finite))


@pytest.mark.parametrize("T,H,K,S,d", [(320, 8, 2, 340, 128), (300, 6, 2, 330, 64), (150, 8, 1, 1100, 128),
                                       (90, 3, 1, 1500, 64), (1200, 4, 1, 1300, 128)])
def test_a_left_padded_prompt(gqa, T, H, K, S, d):
    # with one split of the keys and with several: the padding's queries add nothing, and nothing is NaN
    pads, n = (70, 0, T), T
    q, k, finite = padded(3, T, H, K, S, d, pads, 0x3702)
    scores = torch.zeros(3, K, S, device="cuda")
    ws = torch.empty(gqa.gqa_prompt_scores_workspace_bytes(3, T, H, K, S, d), dtype=torch.uint8, device="cuda")
    gqa.gqa_prompt_scores(scores, q, k, torch.full((3,), n, dtype=torch.int32, device="cuda"), d ** -0.5, workspace=ws)
    assert gqa.gqa_get_last_error() == (0, 0)
    # the queries from the first finite key on
    added = np.concatenate([cache_ops.prompt_scores(host(q)[b:b + 1, m:], host(k)[b:b + 1], (n,), d ** -0.5)
                            for b, m in enumerate(pads)])
    assert not added[2].any() and not added[0, :, :70].any() and np.isfinite(added).all()
    rel = 2 * d * 2.0 ** -23 * largest(host(q), host(finite), d ** -0.5) + 2.0 ** -20
    assert_scores(host(scores), np.zeros((3, K, S), np.float32), added, (n,) * 3, rel, T * H // K + S, "left padding")


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("H,K,S,d", [(8, 2, 900, 128), (3, 1, 400, 64), (20, 1, 2500, 128)])
def test_a_decode_step_of_masked_keys_alone(gqa, H, K, S, d, splits):
    # sequence 0 has keys at -inf alone: zeros, and its scores stay; the prompt's form of the same step says the same
    q, k, finite = padded(2, 1, H, K, S, d, (S, 5), 0x3703)
    v = synth.normal((2, K, S, d), synth.BF16, 0x3703, 3)
    before = np.abs(synth.normal((2, K, S), synth.F32, 0x3703, 4)).astype(np.float32)
    out, scores, again = torch.full((2, H, d), 9.0, dtype=torch.bfloat16, device="cuda"), dev(before), dev(before)
    lens = torch.tensor([S, S - 1], dtype=torch.int32, device="cuda")
    ws = torch.empty(max(gqa.gqa_decode_scores_workspace_bytes(2, H, K, S, d, splits),
                         gqa.gqa_prompt_scores_workspace_bytes(2, 1, H, K, S, d)), dtype=torch.uint8, device="cuda")
    gqa.gqa_decode_scores(out, scores, q[:, 0].contiguous(), k, dev(v), lens, d ** -0.5, splits, workspace=ws)
    gqa.gqa_prompt_scores(again, q, k, lens, d ** -0.5, workspace=ws)
    assert gqa.gqa_get_last_error() == (0, 0)
    assert not out[0].any() and np.array_equal(host(scores)[0], before[0]) and np.array_equal(host(again)[0], before[0])
    want, added, spread = cache_ops.decode_scores(host(q)[1:, 0], host(k)[1:], v[1:], (S - 1,), d ** -0.5)
    rel = 2 * d * 2.0 ** -23 * largest(host(q), host(finite), d ** -0.5) + 2.0 ** -20
    for s in (scores, again):
        assert_scores(host(s)[1:], before[1:], added, (S - 1,), rel, H + S, f"splits {splits}")
    assert_out(host(out)[1:], want, spread, rel, f"splits {splits}")
