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


def sink_and_tail(S, far, seed):
    """Key 0 scores 4, key 1 -6, the others 0 (q = 1 in dim 0). V rows of one block scale, but that of key 1, 2^far above."""
    k, v = np.zeros((S, D), np.float32), np.abs(synth.normal((S, D), synth.F32, seed, 1)).clip(0, 2.9).astype(np.float32)
    v[:, ::32] = 3.0
    k[0, 0], k[1, 0] = 4.0, -6.0
    v[1] *= 2.0 ** far
    cache = [a.reshape(1, 1, S, -1) for x in (k, v) for a in cache_ops.mxfp4_quantize(x)]
    q = np.zeros((1, 8, D), np.float32)
    q[..., 0] = 1.0
    return cache, host(torch.from_numpy(q).bfloat16())


@pytest.mark.parametrize("far", [0, 8, 9, 10, 11, 12, 13, 14, 40, 90])
@pytest.mark.parametrize("weight", [1.06, 1.19, 1.94])
def test_decode_a_flat_tail_beside_one_large_block(gqa, far, weight):
    # 60000 keys of weight 2^-17 make up half of the result, and what the rounding takes off one of them it takes off
    # all; key 1 weighs 2^-40. 2^-8: bfloat16 weights, for scales that do not fit one fp16 range
    cache, q = sink_and_tail(60000, far, 0x3902)
    check_decode(gqa, q, cache, (60000,), (17 - np.log2(weight)) * np.log(2.0) / 4.0, splits=1, p_step=2.0 ** -8,
                 what=f"{far} {weight}")


@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("where", [0, 37, 699])
@pytest.mark.parametrize("scale_v,lower", [(254, 400.0), (254, 80.0), (240, 60.0), (180, 45.0), (254, 87.5), (150, 12.0)])
def test_decode_a_huge_value_of_no_weight(gqa, scale_v, lower, where, splits):
    # one key's V block lies up to 2^127 above the others', and its weight as far below: what counts is their product,
    # and the other keys' values keep theirs. Half of the heads give it next to no weight at all
    B, H, K, S = 1, 8, 1, 700
    cache = quantised(B, K, S, 0x3903, spread=0.0)
    k = oracle.widen(synth.normal((B, K, S, D), synth.BF16, 0x3904, 1)).astype(np.float32)
    k[..., 0] = 0.0
    k[0, 0, where, 0] = -4.0
    cache[0], cache[1] = cache_ops.mxfp4_quantize(k)
    cache[3] = cache[3].copy()
    cache[3][0, 0, where, [1, 3]] = scale_v
    q = oracle.widen(synth.normal((B, H, D), synth.BF16, 0x3904, 2)) * 0.25
    q[..., 0] = lower / 4.0
    q[:, ::2, 0] = 100.0
    q = host(torch.from_numpy(q).float().bfloat16())
    check_decode(gqa, q, cache, (S,), 1.0, splits, 2.0 ** -8, f"{scale_v} {lower} {where}")


def test_decode_values_of_every_size(gqa):
    # blocks from 2^-127 to 2^127 in no order, weights from 1 down to 2^-120: in bfloat16 every product counts
    B, H, K, S = 2, 8, 2, 600
    cache = quantised(B, K, S, 0x3905, spread=0.0)
    rnd = synth.normal((B, K, S, 4), synth.F64, 0x3906, 1)
    k = np.zeros((B, K, S, D), np.float32)
    k[..., 0] = synth.normal((B, K, S), synth.F32, 0x3906, 2)
    cache[0], cache[1] = cache_ops.mxfp4_quantize(k)
    cache[3] = np.clip(127 + 45 * rnd, 0, 240).astype(np.uint8)
    q = np.zeros((B, H, D), np.float32)
    q[..., 0] = np.linspace(1.0, 12.0, H)
    check_decode(gqa, host(torch.from_numpy(q).bfloat16()), cache, (S, S - 5), 1.0, 1, 2.0 ** -8, "every size")


@pytest.mark.parametrize("splits", [0, 1, 2, 7])
def test_decode_scores_below_float32(gqa, splits):
    # keys of scale 2^127 against q: scores of -2^130 and beyond. They weigh nothing: the first 128 and a few others of
    # head group 0, all of group 1 (zeros, whether one split holds them or several)
    B, H, K, S = 2, 6, 2, 1400
    cache = quantised(B, K, S, 0x3907, spread=0.0)
    k = oracle.widen(synth.normal((B, K, S, D), synth.BF16, 0x3908, 1)).astype(np.float32)
    k[..., 0] = 0.0
    masked = np.zeros((B, K, S), bool)
    masked[:, 0, [*range(130), 700, 1390]] = True
    masked[:, 1] = True
    k[masked] = 0.0
    k[masked, 0] = -6.0
    cache[0], cache[1] = cache_ops.mxfp4_quantize(k)
    cache[1] = np.where(masked[..., None] & (np.arange(4) == 0), 254, cache[1]).astype(np.uint8)
    q = oracle.widen(synth.normal((B, H, D), synth.BF16, 0x3908, 2))
    q[..., 0] = 4.0
    q = host(torch.from_numpy(q).float().bfloat16())
    out = torch.full((B, H, D), 9.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(gqa.gqa_decode_mxfp4_workspace_bytes(B, H, K, S, D, splits), dtype=torch.uint8, device="cuda")
    lens = (S, 129)
    gqa.gqa_decode_mxfp4(out, dev(q), *(dev(c) for c in cache), dev(np.array(lens, np.int32)), D ** -0.5, splits, ws)
    assert gqa.gqa_get_last_error() == (0, 0)
    assert not out[:, 3:].any() and not out[1].any()  # sequence 1 ends before its first other key
    kv, v = cache_ops.mxfp4_values(cache[0], cache[1]), cache_ops.mxfp4_values(cache[2], cache[3])
    want, _, spread = cache_ops.decode_scores(q[:1, :3], kv[:1, :1], v[:1, :1], (S,), D ** -0.5)
    a = np.sqrt((oracle.widen(q) ** 2).sum(-1).max() * (k[~masked].astype(np.float64) ** 2).sum(-1).max()) * D ** -0.5
    tol = (2.0 ** -8 + 2 * D * 2.0 ** -23 * a + 2.0 ** -20) * spread + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(oracle.widen(host(out))[:1, :3] - want) <= tol)


@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("scale_v", [235, 243, 248, 252, 253])
def test_decode_values_near_the_end_of_float32(gqa, scale_v, splits):
    # few keys, so that sum p v stays in range: 2^126 of weight 1, smaller ones beside it
    B, H, K, S = 1, 8, 2, 260
    cache = quantised(B, K, S, 0x3909, spread=0.0)
    k = np.zeros((B, K, S, D), np.float32)
    k[:, :, [3, 200], 0] = 6.0, 5.0
    cache[0], cache[1] = cache_ops.mxfp4_quantize(k)
    cache[3] = np.full_like(cache[3], 127)
    cache[3][:, :, 3] = scale_v
    cache[2][:, :, 3] = 0x1A  # -1, 0.5
    cache[3][:, :, 200, 2] = scale_v - 9
    q = np.zeros((B, H, D), np.float32)
    q[..., 0] = np.linspace(2.0, 16.0, H)
    check_decode(gqa, host(torch.from_numpy(q).bfloat16()), cache, (S,), 1.0, splits, 2.0 ** -8, f"{scale_v}")
