"""Pins for the oracle of the cache operators (oracle/cache_ops.py): rows worked
by hand, closed forms, and torch's own float64 softmax and sort."""
import numpy as np
import pytest
import torch

import oracle
import synth
from oracle import cache_ops


def test_rotation_by_hand():
    # dims 0 and 2 are a pair (half a rotary dim apart), 1 and 3 the other; a quarter turn takes (a, b) to (-b, a)
    table = np.array([[1.0, 1.0, 0.0, 0.0], [0.0, 1.0, 1.0, 0.0]])
    y = np.arange(1.0, 6.0).reshape(1, 1, 1, 5)
    assert cache_ops.rotate(y, table, [[1]], False).ravel().tolist() == [-3.0, 2.0, 1.0, 4.0, 5.0]
    assert cache_ops.rotate(y, table, [[1]], True).ravel().tolist() == [-2.0, 1.0, 3.0, 4.0, 5.0]
    assert cache_ops.rotate(y, table, [[0]], False).ravel().tolist() == y.ravel().tolist()


def test_rotation_depends_on_the_distance_alone():
    table = cache_ops.rope_table(500, 32, 10000.0)
    q, k = (synth.normal((1, 1, 1, 32), synth.F64, 5, s) for s in (1, 2))
    for il in (False, True):
        dots = [(cache_ops.rotate(q, table, [[p + 7]], il) * cache_ops.rotate(k, table, [[p]], il)).sum()
                for p in (0, 100, 492)]
        assert np.allclose(dots, dots[0], rtol=0, atol=1e-10)
    assert table[0].tolist() == [1.0] * 16 + [0.0] * 16
    assert np.isclose(table[3, 16], np.sin(3.0)) and np.isclose(table[3, 15], np.cos(3.0 * 10000.0 ** (-30 / 32)))


def test_norm_by_hand():
    y = cache_ops.norm_heads(np.array([[3.0, 4.0, 0.0, 0.0]], np.float32), np.array([1, 2, 1, 1], np.float32), 0.0)
    assert np.allclose(y, [[3 / 2.5, 8 / 2.5, 0, 0]])
    assert cache_ops.norm_heads(np.zeros((1, 4), np.float32), np.ones(4, np.float32), 1e-6).tolist() == [[0.0] * 4]


def test_scores_are_the_columns_of_the_softmax():
    B, T, H, K, S, d = 2, 5, 4, 2, 9, 16
    q, k = synth.normal((B, T, H, d), synth.F64, 6, 1), synth.normal((B, K, S, d), synth.F64, 6, 2)
    lens = [9, 3]
    got = cache_ops.prompt_scores(q, k, lens, 0.3)
    for b, n in enumerate(lens):
        # as many weights of one as queries and heads that count
        assert np.allclose(got[b].sum(-1), min(T, n) * (H // K))
        assert np.all(got[b, :, n:] == 0)
        x = 0.3 * torch.einsum("thd,hsd->hts", torch.from_numpy(q[b]), torch.from_numpy(k[b].repeat(H // K, 0)))
        at = n - T + torch.arange(T)
        x = x.masked_fill(torch.arange(S)[None, None, :] > at[None, :, None], -float("inf"))
        p = torch.softmax(x, -1)[:, at >= 0]
        assert np.allclose(got[b], p.reshape(K, H // K, -1, S).sum((1, 2)).numpy())
    # the last query alone is a decode step
    out, added, _ = cache_ops.decode_scores(q[:, -1], k, k, lens, 0.3)
    assert np.allclose(added, cache_ops.prompt_scores(q[:, -1:], k, lens, 0.3))
    assert np.allclose(out, oracle.decode(q[:, -1], k, k, np.array(lens, np.int32), 0.3))


def test_evict_by_hand():
    k = np.arange(6, dtype=np.float32).reshape(1, 1, 6, 1) * 10
    s = np.array([[[0.5, 9.0, 0.1, 0.5, 7.0, 0.5]]], np.float32)
    pos = np.arange(6, dtype=np.int32).reshape(1, 1, 6)
    # keep 3: rows 1 and 4 by score, row 0 the first of the equal ones; row 4 moves into the hole at 2
    k1, v1, s1, p1, n1 = cache_ops.evict(k, k + 1, s, pos, [6], 3, 0, None)
    assert k1.ravel().tolist() == [0, 10, 40, 30, 40, 50] and v1.ravel().tolist() == [1, 11, 41, 31, 41, 51]
    assert s1.ravel().tolist() == [0.5, 9.0, 7.0, 0, 0, 0] and p1.ravel().tolist() == [0, 1, 4, -1, -1, -1]
    assert n1.tolist() == [3]
    # sinks hold row 0, age holds row 5: they come before the heaviest
    k1, _, s1, p1, _ = cache_ops.evict(k, k, s, pos, [6], 3, 1, [5])
    assert p1.ravel()[:3].tolist() == [0, 1, 5] and k1.ravel()[:3].tolist() == [0, 10, 50]
    s1 = s.copy()
    s1[0, 0, 1] = np.nan  # below every number
    assert cache_ops.evict(k, k, s1, pos, [6], 3, 0, None)[3].ravel()[:3].tolist() == [0, 3, 4]
    assert cache_ops.evict(k, k, s, None, [2], 3, 0, None)[2].tolist() == s.tolist()  # short enough already


def test_quantizer_by_hand():
    x = np.zeros(64, np.float32)
    x[:9] = [6.0, -6.0, 0.25, 0.75, 2.5, 5.0, -3.5, 7.9, 0.2]  # largest 7.9: scale 2^(2 - 2)
    x[32:35] = [0.375, -0.09375, 0.01]  # largest 0.375: 2^-2 / 4
    codes, scales = cache_ops.mxfp4_quantize(x)
    assert scales.tolist() == [127, 123]
    got = cache_ops.mxfp4_values(codes, scales)
    # 0.25 ties to 0, 0.75 to 1, 2.5 to 2, 5 to 4, 3.5 to 4; 7.9 saturates
    assert got[:9].tolist() == [6.0, -6.0, 0.0, 1.0, 2.0, 4.0, -4.0, 6.0, 0.0]
    assert got[32:35].tolist() == [0.375, -0.09375, 0.0]
    assert codes[1] == (2 << 4) | 0 and codes[0] == (15 << 4) | 7


def test_quantizer_bounds_and_edges():
    x = synth.normal((200, 128), synth.BF16, 7, 1)
    codes, scales = cache_ops.mxfp4_quantize(x)
    w, v = oracle.widen(x), cache_ops.mxfp4_values(codes, scales)
    step = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, axis=-1)
    # half the widest gap (4 .. 6), and up to 2 steps above 6 where the largest value saturates
    assert np.all(np.abs(w - v) <= np.where(np.abs(w) > 6 * step, 2, 1) * step)
    # values that the format holds come back as they are
    c2, s2 = cache_ops.mxfp4_quantize(v.astype(np.float32))
    assert np.array_equal(cache_ops.mxfp4_values(c2, s2), v)
    bad = np.zeros(96, np.float32)
    bad[3], bad[40] = np.nan, -np.inf
    codes, scales = cache_ops.mxfp4_quantize(bad)
    assert scales.tolist() == [255, 255, 0] and not codes.any()
    tiny = np.full(32, 2.0 ** -130, np.float32)  # below the smallest scale's 4
    codes, scales = cache_ops.mxfp4_quantize(tiny)
    assert scales.tolist() == [0] and np.all(cache_ops.mxfp4_values(codes, scales) == 0.0)


@pytest.mark.parametrize("value", [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
def test_ties_go_to_the_even_code(value):
    x = np.zeros(32, np.float32)
    x[0], x[1], x[2] = 4.0, value, -value
    codes, scales = cache_ops.mxfp4_quantize(x)
    assert scales[0] == 127
    low, high = int(codes[0]) >> 4, int(codes[1]) & 15
    assert low % 2 == 0 and high == low + 8
