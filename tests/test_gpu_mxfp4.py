"""GPU parity of the 4-bit cache: the append and the read are exact, the decode
is compared with the float64 decode of the values the cache holds.

Tolerance of the decode: the result's rounding to bfloat16 is 2^-8 of it. The
weight p meets the V codes in fp16 (2^-11 of sum p |v|) where the block scales
of a step's keys lie within 2^15 of each other, else in bfloat16 (2^-8). A
score is a float32 sum of d products (a step of 2^-23 each) times the block's
scale: p is within REL = 2 d 2^-23 A + 2^-20, A the largest scale * sum |q k|.
fp16 drops what is below 2^(j - 39) of the largest weight at j bits below the
reference scale: nothing at these lengths.
"""
import numpy as np
import pytest
import torch

import oracle
import synth
from _helpers import Guarded, dev, host
from oracle import cache_ops

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def gqa():
    from kv_cache_02_b200 import gqa as g

    return g


def quantised(B, K, S, seed, spread=1.0):
    """Caches of N(0, 1) rows whose channels differ in size by exp(spread N(0, 1))."""
    out = []
    for stream in (2, 3):
        x = oracle.widen(synth.normal((B, K, S, D), synth.BF16, seed, stream))
        x = x * np.exp(spread * synth.normal((K, 1, D), synth.F64, seed, stream + 10))
        out += list(cache_ops.mxfp4_quantize(x.astype(np.float32)))
    return out


def poison(codes, scales, lens):
    """Rows past each length: scale 255, which is NaN."""
    for b, n in enumerate(lens):
        codes[b, :, n:], scales[b, :, n:] = 0x77, 255


def check_decode(gqa, q, cache, lens, scale, splits=0, p_step=2.0 ** -11, what=""):
    B, H, _ = q.shape
    K, S = cache[0].shape[1:3]
    out = Guarded((B, H, D), torch.bfloat16)
    n = gqa.gqa_decode_mxfp4_workspace_bytes(B, H, K, S, D, splits)
    ws = torch.full((n + 64,), 0xEE, dtype=torch.uint8, device="cuda")
    gqa.gqa_decode_mxfp4(out.t, dev(q), *(dev(c) for c in cache), dev(np.array(lens, np.int32)), scale, splits, ws[:n])
    assert gqa.gqa_get_last_error() == (0, 0) and out.intact() and bool((ws[n:] == 0xEE).all())
    with np.errstate(invalid="ignore"):
        k, v = cache_ops.mxfp4_values(cache[0], cache[1]), cache_ops.mxfp4_values(cache[2], cache[3])
    want, _, spread = cache_ops.decode_scores(q, k, v, lens, scale)
    norms = [np.sqrt((np.nan_to_num(oracle.widen(x)) ** 2).sum(-1).max()) for x in (q, k)]
    rel = 2 * D * 2.0 ** -23 * abs(scale) * norms[0] * norms[1] + 2.0 ** -20
    err = np.abs(oracle.widen(host(out.t)) - want)
    tol = (p_step + rel) * spread + 2.0 ** -8 * np.abs(want) + 1e-37
    assert np.all(err <= tol), f"{what}: {np.nanmax(err / tol)} of the tolerance"
    return host(out.t)


CASES = [
    # B, H, K, S_max, lens
    (1, 1, 1, 4, (1,)),
    (3, 16, 4, 320, (300, 1, 77)),
    (4, 64, 8, 1024, (0, 999, 1024, 513)),
    (2, 8, 8, 192, (192, 65)),
    (2, 66, 1, 704, (700, 129)),
    (1, 21, 3, 2100, (2099,)),
    (2, 24, 2, 6000, (5999, 128)),
]


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_decode(gqa, case, splits):
    B, H, K, S, lens = case
    cache = quantised(B, K, S, 0x3401 + S)
    poison(cache[0], cache[1], lens)
    poison(cache[2], cache[3], lens)
    q = synth.normal((B, H, D), synth.BF16, 0x3402, 1)
    got = check_decode(gqa, q, cache, lens, D ** -0.5, splits, what=f"{case} {splits}")
    for b, n in enumerate(lens):
        assert n or not got[b].any()


def test_decode_extreme_queries(gqa):
    # heads whose elements differ by 2^20, tiny and huge heads, zero heads, a negative softmax scale
    B, H, K, S = 1, 16, 2, 200
    cache = quantised(B, K, S, 0x3403, spread=0.2)
    q = oracle.widen(synth.normal((B, H, D), synth.BF16, 0x3403, 1))
    q[0, 0] *= 2.0 ** -120
    q[0, 1] = 0.0
    q[0, 2, :64] *= 2.0 ** -20
    q[0, 3] *= 2.0 ** 6
    q[0, 4, 1:] = 0.0
    q = host(torch.from_numpy(q).float().bfloat16())
    for scale in (0.05, -0.05):
        check_decode(gqa, q, cache, (S,), scale, what=f"scale {scale}")


@pytest.mark.parametrize("kind", ["steps", "keys", "wide", "zeros", "rising", "ends"])
def test_decode_block_scales_far_apart(gqa, kind):
    """V scales that do not fit one fp16 range: other exponents are another value, not another order of keys."""
    B, H, K, S = 2, 12, 2, 700
    cache = quantised(B, K, S, 0x3404)
    vs = cache[3].astype(int)
    t = np.arange(S)[None, None, :, None]
    rnd = np.abs(synth.normal((B, K, S, 4), synth.F64, 0x3405, 1))
    if kind == "steps":      # every 32-key step has its own magnitude
        vs = vs + (t // 32 % 5 - 2) * 9
    elif kind == "keys":     # neighbours 2^40 apart
        vs = vs + np.where(t % 3 == 0, -40, 0)
    elif kind == "wide":     # anything at all
        vs = 127 + np.clip(rnd * 30 - 30, -100, 60).astype(int)
    elif kind == "zeros":    # rows of zeros, scale 0
        vs = np.where(t % 7 == 0, 0, vs)
        cache[2] = np.where(t % 7 == 0, 0, cache[2]).astype(np.uint8)
    elif kind == "rising":   # the reference has to follow
        vs = vs - 60 + t // 8
    else:                    # the first key far above all the others
        vs = np.where(t == 0, 200, vs)
    cache[3] = np.clip(vs, 0, 254).astype(np.uint8)
    q = synth.normal((B, H, D), synth.BF16, 0x3404, 1)
    for splits in (1, 2):
        check_decode(gqa, q, cache, (S, S - 13), 0.3 * D ** -0.5, splits, 2.0 ** -8, kind)


def test_decode_a_light_sink_and_a_long_flat_tail(gqa):
    # one key of weight 1 and small values, thousands of keys of weight 2^-17 that make up half of the result
    B, H, K, S = 1, 8, 1, 60000
    cache = quantised(B, K, S, 0x3406, spread=0.0)
    k = np.zeros((S, D), np.float32)
    k[0, 0] = 4.0
    c, s = cache_ops.mxfp4_quantize(k)
    cache[0], cache[1] = c.reshape(1, 1, S, -1), s.reshape(1, 1, S, -1)
    v = np.abs(synth.normal((S, D), synth.F32, 0x3407, 1)).astype(np.float32)
    v[0] /= 64
    c, s = cache_ops.mxfp4_quantize(v)
    cache[2], cache[3] = c.reshape(1, 1, S, -1), s.reshape(1, 1, S, -1)
    q = np.zeros((B, H, D), np.float32)
    q[..., 0] = 17 * np.log(2.0) / 4.0
    check_decode(gqa, host(torch.from_numpy(q).bfloat16()), cache, (S,), 1.0, what="sink")


def test_decode_nan_blocks(gqa):
    # a NaN block of a cached V row makes its 32 dims NaN, of a K row everything; other heads and sequences stay
    B, H, K, S = 2, 8, 2, 96
    cache = quantised(B, K, S, 0x3408)
    cache[3][0, 1, 50, 2] = 255
    q = synth.normal((B, H, D), synth.BF16, 0x3408, 1)
    out = torch.empty(B, H, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(gqa.gqa_decode_mxfp4_workspace_bytes(B, H, K, S, D), dtype=torch.uint8, device="cuda")
    lens = torch.tensor([96, 90], dtype=torch.int32, device="cuda")
    gqa.gqa_decode_mxfp4(out, dev(q), *(dev(c) for c in cache), lens, 0.1, workspace=ws)
    bad = torch.zeros(B, H, D, dtype=torch.bool, device="cuda")
    bad[0, 4:, 64:96] = True
    assert torch.equal(torch.isnan(out), bad)
    cache[1][1, 0, 3, 0] = 255
    gqa.gqa_decode_mxfp4(out, dev(q), *(dev(c) for c in cache), lens, 0.1, workspace=ws)
    bad[1, :4] = True
    assert torch.equal(torch.isnan(out), bad) and gqa.gqa_get_last_error() == (0, 0)


def test_decode_bad_lengths(gqa):
    B, H, K, S = 3, 8, 2, 64
    cache = quantised(B, K, S, 0x3409)
    out = torch.full((B, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(gqa.gqa_decode_mxfp4_workspace_bytes(B, H, K, S, D), dtype=torch.uint8, device="cuda")
    gqa.gqa_decode_mxfp4(out, dev(synth.normal((B, H, D), synth.BF16, 0x3409, 1)), *(dev(c) for c in cache),
                         torch.tensor([65, -1, 64], dtype=torch.int32, device="cuda"), 0.1, workspace=ws)
    assert gqa.gqa_get_last_error() == (gqa.GQA_ERR_DEVICE, gqa.GQA_DEVERR_SEQLEN)
    assert not out[:2].any() and bool(torch.isfinite(out).all())


def empty_cache(B, K, S):
    return [torch.full((B, K, S, w), 0xA5, dtype=torch.uint8, device="cuda") for w in (D // 2, D // 32, D // 2, D // 32)]


@pytest.mark.parametrize("B,T,K,S,pos", [(1, 1, 1, 4, (3,)), (3, 1, 8, 64, (0, 63, 17)), (2, 37, 3, 100, (63, 0)),
                                         (2, 300, 2, 304, (0, 4)), (70, 2, 5, 8, tuple(range(7)) * 10)])
def test_append_and_read_are_exact(gqa, B, T, K, S, pos):
    new = []
    for stream in (5, 6):
        x = oracle.widen(synth.normal((B, T, K, D), synth.BF16, 0x3410, stream))
        x = x * np.exp2(np.round(10 * synth.normal((B, T, K, 4, 1), synth.F64, 0x3410, stream + 2))).repeat(32, -1).reshape(x.shape)
        new.append(host(torch.from_numpy(x).float().bfloat16()))
    cache = empty_cache(B, K, S)
    tpos = dev(np.array(pos, np.int32))
    gqa.gqa_kv_append_mxfp4(*cache, dev(new[0]), dev(new[1]), tpos)
    assert gqa.gqa_get_last_error() == (0, 0)
    out = [torch.empty(B, T, K, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    gqa.gqa_kv_read_mxfp4(*out, *cache, tpos)
    for i, x in enumerate(new):
        codes, scales = cache_ops.mxfp4_quantize(x)
        want = [np.full((B, K, S, w), 0xA5, np.uint8) for w in (D // 2, D // 32)]
        for b in range(B):
            want[0][b, :, pos[b]:pos[b] + T] = codes[b].swapaxes(0, 1)
            want[1][b, :, pos[b]:pos[b] + T] = scales[b].swapaxes(0, 1)
        assert np.array_equal(host(cache[2 * i]), want[0]) and np.array_equal(host(cache[2 * i + 1]), want[1])
        assert np.array_equal(oracle.widen(host(out[i])), cache_ops.mxfp4_values(codes, scales))


def test_append_edges(gqa):
    rows = np.zeros((9, D), np.float32)
    rows[0, :8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0]      # ties
    rows[1, :8] = [-0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 7.9]
    rows[2, 5], rows[2, 40] = np.nan, np.inf
    rows[3] = 2.0 ** -126
    rows[3, 3] = 2.0 ** -133                                         # bfloat16's smallest
    rows[4] = 3e38
    rows[5, 0] = -0.0
    rows[6] = 2.0 ** -128
    rows[7] = np.ldexp(1.0, np.arange(D) - 64)
    rows[8] = -np.ldexp(1.0, -np.arange(D))
    x = host(torch.from_numpy(rows).bfloat16()).reshape(1, 9, 1, D)
    cache = empty_cache(1, 1, 12)
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    gqa.gqa_kv_append_mxfp4(*cache, dev(x), dev(x), pos)
    codes, scales = cache_ops.mxfp4_quantize(x)
    assert np.array_equal(host(cache[0])[0, 0, :9], codes[0, :, 0]) and np.array_equal(host(cache[1])[0, 0, :9], scales[0, :, 0])
    assert np.array_equal(host(cache[2])[0, 0, :9], codes[0, :, 0]) and np.array_equal(host(cache[3])[0, 0, :9], scales[0, :, 0])
    out = [torch.empty(1, 9, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    gqa.gqa_kv_read_mxfp4(*out, *cache, pos)
    assert np.array_equal(oracle.widen(host(out[0])), cache_ops.mxfp4_values(codes, scales), equal_nan=True)


def test_read_every_code_at_every_scale(gqa):
    # 256 scales x 16 codes, the subnormal results among them
    cache = empty_cache(1, 1, 256)
    c = np.arange(D, dtype=np.uint8) % 16
    for i in (0, 2):
        cache[i][:] = dev((c[0::2] | (c[1::2] << 4)).astype(np.uint8))
        cache[i + 1][:] = torch.arange(256, device="cuda").to(torch.uint8).view(1, 1, 256, 1)
    out = [torch.empty(1, 256, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    gqa.gqa_kv_read_mxfp4(*out, *cache, torch.zeros(1, dtype=torch.int32, device="cuda"))
    want = cache_ops.mxfp4_values(host(cache[0]), host(cache[1]))[0, 0]
    for o in out:
        got = oracle.widen(host(o))[0, :, 0]
        assert np.array_equal(got[:253], want[:253]) and np.isnan(got[255]).all()
        # 2^126 * 4 and beyond are past bfloat16
        big = np.abs(want) > 3.3895313892515355e38
        assert np.array_equal(got[~big & ~np.isnan(want)], want[~big & ~np.isnan(want)]) and np.isinf(got[big]).all()


def test_positions_out_of_range(gqa):
    B, T, K, S = 4, 3, 2, 16
    x = dev(synth.normal((B, T, K, D), synth.BF16, 0x3411, 1))
    cache = empty_cache(B, K, S)
    pos = torch.tensor([14, -1, 2 ** 31 - 1, 13], dtype=torch.int32, device="cuda")
    gqa.gqa_kv_append_mxfp4(*cache, x, x, pos)
    assert gqa.gqa_get_last_error() == (gqa.GQA_ERR_DEVICE, gqa.GQA_DEVERR_APPEND_POS)
    assert all(bool((c[:3] == 0xA5).all()) and bool((c[3, :, :13] == 0xA5).all()) for c in cache)
    out = [torch.full((B, T, K, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    gqa.gqa_kv_read_mxfp4(*out, *cache, pos)
    assert gqa.gqa_get_last_error() == (gqa.GQA_ERR_DEVICE, gqa.GQA_DEVERR_APPEND_POS)
    assert not out[0][:3].any() and out[0][3].any() and not out[1][:3].any()
