"""GPU parity of gqa_decode_scores and gqa_prompt_scores with the float64 oracle.

Tolerances. A weight p = 2^(x - m) / L: x is a sum of d products of bfloat16
values in float32, off by at most d 2^-23 sum |q k| (a step for each addition),
times the scale; m and L carry the same error, ex2.approx 2^-22, the rest less.
With A = scale * max sum |q k| every weight is within a relative
REL = 2 d 2^-23 A + 2^-20. Weights add up in float32 in a chain of at most N
terms: N 2^-24 of the sum. The score's own last addition: 2^-24 of it.

Outputs: the decode rounds p to bfloat16 (2^-8 of sum p |v|), and the result
(2^-8 of it).
"""
import numpy as np
import pytest
import torch

import oracle
import synth
from _helpers import Guarded, dev, host
from oracle import cache_ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gqa():
    from kv_cache_02_b200 import gqa as g

    return g


def largest(q, k, scale):
    """scale * an upper bound of sum |q k|."""
    q, k = np.abs(oracle.widen(q)), np.abs(np.nan_to_num(oracle.widen(k)))
    return abs(scale) * np.sqrt((q * q).sum(-1).max() * (k * k).sum(-1).max())


def assert_scores(got, before, added, lens, rel, chain, what):
    B, K, S = got.shape
    live = np.arange(S)[None, None, :] < np.asarray(lens)[:, None, None]
    live = np.broadcast_to(live, got.shape)
    assert np.array_equal(got[~live].view(np.uint32), before[~live].view(np.uint32)), f"{what}: rows past the length"
    want = before.astype(np.float64) + added
    tol = (rel + chain * 2.0 ** -24) * added + 2.0 ** -23 * np.abs(want) + 1e-37
    err = np.abs(got - want)
    assert np.all(err[live] <= tol[live]), f"{what}: {np.max((err / tol)[live])} of the tolerance"


def assert_out(got, out, spread, rel, what):
    err = np.abs(oracle.widen(got) - out)
    tol = (2.0 ** -8 + rel) * spread + 2.0 ** -8 * np.abs(out) + 1e-37
    assert np.all(err <= tol), f"{what}: {np.max(err / tol)} of the tolerance"


def caches(B, K, S_max, d, lens, seed):
    """NaN past the lengths."""
    return [synth.cache(B * K, S_max, d, synth.BF16, seed, s, np.asarray(lens, np.int32), K).reshape(B, K, S_max, d)
            for s in (2, 3)]


def start_scores(B, K, S, lens, seed):
    s = np.abs(synth.normal((B, K, S), synth.F32, seed, 9)).astype(np.float32)
    for b, n in enumerate(lens):
        s[b, :, n:] = np.nan  # never read
    return s


DECODE = [
    # B, H, K, d, S_max, lens
    (1, 1, 1, 128, 1, (1,)),
    (3, 16, 4, 128, 333, (300, 1, 77)),
    (4, 64, 8, 128, 1024, (0, 999, 1024, 513)),
    (2, 8, 8, 64, 192, (192, 65)),
    (2, 66, 1, 128, 704, (700, 129)),   # one KV head, 66 query heads: nine head slices, the last of two
    (1, 21, 3, 64, 2100, (2100,)),      # an odd group
    (2, 24, 2, 128, 5000, (4999, 3)),
]


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("case", DECODE, ids=str)
def test_decode_scores(gqa, case, splits):
    B, H, K, d, S, lens = case
    kc, vc = caches(B, K, S, d, lens, 0x3201)
    q, before = synth.normal((B, H, d), synth.BF16, 0x3201, 1), start_scores(B, K, S, lens, 0x3202)
    scale = 1.5 / np.sqrt(d)
    out, scores = Guarded((B, H, d), torch.bfloat16), Guarded((B, K, S), torch.float32)
    scores.t.copy_(dev(before))
    n = gqa.gqa_decode_scores_workspace_bytes(B, H, K, S, d, splits)
    ws = torch.full((n,), 0xEE, dtype=torch.uint8, device="cuda")
    args = (dev(q), dev(kc), dev(vc), dev(np.array(lens, np.int32)))
    gqa.gqa_decode_scores(out.t, scores.t, *args, scale, splits, ws)
    assert gqa.gqa_get_last_error() == (0, 0) and out.intact() and scores.intact()
    want, added, spread = cache_ops.decode_scores(q, kc, vc, lens, scale)
    rel = 2 * d * 2.0 ** -23 * largest(q, kc, scale) + 2.0 ** -20
    assert_scores(host(scores.t), before, added, lens, rel, H // K + S, f"{case}")
    assert_out(host(out.t), want, spread, rel, f"{case}")
    # the same call again repeats bit for bit
    again, out2 = dev(before), torch.empty_like(out.t)
    gqa.gqa_decode_scores(out2, again, *args, scale, splits, ws)
    assert np.array_equal(host(again).view(np.uint32), host(scores.t).view(np.uint32)) and torch.equal(out2, out.t)


@pytest.mark.parametrize("bs", [16, 48, 64])
def test_decode_scores_paged(gqa, bs):
    B, H, K, d, lens = 3, 24, 4, 128, (700, 0, 353)
    mb = -(-720 // bs)
    S = mb * bs
    kc, vc = caches(B, K, S, d, lens, 0x3203)
    order = np.argsort(synth.normal((B * mb + 2,), synth.F64, 0x3203, 4))
    table = order[:B * mb].astype(np.int32).reshape(B, mb)
    pools = []
    for c in (kc, vc):
        pool = np.full((B * mb + 2, K, bs, d), 0x7FC0, np.uint16)
        for b in range(B):
            for i in range(mb):
                pool[table[b, i]] = c[b, :, i * bs:(i + 1) * bs]
        pools.append(dev(pool))
    q, before = synth.normal((B, H, d), synth.BF16, 0x3203, 1), start_scores(B, K, S, lens, 0x3204)
    out, scores = torch.empty(B, H, d, dtype=torch.bfloat16, device="cuda"), dev(before)
    ws = torch.empty(gqa.gqa_decode_scores_paged_workspace_bytes(B, H, K, d, bs, mb), dtype=torch.uint8, device="cuda")
    gqa.gqa_decode_scores_paged(out, scores, dev(q), *pools, dev(table), dev(np.array(lens, np.int32)), d ** -0.5,
                                workspace=ws)
    assert gqa.gqa_get_last_error() == (0, 0)
    want, added, spread = cache_ops.decode_scores(q, kc, vc, lens, d ** -0.5)
    rel = 2 * d * 2.0 ** -23 * largest(q, kc, d ** -0.5) + 2.0 ** -20
    assert_scores(host(scores), before, added, lens, rel, H // K + S, f"paged {bs}")
    assert_out(host(out), want, spread, rel, f"paged {bs}")


def test_decode_scores_bad_lengths(gqa):
    B, H, K, d, S = 3, 8, 2, 128, 64
    kc, vc = caches(B, K, S, d, (64, 64, 64), 0x3205)
    q, scores = dev(synth.normal((B, H, d), synth.BF16, 0x3205, 1)), torch.zeros(B, K, S, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(gqa.gqa_decode_scores_workspace_bytes(B, H, K, S, d), dtype=torch.uint8, device="cuda")
    lens = torch.tensor([65, -1, 64], dtype=torch.int32, device="cuda")
    gqa.gqa_decode_scores(out, scores, q, dev(kc), dev(vc), lens, 1.0, workspace=ws)
    assert gqa.gqa_get_last_error() == (gqa.GQA_ERR_DEVICE, gqa.GQA_DEVERR_SEQLEN)
    assert not scores[:2].any() and not out[:2].any() and abs(float(scores[2].sum()) - H) < 1e-3


def test_a_peaked_softmax_keeps_its_tail(gqa):
    # one key takes all but 2^-40 of the weight: the others' weights are as exact, relatively, as any
    B, H, K, d, S = 1, 8, 1, 128, 1000
    kc, vc = caches(B, K, S, d, (S,), 0x3206)
    k = oracle.widen(kc) * 0.01
    q = np.zeros((B, H, d), np.float32)
    q[..., 0] = 1.0
    k[0, 0, 500, 0] = 27.0
    kc, q = dev(k.astype(np.float32)).bfloat16(), dev(q).bfloat16()
    scores, out = torch.zeros(B, K, S, device="cuda"), torch.empty_like(q)
    ws = torch.empty(gqa.gqa_decode_scores_workspace_bytes(B, H, K, S, d), dtype=torch.uint8, device="cuda")
    gqa.gqa_decode_scores(out, scores, q, kc, dev(vc), torch.tensor([S], dtype=torch.int32, device="cuda"), 1.0,
                          workspace=ws)
    _, added, _ = cache_ops.decode_scores(host(q), host(kc), vc, (S,), 1.0)
    rel = 2 * d * 2.0 ** -23 * largest(host(q), host(kc), 1.0) + 2.0 ** -20
    assert_scores(host(scores), np.zeros((B, K, S), np.float32), added, (S,), rel, H + S, "peaked")
    assert added[0, 0].min() < 1e-10


PROMPT = [
    # B, T, H, K, d, S_max, lens
    (1, 1, 1, 1, 128, 1, (1,)),
    (2, 1, 8, 2, 128, 300, (300, 17)),          # a single query: a decode step's weights
    (3, 40, 8, 2, 64, 200, (200, 40, 41)),
    (2, 130, 12, 4, 128, 130, (130, 100)),      # a whole prompt, and one shorter than T
    (4, 33, 5, 1, 128, 260, (0, 1, 32, 260)),   # 25 tokens a tile, an empty sequence
    (1, 17, 128, 1, 64, 140, (140,)),           # one token a tile
    (1, 9, 130, 2, 128, 64, (64,)),             # 65 heads a token: 1 token a tile, the rest of it zero
    (1, 300, 16, 2, 128, 4000, (3999,)),        # the keys are split
    (1, 900, 8, 1, 64, 900, (900,)),            # the rows are split
    (2, 64, 7, 7, 64, 513, (513, 512)),
]


@pytest.mark.parametrize("case", PROMPT, ids=str)
def test_prompt_scores(gqa, case):
    B, T, H, K, d, S, lens = case
    kc, _ = caches(B, K, S, d, lens, 0x3207)
    q = synth.normal((B, T, H, d), synth.BF16, 0x3207, 1)
    for b, n in enumerate(lens):
        q[b, :max(0, T - n)] = 0x7FC0  # queries before the sequence: NaN, not read into anything
    before = start_scores(B, K, S, lens, 0x3208)
    scale = 1.3 / np.sqrt(d)
    scores = Guarded((B, K, S), torch.float32)
    scores.t.copy_(dev(before))
    n = gqa.gqa_prompt_scores_workspace_bytes(B, T, H, K, S, d)
    ws = torch.full((n + 256,), 0xEE, dtype=torch.uint8, device="cuda")
    args = (dev(q), dev(kc), dev(np.array(lens, np.int32)), scale)
    gqa.gqa_prompt_scores(scores.t, *args, workspace=ws[:n])
    assert gqa.gqa_get_last_error() == (0, 0) and scores.intact() and bool((ws[n:] == 0xEE).all())
    real = q.copy()
    real[real == 0x7FC0] = 0
    added = cache_ops.prompt_scores(real, kc, lens, scale)
    rel = 2 * d * 2.0 ** -23 * largest(real, kc, scale) + 2.0 ** -20
    assert_scores(host(scores.t), before, added, lens, rel, T * H // K + S, f"{case}")
    again = dev(before)
    gqa.gqa_prompt_scores(again, *args, workspace=ws[:n])
    assert np.array_equal(host(again).view(np.uint32), host(scores.t).view(np.uint32))


def test_prompt_scores_bad_lengths(gqa):
    B, T, H, K, d, S = 3, 5, 8, 2, 128, 64
    kc, _ = caches(B, K, S, d, (64, 64, 64), 0x3209)
    scores = torch.zeros(B, K, S, device="cuda")
    ws = torch.empty(gqa.gqa_prompt_scores_workspace_bytes(B, T, H, K, S, d), dtype=torch.uint8, device="cuda")
    gqa.gqa_prompt_scores(scores, dev(synth.normal((B, T, H, d), synth.BF16, 0x3209, 1)), dev(kc),
                          torch.tensor([65, -1, 64], dtype=torch.int32, device="cuda"), 0.1, workspace=ws)
    assert gqa.gqa_get_last_error() == (gqa.GQA_ERR_DEVICE, gqa.GQA_DEVERR_SEQLEN)
    assert not scores[:2].any() and abs(float(scores[2].sum()) - T * H) < 1e-3


def test_the_last_query_is_the_decode_step(gqa):
    B, H, K, d, S = 2, 32, 8, 128, 700
    lens = dev(np.array([700, 5], np.int32))
    kc, vc = caches(B, K, S, d, (700, 5), 0x320A)
    q = dev(synth.normal((B, H, d), synth.BF16, 0x320A, 1))
    a, b = torch.zeros(B, K, S, device="cuda"), torch.zeros(B, K, S, device="cuda")
    ws = torch.empty(max(gqa.gqa_prompt_scores_workspace_bytes(B, 1, H, K, S, d),
                         gqa.gqa_decode_scores_workspace_bytes(B, H, K, S, d)), dtype=torch.uint8, device="cuda")
    gqa.gqa_prompt_scores(a, q[:, None].contiguous(), dev(kc), lens, d ** -0.5, workspace=ws)
    gqa.gqa_decode_scores(torch.empty_like(q), b, q, dev(kc), dev(vc), lens, d ** -0.5, workspace=ws)
    assert torch.allclose(a, b, rtol=2e-3, atol=1e-9)
