"""GPU parity of gqa_kv_evict with the oracle: every byte equal."""
import numpy as np
import pytest
import torch

import synth
from _helpers import Guarded, dev, host
from oracle import cache_ops

pytestmark = pytest.mark.gpu
TORCH = {synth.BF16: torch.bfloat16, synth.F32: torch.float32}


@pytest.fixture(scope="module")
def gqa():
    from kv_cache_02_b200 import gqa as g

    return g


def same(got, want, what):
    assert np.array_equal(got.view(np.uint8), want.view(np.uint8)), what


def make(B, K, S, d, dt, seed, ties=False):
    kc, vc = (synth.normal((B, K, S, d), dt, seed, s) for s in (1, 2))
    s = np.abs(synth.normal((B, K, S), synth.F32, seed, 3)).astype(np.float32)
    if ties:
        s = np.round(s * 4) / 4
    order = np.argsort(synth.normal((B, K, S), synth.F64, seed, 4), axis=-1)
    return kc, vc, s, order.astype(np.int32)


def run(gqa, kc, vc, s, pos, lens, keep, sinks, recent):
    B, K, S, d = kc.shape
    t = torch.bfloat16 if kc.dtype == np.uint16 else torch.float32
    gk, gv, gs = Guarded(kc.shape, t), Guarded(vc.shape, t), Guarded(s.shape, torch.float32)
    for g, a in ((gk, kc), (gv, vc), (gs, s)):
        g.t.copy_(dev(a))
    tp, tl = None if pos is None else dev(pos), dev(np.array(lens, np.int32))
    n = gqa.gqa_kv_evict_workspace_bytes(B, K, S, keep)
    ws = torch.full((n + 64,), 0xEE, dtype=torch.uint8, device="cuda")
    gqa.gqa_kv_evict(gk.t, gv.t, gs.t, tp, tl, keep, sinks, None if recent is None else dev(np.array(recent, np.int32)),
                     ws[:n])
    status = gqa.gqa_get_last_error()
    assert gk.intact() and gv.intact() and gs.intact() and bool((ws[n:] == 0xEE).all())
    return (host(gk.t), host(gv.t), host(gs.t), None if pos is None else host(tp), host(tl)), status


def compare(gqa, kc, vc, s, pos, lens, keep, sinks, recent, what):
    got, status = run(gqa, kc, vc, s, pos, lens, keep, sinks, recent)
    assert status == (0, 0), what
    want = cache_ops.evict(kc, vc, s, pos, lens, keep, sinks, recent)
    for g, w, n in zip(got, want, ("keys", "values", "scores", "positions", "lengths")):
        if w is not None:
            same(g, w, f"{what}: {n}")


CASES = [
    # B, K, S, d, dtype, lens, keep, sinks, recent (rows), ties
    (1, 1, 1, 128, synth.BF16, (1,), 1, 0, 0, False),
    (3, 2, 100, 64, synth.BF16, (100, 0, 33), 32, 4, 8, False),
    (2, 3, 777, 128, synth.F32, (777, 776), 1, 0, 0, False),
    (2, 2, 777, 64, synth.F32, (777, 500), 776, 0, 0, True),
    (2, 4, 2048, 128, synth.BF16, (2048, 2047), 1024, 2000, 5, True),   # more held than kept
    (1, 2, 8193, 128, synth.BF16, (8193,), 700, 4, 64, True),           # a cluster of CTAs
    (2, 1, 9000, 128, synth.BF16, (40, 9000), 39, 0, 0, False),         # a long cache, a short sequence
    (1, 2, 20000, 64, synth.BF16, (19999,), 15000, 1, 1000, False),
    (3, 8, 10004, 64, synth.BF16, (10004, 9000, 12), 9000, 4, 64, True),  # more heads than clusters fit: 16 rows a thread
    (3, 8, 16384, 64, synth.BF16, (16384, 16000, 9), 16200, 4, 64, False),
]


@pytest.mark.parametrize("positions", [True, False])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_the_oracle(gqa, case, positions):
    B, K, S, d, dt, lens, keep, sinks, recent, ties = case
    kc, vc, s, pos = make(B, K, S, d, dt, 0x3301 + S, ties)
    since = [max(0, n - recent) for n in lens] if recent else None
    compare(gqa, kc, vc, s, pos if positions else None, lens, keep, sinks, since, f"{case}")


def test_every_kind_of_score(gqa):
    B, K, S = 1, 1, 64
    kc, vc, s, pos = make(B, K, S, 128, synth.BF16, 0x3302)
    s[0, 0, :16] = [np.inf, -np.inf, np.nan, 0.0, -0.0, -1.0, 1e-45, -1e-45, np.inf, np.nan, 3e38, -3e38, 0.0, -0.0, 1.0, 1.0]
    s[0, 0, 16:] = s[0, 0, :48]
    for keep in range(1, 64, 3):
        compare(gqa, kc, vc, s, None, (S,), keep, 0, None, f"keep {keep}")
    s[:] = 0.25  # all equal: the first rows stay, nothing moves
    compare(gqa, kc, vc, s, pos, (S,), 20, 0, None, "equal")
    s[:] = np.nan
    compare(gqa, kc, vc, s, pos, (S,), 20, 0, [60], "nan")


def test_held_rows_at_the_ends_of_the_positions(gqa):
    kc, vc, s, pos = make(2, 2, 300, 64, synth.BF16, 0x3303)
    pos[0, 0, 5], pos[1, 1, 250] = 2 ** 31 - 1, -(2 ** 31)
    compare(gqa, kc, vc, s, pos, (300, 299), 100, 3, [2 ** 31 - 1, -(2 ** 31)], "extremes")


def test_a_cut_cache_can_be_cut_again(gqa):
    kc, vc, s, pos = make(2, 2, 400, 128, synth.BF16, 0x3304)
    lens = np.array((400, 380), np.int32)
    for keep in (300, 200, 64, 64):
        compare(gqa, kc, vc, s, pos, lens, keep, 4, [390, 370], f"keep {keep}")
        kc, vc, s, pos, lens = cache_ops.evict(kc, vc, s, pos, lens, keep, 4, [390, 370])


def test_bad_lengths_leave_the_sequence(gqa):
    kc, vc, s, pos = make(3, 2, 100, 128, synth.BF16, 0x3305)
    got, status = run(gqa, kc, vc, s, pos, (101, -1, 100), 50, 0, None)
    assert status == (gqa.GQA_ERR_DEVICE, gqa.GQA_DEVERR_SEQLEN)
    want = cache_ops.evict(kc, vc, s, pos, (101, -1, 100), 50, 0, None)
    for b in range(2):
        for g, w in zip(got[:4], (kc, vc, s, pos)):
            same(g[b], w[b], "left alone")
    assert got[4].tolist() == [101, -1, 50]
    for g, w in zip(got[:4], want[:4]):
        same(g[2], w[2], "the good one")


def test_a_cache_longer_than_a_cluster_holds(gqa):
    # more than 8 x 40960 rows: the last keys of each CTA's segment are not kept in shared memory
    S, keep = 400000, 70000
    kc = torch.zeros(1, 1, S, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.from_numpy(np.round(np.abs(synth.normal((1, 1, S), synth.F32, 0x3306, 1)) * 1000) / 1000).float().cuda()
    pos, lens = torch.arange(S, dtype=torch.int32, device="cuda").view(1, 1, S).clone(), torch.tensor([S], dtype=torch.int32, device="cuda")
    kc[0, 0, :, 0] = (torch.arange(S, device="cuda") % 251).bfloat16()
    vc, first, rows = kc.clone(), s.clone(), kc.clone()
    ws = torch.empty(gqa.gqa_kv_evict_workspace_bytes(1, 1, S, keep), dtype=torch.uint8, device="cuda")
    gqa.gqa_kv_evict(kc, vc, s, pos, lens, keep, workspace=ws)
    assert gqa.gqa_get_last_error() == (0, 0)
    stay = torch.sort(first[0, 0], descending=True, stable=True).indices[:keep].sort().values
    got = pos[0, 0, :keep].long()
    assert torch.equal(got.sort().values, stay) and bool((pos[0, 0, keep:] == -1).all())
    assert torch.equal(s[0, 0, :keep], first[0, 0, got]) and not s[0, 0, keep:].any()
    assert torch.equal(kc[0, 0, :keep], rows[0, 0, got]) and torch.equal(vc[0, 0, :keep], rows[0, 0, got])
    assert torch.equal(got[stay[stay < keep]], stay[stay < keep])  # rows below keep that stay do not move


@pytest.mark.parametrize("bs,dt", [(16, synth.BF16), (48, synth.F32)])
def test_paged(gqa, bs, dt):
    B, K, d, lens, keep = 3, 2, 128, (650, 30, 401), 200
    mb = -(-660 // bs)
    S = mb * bs
    kc, vc, s, pos = make(B, K, S, d, dt, 0x3307)
    table = np.argsort(synth.normal((B * mb + 2,), synth.F64, 0x3307, 7))[:B * mb].astype(np.int32).reshape(B, mb)
    pools = []
    for c in (kc, vc):
        pool = torch.zeros(B * mb + 2, K, bs, d, dtype=TORCH[dt], device="cuda")
        pool[dev(table).long()] = dev(c).view(B, K, mb, bs, d).transpose(1, 2)
        pools.append(pool)
    ts, tp, tl = dev(s), dev(pos), dev(np.array(lens, np.int32))
    ws = torch.empty(gqa.gqa_kv_evict_workspace_bytes(B, K, S, keep), dtype=torch.uint8, device="cuda")
    gqa.gqa_kv_evict_paged(*pools, dev(table), ts, tp, tl, keep, 2, dev(np.array([640, 0, 390], np.int32)), ws)
    assert gqa.gqa_get_last_error() == (0, 0)
    want = cache_ops.evict(kc, vc, s, pos, lens, keep, 2, [640, 0, 390])
    for pool, w in zip(pools, want):
        same(host(pool[dev(table).long()].transpose(1, 2).reshape(B, K, S, d)), w, "rows")
    for g, w in zip((ts, tp, tl), want[2:]):
        same(host(g), w, "state")


def test_paged_entries_outside_the_pool(gqa):
    B, K, d, bs, mb = 1, 1, 64, 16, 4
    pools = [torch.arange(3 * bs, device="cuda").float().view(3, 1, bs, 1).expand(3, 1, bs, d).contiguous() for _ in range(2)]
    s = torch.arange(64, device="cuda").float().view(1, 1, 64).contiguous()  # the last rows stay
    lens = torch.tensor([64], dtype=torch.int32, device="cuda")
    ws = torch.empty(gqa.gqa_kv_evict_workspace_bytes(1, 1, 64, 16), dtype=torch.uint8, device="cuda")
    gqa.gqa_kv_evict_paged(*pools, torch.tensor([[1, 0, 2, 3]], dtype=torch.int32, device="cuda"), s, None, lens, 16, workspace=ws)
    assert gqa.gqa_get_last_error() == (gqa.GQA_ERR_DEVICE, gqa.GQA_DEVERR_BLOCK)
    want = torch.arange(3 * bs, device="cuda").float().view(3, bs, 1).expand(3, bs, d)
    assert torch.equal(pools[0][:, 0], want) and int(lens[0]) == 16
