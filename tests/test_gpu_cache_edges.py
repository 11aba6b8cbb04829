"""Calls of the cache operators at the edges of what their documentation
allows: offsets past 2^31 elements, buffers that start 16 bytes into an
allocation, host threads that call at once, rows of the largest capacity."""
import threading

import numpy as np
import pytest
import torch

import oracle
import synth
from _helpers import dev, host
from oracle import cache_ops
from test_gpu_scores import assert_out, assert_scores, largest

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def gqa():
    from kv_cache_02_b200 import gqa as g

    return g


def shifted(*shape, dtype=torch.bfloat16, by=16):
    """A tensor that starts `by` bytes into its allocation."""
    n = int(np.prod(shape)) * torch.tensor([], dtype=dtype).element_size()
    return torch.zeros(n + by, dtype=torch.uint8, device="cuda")[by:].view(dtype).view(shape)


def test_rows_past_2_to_31_elements(gqa):
    # 2 x 8.6 GB: the last KV head's last rows lie past 2^32 bytes and 2^31 elements
    B, K, S, H = 1, 16, 2_100_000, 32
    kc, vc = (torch.zeros(B, K, S, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x = dev(synth.normal((B, 3, H + 2 * K, D), synth.BF16, 0x3601, 1))
    q, k, v = x[:, :, :H], x[:, :, H:H + K], x[:, :, H + K:]
    rows, out = torch.tensor([S - 3], dtype=torch.int32, device="cuda"), torch.empty(B, 3, H, D, dtype=torch.bfloat16, device="cuda")
    row_pos = torch.arange(S, dtype=torch.int32, device="cuda").repeat(B, K, 1)
    positions = torch.arange(3, dtype=torch.int32, device="cuda").view(1, 3) + 7
    gqa.gqa_qk_norm_rope(out, q, k, None, positions, v=v, k_cache=kc, v_cache=vc, rows=rows, row_pos=row_pos)
    assert gqa.gqa_get_last_error() == (0, 0)
    assert torch.equal(kc[0, :, S - 3:], k[0].transpose(0, 1)) and torch.equal(vc[0, :, S - 3:], v[0].transpose(0, 1))
    assert not kc[0, :, S - 10:S - 3].any() and torch.equal(row_pos[0, :, S - 3:], positions.expand(K, 3))
    # those three rows are the heaviest: they come down to the first three holes
    scores = torch.zeros(B, K, S, device="cuda")
    scores[:, :, S - 3:] = torch.tensor([3.0, 1.0, 2.0], device="cuda")
    lens = torch.tensor([S], dtype=torch.int32, device="cuda")
    ws = torch.empty(gqa.gqa_kv_evict_workspace_bytes(B, K, S, 8), dtype=torch.uint8, device="cuda")
    gqa.gqa_kv_evict(kc, vc, scores, None, lens, 8, workspace=ws)
    assert gqa.gqa_get_last_error() == (0, 0) and int(lens[0]) == 8
    assert torch.equal(kc[0, :, 5:8], k[0].transpose(0, 1)) and torch.equal(vc[0, :, 5:8], v[0].transpose(0, 1))
    assert scores[0, :, 5:8].tolist() == [[3.0, 1.0, 2.0]] * K and not scores[0, :, 8:].any()
    # weights over all of a far head's rows: keys of zero but for three
    kc[0, K - 1, S - 3:] = k[0, :, K - 1]
    lens.fill_(S)
    scores.zero_()
    one = out[:, 0].contiguous()
    ws = torch.empty(gqa.gqa_decode_scores_workspace_bytes(B, H, K, S, D), dtype=torch.uint8, device="cuda")
    got = torch.empty_like(one)
    gqa.gqa_decode_scores(got, scores, one, kc, vc, lens, 0.5, workspace=ws)
    assert gqa.gqa_get_last_error() == (0, 0)
    x3 = 0.5 * (one[0, -2:].double() @ kc[0, K - 1, S - 3:].double().T)
    x8 = 0.5 * (one[0, -2:].double() @ kc[0, K - 1, :8].double().T)
    total = torch.cat([x3.exp(), x8.exp()], 1).sum(1, keepdim=True) + (S - 11)
    want = (x3.exp() / total).sum(0)
    assert torch.allclose(scores[0, K - 1, S - 3:].double(), want, rtol=1e-4, atol=0)


def test_four_bit_rows_past_2_to_31_bytes(gqa):
    B, K, S, H = 1, 2, 20_000_000, 8
    cache = [torch.zeros(B, K, S, n, dtype=torch.uint8, device="cuda") for n in (D // 2, D // 32, D // 2, D // 32)]
    new = [synth.normal((B, 4, K, D), synth.BF16, 0x3602, s) for s in (1, 2)]
    pos = torch.tensor([S - 4], dtype=torch.int32, device="cuda")
    gqa.gqa_kv_append_mxfp4(*cache, dev(new[0]), dev(new[1]), pos)
    back = [torch.empty(B, 4, K, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    gqa.gqa_kv_read_mxfp4(*back, *cache, pos)
    values = [cache_ops.mxfp4_values(*cache_ops.mxfp4_quantize(x)) for x in new]
    for b, v in zip(back, values):
        assert np.array_equal(oracle.widen(host(b)), v)
    # every other key and value is zero: the result is the four rows' share
    q = synth.normal((B, H, D), synth.BF16, 0x3602, 3)
    ws = torch.empty(gqa.gqa_decode_mxfp4_workspace_bytes(B, H, K, S, D), dtype=torch.uint8, device="cuda")
    out = torch.empty(B, H, D, dtype=torch.bfloat16, device="cuda")
    gqa.gqa_decode_mxfp4(out, dev(q), *cache, pos + 4, 1.0, workspace=ws)
    assert gqa.gqa_get_last_error() == (0, 0)
    for h in range(H):
        x = values[0][0, :, h // (H // K)] @ oracle.widen(q)[0, h]
        w = np.exp(x - x.max())
        want = (w / (w.sum() + (S - 4) * np.exp(-x.max()))) @ values[1][0, :, h // (H // K)]
        # the weights' rounding to fp16 and the result's, and 2 d 2^-23 of the scores' magnitudes (below 2^-10)
        spread = (w / (w.sum() + (S - 4) * np.exp(-x.max()))) @ np.abs(values[1][0, :, h // (H // K)])
        assert np.all(np.abs(oracle.widen(host(out))[0, h] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * spread)


def test_buffers_that_start_16_bytes_in(gqa):
    B, T, H, K, S = 2, 9, 16, 4, 64
    def put(a, **kw):
        t = shifted(*a.shape, dtype=torch.from_numpy(a).dtype if a.dtype != np.uint16 else torch.bfloat16, **kw)
        t.copy_(dev(a))
        return t
    q, k, v = (synth.normal((B, T, n, D), synth.BF16, 0x3603, s) for n, s in ((H, 1), (K, 2), (K, 3)))
    kc, vc = (synth.normal((B, K, S, D), synth.BF16, 0x3603, s) for s in (4, 5))
    lens = np.array([50, 64], np.int32)
    results = []
    for place in (dev, put):
        tq, tk, tv, tkc, tvc = (place(a) for a in (q, k, v, kc, vc))
        table = place(np.zeros((64, D), np.float32))
        gqa.gqa_rope_table(table)
        pos = torch.arange(T, dtype=torch.int32, device="cuda").repeat(B, 1)
        w = place(synth.normal((D,), synth.BF16, 0x3603, 6))
        tl = dev(lens)
        tq2, tk2 = place(q), place(k)
        gqa.gqa_qk_norm_rope(tq2, tq, tk, table, pos, w, w, k_out=tk2, v=tv, k_cache=tkc, v_cache=tvc, rows=tl - 50)
        scores, out = place(np.zeros((B, K, S), np.float32)), place(q[:, 0])
        n = max(gqa.gqa_decode_scores_workspace_bytes(B, H, K, S, D), gqa.gqa_prompt_scores_workspace_bytes(B, T, H, K, S, D),
                gqa.gqa_kv_evict_workspace_bytes(B, K, S, 32), gqa.gqa_decode_mxfp4_workspace_bytes(B, H, K, S, D))
        ws = place(np.zeros(n, np.uint8))
        gqa.gqa_decode_scores(out, scores, tq2[:, 0].contiguous() if place is dev else put(host(tq2[:, 0])), tkc, tvc, tl, 0.1, workspace=ws)
        gqa.gqa_prompt_scores(scores, tq2, tkc, tl, 0.1, workspace=ws)
        c4 = [place(np.zeros((B, K, S, m), np.uint8)) for m in (D // 2, D // 32, D // 2, D // 32)]
        gqa.gqa_kv_append_mxfp4(*c4, tk2, tv, tl - 50)
        back, back2, out4 = place(k), place(k), place(q[:, 0])
        gqa.gqa_kv_read_mxfp4(back, back2, *c4, tl - 50)
        gqa.gqa_decode_mxfp4(out4, tq[:, 0].contiguous() if place is dev else put(q[:, 0]), *c4, tl, 0.1, workspace=ws)
        # positions at any alignment that int32 has
        row_pos = shifted(B, K, S, dtype=torch.int32, by=4 if place is put else 16)
        row_pos.copy_(torch.arange(S, dtype=torch.int32, device="cuda").expand(B, K, S))
        gqa.gqa_kv_evict(tkc, tvc, scores, row_pos, tl, 32, 2, None, ws)
        assert gqa.gqa_get_last_error() == (0, 0)
        results.append([t.clone() for t in (tq2, tk2, tkc, tvc, out, scores, *c4, back, back2, out4, row_pos, tl)])
    for i, (a, b) in enumerate(zip(*results)):
        assert torch.equal(a, b), i
    with pytest.raises(gqa.GqaError):  # 8 bytes in: refused
        gqa.gqa_kv_evict(shifted(B, K, S, D, by=8), vc := torch.zeros(B, K, S, D, dtype=torch.bfloat16, device="cuda"),
                         torch.zeros(B, K, S, device="cuda"), None, dev(lens), 32, workspace=ws)


def test_positions_not_aligned_to_four_in_a_long_cache(gqa):
    # the vector reads of the long cache's select need 16-byte rows: refused here by the pointer, not by the caller
    S, keep = 20000, 300
    kc, vc = (synth.normal((1, 1, S, 64), synth.BF16, 0x3604, s) for s in (1, 2))
    s = np.abs(synth.normal((1, 1, S), synth.F32, 0x3604, 3)).astype(np.float32)
    pos = np.argsort(s, axis=-1).astype(np.int32)
    want = cache_ops.evict(kc, vc, s, pos, [S], keep, 3, [S - 50])
    tp = shifted(1, 1, S, dtype=torch.int32, by=4)
    tp.copy_(dev(pos))
    tk, tv, ts, tl = dev(kc), dev(vc), dev(s), torch.tensor([S], dtype=torch.int32, device="cuda")
    ws = torch.empty(gqa.gqa_kv_evict_workspace_bytes(1, 1, S, keep), dtype=torch.uint8, device="cuda")
    gqa.gqa_kv_evict(tk, tv, ts, tp, tl, keep, 3, torch.tensor([S - 50], dtype=torch.int32, device="cuda"), ws)
    assert gqa.gqa_get_last_error() == (0, 0)
    for got, w in zip((tk, tv, ts, tp, tl), want):
        assert np.array_equal(host(got).view(np.uint8), w.view(np.uint8))


def test_host_threads_call_at_once(gqa):
    B, H, K, S = 2, 16, 4, 500
    lens = (500, 311)
    kc, vc = (synth.normal((B, K, S, D), synth.BF16, 0x3605, s) for s in (1, 2))
    q = synth.normal((B, H, D), synth.BF16, 0x3605, 3)
    want, added, spread = cache_ops.decode_scores(q, kc, vc, lens, 0.1)
    rel = 2 * D * 2.0 ** -23 * largest(q, kc, 0.1) + 2.0 ** -20
    found, errors = [None] * 4, []
    shared = dev(q), dev(kc), dev(vc), dev(np.array(lens, np.int32))
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    scores, out = torch.zeros(B, K, S, device="cuda"), torch.empty(B, H, D, dtype=torch.bfloat16, device="cuda")
                    ws = torch.empty(gqa.gqa_decode_scores_workspace_bytes(B, H, K, S, D, 1 + i), dtype=torch.uint8, device="cuda")
                    gqa.gqa_decode_scores(out, scores, *shared, 0.1, 1 + i, ws)
                found[i] = scores, out
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors and gqa.gqa_get_last_error() == (0, 0)
    for scores, out in found:
        assert_scores(host(scores), np.zeros((B, K, S), np.float32), added, lens, rel, H // K + S, "threads")
        assert_out(host(out), want, spread, rel, "threads")


def test_empty_calls(gqa):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    i32 = torch.int32
    gqa.gqa_qk_norm_rope(z(0, 3, 8, D), z(0, 3, 8, D), z(0, 3, 2, D), None, None)
    gqa.gqa_qk_norm_rope(z(2, 0, 8, D), z(2, 0, 8, D), z(2, 0, 2, D), None, None)
    gqa.gqa_prompt_scores(torch.zeros(2, 2, 16, device="cuda"), z(2, 0, 8, D), z(2, 2, 16, D), z(2, dtype=i32), 1.0)
    gqa.gqa_decode_scores(z(0, 8, D), z(0, 2, 16, dtype=torch.float32), z(0, 8, D), z(0, 2, 16, D), z(0, 2, 16, D), z(0, dtype=i32), 1.0)
    gqa.gqa_kv_evict(z(0, 2, 16, D), z(0, 2, 16, D), z(0, 2, 16, dtype=torch.float32), None, z(0, dtype=i32), 4)
    c = [z(0, 2, 16, n, dtype=torch.uint8) for n in (64, 4, 64, 4)]
    gqa.gqa_kv_append_mxfp4(*c, z(0, 3, 2, D), z(0, 3, 2, D), z(0, dtype=i32))
    gqa.gqa_decode_mxfp4(z(0, 8, D), z(0, 8, D), *c, z(0, dtype=i32), 1.0)
    assert gqa.gqa_get_last_error() == (0, 0)


@pytest.mark.parametrize("H,d", [(4, 128), (3, 128), (5, 64), (7, 128)])  # 7 heads: 126 rows of a tile are queries
def test_prompt_scores_of_keys_at_minus_infinity(gqa, H, d):
    # such a key weighs nothing, whether it is alone among others or all that a query sees of the first tiles
    B, T, K, S, n = 1, 60, 1, 800, 777
    k = synth.normal((B, K, S, d), synth.F32, 0x3620, 2)
    q = synth.normal((B, T, H, d), synth.F32, 0x3620, 1)
    q[..., 0] = 1.0
    k[..., 0] = 0.0
    finite = host(dev(k).bfloat16())
    k[0, 0, [*range(200), 333, 650], 0] = -np.inf
    kb, qb = dev(k).bfloat16(), dev(q).bfloat16()
    scores = torch.zeros(B, K, S, device="cuda")
    ws = torch.empty(gqa.gqa_prompt_scores_workspace_bytes(B, T, H, K, S, d), dtype=torch.uint8, device="cuda")
    gqa.gqa_prompt_scores(scores, qb, kb, torch.tensor([n], dtype=torch.int32, device="cuda"), d ** -0.5, workspace=ws)
    assert gqa.gqa_get_last_error() == (0, 0)
    added = cache_ops.prompt_scores(host(qb), host(kb), (n,), d ** -0.5)
    assert not added[0, 0, :200].any() and added[0, 0, 200:333].all() and np.isfinite(added).all()
    rel = 2 * d * 2.0 ** -23 * largest(host(qb), finite, d ** -0.5) + 2.0 ** -20
    assert_scores(host(scores), np.zeros((B, K, S), np.float32), added, (n,), rel, T * H + S, "keys at -inf")


@pytest.mark.parametrize("splits", [0, 1, 2])
@pytest.mark.parametrize("H,d", [(8, 128), (3, 64)])
def test_decode_scores_of_keys_at_minus_infinity(gqa, H, d, splits):
    B, K, S, n = 1, 1, 800, 777
    k, v, q = (synth.normal(shape, synth.F32, 0x3622, s) for s, shape in ((2, (B, K, S, d)), (3, (B, K, S, d)),
                                                                          (1, (B, H, d))))
    q[..., 0] = 1.0
    k[..., 0] = 0.0
    finite = host(dev(k).bfloat16())
    k[0, 0, [*range(450), 500, 776], 0] = -np.inf
    kb, vb, qb = (dev(x).bfloat16() for x in (k, v, q))
    scores, out = torch.zeros(B, K, S, device="cuda"), torch.empty_like(qb)
    ws = torch.empty(gqa.gqa_decode_scores_workspace_bytes(B, H, K, S, d, splits), dtype=torch.uint8, device="cuda")
    gqa.gqa_decode_scores(out, scores, qb, kb, vb, torch.tensor([n], dtype=torch.int32, device="cuda"), d ** -0.5,
                          splits, workspace=ws)
    assert gqa.gqa_get_last_error() == (0, 0)
    want, added, spread = cache_ops.decode_scores(host(qb), host(kb), host(vb), (n,), d ** -0.5)
    assert not added[0, 0, :450].any() and added[0, 0, 450:500].all() and np.isfinite(want).all()
    rel = 2 * d * 2.0 ** -23 * largest(host(qb), finite, d ** -0.5) + 2.0 ** -20
    assert_scores(host(scores), np.zeros((B, K, S), np.float32), added, (n,), rel, H + S, "keys at -inf")
    assert_out(host(out), want, spread, rel, "keys at -inf")


@pytest.mark.parametrize("splits", [1, 2])
def test_a_split_of_nan_keys_is_not_lost(gqa, splits):
    # every query sees them: outputs and weights are NaN, whatever the other splits hold
    B, H, K, d, S, n, bad = 1, 6, 2, 128, 4000, 3999, 2100
    k = synth.normal((B, K, S, d), synth.F32, 0x3623, 2)
    k[0, 0, :bad] = np.nan
    kb, q = dev(k).bfloat16(), dev(synth.normal((B, 4, H, d), synth.BF16, 0x3623, 1))
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    a, b, out = torch.zeros(B, K, S, device="cuda"), torch.zeros(B, K, S, device="cuda"), torch.empty_like(q[:, 0])
    ws = torch.empty(max(gqa.gqa_decode_scores_workspace_bytes(B, H, K, S, d, splits),
                         gqa.gqa_prompt_scores_workspace_bytes(B, 4, H, K, S, d)), dtype=torch.uint8, device="cuda")
    gqa.gqa_decode_scores(out, a, q[:, 0].contiguous(), kb, kb.nan_to_num(), lens, 0.1, splits, workspace=ws)
    gqa.gqa_prompt_scores(b, q, kb, lens, 0.1, workspace=ws)
    assert out[0, :H // K].isnan().all() and out[0, H // K:].isfinite().all()
    for s, seen in ((a, n), (b, n - 3)):
        assert s[0, 0, :seen].isnan().all() and s[0, 1].isfinite().all() and not s[0, :, n:].any()


def test_decode_scores_paged_entries_outside_the_pool(gqa):
    # block 0 is read in place of a bad entry; the other sequence, and entries past the length, do not mind
    B, H, K, d, bs, mb = 2, 8, 2, 128, 16, 8
    pools = [dev(synth.normal((B * mb, K, bs, d), synth.BF16, 0x3621, s)) for s in (2, 3)]
    q = dev(synth.normal((B, H, d), synth.BF16, 0x3621, 1))
    table = torch.arange(B * mb, dtype=torch.int32, device="cuda").reshape(B, mb).contiguous()
    lens = torch.tensor([128, 70], dtype=torch.int32, device="cuda")
    ws = torch.empty(gqa.gqa_decode_scores_paged_workspace_bytes(B, H, K, d, bs, mb), dtype=torch.uint8, device="cuda")

    def run():
        out, scores = torch.empty_like(q), torch.zeros(B, K, mb * bs, device="cuda")
        gqa.gqa_decode_scores_paged(out, scores, q, *pools, table, lens, 0.1, workspace=ws)
        return out, scores, gqa.gqa_get_last_error()

    out, scores, err = run()
    assert err == (0, 0)
    table[1, 5:] = -1  # past the length
    table[0, 3] = B * mb
    out2, scores2, err = run()
    assert err == (gqa.GQA_ERR_DEVICE, gqa.GQA_DEVERR_BLOCK)
    assert torch.equal(out2[1], out[1]) and torch.equal(scores2[1], scores[1])
    table[0, 3] = 0
    out3, scores3, err = run()
    assert err == (0, 0) and torch.equal(out2, out3) and torch.equal(scores2, scores3)
