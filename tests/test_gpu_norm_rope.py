"""GPU parity of gqa_qk_norm_rope with the float64 oracle.

Tolerance: float32 arithmetic, one rounding to dtype. The mean of d squares is
a sum of positive terms in at most 12 rounded steps, then a division, a square
root, a reciprocal and two products: under 20 half steps of 2^-24 relative for
y, and the rotation's three roundings act on |y_i| + |y_j|: 32 * 2^-24 (|y_i| +
|y_j|) covers both. The result's rounding adds half a step, 2^-8 |y| for
bfloat16 and 2^-24 |y| for float32.
"""
import numpy as np
import pytest
import torch

import oracle
import synth
from _helpers import Guarded, dev, host
from oracle import cache_ops

pytestmark = pytest.mark.gpu
TORCH = {synth.BF16: torch.bfloat16, synth.F32: torch.float32}


@pytest.fixture(scope="module")
def gqa():
    from kv_cache_02_b200 import gqa as g

    return g


def check(got, y, z, table, interleaved, what):
    """got against z, the rotation of y."""
    r = 0 if table is None else table.shape[1]
    other = np.zeros_like(y)
    if r:
        if interleaved:
            other[..., 0:r:2], other[..., 1:r:2] = y[..., 1:r:2], y[..., 0:r:2]
        else:
            other[..., :r // 2], other[..., r // 2:r] = y[..., r // 2:r], y[..., :r // 2]
    half = 2.0 ** -8 if got.dtype == np.uint16 else 2.0 ** -24
    err = np.abs(oracle.widen(got) - z)
    tol = half * np.abs(z) + 32 * 2.0 ** -24 * (np.abs(y) + np.abs(other)) + 1e-38
    assert np.all(err <= tol), f"{what}: {np.max(err / tol)} of the tolerance"


def inputs(B, T, H, K, d, dt, seed, fused=True):
    """q, k, v as slices of one fused [B, T, (H + 2 K) d] tensor, and on their own on the host."""
    x = synth.normal((B, T, (H + 2 * K) * d), dt, seed, 1)
    t = dev(x).view(B, T, H + 2 * K, d)
    n = x.reshape(B, T, H + 2 * K, d)
    cut = (slice(0, H), slice(H, H + K), slice(H + K, None))
    return [t[:, :, c] for c in cut], [n[:, :, c] for c in cut]


CASES = [
    # B, T, H, K, d, dtype, rotary, interleaved, norm
    (1, 1, 1, 1, 128, synth.BF16, 128, False, True),
    (2, 3, 8, 2, 128, synth.BF16, 128, True, True),
    (3, 5, 12, 4, 128, synth.BF16, 64, False, True),
    (2, 7, 6, 6, 64, synth.BF16, 64, False, True),
    (2, 7, 10, 2, 64, synth.BF16, 16, True, False),
    (1, 300, 32, 8, 128, synth.BF16, 128, False, True),
    (700, 1, 16, 2, 128, synth.BF16, 16, False, True),
    (2, 9, 8, 2, 128, synth.F32, 128, False, True),
    (2, 9, 5, 1, 64, synth.F32, 32, True, True),
    (2, 257, 7, 7, 64, synth.F32, 0, False, True),
    (1, 2, 4, 2, 128, synth.BF16, 0, False, False),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_the_oracle(gqa, case):
    B, T, H, K, d, dt, rd, il, norm = case
    (q, k, v), (nq, nk, nv) = inputs(B, T, H, K, d, dt, 0x3101 + H + d)
    wq, wk = (synth.normal((d,), dt, 0x3102, s) if norm else None for s in (2, 3))
    S_max, max_pos = T + 9, 5000
    rows = synth.uniform_int(B, 0, S_max - T, 0x3103, 4).astype(np.int32)
    positions = (rows[:, None] * 3 + 4 * np.arange(T)[None, :] + np.arange(B)[:, None]).astype(np.int32) % max_pos
    table = torch.empty(max_pos, rd, device="cuda") if rd else None
    if rd:
        gqa.gqa_rope_table(table, 500000.0)
    t = TORCH[dt]
    q_out, k_out = Guarded((B, T, H, d), t), Guarded((B, T, K, d), t)
    kc, vc = Guarded((B, K, S_max, d), t), Guarded((B, K, S_max, d), t)
    row_pos = torch.full((B, K, S_max), -7, dtype=torch.int32, device="cuda")
    before = host(kc.t).copy(), host(vc.t).copy()
    gqa.gqa_qk_norm_rope(q_out.t, q, k, table, dev(positions), None if wq is None else dev(wq),
                         None if wk is None else dev(wk), 1e-6, il, k_out.t, v, kc.t, vc.t, dev(rows), row_pos)
    assert gqa.gqa_get_last_error() == (0, 0)
    assert all(g.intact() for g in (q_out, k_out, kc, vc))
    tab = None if table is None else host(table)
    for x, w, got, what in ((nq, wq, host(q_out.t), "q"), (nk, wk, host(k_out.t), "k")):
        y = cache_ops.norm_heads(x, w, 1e-6)
        check(got, y, cache_ops.rotate(y, tab, positions, il), tab, il, f"{case} {what}")
    # the cache: finished keys and v at the rows, every other row as it was
    want_k, want_v = before
    want_pos = np.full((B, K, S_max), -7, np.int32)
    for b in range(B):
        for i in range(T):
            want_k[b, :, rows[b] + i], want_v[b, :, rows[b] + i] = host(k_out.t)[b, i], nv[b, i]
            want_pos[b, :, rows[b] + i] = positions[b, i]
    assert np.array_equal(host(kc.t).view(np.uint8), want_k.view(np.uint8))
    assert np.array_equal(host(vc.t).view(np.uint8), want_v.view(np.uint8))
    assert np.array_equal(host(row_pos), want_pos)


@pytest.mark.parametrize("bs", [16, 48])
def test_paged_equals_contiguous(gqa, bs):
    B, T, H, K, d = 3, 40, 8, 2, 128
    (q, k, v), _ = inputs(B, T, H, K, d, synth.BF16, 0x3104)
    mb = -(-70 // bs)
    order = np.argsort(synth.normal((B * mb + 2,), synth.F64, 0x3105, 1))
    blocks = order[:B * mb].astype(np.int32).reshape(B, mb)
    rows, positions = np.array([0, 13, mb * bs - T], np.int32), np.arange(B * T, dtype=np.int32).reshape(B, T)
    table = torch.empty(1000, d, device="cuda")
    gqa.gqa_rope_table(table, 10000.0)
    w = dev(synth.normal((d,), synth.BF16, 0x3106, 1))
    out = [torch.empty(B, T, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kp, vp = (torch.zeros(B * mb + 2, K, bs, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kc, vc = (torch.zeros(B, K, mb * bs, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rp = [torch.zeros(B, K, mb * bs, dtype=torch.int32, device="cuda") for _ in range(2)]
    gqa.gqa_qk_norm_rope_paged(out[0], q, k, v, table, dev(positions), kp, vp, dev(blocks), dev(rows), w, w,
                               row_pos=rp[0])
    gqa.gqa_qk_norm_rope(out[1], q, k, table, dev(positions), w, w, v=v, k_cache=kc, v_cache=vc, rows=dev(rows),
                         row_pos=rp[1])
    assert gqa.gqa_get_last_error() == (0, 0)
    assert torch.equal(out[0], out[1]) and torch.equal(rp[0], rp[1])
    for pool, cache in ((kp, kc), (vp, vc)):
        gathered = pool[dev(blocks).long()].transpose(1, 2).reshape(B, K, mb * bs, d)
        assert torch.equal(gathered, cache)
        unused = torch.ones(B * mb + 2, dtype=torch.bool, device="cuda")
        unused[dev(blocks).long().flatten()] = False
        assert not pool[unused].any()


def test_in_place(gqa):
    B, T, H, K, d = 2, 33, 8, 2, 128
    q, k = (dev(synth.normal((B, T, n, d), synth.BF16, 0x3107, s)) for n, s in ((H, 1), (K, 2)))
    table = torch.empty(64, d, device="cuda")
    gqa.gqa_rope_table(table, 10000.0)
    pos = torch.arange(T, dtype=torch.int32, device="cuda").repeat(B, 1)
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    q1, k1 = torch.empty_like(q), torch.empty_like(k)
    gqa.gqa_qk_norm_rope(q1, q, k, table, pos, w, w, k_out=k1)
    gqa.gqa_qk_norm_rope(q, q, k, table, pos, w, w, k_out=k)
    assert torch.equal(q, q1) and torch.equal(k, k1)


def test_out_of_range_rows_positions_and_blocks(gqa):
    B, T, H, K, d, S = 4, 2, 4, 2, 128, 32
    (q, k, v), (nq, nk, _) = inputs(B, T, H, K, d, synth.BF16, 0x3108)
    table = torch.empty(16, d, device="cuda")
    gqa.gqa_rope_table(table, 10000.0)
    pos = torch.tensor([[0, 1], [-5, 15], [16, 2 ** 31 - 1], [3, 4]], dtype=torch.int32, device="cuda")
    out = torch.empty(B, T, H, d, dtype=torch.bfloat16, device="cuda")
    kc, vc = (torch.zeros(B, K, S, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rp = torch.full((B, K, S), -3, dtype=torch.int32, device="cuda")
    rows = torch.tensor([30, 31, -1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    gqa.gqa_qk_norm_rope(out, q, k, table, pos, v=v, k_cache=kc, v_cache=vc, rows=rows, row_pos=rp)
    assert gqa.gqa_get_last_error() == (gqa.GQA_ERR_DEVICE, gqa.GQA_DEVERR_ROPE_POS | gqa.GQA_DEVERR_APPEND_POS)
    y = oracle.widen(nq)
    check(host(out), y, cache_ops.rotate(y, host(table), np.clip(host(pos), 0, 15), False), host(table), False, "q")
    assert not kc[1:].any() and not vc[1:].any() and (rp[1:] == -3).all() and not kc[0, :, :30].any()
    assert torch.equal(vc[0, :, 30:], v[0].transpose(0, 1))
    # a table entry outside the pool drops its rows alone
    kp, vp = (torch.zeros(3, K, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    blocks = torch.tensor([[0, 3], [-1, 1], [2, 9], [9, 9]], dtype=torch.int32, device="cuda")
    rows = torch.tensor([15, 16, 3, 40], dtype=torch.int32, device="cuda")
    pos.zero_()
    gqa.gqa_qk_norm_rope_paged(out, q, k, v, table, pos, kp, vp, blocks, rows)
    assert gqa.gqa_get_last_error() == (gqa.GQA_ERR_DEVICE, gqa.GQA_DEVERR_BLOCK | gqa.GQA_DEVERR_APPEND_POS)
    want = torch.zeros_like(vp)
    want[0, :, 15], want[1, :, 0], want[1, :, 1], want[2, :, 3], want[2, :, 4] = v[0, 0], v[1, 0], v[1, 1], v[2, 0], v[2, 1]
    assert torch.equal(vp, want)


def test_values_that_overflow_stay_where_they_are(gqa):
    # zeros, an infinity in dims that are not rotated, a NaN row: the other rows and dims are theirs alone
    B, T, H, K, d = 1, 1, 4, 1, 128
    q = dev(synth.normal((B, T, H, d), synth.BF16, 0x3109, 1))
    q[0, 0, 0] = 0
    q[0, 0, 1, 100] = float("inf")
    q[0, 0, 2, 5] = float("nan")
    k = dev(synth.normal((B, T, K, d), synth.BF16, 0x3109, 2))
    table = torch.empty(64, 64, device="cuda")
    gqa.gqa_rope_table(table, 10000.0)
    pos = torch.full((1, 1), 9, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    gqa.gqa_qk_norm_rope(out, q, k, table, pos)
    assert not out[0, 0, 0].any() and out[0, 0, 1, 100] == float("inf")
    assert torch.isfinite(out[0, 0, 1]).sum() == d - 1 and torch.isnan(out[0, 0, 2]).sum() == 2
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    gqa.gqa_qk_norm_rope(out, q, k, table, pos, w, w)
    assert not out[0, 0, 0].any() and torch.isnan(out[0, 0, 2]).all() and torch.isfinite(out[0, 0, 3]).all()


def test_table_of_far_positions(gqa):
    # cosines and sines of 64-bit angles, rounded once: half a step of float32, 2^-25 below 1, and the 64-bit angle's own error
    table = torch.empty(140000, 32, device="cuda")
    gqa.gqa_rope_table(table, 10000.0)
    want = cache_ops.rope_table(140000, 32, 10000.0)
    assert np.max(np.abs(host(table).astype(np.float64) - want)) <= 2.0 ** -25 + 1e-10


def test_tokens_at_any_one_stride(gqa):
    x = dev(synth.normal((2, 6, 3, 8, 64), synth.BF16, 0x310A, 1))
    q, k = x[:, :, 0], x[:, :, 2, :4]
    out, k_out = torch.empty(2, 6, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 6, 4, 64, dtype=torch.bfloat16, device="cuda")
    gqa.gqa_qk_norm_rope(out, q, k, None, None, k_out=k_out)
    assert torch.equal(out, q) and torch.equal(k_out, k)
    with pytest.raises(ValueError):
        gqa.gqa_qk_norm_rope(out[:, :3], q[:, :3], k[:, :3], None, None)  # the batch is at another stride
    with pytest.raises(ValueError):
        gqa.gqa_qk_norm_rope(out, q.transpose(2, 3).contiguous().transpose(2, 3), k, None, None)  # heads not contiguous
