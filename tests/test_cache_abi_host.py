"""The C ABI of include/gqa_cache.h on the host: every symbol is exported and
bound, and bad arguments are refused before anything touches the GPU."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gqa_cache.h")
P = 0x10000  # a fake, 16-byte-aligned device address: never dereferenced by these calls
OK, ARG, SHAPE, ALIGN, UNSUPPORTED = 0, -1, -2, -3, -6
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    from kv_cache_02_b200 import build

    build.build()
    from kv_cache_02_b200 import gqa

    return gqa.library()


def test_every_declared_symbol_is_exported_and_bound(lib):
    from kv_cache_02_b200 import gqa

    names = set(re.findall(r"GQA_API\s+[\w\s\*]+?\b(gqa_\w+)\s*\(", open(HEADER).read()))
    assert len(names) == 16
    for n in names:
        assert hasattr(lib, n) and callable(getattr(gqa, n)) and n in gqa.EXPORTED, n


def test_rope_table(lib):
    f = lib.gqa_rope_table  # rope, max_pos, rotary_dim, theta, stream
    assert f(P, 16, 7, 1e4, None) == SHAPE and f(P, 16, 0, 1e4, None) == SHAPE
    assert f(P, 16, 8, 0.0, None) == ARG and f(P, -1, 8, 1e4, None) == ARG and f(None, 16, 8, 1e4, None) == ARG
    assert f(P + 4, 16, 8, 1e4, None) == ALIGN and f(None, 0, 8, 1e4, None) == OK
    assert f(P, 16, 8, float("nan"), None) == ARG


def norm_rope(lib, q_out=P, k_out=None, kc=None, vc=None, row_pos=None, q=P, k=P, v=None, wq=P, wk=P, rope=P, pos=P,
              rows=None, B=2, T=3, H=8, K=2, S=16, d=128, qs=1024, ks=256, vs=256, rd=128, mp=64, il=0, eps=1e-6,
              dt=BF16):
    return lib.gqa_qk_norm_rope(q_out, k_out, kc, vc, row_pos, q, k, v, wq, wk, rope, pos, rows, B, T, H, K, S, d, qs,
                                ks, vs, rd, mp, il, eps, dt, None)


@pytest.mark.parametrize("status,bad", [
    (ARG, dict(dt=5)), (ARG, dict(B=-1)), (ARG, dict(T=-1)), (ARG, dict(H=0)), (ARG, dict(eps=-1.0)),
    (ARG, dict(eps=float("nan"))), (SHAPE, dict(d=96)), (SHAPE, dict(H=7)), (SHAPE, dict(rd=136)),
    (SHAPE, dict(rd=24)), (ARG, dict(rd=-16)), (ARG, dict(kc=P, rows=P, v=P)), (ARG, dict(kc=P, vc=P, rows=P)),
    (ARG, dict(kc=P, vc=P, v=P)), (SHAPE, dict(kc=P, vc=P, v=P, rows=P, T=17)), (ARG, dict(row_pos=P)),
    (SHAPE, dict(qs=1016)), (SHAPE, dict(qs=1028)), (SHAPE, dict(ks=255)), (SHAPE, dict(kc=P, vc=P, v=P, rows=P, vs=8)),
    (ARG, dict(mp=0)), (ARG, dict(q_out=None)), (ARG, dict(rope=None)), (ARG, dict(pos=None)),
    (ALIGN, dict(q=P + 2)), (ALIGN, dict(wq=P + 8)), (ALIGN, dict(rope=P + 4)), (OK, dict(B=0, q=None)),
    (OK, dict(T=0, q=None)), (ARG, dict(kc=P, vc=P, v=P, rows=P, S=0))], ids=str)
def test_norm_rope(lib, status, bad):
    assert norm_rope(lib, **bad) == status


def test_norm_rope_paged(lib):
    def f(table=P, kp=P, v=P, nb=8, bs=16, mb=2, T=3, B=2):
        return lib.gqa_qk_norm_rope_paged(P, None, kp, P, None, P, P, v, P, P, P, P, table, P, B, T, 8, 2, 128, nb, bs,
                                          mb, 1024, 256, 256, 128, 64, 0, 1e-6, BF16, None)
    assert f(bs=24) == SHAPE and f(nb=0) == SHAPE and f(mb=0) == SHAPE and f(T=33) == SHAPE
    assert f(table=None) == ARG and f(kp=None) == ARG and f(v=None) == ARG and f(B=0, table=None) == OK


def test_decode_scores(lib):
    ws = lib.gqa_decode_scores_workspace_bytes
    n = ws(2, 8, 2, 64, 128, 0)
    # the partials' (m, l) of one split, the queue and a float per query head and row
    assert n == 16 * 8 + 16 + 2 * 8 * 64 * 4
    assert ws(2, 6, 4, 64, 128, 0) == 0 and ws(2, 8, 2, 64, 96, 0) == 0 and ws(2, 8, 2, 64, 128, -1) == 0

    def f(out=P, scores=P, q=P, B=2, H=8, K=2, S=64, d=128, splits=0, w=P, wb=n, dt=BF16):
        return lib.gqa_decode_scores(out, scores, q, P, P, P, B, H, K, S, d, 1.0, splits, w, wb, dt, None)
    assert f(H=6, K=4) == SHAPE and f(d=96) == SHAPE and f(S=0) == ARG and f(splits=-1) == ARG and f(dt=9) == ARG
    assert f(dt=F32) == UNSUPPORTED and f(scores=None) == ARG and f(w=None) == ARG and f(wb=n - 1) == ARG
    assert f(q=P + 2) == ALIGN and f(scores=P + 4) == ALIGN and f(w=P + 8) == ALIGN and f(B=0, out=None) == OK
    assert f(B=1 << 12, H=8, K=8, S=1 << 16) == SHAPE

    pws = lib.gqa_decode_scores_paged_workspace_bytes
    assert pws(2, 8, 2, 128, 24, 4, 0) == 0 and pws(2, 8, 2, 128, 16, 4, 0) == n

    def g(table=P, nb=16, bs=16, mb=4, dt=BF16):
        return lib.gqa_decode_scores_paged(P, P, P, P, P, table, P, 2, 8, 2, 128, nb, bs, mb, 1.0, 0, P, n, dt, None)
    assert g(bs=24) == SHAPE and g(mb=0) == SHAPE and g(nb=0) == SHAPE and g(table=None) == ARG
    assert g(dt=F32) == UNSUPPORTED


def test_prompt_scores(lib):
    ws = lib.gqa_prompt_scores_workspace_bytes
    n = ws(2, 40, 8, 2, 64, 128)
    assert n >= 2 * 2 * 2 * 128 * 4  # a log-sum-exp per row of two 32-token tiles
    assert ws(2, 40, 6, 4, 64, 128) == 0 and ws(2, 40, 256, 1, 64, 128) == 0 and ws(2, -1, 8, 2, 64, 128) == 0

    def f(scores=P, q=P, B=2, T=40, H=8, K=2, S=64, d=128, w=P, wb=n, dt=BF16):
        return lib.gqa_prompt_scores(scores, q, P, P, B, T, H, K, S, d, 1.0, w, wb, dt, None)
    assert f(H=6, K=4) == SHAPE and f(d=32) == SHAPE and f(H=258, K=2) == SHAPE and f(T=-1) == ARG and f(S=0) == ARG
    assert f(dt=F32) == UNSUPPORTED and f(dt=4) == ARG and f(q=None) == ARG and f(w=None) == ARG and f(wb=n - 4) == ARG
    assert f(q=P + 8) == ALIGN and f(w=P + 4) == ALIGN and f(B=0, q=None) == OK and f(T=0, q=None) == OK
    assert f(B=1 << 12, H=8, K=8, S=1 << 16) == SHAPE


def test_evict(lib):
    ws = lib.gqa_kv_evict_workspace_bytes
    n = ws(2, 3, 64, 16)
    assert n >= 2 * 8
    # lists of the moves, at most keep and at most what lies past it
    assert ws(2, 3, 20000, 9000) >= 2 * 3 * 2 * 9000 * 4 > ws(2, 3, 20000, 19000) >= 2 * 3 * 2 * 1000 * 4
    assert ws(2, 3, 64, 0) == 0 and ws(2, 3, 64, 65) == 0

    def f(kc=P, scores=P, B=2, K=3, S=64, d=128, keep=16, sinks=0, w=P, wb=n, dt=BF16):
        return lib.gqa_kv_evict(kc, P, scores, None, P, None, B, K, S, d, keep, sinks, w, wb, dt, None)
    assert f(keep=0) == SHAPE and f(keep=65) == SHAPE and f(d=96) == SHAPE and f(sinks=-1) == ARG and f(dt=2) == ARG
    assert f(kc=None) == ARG and f(scores=None) == ARG and f(w=None) == ARG and f(wb=n - 1) == ARG and f(S=0) == ARG
    assert f(kc=P + 8) == ALIGN and f(scores=P + 4) == ALIGN and f(w=P + 4) == ALIGN and f(B=0, kc=None) == OK

    def g(table=P, nb=16, bs=16, mb=4):
        return lib.gqa_kv_evict_paged(P, P, table, P, None, P, None, 2, 3, 128, nb, bs, mb, 16, 0, P, n, BF16, None)
    assert g(bs=8) == SHAPE and g(nb=0) == SHAPE and g(mb=0) == SHAPE and g(table=None) == ARG


def test_mxfp4(lib):
    for f in (lib.gqa_kv_append_mxfp4, lib.gqa_kv_read_mxfp4):
        def call(a=P, b=P, B=2, T=3, K=2, S=64, d=128):
            return f(a, b, P, P, P, P, P, B, T, K, S, d, None)
        assert call(d=64) == UNSUPPORTED and call(S=66) == SHAPE and call(T=65) == SHAPE and call(K=0) == ARG
        assert call(T=-1) == ARG and call(a=None) == ARG and call(b=P + 4) == ALIGN
        assert call(B=0, a=None) == OK and call(T=0, a=None) == OK
    ws = lib.gqa_decode_mxfp4_workspace_bytes
    n = ws(2, 8, 2, 64, 128, 0)
    assert n == 16 and ws(2, 8, 2, 64, 64, 0) == 0 and ws(2, 8, 2, 66, 128, 0) == 0 and ws(2, 7, 2, 64, 128, 0) == 0

    def f(out=P, ks=P, H=8, K=2, S=64, d=128, splits=0, w=P, wb=n, B=2):
        return lib.gqa_decode_mxfp4(out, P, P, ks, P, P, P, B, H, K, S, d, 1.0, splits, w, wb, None)
    assert f(d=64) == UNSUPPORTED and f(S=66) == SHAPE and f(H=7) == SHAPE and f(splits=-1) == ARG and f(K=0) == ARG
    assert f(ks=None) == ARG and f(ks=P + 4) == ALIGN and f(w=None) == ARG and f(wb=n - 1) == ARG and f(w=P + 8) == ALIGN
    assert f(B=0, out=None) == OK and f(B=1 << 12, H=8, K=8, S=1 << 16) == SHAPE


def test_binding_refuses_what_the_library_cannot_see(lib):
    import torch

    from kv_cache_02_b200 import gqa

    q = torch.zeros(1, 2, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not on the GPU
        gqa.gqa_qk_norm_rope(q, q, q[:, :, :2], None, None)
    with pytest.raises(ValueError):
        gqa.gqa_rope_table(torch.zeros(4, 16), 1e4)
    c = torch.zeros(1, 2, 64, 128, dtype=torch.bfloat16)
    s, n = torch.zeros(1, 2, 64), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(AssertionError):  # scores of another dtype
        gqa.gqa_decode_scores(q[:, 0], s.double(), q[:, 0], c, c, n, 1.0)
    with pytest.raises(AssertionError):  # caches of unequal dtype
        gqa.gqa_kv_evict(c, c.float(), s, None, n, 8)
    with pytest.raises(AssertionError):  # lengths of another type
        gqa.gqa_prompt_scores(s, q, c, n.long(), 1.0)
    with pytest.raises(AssertionError):  # scales of another shape
        gqa.gqa_decode_mxfp4(q[:, 0], q[:, 0], *(torch.zeros(1, 2, 64, w, dtype=torch.uint8) for w in (64, 4, 64, 2)), n, 1.0)
