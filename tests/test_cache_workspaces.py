"""Workspace sizes of include/gqa_cache.h on the host: a buffer made for the
largest batch serves every smaller one, and the calls take it."""
import pytest

P = 0x10000  # a fake, 16-byte-aligned device address: never dereferenced by these calls
ARG, BF16 = -1, 1


@pytest.fixture(scope="module")
def lib():
    from kv_cache_02_b200 import build

    build.build()
    from kv_cache_02_b200 import gqa

    return gqa.library()


QUERIES = {
    "evict 16384 -> 16000": lambda lib, B: lib.gqa_kv_evict_workspace_bytes(B, 8, 16384, 16000),
    "evict 12000 -> 3000": lambda lib, B: lib.gqa_kv_evict_workspace_bytes(B, 2, 12000, 3000),
    "evict 9000 -> 8999": lambda lib, B: lib.gqa_kv_evict_workspace_bytes(B, 1, 9000, 8999),
    "prompt 512 of 8192": lambda lib, B: lib.gqa_prompt_scores_workspace_bytes(B, 512, 64, 8, 8192, 128),
    "prompt 32 of 32768": lambda lib, B: lib.gqa_prompt_scores_workspace_bytes(B, 32, 64, 8, 32768, 128),
    "prompt 700 of 700": lambda lib, B: lib.gqa_prompt_scores_workspace_bytes(B, 700, 3, 1, 700, 64),
    "4-bit decode": lambda lib, B: lib.gqa_decode_mxfp4_workspace_bytes(B, 64, 8, 16384, 128, 0),
    "4-bit decode, short": lambda lib, B: lib.gqa_decode_mxfp4_workspace_bytes(B, 8, 1, 640, 128, 0),
    "scores": lambda lib, B: lib.gqa_decode_scores_workspace_bytes(B, 32, 8, 640, 128, 0),
    "scores, one head": lambda lib, B: lib.gqa_decode_scores_workspace_bytes(B, 1, 1, 513, 64, 0),
    "scores, paged": lambda lib, B: lib.gqa_decode_scores_paged_workspace_bytes(B, 32, 8, 128, 16, 60, 0),
}


@pytest.mark.parametrize("query", QUERIES)
def test_sizes_do_not_fall_as_the_batch_grows(lib, query):
    sizes = [QUERIES[query](lib, B) for B in [*range(1, 400), 600, 900, 1300, 1777, 2000, 2400, 3000]]
    assert all(s > 0 for s in sizes)
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_the_batch_that_shrank_takes_the_buffer(lib):
    # a wrong alignment is looked for after the size: what is refused as misaligned was large enough
    n = lib.gqa_kv_evict_workspace_bytes(3, 8, 16384, 16000)
    for B in (1, 2, 3):
        status = lib.gqa_kv_evict(P, P, P, None, P, None, B, 8, 16384, 128, 16000, 0, P + 4, n, BF16, None)
        assert status == -3, B
    n = lib.gqa_prompt_scores_workspace_bytes(8, 512, 64, 8, 8192, 128)
    for B in range(1, 9):
        assert lib.gqa_prompt_scores(P, P, P, P, B, 512, 64, 8, 8192, 128, 1.0, P + 4, n, BF16, None) == -3, B
    n = lib.gqa_decode_mxfp4_workspace_bytes(200, 64, 8, 16384, 128, 0)
    for B in (1, 7, 15, 16, 17, 100, 200):
        assert lib.gqa_decode_mxfp4(P, P, P, P, P, P, P, B, 64, 8, 16384, 128, 1.0, 0, P + 4, n, None) == -3, B
    # and one byte less than a batch of its own takes is still refused
    need = min(lib.gqa_decode_mxfp4_workspace_bytes(1, 64, 8, 16384, 128, 0), n)
    assert lib.gqa_decode_mxfp4(P, P, P, P, P, P, P, 1, 64, 8, 16384, 128, 1.0, 0, P, need - 1, None) == ARG
