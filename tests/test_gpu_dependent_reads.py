"""Calls that read what the call right before them wrote: a chain that goes out
without a pause, and replayed as a graph, gives bit for bit what the same calls
give with a synchronisation after each."""
import pytest
import torch

import synth
from _helpers import dev

pytestmark = pytest.mark.gpu
B, H, K, D, S, KEEP, N = 8, 16, 4, 128, 320, 256, 24


@pytest.fixture(scope="module")
def gqa():
    from kv_cache_02_b200 import gqa as g

    return g


def make(i):
    """One link's buffers: a cache over its budget, its lengths, a 4-bit cache and an 8-bit row's way in."""
    x = dev(synth.normal((B, 1, H + 2 * K, D), synth.BF16, 0x3800 + i, 1))
    s = dict(x=x, kc=dev(synth.normal((B, K, S, D), synth.BF16, 0x3800 + i, 2)),
             vc=dev(synth.normal((B, K, S, D), synth.BF16, 0x3800 + i, 3)),
             scores=dev(synth.normal((B, K, S), synth.F32, 0x3800 + i, 4)).abs(),
             row_pos=torch.arange(S, dtype=torch.int32, device="cuda").repeat(B, K, 1),
             lens=torch.tensor([S - 1 - (i + b) % 60 for b in range(B)], dtype=torch.int32, device="cuda"),
             positions=torch.full((B, 1), S, dtype=torch.int32, device="cuda"))
    for name in ("q", "out", "out4", "out1"):
        s[name] = torch.zeros(B, 1, H, D, dtype=torch.bfloat16, device="cuda")
    for name in ("k", "back_k", "back_v"):
        s[name] = torch.zeros(B, 1, K, D, dtype=torch.bfloat16, device="cuda")
    s["v"] = x[:, :, H + K:].contiguous()
    s["c4"] = [torch.zeros(B, K, S, n, dtype=torch.uint8, device="cuda") for n in (D // 2, D // 32, D // 2, D // 32)]
    return s


def calls(gqa, s, table, ws):
    """The link's calls, each reading what the one before wrote: lengths, rows, queries, codes."""
    x = s["x"]
    yield lambda: gqa.gqa_kv_evict(s["kc"], s["vc"], s["scores"], s["row_pos"], s["lens"], KEEP, 2, None, ws)
    yield lambda: gqa.gqa_qk_norm_rope(s["q"], x[:, :, :H], x[:, :, H:H + K], table, s["positions"], k_out=s["k"],
                                       v=s["v"], k_cache=s["kc"], v_cache=s["vc"], rows=s["lens"], row_pos=s["row_pos"])
    yield lambda: gqa.gqa_decode_scores(s["out"][:, 0], s["scores"], s["q"][:, 0], s["kc"], s["vc"], s["lens"], 0.1,
                                        workspace=ws)
    yield lambda: gqa.gqa_kv_append_mxfp4(*s["c4"], s["k"], s["v"], s["lens"])
    yield lambda: gqa.gqa_kv_read_mxfp4(s["back_k"], s["back_v"], *s["c4"], s["lens"])
    yield lambda: gqa.gqa_decode_mxfp4(s["out4"][:, 0], s["q"][:, 0], *s["c4"], s["lens"], 0.1, workspace=ws)
    # the token once more, at the row after the cut
    yield lambda: gqa.gqa_decode_append(s["out1"][:, 0], s["q"][:, 0], s["kc"], s["vc"], s["k"][:, 0], s["v"][:, 0],
                                        s["lens"], 0.1, workspace=ws)


def tensors(s):
    return [t for v in s.values() for t in (v if isinstance(v, list) else [v])]


def test_a_chain_without_a_pause(gqa):
    table = torch.empty(S + 8, D, device="cuda")
    gqa.gqa_rope_table(table)
    ws = torch.empty(max(gqa.gqa_kv_evict_workspace_bytes(B, K, S, KEEP), gqa.gqa_decode_workspace_bytes(B, H, K, S, D),
                         gqa.gqa_decode_scores_workspace_bytes(B, H, K, S, D),
                         gqa.gqa_decode_mxfp4_workspace_bytes(B, H, K, S, D)), dtype=torch.uint8, device="cuda")
    slow, fast, kept = ([make(i) for i in range(N)] for _ in range(3))
    for s in slow:
        for call in calls(gqa, s, table, ws):
            call()
            torch.cuda.synchronize()
        assert s["lens"].tolist() == [KEEP] * B
    ready = [c for s in fast for c in calls(gqa, s, table, ws)]
    torch.cuda.synchronize()
    for call in ready:
        call()
    torch.cuda.synchronize()
    assert gqa.gqa_get_last_error() == (0, 0)
    for a, b in zip(slow, fast):
        assert all(torch.equal(x, y) for x, y in zip(tensors(a), tensors(b)))
    # the same as one graph, replayed on the buffers as they were
    graph = torch.cuda.CUDAGraph()
    replayed = [make(i) for i in range(N)]
    with torch.cuda.graph(graph):
        for s in replayed:
            for call in calls(gqa, s, table, ws):
                call()
    for _ in range(3):
        for s, fresh in zip(replayed, kept):
            for x, y in zip(tensors(s), tensors(fresh)):
                x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(slow, replayed):
            assert all(torch.equal(x, y) for x, y in zip(tensors(a), tensors(b)))
    assert gqa.gqa_get_last_error() == (0, 0)
