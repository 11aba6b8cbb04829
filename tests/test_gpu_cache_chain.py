"""The cache operators one after another, as a serving loop calls them, with no
synchronisation in between; captured and replayed; on other streams."""
import numpy as np
import pytest
import torch

import oracle
import synth
from _helpers import assert_close, dev, host
from oracle import cache_ops
from test_gpu_norm_rope import check as check_rope
from test_gpu_scores import assert_out, assert_scores, largest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gqa():
    from kv_cache_02_b200 import gqa as g

    return g


def empty(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def test_prompt_cut_and_steps(gqa):
    """A prompt: norm and rotation into the cache, prefill, its weights, a cut; then steps over the cut cache."""
    B, T, H, K, d, S, keep, steps = 2, 150, 16, 4, 128, 160, 64, 4
    table = empty(1000, d, dtype=torch.float32)
    gqa.gqa_rope_table(table, 10000.0)
    w = dev(synth.normal((d,), synth.BF16, 0x3501, 9))
    scale = d ** -0.5
    kc, vc = torch.zeros(B, K, S, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, K, S, d, dtype=torch.bfloat16, device="cuda")
    scores, row_pos = torch.zeros(B, K, S, device="cuda"), torch.full((B, K, S), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = empty(max(gqa.gqa_prompt_scores_workspace_bytes(B, T, H, K, S, d), gqa.gqa_kv_evict_workspace_bytes(B, K, S, keep),
                   gqa.gqa_decode_scores_workspace_bytes(B, H, K, S, d)), dtype=torch.uint8)
    log = []  # device copies, read when all is done

    def step(t, first, cut):
        x = dev(synth.normal((B, t, H + 2 * K, d), synth.BF16, 0x3502 + first, 1))
        q, k, v = x[:, :, :H], x[:, :, H:H + K], x[:, :, H + K:]
        pos = (first + torch.arange(t, dtype=torch.int32, device="cuda")).repeat(B, 1)
        q_out, k_out, out = empty(B, t, H, d), empty(B, t, K, d), empty(B, t, H, d)
        gqa.gqa_qk_norm_rope(q_out, q, k, table, pos, w, w, k_out=k_out, v=v, k_cache=kc, v_cache=vc, rows=lens,
                             row_pos=row_pos)
        lens.add_(t)
        before = scores.clone()
        if t > 1:
            gqa.gqa_prefill_causal(out, q_out, k_out, v.contiguous(), scale)
            gqa.gqa_prompt_scores(scores, q_out, kc, lens, scale, workspace=ws)
        else:
            gqa.gqa_decode_scores(out[:, 0], scores, q_out[:, 0], kc, vc, lens, scale, workspace=ws)
        full = [a.clone() for a in (kc, vc, scores, row_pos, lens)]
        if cut:
            gqa.gqa_kv_evict(kc, vc, scores, row_pos, lens, keep, 2, pos[:, -1] - 7, workspace=ws)
        log.append((x, pos, q_out, k_out, out, before, full, [a.clone() for a in (kc, vc, scores, row_pos, lens)], cut))

    step(T, 0, True)
    for i in range(steps):
        step(1, T + i, i % 2 == 1)
    assert gqa.gqa_get_last_error() == (0, 0)
    for x, pos, q_out, k_out, out, before, full, after, cut in log:
        t = x.shape[1]
        for part, got in ((x[:, :, :H], q_out), (x[:, :, H:H + K], k_out)):
            y = cache_ops.norm_heads(host(part), host(w), 1e-6)
            check_rope(host(got), y, cache_ops.rotate(y, host(table), host(pos), False), host(table), False, f"{t} rows")
        fk, fv, fs, fp, fl = (host(a) for a in full)
        rel = 2 * d * 2.0 ** -23 * largest(host(q_out), fk, scale) + 2.0 ** -20
        if t > 1:
            assert_close(host(out), oracle.prefill_causal(host(q_out), host(k_out), host(x[:, :, H + K:]), scale), "prefill")
            added = cache_ops.prompt_scores(host(q_out), fk, fl, scale)
        else:
            want, added, spread = cache_ops.decode_scores(host(q_out[:, 0]), fk, fv, fl, scale)
            assert_out(host(out[:, 0]), want, spread, rel, "decode")
        assert_scores(fs, host(before), added, fl, rel, t * H // K + S, f"{t} rows")
        if cut:
            want = cache_ops.evict(fk, fv, fs, fp, fl, keep, 2, host(pos)[:, -1] - 7)
            for g, e in zip(after, want):
                assert np.array_equal(host(g).view(np.uint8), e.view(np.uint8))
    # every row still holds the key of the position that its row_pos says
    keys = np.concatenate([host(entry[3]) for entry in log], axis=1)
    final_k, final_p, final_n = host(kc), host(row_pos), host(lens)
    for b in range(B):
        for g in range(K):
            n = final_n[b]
            assert len(set(final_p[b, g, :n])) == n
            assert np.array_equal(final_k[b, g, :n], keys[b, final_p[b, g, :n], g])


def test_four_bit_steps(gqa):
    """A prompt into the 4-bit cache, read back, then append and decode, one step right after the other."""
    B, T, H, K, d, S, steps = 2, 70, 16, 2, 128, 80, 5
    cache = [torch.zeros(B, K, S, n, dtype=torch.uint8, device="cuda") for n in (d // 2, d // 32, d // 2, d // 32)]
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    new = [dev(synth.normal((B, T + steps, K, d), synth.BF16, 0x3503, s)) for s in (1, 2)]
    q = dev(synth.normal((B, steps, H, d), synth.BF16, 0x3503, 3))
    gqa.gqa_kv_append_mxfp4(*cache, *(x[:, :T].contiguous() for x in new), pos)
    back = [empty(B, T, K, d) for _ in range(2)]
    gqa.gqa_kv_read_mxfp4(*back, *cache, pos)
    pos.add_(T)
    ws = empty(gqa.gqa_decode_mxfp4_workspace_bytes(B, H, K, S, d), dtype=torch.uint8)
    outs = [empty(B, H, d) for _ in range(steps)]
    for i in range(steps):
        gqa.gqa_kv_append_mxfp4(*cache, *(x[:, T + i:T + i + 1].contiguous() for x in new), pos)
        pos.add_(1)
        gqa.gqa_decode_mxfp4(outs[i], q[:, i].contiguous(), *cache, pos, d ** -0.5, workspace=ws)
    assert gqa.gqa_get_last_error() == (0, 0)
    values = [cache_ops.mxfp4_values(*cache_ops.mxfp4_quantize(host(x))) for x in new]
    for g, e in zip(back, values):
        assert np.array_equal(oracle.widen(host(g)), e[:, :T])
    k, v = (x.swapaxes(1, 2) for x in values)
    for i in range(steps):
        n = T + i + 1
        want, _, spread = cache_ops.decode_scores(host(q[:, i]), k, v, [n] * B, d ** -0.5)
        rel = 2 * d * 2.0 ** -23 * largest(host(q), k.astype(np.float32), d ** -0.5) + 2.0 ** -20
        assert_out(host(outs[i]), want, spread, rel, f"step {i}")


def serving(gqa, B=2, H=16, K=4, d=128, S=512):
    """Inputs and one step of everything, on whatever stream is current."""
    s = dict(x=dev(synth.normal((B, 1, H + 2 * K, d), synth.BF16, 0x3504, 1)), table=empty(1024, d, dtype=torch.float32),
             kc=dev(synth.normal((B, K, S, d), synth.BF16, 0x3504, 2)), vc=dev(synth.normal((B, K, S, d), synth.BF16, 0x3504, 3)),
             scores=dev(np.abs(synth.normal((B, K, S), synth.F32, 0x3504, 4)).astype(np.float32)), lens=torch.tensor([300, 222], dtype=torch.int32, device="cuda"),
             q=empty(B, 1, H, d), out=empty(B, H, d), out4=empty(B, H, d), k=empty(B, 1, K, d),
             row_pos=torch.arange(S, dtype=torch.int32, device="cuda").repeat(B, K, 1),
             pos=torch.tensor([[300], [222]], dtype=torch.int32, device="cuda"),
             cache=[torch.zeros(B, K, S, n, dtype=torch.uint8, device="cuda") for n in (d // 2, d // 32, d // 2, d // 32)])
    gqa.gqa_rope_table(s["table"])
    sizes = (gqa.gqa_decode_scores_workspace_bytes(B, H, K, S, d), gqa.gqa_kv_evict_workspace_bytes(B, K, S, 200),
             gqa.gqa_prompt_scores_workspace_bytes(B, 1, H, K, S, d), gqa.gqa_decode_mxfp4_workspace_bytes(B, H, K, S, d))
    s["ws"] = empty(max(sizes), dtype=torch.uint8)
    for _ in range(2):
        gqa.gqa_kv_append_mxfp4(*s["cache"], s["kc"].transpose(1, 2).contiguous(), s["vc"].transpose(1, 2).contiguous(),
                                torch.zeros(B, dtype=torch.int32, device="cuda"))
    s["state"] = [s["scores"], s["lens"], s["row_pos"], s["kc"], s["vc"], *s["cache"]]

    def step(ws=s["ws"]):
        x = s["x"]
        gqa.gqa_qk_norm_rope(s["q"], x[:, :, :H], x[:, :, H:H + K], s["table"], s["pos"], k_out=s["k"], v=x[:, :, H + K:],
                             k_cache=s["kc"], v_cache=s["vc"], rows=s["lens"], row_pos=s["row_pos"])
        gqa.gqa_kv_append_mxfp4(*s["cache"], s["k"], x[:, :, H + K:].contiguous(), s["lens"])
        s["lens"].add_(1)
        gqa.gqa_decode_scores(s["out"], s["scores"], s["q"][:, 0], s["kc"], s["vc"], s["lens"], d ** -0.5, workspace=ws)
        gqa.gqa_prompt_scores(s["scores"], s["q"], s["kc"], s["lens"], d ** -0.5, workspace=ws)
        gqa.gqa_decode_mxfp4(s["out4"], s["q"][:, 0], *s["cache"], s["lens"], d ** -0.5, workspace=ws)
        gqa.gqa_kv_evict(s["kc"], s["vc"], s["scores"], s["row_pos"], s["lens"], 200, 4, None, ws)
        s["pos"].add_(1)

    def results():
        return [t.clone() for t in (s["out"], s["out4"], s["q"], s["pos"], *s["state"])]
    return s, step, results


def test_captured_and_replayed(gqa):
    s, step, results = serving(gqa)
    for _ in range(3):
        step()
    want = results()
    s, step, results = serving(gqa)
    first = [t.clone() for t in (*s["state"], s["pos"])]
    graphs = []
    for _ in range(2):  # two graphs that share a workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for t, f in zip((*s["state"], s["pos"]), first):
        t.copy_(f)
    s["ws"].fill_(0xEE)
    graphs[0].replay()
    graphs[1].replay()
    graphs[0].replay()
    got = results()
    assert gqa.gqa_get_last_error() == (0, 0)
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), i


def test_two_streams(gqa):
    s, step, results = serving(gqa)
    step()
    want = results()
    runs = [serving(gqa) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for st, (_, f, _) in zip(streams, runs):  # two calls of each operator at once, each with its own workspace
        with torch.cuda.stream(st):
            f()
    torch.cuda.synchronize()
    assert gqa.gqa_get_last_error() == (0, 0)
    for _, _, r in runs:
        for a, b in zip(r(), want):
            assert torch.equal(a, b)


def test_the_stream_that_is_given(gqa):
    # the call waits for what its own stream holds, whichever stream is current
    st = torch.cuda.Stream()
    q = dev(synth.normal((64, 8, 8, 128), synth.BF16, 0x3505, 1))
    k = q[:, :, :2].contiguous()
    x = torch.zeros_like(q)
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
        x.copy_(q)
    gqa.gqa_qk_norm_rope(out, x, k, None, None, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(out, q)
