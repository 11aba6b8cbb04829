"""The cache operators' cases: inputs, plain forms, exact values and floors.

Six operators that keep a GQA key-value cache (see include/gqa_cache.h):

  rope    norm of every query and key head, position rotation, cache write     gqa_qk_norm_rope[_paged]
  scores  one new token's attention, its weights added up per cached row       gqa_decode_scores[_paged]
  prompt  the weights of a prompt's (or its last queries') attention, added up  gqa_prompt_scores
  evict   the rows of lowest accumulated weight leave the cache                gqa_kv_evict[_paged]
  quant   rows into a microscaled 4-bit cache, and read back as bf16           gqa_kv_append_mxfp4, gqa_kv_read_mxfp4
  mxdec   one new token's attention over the 4-bit cache                       gqa_decode_mxfp4

Notation as in gqa.h: B sequences, H query heads, K KV heads, G = H / K, d the
head dimension, S the cache's capacity in tokens.
"""
import math
import random

import numpy as np
import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
CODE_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # e2m1 magnitudes of codes 0..7; bit 3 is the sign


# ----------------------------------------------------------------------------
# cases

def listed():
    return [
        # a serving step's new tokens: 8 sequences of a 32-query-head layer, into a paged cache (latency)
        dict(name="rope-step-paged", op="rope", B=8, T=1, H=32, K=8, d=128, S=8192, page=16, dtype="bf16", rotary=128,
             interleaved=False, norm=True, cache=True, theta=500000.0),
        # a prompt of 4 x 4096 tokens out of a fused QKV projection, for the prefill that follows (it writes the cache)
        dict(name="rope-prompt", op="rope", B=4, T=4096, H=32, K=8, d=128, S=4096, page=0, dtype="bf16", rotary=128,
             interleaved=False, norm=True, cache=False, theta=500000.0),
        # a decode step at 8192 tokens of context
        dict(name="scores-8k", op="scores", B=8, H=32, K=8, d=128, S=8192, lo=8192, hi=8192, page=0),
        # one long document: the cache's length is what the work is split over
        dict(name="scores-128k", op="scores", B=1, H=64, K=8, d=128, S=131072, lo=131072, hi=131072, page=0),
        # the weights of a whole prompt, batch 4 x 4096
        dict(name="prompt-4k", op="prompt", B=4, T=4096, H=32, K=8, d=128, S=4096, lo=4096, hi=4096),
        # the last 32 queries of two long prompts of unequal length
        dict(name="prompt-window", op="prompt", B=2, T=32, H=64, K=8, d=128, S=32768, lo=20000, hi=32768),
        # the steady state of a bounded cache: a few rows over the budget leave it
        dict(name="evict-step", op="evict", B=8, K=8, d=128, S=2304, lo=2049, hi=2112, keep=2048, sinks=4, recent=256,
             page=0, dtype="bf16"),
        # a long prompt cut down to its heavy rows
        dict(name="evict-long", op="evict", B=1, K=8, d=128, S=131072, lo=131072, hi=131072, keep=8192, sinks=4,
             recent=1024, page=0, dtype="bf16"),
        # one new token of 8 sequences (latency)
        dict(name="quant-step", op="quant", B=8, T=1, K=8, d=128, S=8192),
        # a prompt into the 4-bit cache, read back for a prefill that goes on
        dict(name="quant-prompt", op="quant", B=4, T=4096, K=8, d=128, S=4096),
        # the decode step at 8192 tokens over the 4-bit cache
        dict(name="mxdec-8k", op="mxdec", B=8, H=32, K=8, d=128, S=8192, lo=8192, hi=8192),
        # a ragged serving batch, 1K to 16K tokens
        dict(name="mxdec-ragged", op="mxdec", B=32, H=64, K=8, d=128, S=16384, lo=1024, hi=16384),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "scores", "prompt", "evict", "quant", "mxdec"))
    K = rng.choice((1, 2, 3, 4, 8))
    G = rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 12, 16))
    d = rng.choice((64, 128))
    page = rng.choice((0, 0, 16, 48, 64, 128))
    if op == "rope":
        T = _log_int(rng, 1, 2048)
        B = _log_int(rng, 1, max(1, min(64, 8192 // T)))
        S = T + _log_int(rng, 1, 4096)
        return dict(op=op, B=B, T=T, H=K * G, K=K, d=d, S=S, page=page, dtype=rng.choice(("bf16", "bf16", "f32")),
                    rotary=rng.choice((d, d, d // 2, 16, 0)), interleaved=rng.random() < 0.3, norm=rng.random() < 0.8,
                    cache=rng.random() < 0.7, theta=rng.choice((10000.0, 500000.0)))
    if op in ("scores", "mxdec"):
        S = _log_int(rng, 1, 40000)
        B = _log_int(rng, 1, max(1, min(32, 262144 // S)))
        if op == "mxdec":
            return dict(op=op, B=B, H=K * G, K=K, d=128, S=(S + 3) // 4 * 4, lo=rng.randint(0, S), hi=S)
        return dict(op=op, B=B, H=K * G, K=K, d=d, S=S, lo=rng.randint(0, S), hi=S, page=page)
    if op == "prompt":
        S = _log_int(rng, 1, 16384)
        T = _log_int(rng, 1, min(S, 4096))
        B = _log_int(rng, 1, max(1, min(8, 16777216 // (S * T))))
        return dict(op=op, B=B, T=T, H=K * G, K=K, d=d, S=S, lo=rng.randint(0, S), hi=S)
    if op == "evict":
        S = _log_int(rng, 16, 65536)
        B = _log_int(rng, 1, max(1, min(16, 131072 // S)))
        keep = _log_int(rng, 1, S)
        sinks = rng.randint(0, min(8, keep))
        return dict(op=op, B=B, K=K, d=d, S=S, lo=rng.randint(0, S), hi=S, keep=keep, sinks=sinks,
                    recent=rng.randint(0, (keep - sinks) // 2), page=page, dtype=rng.choice(("bf16", "bf16", "f32")))
    T = _log_int(rng, 1, 4096)
    B = _log_int(rng, 1, max(1, min(64, 16384 // T)))
    return dict(op=op, B=B, T=T, K=K, d=128, S=(T + _log_int(rng, 1, 2048) + 3) // 4 * 4)


def _lens(c):
    """The sequences' lengths: part of the case, so that work() knows them."""
    r = random.Random("%d %d %d" % (c["B"], c["lo"], c["hi"]))
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]


def _moved(c):
    """Rows per KV head that eviction moves, expected over equally likely orders of the scores."""
    n = 0.0
    for length in _lens(c):
        over = length - c["keep"]
        if over <= 0:
            continue
        fresh = min(c["recent"], over)
        others = length - c["recent"] - c["sinks"]
        share = (c["keep"] - c["recent"] - c["sinks"]) / others if others > 0 else 0.0
        n += fresh + (over - fresh) * min(1.0, max(0.0, share))
    return n


def work(case):
    c = case
    op = c["op"]
    if op == "rope":
        e = 4 if c["dtype"] == "f32" else 2
        n = c["B"] * c["T"]
        rows = 2 * (c["H"] + c["K"]) + (2 * c["K"] if c["cache"] else 0)
        table = 4 * c["rotary"] * min(n, 8192 if c["T"] == 1 else n)
        return {"bytes": n * rows * c["d"] * e + table + 4 * n + (4 * n * c["K"] if c["cache"] else 0),
                "flops": n * (c["H"] + c["K"]) * c["d"] * 8.0}
    if op == "quant":
        n = 2 * c["B"] * c["T"] * c["K"]
        return {"bytes": n * (2 * c["d"] * 2 + 2 * (c["d"] // 2 + c["d"] // 32)), "flops": n * c["d"] * 4.0}
    if op == "evict":
        tot = sum(_lens(c)) * c["K"]
        e = 4 if c["dtype"] == "f32" else 2
        over = sum(max(0, x - c["keep"]) for x in _lens(c)) * c["K"]
        return {"bytes": 8.0 * tot + 8.0 * over + _moved(c) * c["K"] * (2 * 2 * c["d"] * e + 8), "flops": tot * 1.0}
    keys = sum(_lens(c))
    if op == "scores":
        return {"bytes": keys * c["K"] * (4 * c["d"] + 8) + 4 * c["B"] * c["H"] * c["d"],
                "flops": 4.0 * keys * c["H"] * c["d"]}
    if op == "mxdec":
        row = c["d"] // 2 + c["d"] // 32
        return {"bytes": keys * c["K"] * 2 * row + 4 * c["B"] * c["H"] * c["d"] + 2 * c["B"] * c["K"] * (2 * c["d"] + row),
                "flops": 4.0 * keys * c["H"] * c["d"]}
    pairs = 0
    for n in _lens(c):
        t = min(c["T"], n)
        pairs += t * n - t * (t - 1) // 2
    return {"bytes": 2 * c["d"] * (keys * c["K"] + c["B"] * c["T"] * c["H"]) + 8 * keys * c["K"],
            "flops": 2.0 * pairs * c["H"] * c["d"]}


# ----------------------------------------------------------------------------
# inputs

def _table(max_pos, rotary, theta):
    """cos of the rotary / 2 angles, then their sines, of every position (angles in 64 bits)."""
    inv = theta ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / max(rotary, 1))
    a = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * inv[None, :]
    return torch.cat([a.cos(), a.sin()], 1).float()


def _pages(g, B, S, page):
    """A block table whose pages lie in no order, and the number of blocks of its pool."""
    n = -(-S // page)
    order = torch.randperm(B * n + 3, generator=g, device="cuda")
    return order[:B * n].to(torch.int32).view(B, n).contiguous(), B * n + 3


def _power(e):
    """2^(e - 127) in 32 bits, for whole e from 0 to 254 (made from its bits: a call of exp2 may round)."""
    e = e.to(torch.int32)
    return torch.where(e > 0, e << 23, 1 << 22).to(torch.int32).view(F32)


def _quantise(x):
    """bf16 rows [..., d] -> (codes [..., d/2] uint8, scales [..., d/32] uint8): blocks of 32 share the scale
    2^(floor(log2 amax) - 2), stored with bias 127; each value over its scale goes to the nearest e2m1 value, ties
    to the even code, beyond 6 to 6; the even element of a byte is its low half."""
    b = x.float().unflatten(-1, (-1, 32))
    e = (b.abs().amax(-1).view(torch.int32) >> 23) - 2  # a subnormal maximum has exponent field 0, as zero has
    e = e.clamp(min=0)
    step = _power(e).double()[..., None]
    a = (b.double() / step).abs().float()
    m = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    m = (m + 8 * (b < 0) * (m > 0)).to(torch.uint8).flatten(-2)
    return m[..., 0::2] | (m[..., 1::2] << 4), e.to(torch.uint8)


def _values(codes, scales):
    """What a 4-bit cache holds, in 32 bits."""
    table = torch.tensor(CODE_VALUES + tuple(-v for v in CODE_VALUES), device=codes.device)
    two = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    return (two.unflatten(-1, (-1, 32)) * _power(scales)[..., None]).flatten(-2)


def prepare(case, seed):
    c, op = case, case["op"]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(c)
    B, K, d, S = c["B"], c["K"], c["d"], c["S"]

    def normal(*shape, dtype=BF16, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(std)

    i32 = dict(dtype=torch.int32, device="cuda")
    if op == "rope":
        t = F32 if c["dtype"] == "f32" else BF16
        T, H = c["T"], c["H"]
        s["qkv"] = normal(B, T, (H + 2 * K) * d, dtype=t, std=2.0)  # one projection's output: strided heads
        s["q"], s["k"], s["v"] = (x.unflatten(-1, (-1, d)) for x in s["qkv"].split([H * d, K * d, K * d], -1))
        s["wq"], s["wk"] = ((1 + normal(d, dtype=t, std=0.1), 1 + normal(d, dtype=t, std=0.1)) if c["norm"] else (None, None))
        s["rows"] = torch.randint(0, S - T + 1, (B,), generator=g, **i32)
        first = s["rows"] + (torch.randint(0, 1000, (B,), generator=g, **i32) if c["cache"] else 0)  # rows that left
        s["positions"] = (first[:, None] + torch.arange(T, **i32)[None, :]).contiguous()
        s["rope"] = _table(S + 1000, c["rotary"], c["theta"]) if c["rotary"] else None
        s["q_out"], s["k_out"] = torch.empty(B, T, H, d, dtype=t, device="cuda"), torch.empty(B, T, K, d, dtype=t, device="cuda")
        if c["cache"]:
            if c["page"]:
                s["table"], blocks = _pages(g, B, S, c["page"])
                shape, cap = (blocks, K, c["page"], d), s["table"].shape[1] * c["page"]
            else:
                shape, cap = (B, K, S, d), S
            s["kc"], s["vc"] = torch.zeros(shape, dtype=t, device="cuda"), torch.zeros(shape, dtype=t, device="cuda")
            s["row_pos"] = torch.full((B, K, cap), -1, **i32)
        return s
    if op in ("scores", "prompt"):
        s["lens"] = torch.tensor(_lens(c), **i32)
        H = c["H"]
        s["q"] = normal(B, H, d, std=1.5) if op == "scores" else normal(B, c["T"], H, d, std=1.5)
        cap = S
        if c.get("page"):
            s["table"], blocks = _pages(g, B, S, c["page"])
            cap = s["table"].shape[1] * c["page"]
            s["kc"] = normal(blocks, K, c["page"], d)
        else:
            s["kc"] = normal(B, K, S, d)
        s["scores"] = torch.zeros(B, K, cap, device="cuda")
        live = torch.arange(cap, device="cuda")[None, None, :] < s["lens"][:, None, None]
        s["scores"] += torch.rand(B, K, cap, generator=g, device="cuda") * live * (4.0 * c.get("T", 1) * H / (K * S))
        if op == "scores":
            s["vc"] = normal(*s["kc"].shape)
            s["out"] = torch.empty_like(s["q"])
        if own:
            from kv_cache_02_b200 import gqa
            if op == "prompt":
                n = gqa.gqa_prompt_scores_workspace_bytes(B, c["T"], H, K, S, d)
            elif c["page"]:
                n = gqa.gqa_decode_scores_paged_workspace_bytes(B, H, K, d, c["page"], s["table"].shape[1])
            else:
                n = gqa.gqa_decode_scores_workspace_bytes(B, H, K, S, d)
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        return s
    if op == "evict":
        t = F32 if c["dtype"] == "f32" else BF16
        lens = torch.tensor(_lens(c), **i32)
        cap = S
        if c["page"]:
            s["table"], blocks = _pages(g, B, S, c["page"])
            cap = s["table"].shape[1] * c["page"]
            s["kc"] = normal(blocks, K, c["page"], d, dtype=t)
        else:
            s["kc"] = normal(B, K, S, d, dtype=t)
        s["vc"] = normal(*s["kc"].shape, dtype=t)
        live = torch.arange(cap, device="cuda")[None, None, :] < lens[:, None, None]
        weight = torch.exp(2.0 * torch.randn(B, K, cap, generator=g, device="cuda")) * live  # heavy-tailed, as sums of weights are
        pos = torch.where(live, torch.arange(cap, **i32)[None, None, :] + lens[:, None, None] // 3, -1).to(torch.int32)
        pos = pos.expand(-1, K, -1)
        # the rows of a cache that has been cut before lie in no order
        mix = torch.argsort(torch.where(live, torch.rand(B, K, cap, generator=g, device="cuda"), 2.0), -1)
        pos = torch.gather(pos, -1, mix)
        n = B * K * cap
        # lengths, scores and positions in one buffer: a pass begins with a copy of them, and ends with them changed
        s["saved"] = torch.cat([weight.view(-1).view(torch.int32), pos.view(-1), lens])
        s["live"] = torch.empty_like(s["saved"])
        s["scores"] = s["live"][:n].view(torch.float32).view(B, K, cap)
        s["row_pos"] = s["live"][n:2 * n].view(B, K, cap)
        s["lens"] = s["live"][2 * n:]
        s["recent_from"] = (pos.amax((1, 2)) + 1 - c["recent"]).to(torch.int32).contiguous()
        if own:
            from kv_cache_02_b200 import gqa
            s["ws"] = torch.empty(gqa.gqa_kv_evict_workspace_bytes(B, K, cap, c["keep"]), dtype=torch.uint8, device="cuda")
        return s
    if op == "quant":
        T = c["T"]
        # channels of unequal size, as keys have
        size = torch.exp(torch.randn(K, d, generator=g, device="cuda"))
        s["k"] = (normal(B, T, K, d, dtype=F32) * size).to(BF16)
        s["v"] = normal(B, T, K, d)
        s["pos"] = torch.randint(0, S - T + 1, (B,), generator=g, **i32)
        s["k_out"], s["v_out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        for n in "kv":
            s[n + "c"] = torch.zeros(B, K, S, d // 2, dtype=torch.uint8, device="cuda")
            s[n + "s"] = torch.zeros(B, K, S, d // 32, dtype=torch.uint8, device="cuda")
        return s
    # mxdec: one step, the new token's rows first
    H = c["H"]
    lens = _lens(c)
    s["lens"] = torch.tensor(lens, **i32)
    s["pos"] = torch.tensor([max(0, x - 1) for x in lens], **i32)
    s["q"] = normal(B, H, d, std=1.5)
    s["k"], s["v"] = normal(B, 1, K, d), normal(B, 1, K, d)
    size = torch.exp(0.7 * torch.randn(K, 1, d, generator=g, device="cuda")).to(BF16)
    for n in "kv":
        x = normal(B, K, S, d)
        if n == "k":
            x *= size
        parts = [_quantise(x[b]) for b in range(B)]
        s[n + "c"], s[n + "s"] = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
        del x, parts
    s["out"] = torch.empty_like(s["q"])
    if own:
        from kv_cache_02_b200 import gqa
        s["ws"] = torch.empty(gqa.gqa_decode_mxfp4_workspace_bytes(B, H, K, S, d), dtype=torch.uint8, device="cuda")
    return s


# ----------------------------------------------------------------------------
# one pass

def run(state):
    s = state
    return {"rope": _run_rope, "scores": _run_scores, "prompt": _run_prompt, "evict": _run_evict,
            "quant": _run_quant, "mxdec": _run_mxdec}[s["op"]](s)


def _gathered(cache, s):
    """A paged cache as [B, K, cap, d]."""
    if not s.get("page"):
        return cache
    return cache[s["table"].long()].transpose(1, 2).flatten(2, 3)


def _norm_rotate(x, w, s):
    x = x.float()
    if w is not None:
        x = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)) * w.float()
    r = s["rotary"]
    if not r:
        return x
    cs = s["rope"][s["positions"].long()][:, :, None, :]
    cos, sin = cs[..., :r // 2], cs[..., r // 2:]
    if s["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _run_rope(s):
    if own:
        from kv_cache_02_b200 import gqa
        rot = dict(q_weight=s["wq"], k_weight=s["wk"], eps=1e-6, interleaved=s["interleaved"])
        if not s["cache"]:
            gqa.gqa_qk_norm_rope(s["q_out"], s["q"], s["k"], s["rope"], s["positions"], k_out=s["k_out"], **rot)
            return [s["q_out"], s["k_out"]]
        if s["page"]:
            gqa.gqa_qk_norm_rope_paged(s["q_out"], s["q"], s["k"], s["v"], s["rope"], s["positions"], s["kc"], s["vc"],
                                       s["table"], s["rows"], row_pos=s["row_pos"], **rot)
        else:
            gqa.gqa_qk_norm_rope(s["q_out"], s["q"], s["k"], s["rope"], s["positions"], v=s["v"], k_cache=s["kc"],
                                 v_cache=s["vc"], rows=s["rows"], row_pos=s["row_pos"], **rot)
        return [s["q_out"], s["kc"], s["vc"], s["row_pos"]]
    q = _norm_rotate(s["q"], s["wq"], s).to(s["q"].dtype)
    k = _norm_rotate(s["k"], s["wk"], s).to(s["k"].dtype)
    if not s["cache"]:
        return [q, k]
    b = torch.arange(s["B"], device="cuda")[:, None]
    at = s["rows"].long()[:, None] + torch.arange(s["T"], device="cuda")[None, :]
    if s["page"]:
        block = s["table"].long()[b, at // s["page"]]
        s["kc"][block, :, at % s["page"]] = k
        s["vc"][block, :, at % s["page"]] = s["v"]
    else:
        s["kc"][b, :, at] = k
        s["vc"][b, :, at] = s["v"]
    s["row_pos"][b, :, at] = s["positions"][..., None].expand(-1, -1, s["K"])
    return [q, s["kc"], s["vc"], s["row_pos"]]


def _weights(q, keys, mask, scale):
    """Softmax weights of q [..., n, d] over keys [..., S, d]; a row whose mask leaves nothing has none."""
    x = torch.matmul(q.float(), keys.float().transpose(-1, -2)).mul_(scale).masked_fill_(~mask, -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True).clamp_(min=-3e38)).exp_()
    return x.div_(x.sum(-1, keepdim=True).clamp_(min=1e-38))


def _run_scores(s):
    if own:
        from kv_cache_02_b200 import gqa
        if s["page"]:
            gqa.gqa_decode_scores_paged(s["out"], s["scores"], s["q"], s["kc"], s["vc"], s["table"], s["lens"],
                                        s["d"] ** -0.5, workspace=s["ws"])
        else:
            gqa.gqa_decode_scores(s["out"], s["scores"], s["q"], s["kc"], s["vc"], s["lens"], s["d"] ** -0.5,
                                  workspace=s["ws"])
        return [s["out"], s["scores"]]
    B, H, K, d = s["B"], s["H"], s["K"], s["d"]
    keys, values = _gathered(s["kc"], s), _gathered(s["vc"], s)
    mask = (torch.arange(keys.shape[2], device="cuda")[None, :] < s["lens"][:, None])[:, None, None, :]
    p = _weights(s["q"].view(B, K, H // K, d), keys, mask, d ** -0.5)
    s["scores"] += p.sum(2)
    return [torch.matmul(p, values.float()).view(B, H, d).to(BF16), s["scores"]]


def _run_prompt(s):
    if own:
        from kv_cache_02_b200 import gqa
        gqa.gqa_prompt_scores(s["scores"], s["q"], s["kc"], s["lens"], s["d"] ** -0.5, workspace=s["ws"])
        return [s["scores"]]
    B, T, H, K, d, S = s["B"], s["T"], s["H"], s["K"], s["d"], s["S"]
    q = s["q"].view(B, T, K, H // K, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    at = s["lens"][:, None] - T + torch.arange(T, device="cuda")[None, :]  # the queries' keys; below 0: no query
    mask = (torch.arange(S, device="cuda")[None, None, :] <= at[:, :, None])[:, None, :, :].repeat(1, 1, H // K, 1)
    s["scores"] += _weights(q, s["kc"], mask, d ** -0.5).sum(2)
    return [s["scores"]]


def _run_evict(s):
    s["live"].copy_(s["saved"])
    if own:
        from kv_cache_02_b200 import gqa
        args = (s["scores"], s["row_pos"], s["lens"], s["keep"], s["sinks"], s["recent_from"], s["ws"])
        if s["page"]:
            gqa.gqa_kv_evict_paged(s["kc"], s["vc"], s["table"], *args)
        else:
            gqa.gqa_kv_evict(s["kc"], s["vc"], *args)
        return [s["kc"], s["vc"], s["scores"], s["row_pos"], s["lens"]]
    B, K, keep, cap = s["B"], s["K"], s["keep"], s["scores"].shape[2]
    at = torch.arange(cap, device="cuda")
    full = s["lens"][:, None, None]
    live, over = at < full, full > keep
    held = (s["row_pos"] < s["sinks"]) | (s["row_pos"] >= s["recent_from"][:, None, None])
    rank = torch.where(live, torch.where(held, math.inf, s["scores"]), -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(held).scatter_(-1, order[..., :keep], True)
    hole = over & (at < keep) & ~kept
    mover = over & (at >= keep) & kept
    # the i-th mover goes to the i-th hole: both in order of their rows, unit by unit
    src, dst = mover.flatten(0, 1).nonzero(), hole.flatten(0, 1).nonzero()
    s["scores"].view(B * K, cap)[dst[:, 0], dst[:, 1]] = s["scores"].view(B * K, cap)[src[:, 0], src[:, 1]]
    s["row_pos"].view(B * K, cap)[dst[:, 0], dst[:, 1]] = s["row_pos"].view(B * K, cap)[src[:, 0], src[:, 1]]
    b, h = src[:, 0] // K, src[:, 0] % K
    if s["page"]:
        f, t = s["table"].long()[b, src[:, 1] // s["page"]], s["table"].long()[b, dst[:, 1] // s["page"]]
        s["kc"][t, h, dst[:, 1] % s["page"]] = s["kc"][f, h, src[:, 1] % s["page"]]
        s["vc"][t, h, dst[:, 1] % s["page"]] = s["vc"][f, h, src[:, 1] % s["page"]]
    else:
        s["kc"][b, h, dst[:, 1]] = s["kc"][b, h, src[:, 1]]
        s["vc"][b, h, dst[:, 1]] = s["vc"][b, h, src[:, 1]]
    gone = over & live & (at >= keep)
    s["scores"].masked_fill_(gone, 0.0)
    s["row_pos"].masked_fill_(gone, -1)
    s["lens"].clamp_(max=keep)
    return [s["kc"], s["vc"], s["scores"], s["row_pos"], s["lens"]]


def _store(s, n):
    """The new rows of k or v into the plain form's 4-bit cache."""
    codes, scales = _quantise(s[n])
    b = torch.arange(codes.shape[0], device="cuda")[:, None]
    at = s["pos"].long()[:, None] + torch.arange(codes.shape[1], device="cuda")[None, :]
    s[n + "c"][b, :, at] = codes
    s[n + "s"][b, :, at] = scales
    return b, at


def _run_quant(s):
    if own:
        from kv_cache_02_b200 import gqa
        cache = (s["kc"], s["ks"], s["vc"], s["vs"])
        gqa.gqa_kv_append_mxfp4(*cache, s["k"], s["v"], s["pos"])
        gqa.gqa_kv_read_mxfp4(s["k_out"], s["v_out"], *cache, s["pos"])
        return [s["k_out"], s["v_out"]]
    b, at = _store(s, "k")
    _store(s, "v")
    return [_values(s["kc"][b, :, at], s["ks"][b, :, at]).to(BF16), _values(s["vc"][b, :, at], s["vs"][b, :, at]).to(BF16)]


def _run_mxdec(s):
    if own:
        from kv_cache_02_b200 import gqa
        cache = (s["kc"], s["ks"], s["vc"], s["vs"])
        gqa.gqa_kv_append_mxfp4(*cache, s["k"], s["v"], s["pos"])
        gqa.gqa_decode_mxfp4(s["out"], s["q"], *cache, s["lens"], s["d"] ** -0.5, workspace=s["ws"])
        return [s["out"]]
    _store(s, "k")
    _store(s, "v")
    B, H, K, d = s["B"], s["H"], s["K"], s["d"]
    mask = (torch.arange(s["S"], device="cuda")[None, :] < s["lens"][:, None])[:, None, None, :]
    p = _weights(s["q"].view(B, K, H // K, d), _values(s["kc"], s["ks"]), mask, d ** -0.5)
    return [torch.matmul(p, _values(s["vc"], s["vs"])).view(B, H, d).to(BF16)]


# ----------------------------------------------------------------------------
# exact values

def _exact_quantised(x):
    """bf16 rows -> the values their 4-bit blocks stand for, by search among all candidates."""
    x = x.double().unflatten(-1, (-1, 32))
    top = x.abs().amax(-1, keepdim=True)
    top = top.cpu().numpy()
    e = np.where(top > 0, np.frexp(top)[1] - 1 - 2, -127)  # floor(log2 top) - 2
    step = torch.from_numpy(np.ldexp(1.0, np.maximum(e, -127))).to(x.device)
    best, near = torch.zeros_like(x), torch.full_like(x, math.inf)
    for code in (0, 2, 4, 6, 1, 3, 5, 7):  # even codes first: they win ties
        far = ((x / step).abs() - CODE_VALUES[code]).abs()
        best = torch.where(far < near, CODE_VALUES[code] * torch.sign(x) * step, best)
        near = torch.minimum(far, near)
    return best.flatten(-2)


def _exact_held(codes, scales):
    low, high = (codes % 16).long(), (codes // 16).long()
    size = torch.tensor(CODE_VALUES, dtype=torch.float64, device=codes.device)
    pair = torch.stack([size[h % 8] * (1 - 2 * (h // 8)).double() for h in (low, high)], -1).flatten(-2)
    step = torch.from_numpy(np.ldexp(1.0, np.arange(256) - 127)).to(codes.device)
    return pair * step[scales.long()].repeat_interleave(32, -1)


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op == "rope":
        made = []
        for x, w in ((s["q"].double(), s["wq"]), (s["k"].double(), s["wk"])):
            if w is not None:
                x = x / (x.pow(2).sum(-1, keepdim=True) / c["d"] + 1e-6).sqrt() * w.double()
            r = c["rotary"]
            if r:
                half = r // 2
                z = s["rope"].double()[s["positions"].long()]
                turn = torch.complex(z[..., :half], z[..., half:])[:, :, None, :]
                pair = torch.complex(x[..., 0:r:2].clone(), x[..., 1:r:2].clone()) if c["interleaved"] else torch.complex(x[..., :half].clone(), x[..., half:r].clone())
                pair = pair * turn
                x = x.clone()
                if c["interleaved"]:
                    x[..., 0:r:2], x[..., 1:r:2] = pair.real, pair.imag
                else:
                    x[..., :half], x[..., half:r] = pair.real, pair.imag
            made.append(x)
        if not c["cache"]:
            return made
        kc, vc = torch.zeros(s["kc"].shape, dtype=torch.float64, device="cuda"), torch.zeros(s["vc"].shape, dtype=torch.float64, device="cuda")
        for b, first in enumerate(s["rows"].tolist()):
            rows = torch.arange(first, first + c["T"], device="cuda")
            for cache, new in ((kc, made[1][b]), (vc, s["v"][b].double())):
                if c["page"]:
                    cache[s["table"][b].long()[rows // c["page"]], :, rows % c["page"]] = new
                else:
                    cache[b, :, rows] = new.transpose(0, 1)
        return [made[0], kc, vc, None]
    if op in ("quant", "mxdec"):
        if op == "quant":
            return [_exact_quantised(s["k"]), _exact_quantised(s["v"])]
        B, H, K, d = c["B"], c["H"], c["K"], c["d"]
        out = torch.zeros(B, H, d, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lens(c)):
            if n == 0:
                continue
            k, v = _exact_held(s["kc"][b, :, :n], s["ks"][b, :, :n]), _exact_held(s["vc"][b, :, :n], s["vs"][b, :, :n])
            k[:, n - 1], v[:, n - 1] = _exact_quantised(s["k"][b, 0]), _exact_quantised(s["v"][b, 0])
            x = torch.einsum("kgd,knd->kgn", s["q"][b].double().view(K, -1, d), k) / math.sqrt(d)
            out[b] = torch.einsum("kgn,knd->kgd", torch.softmax(x, -1), v).reshape(H, d)
        return [out]
    if op == "evict":
        s["live"].copy_(s["saved"])
        keep, cap = c["keep"], s["scores"].shape[2]
        scores, pos = s["scores"].cpu(), s["row_pos"].cpu()
        since = s["recent_from"].tolist()
        after = scores.double()
        kc, vc = s["kc"].double(), s["vc"].double()
        for b, n in enumerate(_lens(c)):
            if n <= keep:
                continue
            for h in range(c["K"]):
                held = (pos[b, h, :n] < c["sinks"]) | (pos[b, h, :n] >= since[b])
                best = sorted(range(n), key=lambda i, a=held.tolist(), w=scores[b, h, :n].tolist(): (not a[i], 0.0 if a[i] else -w[i], i))[:keep]
                stay = set(best)
                frm = sorted(i for i in stay if i >= keep)
                to = [i for i in range(keep) if i not in stay]
                after[b, h, to] = scores[b, h, frm].double()
                after[b, h, keep:n] = 0.0
                f, t = torch.tensor(frm, dtype=torch.long), torch.tensor(to, dtype=torch.long)
                for cache in (kc, vc):
                    if c["page"]:
                        tab = s["table"][b].long().cpu()
                        cache[tab[t // c["page"]], h, t % c["page"]] = cache[tab[f // c["page"]], h, f % c["page"]]
                    else:
                        cache[b, h, t] = cache[b, h, f]
        return [kc, vc, after, None, None]
    B, H, K, d = c["B"], c["H"], c["K"], c["d"]
    scores = s["scores"].double()
    out = torch.zeros(B, H, d, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(c)):
        if n == 0:
            continue
        k, v = s["kc"], s.get("vc")
        if c.get("page"):
            tab = s["table"][b].long()
            k, v = (x[tab].permute(1, 0, 2, 3).reshape(K, -1, d)[:, :n].double() for x in (k, v))
        else:
            k, v = k[b, :, :n].double(), v[b, :, :n].double() if v is not None else None
        if op == "scores":
            p = torch.softmax(torch.einsum("kgd,knd->kgn", s["q"][b].double().view(K, -1, d), k) / math.sqrt(d), -1)
            out[b] = torch.einsum("kgn,knd->kgd", p, v).reshape(H, d)
            scores[b, :, :n] += p.sum(1)
            continue
        t = min(c["T"], n)
        last = torch.arange(n - t, n, device="cuda")
        later = torch.arange(n, device="cuda")[None, :] > last[:, None]
        for h in range(H):
            x = s["q"][b, c["T"] - t:, h].double() @ k[h // (H // K)].t() / math.sqrt(d)
            scores[b, h // (H // K), :n] += torch.softmax(x.masked_fill(later, -math.inf), -1).sum(0)
    return [out, scores] if op == "scores" else [scores]
