"""Cases of the attention operators: head norms with rotation and cache append, paged decode, paged prefill.

Three operators of the attention half of a decoder layer, over one paged cache:

* "prepare": RMS norm of each query and key head, the position rotation, and the rows of K and V into the cache;
* "decode": a few new tokens of each sequence against its cached keys and values;
* "prefill": the tokens of prompts (or of pieces of prompts behind a cached prefix), causal.

decode and prefill take a sliding window with a few first tokens that stay visible; window 0 means none.

The cache holds pages of `page` tokens: K as [pages, kv heads, dim / 8, page, 8] and V as
[pages, kv heads, page / 8, dim, 8], both bf16.  A sequence's tokens sit in the pages its row of the page table
names, in order.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
MAX_SCORES = 1 << 31        # scores of one plain pass (8 GiB in 32 bits)
MAX_CACHE_VALUES = 1 << 29  # K and V values of one padded batch


def listed():
    return [
        # one new token of one sequence: the smallest call, latency
        {"name": "prepare_one_token", "op": "prepare", "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16,
         "rotary": 128, "style": "half", "prompt": False},
        # a decode step of 64 sequences, partial rotation of neighbouring pairs
        {"name": "prepare_batch_64", "op": "prepare", "tokens": 64, "heads": 64, "kv_heads": 8, "dim": 128, "page": 64,
         "rotary": 64, "style": "interleaved", "prompt": False},
        # a prompt of an odd length, small heads, odd head counts
        {"name": "prepare_prompt_1531", "op": "prepare", "tokens": 1531, "heads": 15, "kv_heads": 5, "dim": 64,
         "page": 32, "rotary": 32, "style": "half", "prompt": True},
        # a prompt of 4096 tokens
        {"name": "prepare_prompt_4096", "op": "prepare", "tokens": 4096, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 16, "rotary": 128, "style": "half", "prompt": True},
        # one sequence of a short chat: latency
        {"name": "decode_one_short", "op": "decode", "batch": 1, "new": 1, "low": 777, "high": 777, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 16, "window": 0, "sinks": 0},
        # one sequence with a very long cache: few rows, so the length has to be split
        {"name": "decode_one_131071", "op": "decode", "batch": 1, "new": 1, "low": 131071, "high": 131071, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "sinks": 0},
        # a batch of 64 sequences of very different lengths
        {"name": "decode_batch_64_ragged", "op": "decode", "batch": 64, "new": 1, "low": 1, "high": 8192, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 16, "window": 0, "sinks": 0},
        # a verify step of 4 drafted tokens, window with sinks, small heads
        {"name": "decode_verify_window", "op": "decode", "batch": 16, "new": 4, "low": 5000, "high": 32768,
         "heads": 32, "kv_heads": 4, "dim": 64, "page": 32, "window": 4096, "sinks": 4},
        # a one-line prompt: latency
        {"name": "prefill_one_37", "op": "prefill", "batch": 1, "q_low": 37, "q_high": 37, "past_high": 0, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 16, "window": 0, "sinks": 0},
        # pieces of 8 prompts of odd lengths, each behind a cached prefix of its own, small heads
        {"name": "prefill_pieces_8", "op": "prefill", "batch": 8, "q_low": 1, "q_high": 700, "past_high": 4096,
         "heads": 24, "kv_heads": 8, "dim": 64, "page": 32, "window": 0, "sinks": 0},
        # one prompt of 4096 tokens
        {"name": "prefill_one_4096", "op": "prefill", "batch": 1, "q_low": 4096, "q_high": 4096, "past_high": 0,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "window": 0, "sinks": 0},
        # one long prompt with a window and sinks
        {"name": "prefill_one_8192_window", "op": "prefill", "batch": 1, "q_low": 8192, "q_high": 8192, "past_high": 0,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "window": 1024, "sinks": 4},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _draw(rng):
    kv = rng.choice([1, 2, 3, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 5, 8, 16])
    c = {"op": rng.choice(["prepare", "decode", "prefill"]), "heads": heads, "kv_heads": kv,
         "dim": rng.choice([64, 128, 128, 256]), "page": rng.choice([16, 32, 64, 128])}
    if c["op"] == "prepare":
        c.update(tokens=_log(rng, 1, 8192), rotary=c["dim"] // rng.choice([1, 2, 4]),
                 style=rng.choice(["half", "interleaved"]), prompt=rng.random() < 0.5)
        return c
    c.update(window=rng.choice([0, _log(rng, 16, 8192)]))
    c.update(sinks=rng.choice([0, 1, 4, 37]) if c["window"] else 0)
    if c["op"] == "decode":
        high = _log(rng, 16, 131072)
        c.update(batch=_log(rng, 1, 64), new=rng.choice([1, 1, 1, 2, 3, 4]), low=max(4, _log(rng, 4, high)), high=high)
    else:
        high = _log(rng, 16, 8192)
        c.update(batch=rng.choice([1, 1, 2, 3, 8]), q_low=_log(rng, 1, high), q_high=high,
                 past_high=rng.choice([0, _log(rng, 16, 8192)]))
    return c


def draw(rng):
    """Cases of the listed ranges; one that would cost more than the largest listed one is drawn again."""
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] > 1.0e9 or w["flops"] > 1.37e11:
            continue
        if c["op"] == "prepare":
            return c
        lens, qs = _lens(c)
        top = _pages(c, lens) * c["page"]
        if c["batch"] * top * c["kv_heads"] * c["dim"] * 2 > MAX_CACHE_VALUES:
            continue
        if c["batch"] * max(qs) * c["heads"] * top > MAX_SCORES:
            continue
        return c


def _lens(c):
    """Tokens of each sequence, the new ones among them, and the new ones: of the case, whatever the seed."""
    r = random.Random("%(batch)d of %(op)s, page %(page)d, %(heads)d heads" % c)
    if c["op"] == "decode":
        lens = [r.randint(c["low"], c["high"]) for _ in range(c["batch"])]
        lens[-1] = c["high"]
        return [max(n, c["new"]) for n in lens], [c["new"]] * c["batch"]
    qs = [r.randint(c["q_low"], c["q_high"]) for _ in range(c["batch"])]
    qs[-1] = c["q_high"]
    return [q + (r.randint(0, c["past_high"]) if c["past_high"] else 0) for q in qs], qs


def _pages(c, lens):
    return -(-max(lens) // c["page"])


def _scale(c):
    return c["dim"] ** -0.5


def work(case):
    c = case
    H, K, D = c["heads"], c["kv_heads"], c["dim"]
    if c["op"] == "prepare":
        T = c["tokens"]
        rows = T * (H + 2 * K) * D
        return {"bytes": 2 * rows * 2 + T * (c["rotary"] * 4 + 4 + 8) + 2 * D * 4, "flops": 6 * T * (H + K) * D}
    lens, qs = _lens(c)
    W, S = c["window"], c["sinks"]
    keys = pairs = 0
    for n, q in zip(lens, qs):
        at = np.arange(n - q, n, dtype=np.int64)
        if W:
            pairs += int(np.sum(np.minimum(at + 1, W) + np.minimum(S, np.maximum(0, at + 1 - W))))
            first = max(0, n - q - W + 1)
            keys += n - first + min(S, first)
        else:
            pairs += int(np.sum(at + 1))
            keys += n
    return {"bytes": keys * K * D * 4 + 2 * sum(qs) * H * D * 2 + 4 * sum(-(-n // c["page"]) for n in lens),
            "flops": 4 * D * H * pairs}


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    H, K, D, P = c["heads"], c["kv_heads"], c["dim"], c["page"]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(std).to(torch.bfloat16)

    s = {"case": dict(c)}
    if c["op"] == "prepare":
        T, R = c["tokens"], c["rotary"]
        if c["prompt"]:       # one prompt from its start, in pages of any order
            n_pages, places = -(-T // P) + 3, 8192
            order = torch.randperm(n_pages, generator=g, device=DEV)
            at = torch.arange(T, device=DEV)
            s["slots"] = order[at // P] * P + at % P
            s["positions"] = at.to(torch.int32)
        else:                 # one new token of each sequence, each in a page of its own
            n_pages, places = T + 3, 32768
            order = torch.randperm(n_pages, generator=g, device=DEV)
            at = torch.randint(0, places, (T,), generator=g, device=DEV)
            s["slots"] = order[:T] * P + at % P
            s["positions"] = at.to(torch.int32)
        turn = torch.arange(places, device=DEV, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R)[None, :]
        s["cos_sin"] = torch.cat([turn.cos(), turn.sin()], dim=1).to(torch.float32).contiguous()
        s["qkv"] = normal(T, (H + 2 * K) * D, std=0.7)
        s["q_norm"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)
        s["k_norm"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)
        s["k_cache"] = normal(n_pages, K, D // 8, P, 8)
        s["v_cache"] = normal(n_pages, K, P // 8, D, 8)
        s["q"] = torch.empty((T, H, D), dtype=torch.bfloat16, device=DEV)
        return s
    lens, qs = _lens(c)
    B, each = c["batch"], _pages(c, lens)
    need = sum(-(-n // P) for n in lens)
    order = torch.randperm(need + 1, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((B, each), dtype=torch.int32)
    at = 0
    order = order.cpu()
    for b, n in enumerate(lens):
        m = -(-n // P)
        table[b, :m] = order[at:at + m]
        at += m
    s["page_table"] = table.to(DEV)
    s["k_cache"] = normal(need + 1, K, D // 8, P, 8)
    s["v_cache"] = normal(need + 1, K, P // 8, D, 8)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["max_len"], s["max_q"] = max(lens), max(qs)
    T = sum(qs)
    s["q"] = normal(T, H, D, std=1.5)
    s["cu_q"] = torch.tensor([0] + list(np.cumsum(qs)), dtype=torch.int32, device=DEV)
    s["out"] = torch.empty((T, H, D), dtype=torch.bfloat16, device=DEV)
    return s


def _config(c):
    from routed_expert_mlp_amd import attention as A
    return A.AttnConfig(n_heads=c["heads"], n_kv_heads=c["kv_heads"], head_dim=c["dim"], page_size=c["page"],
                        rotary_dim=c.get("rotary", 0),
                        rope_style=A.ROPE_INTERLEAVED if c.get("style") == "interleaved" else A.ROPE_HALF,
                        norm_eps=EPS, scale=_scale(c), window=c.get("window", 0), n_sinks=c.get("sinks", 0))


def _bound(s):
    """The call on this state's buffers, its arguments checked and marshalled once, as a serving loop keeps it."""
    from routed_expert_mlp_amd import attention as A
    c, cfg, cache = s["case"], _config(s["case"]), A.KVCache(s["k_cache"], s["v_cache"])
    if c["op"] == "prepare":
        return A.bind_prepare(cfg, cache, s["qkv"], s["q_norm"], s["k_norm"], s["cos_sin"], s["positions"],
                              s["slots"], s["q"])
    if c["op"] == "decode":
        q = s["q"].view(c["batch"], c["new"], c["heads"], c["dim"])
        return A.bind_decode(cfg, cache, q, s["seq_lens"], s["page_table"], s["max_len"], s["out"].view(q.shape))
    return A.bind_prefill(cfg, cache, s["q"], s["cu_q"], s["max_q"], s["seq_lens"], s["page_table"], s["max_len"],
                          s["out"])


def run(state):
    s = state
    if own:
        call = s.get("call")
        if call is None:
            call = s["call"] = _bound(s)
        call()
    elif s["case"]["op"] == "prepare":
        _plain_prepare(s)
    else:
        _plain_attention(s)
    if s["case"]["op"] == "prepare":
        return {"q": s["q"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return s["out"]


def _plain_prepare(s):
    c = s["case"]
    H, K, D, P, R = c["heads"], c["kv_heads"], c["dim"], c["page"], c["rotary"]
    T = c["tokens"]
    x = s["qkv"].float().view(T, H + 2 * K, D)
    y = x[:, :H + K]
    y = y * (y.square().mean(-1, keepdim=True) + EPS).rsqrt()
    w = torch.cat([s["q_norm"].expand(H, D), s["k_norm"].expand(K, D)])
    y = y * w
    turn = s["cos_sin"][s["positions"].long()]
    cos, sin = turn[:, None, :R // 2], turn[:, None, R // 2:]
    if c["style"] == "half":
        a, b = y[..., :R // 2], y[..., R // 2:R]
        z = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        z = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    y = torch.cat([z, y[..., R:]], dim=-1).to(torch.bfloat16)
    s["q"].copy_(y[:, :H])
    page, at = s["slots"] // P, s["slots"] % P
    s["k_cache"][page, :, :, at] = y[:, H:].reshape(T, K, D // 8, 8)
    s["v_cache"][page, :, at // 8, :, at % 8] = x[:, H + K:].to(torch.bfloat16)


def _plain_attention(s):
    c = s["case"]
    H, K, D, W, S = c["heads"], c["kv_heads"], c["dim"], c["window"], c["sinks"]
    B, G, M = c["batch"], c["heads"] // c["kv_heads"], s["max_q"]
    table, T = s["page_table"].long(), s["q"].shape[0]
    k = s["k_cache"][table].permute(0, 2, 1, 4, 3, 5).reshape(B, K, -1, D).float()
    v = s["v_cache"][table].permute(0, 2, 1, 3, 5, 4).reshape(B, K, -1, D).float()
    L = k.shape[2]
    first, lens = s["cu_q"][:-1].long(), s["seq_lens"].long()
    count = s["cu_q"][1:].long() - first
    i = torch.arange(M, device=DEV)
    row = (first[:, None] + i).clamp(max=T - 1)                                     # [B, M]
    q = s["q"][row].view(B, M, K, G, D).permute(0, 2, 3, 1, 4).reshape(B, K, G * M, D).float()
    p = torch.matmul(q, k.transpose(-1, -2)).view(B, K, G, M, L)
    p *= _scale(c)
    at = (lens - count)[:, None] + i                                               # position of each query
    key = torch.arange(L, device=DEV)
    seen = key <= at[..., None]
    if W:
        seen &= (key > at[..., None] - W) | (key < S)
    p.masked_fill_(~seen[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True).clamp(min=-1e30)
    p -= top
    p.exp_()
    o = torch.matmul(p.view(B, K, G * M, L), v).view(B, K, G, M, D)
    o = o / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, M, H, D)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(s["cu_q"][1:].long(), t, right=True)
    s["out"].copy_(o[b, t - first[b]])


def exact(case, seed):
    """The definitions in 64 bits, one sequence and one key/value head at a time."""
    s = prepare(case, seed)
    c = s["case"]
    return _exact_prepare(s) if c["op"] == "prepare" else _exact_attention(s)


def _exact_prepare(s):
    c = s["case"]
    H, K, D, P, R = c["heads"], c["kv_heads"], c["dim"], c["page"], c["rotary"]
    x = s["qkv"].double().reshape(-1, H + 2 * K, D)
    T = x.shape[0]
    table = s["cos_sin"].double()[s["positions"].long()]
    done = []
    for h in range(H + K):
        y = x[:, h] / torch.sqrt(torch.sum(x[:, h] ** 2, dim=1, keepdim=True) / D + EPS)
        y = y * (s["q_norm"] if h < H else s["k_norm"]).double()
        z = y.clone()
        for j in range(R // 2):
            m, n = (j, j + R // 2) if c["style"] == "half" else (2 * j, 2 * j + 1)
            co, si = table[:, j], table[:, R // 2 + j]
            z[:, m] = co * y[:, m] - si * y[:, n]
            z[:, n] = si * y[:, m] + co * y[:, n]
        done.append(z)
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    flat_k = kc.permute(0, 3, 1, 2, 4).reshape(-1, K, D)           # [page and place, head, dim]
    flat_v = vc.permute(0, 2, 4, 1, 3).reshape(-1, K, D)
    for h in range(K):
        flat_k[s["slots"], h] = done[H + h]
        flat_v[s["slots"], h] = x[:, H + K + h]
    kc = flat_k.view(-1, P, K, D // 8, 8).permute(0, 2, 3, 1, 4).contiguous()
    vc = flat_v.view(-1, P // 8, 8, K, D).permute(0, 3, 1, 4, 2).contiguous()
    return {"q": torch.stack(done[:H], dim=1).view(T, H, D), "k_cache": kc, "v_cache": vc}


def _exact_attention(s):
    c = s["case"]
    H, K, D, P, W, S = c["heads"], c["kv_heads"], c["dim"], c["page"], c["window"], c["sinks"]
    G = H // K
    lens, qs = _lens(c)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    row = 0
    for b, (n, m) in enumerate(zip(lens, qs)):
        where = torch.arange(n, device=DEV)
        page, at = s["page_table"][b].long()[where // P], where % P
        for h in range(K):
            k = s["k_cache"][page, h, :, at].reshape(n, D).double()
            v = s["v_cache"][page, h, at // 8, :, at % 8].double()
            for lo in range(0, m, 2048):
                hi = min(m, lo + 2048)
                pos = torch.arange(n - m + lo, n - m + hi, device=DEV)[:, None]
                hidden = where[None, :] > pos
                if W:
                    hidden |= (pos - where[None, :] >= W) & (where[None, :] >= S)
                for e in range(h * G, h * G + G):
                    a = s["q"][row + lo:row + hi, e].double() @ k.T * _scale(c)
                    a[hidden] = -math.inf
                    out[row + lo:row + hi, e] = torch.softmax(a, dim=1) @ v
        row += m
    return out
