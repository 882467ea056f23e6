"""Cases of the operators around the two halves of a decoder layer, for a server of many requests at once.

Four operators of one step:

* "norm": the residual's addition and the RMS norm of each row, out in bf16, in E4M3 with one scale per 128 columns, or both;
* "fp8": the projection that takes such rows, its weights in E4M3 with one scale per 128 x 128 block;
* "lora": low-rank adapters, one of many for each token, added to what the shared projection gave;
* "shared": a decode step of sequences that begin with the same tokens, whose keys and values are cached once.

The cache of "shared" holds pages of `page` tokens: K as [pages, kv heads, dim / 8, page, 8] and V as
[pages, kv heads, page / 8, dim, 8], both bf16.  Its first `prefix` tokens are in the pages that one list names;
the others of each sequence are in the pages of its row of the page table.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
BLOCK = 128                 # columns of a scale
TOP = 448.0                 # largest E4M3 value
TINY = 2.0 ** -126          # least scale
MAX_SCORES = 1 << 29        # scores of one plain pass (2 GiB in 32 bits)
MAX_CACHE_VALUES = 1 << 29  # K and V values of the prefix and of the padded rest


def listed():
    return [
        # one token between the halves of a layer, for both kinds of projection: latency
        {"name": "norm_one_token", "op": "norm", "tokens": 1, "hidden": 4096, "residual": True, "wide": True,
         "bytes": True},
        # pieces of prompts, rows that end inside a block of 128 and of which only the 8-bit form is wanted
        {"name": "norm_ragged_1037", "op": "norm", "tokens": 1037, "hidden": 1544, "residual": True, "wide": False,
         "bytes": True},
        # a prompt of 4096 tokens
        {"name": "norm_prompt_4096", "op": "norm", "tokens": 4096, "hidden": 4096, "residual": True, "wide": True,
         "bytes": True},
        # queries, keys and values (32 and 2 x 8 heads of 128 dims) of one new token: latency, and the weights' stream
        {"name": "fp8_one_token", "op": "fp8", "tokens": 1, "out": 6144, "hidden": 4096},
        # a piece of a prompt into a narrow latent with a rotated part: an odd number of rows, few columns
        {"name": "fp8_narrow_517", "op": "fp8", "tokens": 517, "out": 576, "hidden": 4096},
        # queries, keys and values of a prompt of 4096 tokens
        {"name": "fp8_prompt_4096", "op": "fp8", "tokens": 4096, "out": 6144, "hidden": 4096},
        # one token of a request with an adapter: latency
        {"name": "lora_one_token", "op": "lora", "tokens": 1, "hidden": 4096, "out": 6144, "rank": 16, "adapters": 8,
         "order": "mixed"},
        # a decode step of 64 requests with adapters of several ranks in any order, some with none
        {"name": "lora_batch_64", "op": "lora", "tokens": 64, "hidden": 4096, "out": 6144, "rank": 64, "adapters": 32,
         "order": "mixed"},
        # prompts of several requests, one after the other
        {"name": "lora_prompts_4096", "op": "lora", "tokens": 4096, "hidden": 4096, "out": 4096, "rank": 32,
         "adapters": 5, "order": "runs"},
        # four chats behind a short system prompt: latency
        {"name": "shared_4_behind_1024", "op": "shared", "batch": 4, "new": 1, "prefix": 1024, "low": 1, "high": 256,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "window": 0, "sinks": 0},
        # verify steps of 4 tokens, small heads, a prefix that ends inside a page
        {"name": "shared_24_verify", "op": "shared", "batch": 24, "new": 4, "prefix": 7919, "low": 4, "high": 2048,
         "heads": 24, "kv_heads": 8, "dim": 64, "page": 32, "window": 0, "sinks": 0},
        # 64 requests about one long document
        {"name": "shared_64_behind_32768", "op": "shared", "batch": 64, "new": 1, "prefix": 32768, "low": 1,
         "high": 1024, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "sinks": 0},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _draw(rng):
    op = rng.choice(["norm", "fp8", "lora", "shared"])
    c = {"op": op}
    if op == "norm":
        wide = rng.random() < 0.7
        c.update(tokens=_log(rng, 1, 8192), hidden=8 * _log(rng, 8, 1024), residual=rng.random() < 0.8, wide=wide,
                 bytes=not wide or rng.random() < 0.6)
    elif op == "fp8":
        c.update(tokens=_log(rng, 1, 8192), out=16 * _log(rng, 1, 768), hidden=128 * _log(rng, 1, 64))
    elif op == "lora":
        c.update(tokens=_log(rng, 1, 8192), hidden=8 * _log(rng, 16, 1024), out=8 * _log(rng, 16, 1024),
                 rank=rng.choice([8, 16, 16, 32, 64, 128]), adapters=_log(rng, 1, 64),
                 order=rng.choice(["mixed", "runs"]))
    else:
        kv = rng.choice([1, 2, 3, 4, 8])
        high = _log(rng, 1, 4096)
        new = min(rng.choice([1, 1, 1, 2, 3, 4]), high)
        c.update(batch=_log(rng, 1, 128), new=new, prefix=_log(rng, 16, 32768), low=max(new, _log(rng, 1, high)),
                 high=high, heads=kv * rng.choice([1, 2, 3, 4, 5, 8, 16]), kv_heads=kv,
                 dim=rng.choice([64, 128, 128, 256]), page=rng.choice([16, 32, 64, 128]),
                 window=rng.choice([0, 0, 0, _log(rng, 64, 32768)]))
        c.update(sinks=min(c["prefix"], rng.choice([0, 4, 37])) if c["window"] else 0)
    return c


def draw(rng):
    """Cases of the listed ranges; one that would cost more than the largest listed one is drawn again."""
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] > 4.2e8 or w["flops"] > (2.1e11 if c["op"] == "fp8" else 5.0e10):
            continue
        if c["op"] == "lora" and c["tokens"] * c["adapters"] * c["rank"] > 1 << 24:
            continue
        if c["op"] == "shared":
            top = c["prefix"] + c["high"] + c["page"]
            if c["batch"] * c["new"] * c["heads"] * top > MAX_SCORES:
                continue
            if (c["prefix"] + c["batch"] * (c["high"] + c["page"])) * c["kv_heads"] * c["dim"] * 2 > MAX_CACHE_VALUES:
                continue
        return c


def _owned(c):
    """Tokens of each sequence behind the prefix, the new ones among them: of the case, whatever the seed."""
    r = random.Random("%(batch)d behind %(prefix)d, page %(page)d, %(heads)d heads" % c)
    n = [r.randint(c["low"], c["high"]) for _ in range(c["batch"])]
    n[-1] = c["high"]
    return n


def _adapter_of(c):
    """The adapter of each token (-1: none) and the rank of each adapter: of the case, whatever the seed."""
    r = random.Random("%(tokens)d of %(adapters)d, rank %(rank)d" % c)
    T, n = c["tokens"], c["adapters"]
    if c["order"] == "runs":        # prompts one after the other, the last adapter's first, one prompt in eight without
        at = sorted(r.randrange(T + 1) for _ in range(2 * n - 1))
        ids = np.zeros(T, np.int64)
        for i, (a, b) in enumerate(zip([0] + at, at + [T])):
            ids[a:b] = (n - 1 - i) % n if r.random() < 0.875 else -1
    else:
        ids = np.array([r.randrange(n) if r.random() < 0.875 else -1 for _ in range(T)])
    if T == 1:
        ids[0] = n - 1
    ranks = [max(1, c["rank"] // r.choice([1, 1, 1, 2, 4])) for _ in range(n)]
    ranks[-1] = c["rank"]
    return ids, ranks


def _scale(c):
    return c["dim"] ** -0.5


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["tokens"] * c["hidden"]
        out = 2 * c["residual"] + 2 * c["wide"] + c["bytes"]
        scales = 4 * c["tokens"] * -(-c["hidden"] // BLOCK) if c["bytes"] else 0
        return {"bytes": n * (2 + 2 * c["residual"] + out) + 4 * c["hidden"] + scales, "flops": 6 * n}
    if c["op"] == "fp8":
        T, N, K = c["tokens"], c["out"], c["hidden"]
        blocks = T * (K // BLOCK) + -(-N // BLOCK) * (K // BLOCK)
        return {"bytes": T * K + N * K + 4 * blocks + 2 * T * N, "flops": 2 * T * N * K}
    if c["op"] == "lora":
        T, N, K = c["tokens"], c["out"], c["hidden"]
        ids, ranks = _adapter_of(c)
        used = sum(ranks[a] for a in set(ids.tolist()) if a >= 0)
        rows = sum(ranks[a] for a in ids.tolist() if a >= 0)
        with_one = int(np.sum(ids >= 0))
        return {"bytes": with_one * K * 2 + 4 * T * N + used * (K + N) * 2 + 4 * T + 8 * c["adapters"],
                "flops": 2 * rows * (K + N)}
    H, K, D, W, S, P = c["heads"], c["kv_heads"], c["dim"], c["window"], c["sinks"], c["prefix"]
    keys = pairs = 0
    first = P
    for n in _owned(c):
        at = np.arange(P + n - c["new"], P + n, dtype=np.int64)
        if W:
            pairs += int(np.sum(np.minimum(at + 1, W) + np.minimum(S, np.maximum(0, at + 1 - W))))
            lo = max(0, P + n - c["new"] - W + 1)
            keys += P + n - max(lo, P)
            first = min(first, lo)
        else:
            pairs += int(np.sum(at + 1))
            keys += n
            first = 0
    keys += P - first + min(S, first)
    rows = c["batch"] * c["new"] * H
    return {"bytes": keys * K * D * 4 + 2 * rows * D * 2 + 4 * (c["batch"] + -(-P // c["page"])),
            "flops": 4 * D * H * pairs}


def _quantised(v, rows):
    """Values [a, b] in E4M3 with one scale per `rows` x 128 block: bytes and scales."""
    a, b = v.shape
    pad = torch.nn.functional.pad(v, (0, -b % BLOCK, 0, -a % rows))
    t = pad.view(pad.shape[0] // rows, rows, pad.shape[1] // BLOCK, BLOCK)
    s = (t.abs().amax(dim=(1, 3)) / TOP).clamp(min=TINY)
    q = (t / s[:, None, :, None]).clamp(-TOP, TOP).view(pad.shape)[:a, :b].contiguous()
    return q.to(torch.float8_e4m3fn).view(torch.uint8), s


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(std)

    def bf16(*shape, std=1.0):
        return normal(*shape, std=std).to(torch.bfloat16)

    s = {"case": dict(c)}
    if c["op"] == "norm":
        T, H = c["tokens"], c["hidden"]
        channel = normal(H, std=0.6).exp()         # some channels are far larger than others
        s["x"] = bf16(T, H, std=0.5)
        s["residual"] = (normal(T, H) * channel).to(torch.bfloat16) if c["residual"] else None
        s["weight"] = 1.0 + 0.2 * normal(H)
        s["h"] = torch.empty_like(s["x"]) if c["residual"] else None
        s["y"] = torch.empty_like(s["x"]) if c["wide"] else None
        s["q"] = torch.empty((T, H), dtype=torch.uint8, device=DEV) if c["bytes"] else None
        s["scale"] = torch.empty((T, -(-H // BLOCK)), dtype=torch.float32, device=DEV) if c["bytes"] else None
        s["e4m3"] = s["q"].view(torch.float8_e4m3fn) if c["bytes"] else None
    elif c["op"] == "fp8":
        T, N, K = c["tokens"], c["out"], c["hidden"]
        s["x"], s["x_scale"] = _quantised(normal(T, K) * normal(K, std=0.6).exp(), 1)
        s["w"], s["w_scale"] = _quantised(normal(N, K, std=K ** -0.5), BLOCK)
        s["y"] = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "lora":
        T, N, K, R, n = c["tokens"], c["out"], c["hidden"], c["rank"], c["adapters"]
        ids, ranks = _adapter_of(c)
        s["ids"] = torch.from_numpy(ids).to(DEV).to(torch.int32)
        s["ranks"] = torch.tensor(ranks, dtype=torch.int32, device=DEV)
        s["scales"] = 0.5 + torch.rand(n, generator=g, device=DEV)
        s["a"], s["b"] = bf16(n, R, K, std=K ** -0.5), bf16(n, N, R, std=0.5 * R ** -0.5)
        s["x"], s["base"] = bf16(T, K), bf16(T, N)
        s["out"] = torch.empty_like(s["base"])
    else:
        H, K, D, P, B, M = c["heads"], c["kv_heads"], c["dim"], c["page"], c["batch"], c["new"]
        lens = [c["prefix"] + n for n in _owned(c)]
        first, width = c["prefix"] // P, -(-max(lens) // P)       # first page of a sequence's own, and pages in all
        shared = -(-c["prefix"] // P)
        need = shared + sum(-(-n // P) - first for n in lens)
        order = torch.randperm(need + 1, generator=g, device=DEV).cpu()
        table = torch.zeros((B, width), dtype=torch.int32)
        table[:, :shared] = order[:shared]        # the prefix's pages, as in a table that knows no sharing
        at = shared
        for b, n in enumerate(lens):
            m = -(-n // P) - first
            table[b, first:first + m] = order[at:at + m]
            at += m
        s["shared_pages"] = order[:shared].to(torch.int32).to(DEV)
        s["page_table"] = table.to(DEV)
        s["k_cache"], s["v_cache"] = bf16(need + 1, K, D // 8, P, 8), bf16(need + 1, K, P // 8, D, 8)
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["max_len"] = max(lens)
        s["q"] = bf16(B, M, H, D, std=1.5)
        s["out"] = torch.empty_like(s["q"])
    return s


def _bound(s):
    """The call on this state's buffers, its arguments checked and marshalled once, as a serving loop keeps it."""
    from routed_expert_mlp_amd import attention as A
    from routed_expert_mlp_amd import projection as P
    c = s["case"]
    if c["op"] == "norm":
        return P.bind_norm(s["x"], s["weight"], EPS, residual=s["residual"], h_out=s["h"], y_out=s["y"], q_out=s["q"],
                           q_scale=s["scale"])
    if c["op"] == "fp8":
        return P.bind_fp8(s["x"], s["x_scale"], s["w"], s["w_scale"], s["y"])
    if c["op"] == "lora":
        return P.bind_lora(P.Adapters(a=s["a"], b=s["b"], ranks=s["ranks"], scales=s["scales"]), s["x"], s["ids"],
                           s["base"], s["out"])
    cfg = A.AttnConfig(n_heads=c["heads"], n_kv_heads=c["kv_heads"], head_dim=c["dim"], page_size=c["page"],
                       rotary_dim=0, rope_style=A.ROPE_HALF, norm_eps=EPS, scale=_scale(c), window=c["window"],
                       n_sinks=c["sinks"])
    return A.bind_decode_shared(cfg, A.KVCache(s["k_cache"], s["v_cache"]), s["q"], s["seq_lens"], s["page_table"],
                                s["max_len"], s["shared_pages"], c["prefix"], s["out"])


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        call = s.get("call")
        if call is None:
            call = s["call"] = _bound(s)
        call()
    else:
        {"norm": _plain_norm, "fp8": _plain_fp8, "lora": _plain_lora, "shared": _plain_shared}[op](s)
    if op == "norm":
        return {"h": s["h"], "y": s["y"], "q": s["e4m3"], "scale": s["scale"]}
    return s["y"] if op == "fp8" else s["out"]


def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
        s["h"].copy_(h)
    y = h * (h.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["weight"]
    if s["y"] is not None:
        s["y"].copy_(y)
    if s["q"] is not None:
        T, H = y.shape
        t = torch.nn.functional.pad(y, (0, -H % BLOCK)).view(T, -1, BLOCK)
        scale = (t.abs().amax(-1, keepdim=True) / TOP).clamp(min=TINY)
        s["scale"].copy_(scale[..., 0])
        s["e4m3"].copy_((t / scale).clamp(-TOP, TOP).view(T, -1)[:, :H])


def _plain_fp8(s):
    N = s["w"].shape[0]
    x = s["x"].view(torch.float8_e4m3fn).float() * s["x_scale"].repeat_interleave(BLOCK, 1)
    w = s["w"].view(torch.float8_e4m3fn).float()
    w = w * s["w_scale"].repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)
    s["y"].copy_(x @ w.T)


def _plain_lora(s):
    c = s["case"]
    n, R, N = c["adapters"], c["rank"], c["out"]
    live = torch.arange(R, device=DEV) < s["ranks"][:, None]                       # [n, R]
    a = s["a"].float().masked_fill(~live[:, :, None], 0.0).view(n * R, -1)
    b = s["b"].float().masked_fill(~live[:, None, :], 0.0).transpose(1, 2).reshape(n * R, N)
    low = (s["x"].float() @ a.T).view(-1, n, R)                                     # of every adapter
    mine = (s["ids"][:, None] == torch.arange(n, device=DEV)) * s["scales"]         # and the token's own, scaled
    s["out"].copy_(s["base"].float() + (low * mine[..., None]).view(-1, n * R) @ b)


def _plain_shared(s):
    c = s["case"]
    H, K, D, W, S, B, M = c["heads"], c["kv_heads"], c["dim"], c["window"], c["sinks"], c["batch"], c["new"]
    G, P = H // K, c["prefix"]
    first = P // c["page"]

    def keys(pages):
        return s["k_cache"][pages].transpose(-2, -3).flatten(-2).float()            # [.., page, K, token, D]

    def values(pages):
        return s["v_cache"][pages].transpose(-1, -2).flatten(-3, -2).float()

    lead, rest = s["shared_pages"].long(), s["page_table"][:, first:].long()
    kp, vp = (t.transpose(0, 1).reshape(K, -1, D)[:, :P] for t in (keys(lead), values(lead)))
    ko, vo = (t.transpose(1, 2).reshape(B, K, -1, D) for t in (keys(rest), values(rest)))
    q = s["q"].float().view(B, M, K, G, D) * _scale(c)
    at = (s["seq_lens"].long() - M)[:, None] + torch.arange(M, device=DEV)          # [B, M]
    key_p = torch.arange(P, device=DEV)
    key_o = torch.arange(ko.shape[2], device=DEV) + first * c["page"]
    sp = torch.matmul(q.permute(2, 0, 1, 3, 4).reshape(K, B * M * G, D), kp.transpose(1, 2)).view(K, B, M, G, P)
    so = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(B, K, M * G, D), ko.transpose(2, 3)).view(B, K, M, G, -1)
    hide_p = key_p > at[..., None]
    hide_o = (key_o > at[..., None]) | (key_o < P)
    if W:
        hide_p = hide_p | ((at[..., None] - key_p >= W) & (key_p >= S))
        hide_o = hide_o | ((at[..., None] - key_o >= W) & (key_o >= S))
    sp.masked_fill_(hide_p[None, :, :, None], -math.inf)
    so.masked_fill_(hide_o[:, None, :, None], -math.inf)
    top = torch.maximum(sp.amax(-1), so.amax(-1).transpose(0, 1)).clamp(min=-1e30)   # [K, B, M, G]
    sp.sub_(top[..., None]).exp_()
    so.sub_(top.transpose(0, 1)[..., None]).exp_()
    o = torch.matmul(sp.view(K, B * M * G, P), vp).view(K, B, M, G, D).transpose(0, 1)
    o = o + torch.matmul(so.view(B, K, M * G, -1), torch.where(key_o[:, None] < P, 0.0, vo)).view(B, K, M, G, D)
    total = sp.sum(-1).transpose(0, 1) + so.sum(-1)
    o = o / total.clamp(min=1e-30)[..., None]
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(B, M, H, D))


def exact(case, seed):
    """The definitions in 64 bits, written block by block and sequence by sequence."""
    s = prepare(case, seed)
    return {"norm": _exact_norm, "fp8": _exact_fp8, "lora": _exact_lora, "shared": _exact_shared}[case["op"]](s)


def _to_e4m3(v):
    """The nearest E4M3 value of each (ties to the even one), for |v| <= 448."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.pow(2.0, e - 3)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def _exact_norm(s):
    h = s["x"].double()
    if s["residual"] is not None:
        h = h + s["residual"].double()
    H = h.shape[1]
    y = s["weight"].double() * h / torch.sqrt(torch.sum(h * h, dim=1, keepdim=True) / H + EPS)
    out = {"h": None if s["h"] is None else h, "y": None if s["y"] is None else y, "q": None, "scale": None}
    if s["q"] is not None:
        q, scales = [], []
        for at in range(0, H, BLOCK):
            part = y[:, at:at + BLOCK]
            scale = torch.clamp(part.abs().max(dim=1).values / TOP, min=TINY)
            scales.append(scale)
            q.append(_to_e4m3(part / scale[:, None]))
        out.update(q=torch.cat(q, dim=1), scale=torch.stack(scales, dim=1))
    return out


def _exact_fp8(s):
    x, w = (s[k].view(torch.float8_e4m3fn).double() for k in ("x", "w"))
    y = torch.zeros((x.shape[0], w.shape[0]), dtype=torch.float64, device=DEV)
    rows = torch.arange(w.shape[0], device=DEV) // BLOCK
    for j in range(x.shape[1] // BLOCK):
        at = slice(j * BLOCK, j * BLOCK + BLOCK)
        y += (x[:, at] @ w[:, at].T) * s["x_scale"][:, j:j + 1].double() * s["w_scale"][rows, j].double()
    return y


def _exact_lora(s):
    out = s["base"].double()
    for a, (rank, scale) in enumerate(zip(s["ranks"].tolist(), s["scales"].double())):
        mine = torch.nonzero(s["ids"] == a)[:, 0]
        if mine.numel():
            low = s["x"][mine].double() @ s["a"][a, :rank].double().T
            out[mine] += scale * (low @ s["b"][a, :, :rank].double().T)
    return out


def _exact_shared(s):
    c = s["case"]
    H, K, D, P, W, S, M = c["heads"], c["kv_heads"], c["dim"], c["page"], c["window"], c["sinks"], c["new"]
    G, lead = H // K, c["prefix"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    where = torch.arange(lead, device=DEV)
    page, at = s["shared_pages"].long()[where // P], where % P
    for h in range(K):
        kp = s["k_cache"][page, h, :, at].reshape(lead, D).double()
        vp = s["v_cache"][page, h, at // 8, :, at % 8].double()
        for b, n in enumerate(s["seq_lens"].tolist()):
            mine = torch.arange(lead, n, device=DEV)
            p, j = s["page_table"][b].long()[mine // P], mine % P
            k = torch.cat([kp, s["k_cache"][p, h, :, j].reshape(n - lead, D).double()])
            v = torch.cat([vp, s["v_cache"][p, h, j // 8, :, j % 8].double()])
            pos = torch.arange(n - M, n, device=DEV)[:, None]
            key = torch.arange(n, device=DEV)[None, :]
            hidden = key > pos
            if W:
                hidden |= (pos - key >= W) & (key >= S)
            a = s["q"][b, :, h * G:h * G + G].double() @ k.T * _scale(c)            # [M, G, n]
            a.masked_fill_(hidden[:, None], -math.inf)
            out[b, :, h * G:h * G + G] = torch.softmax(a, dim=-1) @ v
    return out
