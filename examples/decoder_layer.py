"""One decoder layer out of the library's two halves: attention over a paged cache, then the routed MLP.

    python examples/decoder_layer.py

A few sequences of different lengths go through the layer as a server would
take them: their prompts in two pieces (moe_attn_prepare, moe_attn_prefill,
moe_mlp_prefill), then several steps of one new token each and one verify step
of three (moe_attn_prepare, moe_attn_decode, moe_mlp_decode).  The dense
projections and the row norms around them are plain torch.  Weights are random.

At the end the same tokens go through the layer as whole prompts, and the two
results are compared; the MLP half is compared where both runs route alike,
since a token whose expert scores nearly tie may go to other experts.
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

from routed_expert_mlp_amd import attention as A  # noqa: E402
from routed_expert_mlp_amd import capi  # noqa: E402


class Pages:
    """Hands out pages of a cache; one row of the table per sequence."""

    def __init__(self, n_pages, page_size, sequences, max_pages, device):
        self.free, self.page_size = list(range(n_pages))[::-1], page_size
        self.rows = [[] for _ in range(sequences)]
        self.table = torch.zeros((sequences, max_pages), dtype=torch.int32, device=device)

    def grow(self, b, length):
        """Pages for tokens 0 .. length-1 of sequence b."""
        while len(self.rows[b]) * self.page_size < length:
            self.rows[b].append(self.free.pop())
            self.table[b, len(self.rows[b]) - 1] = self.rows[b][-1]

    def slots(self, b, first, last):
        P = self.page_size
        return [self.rows[b][t // P] * P + t % P for t in range(first, last)]


class DecoderLayer:
    """x + attention(norm(x)), then + MLP(norm(.)); bf16 rows [T, hidden]."""

    def __init__(self, attn: A.AttnConfig, mlp: capi.Config, mlp_weights: capi.Weights, max_positions, device, seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        H, D = mlp.hidden, attn.head_dim

        def mat(rows, cols):
            return (torch.randn((rows, cols), generator=g, device=device) * cols ** -0.5).to(torch.bfloat16)

        self.attn, self.mlp, self.mlp_weights, self.device = attn, mlp, mlp_weights, device
        self.w_qkv = mat((attn.n_heads + 2 * attn.n_kv_heads) * D, H)
        self.w_out = mat(H, attn.n_heads * D)
        self.q_norm = 1.0 + 0.1 * torch.randn(D, generator=g, device=device)
        self.k_norm = 1.0 + 0.1 * torch.randn(D, generator=g, device=device)
        R = attn.rotary_dim
        angle = torch.arange(max_positions, device=device, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, R, 2, device=device, dtype=torch.float64) / R)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()

    @staticmethod
    def row_norm(x):
        f = x.float()
        return (f * (f.square().mean(-1, keepdim=True) + 1e-6).rsqrt()).to(torch.bfloat16)

    def forward(self, x, cache, pages, lens, new):
        """The last `new` tokens of each sequence, of lens[b] tokens with them: x [sum(new), hidden] ->
        (layer output, row after the attention half, expert ids)."""
        c, T = self.attn, x.shape[0]
        slots, positions = [], []
        for b, (n, m) in enumerate(zip(lens, new)):
            pages.grow(b, n)
            slots += pages.slots(b, n - m, n)
            positions += list(range(n - m, n))

        def dev(v, dtype):
            return torch.tensor(v, dtype=dtype, device=self.device)

        qkv = torch.nn.functional.linear(self.row_norm(x), self.w_qkv)
        q = torch.empty((T, c.n_heads, c.head_dim), dtype=torch.bfloat16, device=self.device)
        A.moe_attn_prepare(c, cache, qkv, self.q_norm, self.k_norm, self.cos_sin, dev(positions, torch.int32),
                           dev(slots, torch.int64), q)
        out = torch.empty_like(q)
        decode = len(set(new)) == 1 and new[0] <= A.DECODE_MAX_Q
        if decode:
            shape = (len(new), new[0], c.n_heads, c.head_dim)
            A.moe_attn_decode(c, cache, q.view(shape), dev(lens, torch.int32), pages.table, max(lens), out.view(shape))
        else:
            cu = [0]
            for m in new:
                cu.append(cu[-1] + m)
            A.moe_attn_prefill(c, cache, q, dev(cu, torch.int32), max(new), dev(lens, torch.int32), pages.table,
                               max(lens), out)
        h = x + torch.nn.functional.linear(out.view(T, -1), self.w_out)
        y = torch.empty_like(h)
        ids = torch.empty((T, self.mlp.top_k), dtype=torch.int32, device=self.device)
        mlp = capi.moe_mlp_decode if decode and T <= capi.DECODE_MAX_T else capi.moe_mlp_prefill
        mlp(self.mlp, self.mlp_weights, self.row_norm(h), y, ids)
        return h + y, h, ids


def tiny_mlp(device):
    """A small routed MLP of the synthetic recipe: config and weights."""
    import numpy as np

    import synth
    w = synth.workload("tiny_decode")

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(device)

    def bf(bits):
        return dev(bits.view(np.int16)).view(torch.bfloat16)

    experts = [synth.expert_w13(w, e) + synth.expert_w2(w, e) for e in range(w.E)]
    q13, s13, q2, s2 = (dev(np.stack([x[i] for x in experts])) for i in range(4))
    weights = capi.Weights(router_w=dev(synth.router_weight(w)), router_bias=dev(synth.router_bias(w)), w13_q=q13,
                           w13_s=s13, w13_g=dev(synth.w13_globals(w)), w2_q=q2, w2_s=s2, w2_g=dev(synth.w2_globals(w)),
                           shared_w13=bf(synth.shared_w13(w)), shared_w2=bf(synth.shared_w2(w)))
    cfg = capi.Config(kind=capi.KIND_ROUTED, hidden=w.H, moe_intermediate=w.I, num_experts=w.E, top_k=w.K,
                      n_shared_experts=1, shared_intermediate=w.Is, dense_intermediate=0, routed_scaling_factor=w.rsf,
                      swiglu_limit=w.swiglu_limit)
    return cfg, weights


def serve(device="cuda", prompts=(70, 9, 133), steps=4, verify=3, window=0, n_sinks=0):
    """Runs the sequences step by step and as whole prompts; returns the largest relative differences of the rows
    after the attention half and after the layer, and the share of tokens routed alike."""
    cfg, weights = tiny_mlp(device)
    attn = A.AttnConfig(n_heads=8, n_kv_heads=2, head_dim=64, page_size=16, rotary_dim=64, rope_style=A.ROPE_HALF,
                        norm_eps=1e-6, scale=64 ** -0.5, window=window, n_sinks=n_sinks)
    layer = DecoderLayer(attn, cfg, weights, 4096, device)
    B, total = len(prompts), [p + steps + verify for p in prompts]
    g = torch.Generator(device=device)
    g.manual_seed(1)
    tokens = [torch.randn((n, cfg.hidden), generator=g, device=device).to(torch.bfloat16) for n in total]

    def state():
        need = sum(-(-n // attn.page_size) for n in total)
        return A.new_cache(attn, need, device), Pages(need, attn.page_size, B, -(-max(total) // attn.page_size), device)

    cache, pages = state()
    lens, rows = [0] * B, [[] for _ in range(B)]
    work = [[p // 2 for p in prompts], [p - p // 2 for p in prompts]] + [[1] * B] * steps + [[verify] * B]
    for new in work:
        x = torch.cat([t[n:n + m] for t, n, m in zip(tokens, lens, new)])
        lens = [n + m for n, m in zip(lens, new)]
        res = layer.forward(x, cache, pages, lens, new)
        at = 0
        for b, m in enumerate(new):
            rows[b].append([r[at:at + m] for r in res])
            at += m
    cache, pages = state()
    whole = layer.forward(torch.cat(tokens), cache, pages, total, total)
    stepped = [torch.cat([piece[i] for b in range(B) for piece in rows[b]]) for i in range(3)]
    alike = (whole[2] == stepped[2]).all(dim=1)

    def far(a, b):
        return float((a.float() - b.float()).norm(dim=1).div(b.float().norm(dim=1)).max())

    return far(stepped[1], whole[1]), far(stepped[0][alike], whole[0][alike]), float(alike.float().mean())


if __name__ == "__main__":
    for kw in ({}, {"window": 40, "n_sinks": 4}):
        attention, layer, alike = serve(**kw)
        torch.cuda.synchronize()
        print(f"window {kw.get('window', 0)}: stepped against whole, largest relative difference of a row: "
              f"attention half {attention:.1e}, layer {layer:.1e}; routed alike {100 * alike:.1f}%")
        if attention > 2e-2 or layer > 5e-2 or alike < 0.9:
            sys.exit("the two runs differ")
