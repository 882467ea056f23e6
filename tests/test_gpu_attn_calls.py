"""GPU tests of what a call of the attention operators promises beside its
ordinary use: bounds below the lengths, values that are not finite, batches far
more ragged than usual, one workspace for calls of many sizes, the stream that a
bound call runs on."""
import pytest
import torch

from attn_util import assert_within, make_batch
from routed_expert_mlp_amd import attention as A
from test_gpu_attn import DEV, cache_of, check, config, run_prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kv,dim,new,lens,max_q,window,sinks", [
    (8, 2, 128, [70, 5, 90], [200, 40, 300], 33, 0, 0),
    (8, 2, 64, [70, 5, 90], [200, 40, 300], 33, 40, 3),
    (4, 1, 256, [9], [9], 1, 0, 0),
    (8, 2, 128, [40, 2], [3000, 2], 5, 0, 0),            # in parts
    (8, 2, 64, [40, 30], [4000, 20], 7, 900, 5),         # in parts; the second one's first positions are below zero
])
def test_prefill_of_more_new_tokens_than_max_q(heads, kv, dim, new, lens, max_q, window, sinks):
    """The first max_q new tokens keep their own positions; the others' rows are not written."""
    b = make_batch(config(heads, kv, dim, 16, window=window, sinks=sinks), lens, new, seed=dim + max_q)
    what = f"prefill of {new} new tokens, max_q {max_q}, window {window}+{sinks}"
    print(f"[case] {what}", flush=True)
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    q = b.q.to(DEV)
    out = torch.full_like(q, 7.0)
    A.moe_attn_prefill(b.cfg, cache_of(b), q, torch.tensor(cu, dtype=torch.int32, device=DEV), max_q,
                       torch.tensor(lens, dtype=torch.int32, device=DEV), b.table.to(DEV), max(lens), out)
    got = out.double().cpu().numpy()
    for i, (want, bound) in enumerate(b.expected()):
        n = min(max_q, new[i])
        assert_within(got[cu[i]:cu[i] + n], want[:n], bound[:n], f"{what}, sequence {i}")
        assert (got[cu[i] + n:cu[i + 1]] == 7.0).all(), f"{what}, sequence {i}: a row past max_q was written"


@pytest.mark.parametrize("style", [A.ROPE_HALF, A.ROPE_INTERLEAVED])
@pytest.mark.parametrize("dim,rotary", [(64, 16), (128, 64), (256, 0), (256, 128)])
def test_prepare_passes_dims_past_the_rotation_through(dim, rotary, style):
    """Without a norm, dims that are not rotated go out as they came in, whatever they are: infinities, NaN and
    negative zeros stay in their own places."""
    T, heads, kv, page = 21, 4, 2, 16
    cfg = config(heads, kv, dim, page, rotary=rotary, style=style)
    print(f"[case] prepare, {dim} dims of which {rotary} are rotated, style {style}, values not finite", flush=True)
    g = torch.Generator().manual_seed(dim + rotary)
    x = torch.randn((T, heads + 2 * kv, dim), generator=g).to(torch.bfloat16)
    for i, odd in enumerate((float("inf"), -float("inf"), float("nan"), -0.0)):
        at = torch.randint(rotary, dim, (T, heads + kv), generator=g)
        keep = torch.rand((T, heads + kv), generator=g) < 0.7
        for t, h in keep.nonzero().tolist():
            x[t, h, at[t, h]] = odd
    qkv = x.reshape(T, -1).to(DEV)
    k, v = (torch.zeros(s, dtype=torch.bfloat16, device=DEV) for s in A.cache_shapes(cfg, 2))
    q = torch.zeros((T, heads, dim), dtype=torch.bfloat16, device=DEV)
    angle = torch.randn((32, max(rotary // 2, 1)), generator=g)
    table = torch.cat([angle.cos(), angle.sin()], dim=1)[:, :rotary].contiguous().to(DEV) if rotary else None
    positions = torch.arange(T, dtype=torch.int32, device=DEV) if rotary else None
    A.moe_attn_prepare(cfg, A.KVCache(k, v), qkv, None, None, table, positions, torch.arange(T, device=DEV), q)
    keys = k.permute(0, 3, 1, 2, 4).reshape(-1, kv, dim)[:T]
    for got, want in ((q.cpu(), x[:, :heads]), (keys.cpu(), x[:, heads:heads + kv])):
        assert torch.isfinite(got[..., :rotary].float()).all(), "a value that is not rotated reached the rotated dims"
        got, want = got[..., rotary:].contiguous(), want[..., rotary:].contiguous()
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan)
        assert torch.equal(got.view(torch.int16)[~nan], want.view(torch.int16)[~nan])


def test_prefill_of_one_long_piece_among_thousands_of_sequences():
    """Sequences times the longest piece is past what a call may have of tokens; the tokens themselves are few."""
    B, long = 8192, 1024
    new = [1 if b % 3 else 0 for b in range(B)]
    new[5000] = long
    lens = [n + b % 5 for b, n in enumerate(new)]
    b = make_batch(config(8, 2, 64, 16), lens, new, seed=22)
    print(f"[case] prefill of {sum(new)} tokens of {B} sequences, one of {long}", flush=True)
    got, row = run_prefill(b).double().cpu().numpy(), 0
    worst = 0.0
    for want, bound in b.expected():
        err = abs(got[row:row + want.shape[0]] - want)
        assert (err <= bound).all(), f"row {row} and on"
        worst = max(worst, float((err / bound.clip(min=1e-300)).max(initial=0.0)))
        row += want.shape[0]
    print(f"[parity] prefill, one long piece among {B} sequences: worst error {worst:.3f} of its bound", flush=True)


@pytest.mark.parametrize("heads,kv,dim", [(32, 8, 128), (8, 2, 64), (16, 2, 256)])
def test_one_workspace_for_calls_of_many_sizes(heads, kv, dim):
    """A workspace of the bound of the largest sizes serves smaller calls, whether in parts or whole; what lies behind
    the bytes that a call asks for stays as it was."""
    cfg = config(heads, kv, dim, 32)
    B, max_q, max_len = 4, 600, 6000
    most = [A.moe_attn_workspace_bound(cfg, B * max_q, B, max_q, max_len, True),
            A.moe_attn_workspace_bound(cfg, B * 4, B, 4, max_len, False)]
    ws = torch.full((max(most),), 255, dtype=torch.uint8, device=DEV)      # NaN in every float
    for new, lens in (([1], [6000]), ([7], [5000]), ([90], [3000]), ([20, 0, 3], [2500, 10, 40]), ([200], [200]),
                      ([4, 4, 4, 4], [6000, 3, 900, 4]), ([2, 2], [30, 6000])):
        b = make_batch(cfg, lens, new, seed=dim + sum(lens))
        q, table = b.q.to(DEV), b.table.to(DEV)
        n = torch.tensor(lens, dtype=torch.int32, device=DEV)
        cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=DEV)
        for form in ("prefill", "decode"):
            if form == "decode" and (len(set(new)) > 1 or new[0] > 4):
                continue
            need = A.moe_attn_workspace_size(cfg, sum(new), len(new), max(new), max(lens), form == "prefill")
            print(f"[case] {form} of {new} behind {lens}, {heads}/{kv}x{dim}: {need} bytes of {ws.numel()}", flush=True)
            out = torch.full_like(q, float("nan"))
            ws.fill_(255)
            if form == "prefill":
                A.moe_attn_prefill(cfg, cache_of(b), q, cu, max(new), n, table, max(lens), out, ws)
            else:
                shape = (len(new), new[0], heads, dim)
                A.moe_attn_decode(cfg, cache_of(b), q.view(shape), n, table, max(lens), out.view(shape), ws)
            assert torch.all(ws[need:] == 255), "the call wrote behind the bytes that it asks for"
            check(b, out, f"{form} with one workspace")


def bound_calls(b):
    """Bound decode and prefill (both in parts) of one batch of single tokens, and what they read and write."""
    q = b.q.to(DEV)
    lens, table = torch.tensor(b.lens, dtype=torch.int32, device=DEV), b.table.to(DEV)
    cu = torch.arange(len(b.lens) + 1, dtype=torch.int32, device=DEV)
    outs = [torch.zeros_like(q), torch.zeros_like(q)]
    q4, o4 = q.view(-1, 1, *q.shape[1:]), outs[0].view(-1, 1, *q.shape[1:])
    cache = cache_of(b)
    return q, outs, [A.bind_decode(b.cfg, cache, q4, lens, table, max(b.lens), o4),
                     A.bind_prefill(b.cfg, cache, q, cu, 1, lens, table, max(b.lens), outs[1])]


def test_bound_calls_run_on_the_stream_of_the_call():
    """Bound under one stream and called under another that is still busy making the queries."""
    b = make_batch(config(8, 2, 128, 16), [5000, 333], [1, 1], seed=21)
    print("[case] bound calls under another stream", flush=True)
    q, outs, calls = bound_calls(b)
    first = q.clone()
    q.zero_()
    x = torch.randn((8192, 8192), device=DEV).to(torch.bfloat16)
    x @ x
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(20):
            x @ x                                    # about 20 ms
        q.copy_(first)
        for c in calls:
            c()
    torch.cuda.synchronize()
    for out, name in zip(outs, ("decode", "prefill")):
        got, row = out.double().cpu().numpy(), 0
        for i, (want, bound) in enumerate(b.expected()):
            assert_within(got[row:row + 1], want, bound, f"bound {name} under another stream, sequence {i}")
            row += 1


def test_bound_calls_are_captured_under_the_capturing_stream():
    """Bound before, under the default stream, and captured: every replay writes the outputs."""
    b = make_batch(config(8, 2, 128, 16), [5000, 333], [1, 1], seed=23)
    print("[case] bound calls in a graph", flush=True)
    q, outs, calls = bound_calls(b)
    for c in calls:
        c()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c in calls:
            c()
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o.view(torch.int16), w.view(torch.int16))


def test_bound_calls_refuse_another_device(monkeypatch):
    b = make_batch(config(8, 2, 128, 16), [50], [1], seed=24)
    print("[case] bound calls, another device", flush=True)
    other, now = 0, torch._C._cuda_getDevice
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now() + other)
    calls = bound_calls(b)[2]
    other = 1
    for c in calls:
        with pytest.raises(ValueError):
            c()
    other = 0
    torch.cuda.synchronize()
