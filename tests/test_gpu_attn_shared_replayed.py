"""GPU test of decode behind a shared prefix in a captured graph whose lengths change between the replays: whole batches,
padded rows, sequences that end inside the prefix, with and without a window, and a value of the prefix that is not
finite.  Each replay has the bits of an eager call."""
import pytest
import torch

from routed_expert_mlp_amd import attention as A
from test_gpu_attn_shared import DEV, config

pytestmark = pytest.mark.gpu


# the prefix in the launch of the own keys; in wide blocks of 4 wavefronts, and of 8
@pytest.mark.parametrize("heads,kv,dim,page,shared,B", [(8, 2, 128, 16, 203, 20), (16, 1, 256, 64, 4100, 64),
                                                        (64, 4, 128, 64, 9001, 64)])
@pytest.mark.parametrize("window", [0, 90])
def test_lengths_change_between_replays(heads, kv, dim, page, shared, B, window):
    cfg, own = config(heads, kv, dim, page, window, 3 if window else 0), 128
    g = torch.Generator(device=DEV).manual_seed(B)
    lead, first, width = -(-shared // page), shared // page, -(-(shared + own) // page)
    n = lead + B * (width - first)
    cache = A.KVCache(*(torch.randn(s, generator=g, device=DEV).to(torch.bfloat16) for s in A.cache_shapes(cfg, n)))
    key = shared // 2
    cache.v[key // page, 0, key % page // 8, 5, key % 8] = float("inf")
    pages = torch.arange(lead, dtype=torch.int32, device=DEV)
    table = torch.zeros((B, width), dtype=torch.int32, device=DEV)
    table[:, first:] = lead + torch.arange(n - lead, dtype=torch.int32, device=DEV).view(B, -1)
    q = torch.randn((B, 1, heads, dim), generator=g, device=DEV).to(torch.bfloat16)
    lens, out = torch.full((B,), shared + 1, dtype=torch.int32, device=DEV), torch.empty_like(q)
    call = A.bind_decode_shared(cfg, cache, q, lens, table, shared + own, pages, shared, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    at = torch.arange(B, device=DEV)
    for what, now in (("behind", shared + 1 + at % own), ("padded", torch.where(at % 3 == 0, 0, shared + 1 + at % own)),
                      ("inside", (at * 977) % (shared + own) + 1), ("none", at * 0), ("again", shared + own - at % own)):
        lens.copy_(now)
        out.fill_(float("nan"))
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        want = torch.empty_like(q)
        A.moe_attn_decode_shared(cfg, cache, q, lens, table, shared + own, pages, shared, want)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), what
        sees = (now > key) & ((now - 1 - key < window) if window else True)
        odd = ~torch.isfinite(got.float()).flatten(1).all(1)
        assert torch.equal(odd, sees), f"{what}: who has the value that is not finite"
        assert bool((got[now == 0] == 0).all()), f"{what}: padded rows"
