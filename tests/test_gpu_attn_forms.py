"""GPU parity of the forms of the attention kernels that only long or large calls take: prefill blocks that go
through more tiles than the ring of page ids holds, both block sizes at 128 dims, whole and in parts; wide
groups of 256 dims in decode; prepare with several heads a block; a captured prepare that has to store."""
import numpy as np
import pytest
import torch

from attn_marks import attend_torch, mark_values
from attn_util import assert_within, make_batch
from oracle import attn_oracle as AO
from routed_expert_mlp_amd import attention as A
from test_gpu_attn import DEV, cache_of, check, config, prepare_case, run_decode, run_prefill

pytestmark = pytest.mark.gpu


def check_long(b, out, what):
    got, row = out.double().cpu().numpy().reshape(-1, b.cfg.n_heads, b.cfg.head_dim), 0
    for i, (q, k, v) in enumerate(zip(b.qs, b.keys, b.values)):
        if q.shape[0] and k.shape[0]:
            want, bound = attend_torch(b.cfg, q, k, v, DEV)
            assert_within(got[row:row + q.shape[0]], want, bound, f"{what} sequence {i} of {b.lens[i]}")
        else:
            assert (got[row:row + q.shape[0]] == 0).all()
        row += q.shape[0]


WHOLE = [
    # heads, kv, dim, page, new, lens, window, sinks: more column blocks than places, so no parts
    (32, 8, 64, 32, [2100], [6600], 0, 0),                      # 104 tiles of 64 keys: ids past the 64 held, twice refilled
    (32, 8, 64, 16, [300, 1900, 5], [6400, 6300, 4], 5000, 150),
    (32, 8, 128, 64, [2100], [6700], 0, 0),                     # 8 wavefronts, 105 tiles of 64 keys
    (32, 8, 128, 16, [2100], [9000], 6300, 150),                # the same with a window and sinks
    (32, 8, 128, 16, [900, 1400], [5000, 6500], 0, 0),
    (32, 8, 128, 32, [2048], [2048], 0, 0),                     # 4 wavefronts, 64 tiles of 32 keys
    (32, 8, 128, 16, [3000], [3000], 1024, 4),                  # 4 wavefronts, a window
    (16, 2, 256, 64, [2100], [3500], 0, 0),                     # 110 tiles of 32 keys
    (16, 2, 256, 128, [2100], [5000], 3300, 70),
]


@pytest.mark.parametrize("heads,kv,dim,page,new,lens,window,sinks", WHOLE)
def test_prefill_long_blocks(heads, kv, dim, page, new, lens, window, sinks):
    cfg = config(heads, kv, dim, page, window=window, sinks=sinks)
    assert A.moe_attn_workspace_size(cfg, sum(new), len(new), max(new), max(lens), True) == 0, "not whole"
    what = f"long prefill {heads}/{kv}x{dim} page {page} window {window}+{sinks}"
    print(f"[case] {what} new {new} lens {lens}", flush=True)
    b = mark_values(make_batch(cfg, lens, new, seed=dim + len(new)))
    check_long(b, run_prefill(b, pad=1), what)


PARTS = [
    (32, 8, 64, 64, [500], [20000], 0, 0),                      # parts of about 79 tiles
    (32, 8, 128, 64, [500], [20000], 0, 0),
    (32, 8, 128, 128, [400], [14000], 12000, 99),
    (16, 4, 256, 64, [180], [9000], 0, 0),
    (8, 2, 128, 16, [60], [30001], 0, 0),
]


@pytest.mark.parametrize("heads,kv,dim,page,new,lens,window,sinks", PARTS)
def test_prefill_long_parts(heads, kv, dim, page, new, lens, window, sinks):
    cfg = config(heads, kv, dim, page, window=window, sinks=sinks)
    assert A.moe_attn_workspace_size(cfg, sum(new), len(new), max(new), max(lens), True) > 0, "not in parts"
    what = f"long prefill in parts {heads}/{kv}x{dim} page {page} window {window}+{sinks}"
    print(f"[case] {what} new {new} lens {lens}", flush=True)
    b = mark_values(make_batch(cfg, lens, new, seed=dim + len(new)))
    check_long(b, run_prefill(b), what)


@pytest.mark.parametrize("heads,kv,dim,page,new,lens,window,sinks", [
    (4, 1, 128, 64, 1, [30001], 0, 0),
    (8, 2, 64, 16, 1, [20000, 77], 0, 0),
    (8, 2, 256, 64, 2, [9000, 4097], 0, 0),
    (4, 1, 64, 64, 1, [20000], 9000, 17),
])
def test_decode_long(heads, kv, dim, page, new, lens, window, sinks):
    cfg = config(heads, kv, dim, page, window=window, sinks=sinks)
    what = f"long decode {heads}/{kv}x{dim} page {page} window {window}+{sinks}"
    print(f"[case] {what} lens {lens}", flush=True)
    b = mark_values(make_batch(cfg, lens, [new] * len(lens), seed=dim))
    check(b, run_decode(b), what)


@pytest.mark.parametrize("heads,kv,new,window", [(48, 1, 1, 0), (24, 2, 4, 0), (16, 2, 8, 3000), (35, 1, 1, 40)])
def test_decode_wide_groups_of_256_dims(heads, kv, new, window):
    """More than 32 rows of a key/value head, at 256 dims: several blocks that read the same keys."""
    lens = [8000, 0, 5, 33, 64, 700, 1, 2050, 8]
    b = make_batch(config(heads, kv, 256, 64, window=window, sinks=3), lens, [new] * len(lens), seed=heads)
    print(f"[case] decode of {new * heads // kv} rows a head of 256 dims, window {window}", flush=True)
    check(b, run_decode(b), "decode, wide groups of 256 dims")


# A block of moe_attn_prepare goes through (heads + 2 kv) * ceil(T / (2048 / dim)) / 1536 heads, 1 to 8 of them.
MANY = [
    # T, heads, kv, dim, page, rotary, style, norm, first slot (None: shuffled)
    (1003, 15, 5, 256, 32, 128, A.ROPE_HALF, "both", 3),             # 2: a block with the last query and the first key
    (1531, 35, 7, 128, 16, 128, A.ROPE_INTERLEAVED, "both", 0),      # 3
    (3001, 35, 7, 128, 64, 64, A.ROPE_HALF, "k", None),              # 5: keys and values in a block
    (4100, 15, 5, 64, 32, 64, A.ROPE_HALF, "q", 16),                 # 2
    (4003, 15, 5, 256, 64, 256, A.ROPE_INTERLEAVED, "both", None),   # 8: queries, keys and values over four blocks
    (2500, 29, 1, 128, 128, 0, A.ROPE_HALF, "k", 5),                 # 3: a block with two queries and the key
]


@pytest.mark.parametrize("T,heads,kv,dim,page,rotary,style,norm,first", MANY)
def test_prepare_several_heads_a_block(T, heads, kv, dim, page, rotary, style, norm, first):
    rng = np.random.default_rng(T)
    n_pages = -(-(T + (first or 0)) // page) + 2
    if first is None:
        slots = [int(s) for s in rng.permutation(n_pages * page)[:T]]
        positions = [int(p) for p in rng.integers(0, 5000, T)]
    else:
        order = rng.permutation(n_pages)
        slots = [int(order[(first + t) // page]) * page + (first + t) % page for t in range(T)]
        positions = list(range(first, first + T))
    print(f"[case] prepare T={T} {heads}/{kv}x{dim}, several heads a block", flush=True)
    prepare_case(T, heads, kv, dim, page, rotary, style, norm, slots, n_pages, positions, seed=T + dim)


def test_captured_prepare_stores_at_every_replay():
    """The slots are overwritten before each replay, so that keys and values have to come from it."""
    cfg = config(8, 2, 128, 16, rotary=128)
    T = 35
    print("[case] prepare in a graph, slots overwritten", flush=True)
    cache = A.new_cache(cfg, 4)
    qkv = torch.zeros((T, 12 * 128), dtype=torch.bfloat16, device=DEV)
    table = torch.from_numpy(AO.rope_table(256, 128)).to(DEV)
    w = torch.ones(128, device=DEV)
    slots = torch.randperm(64, device=DEV)[:T]
    positions = torch.arange(T, dtype=torch.int32, device=DEV)
    q = torch.empty((T, 8, 128), dtype=torch.bfloat16, device=DEV)
    call = A.bind_prepare(cfg, cache, qkv, w, w, table, positions, slots, q)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    gen = torch.Generator(device=DEV)
    gen.manual_seed(4)
    for _ in range(3):
        qkv.copy_(torch.randn(qkv.shape, generator=gen, device=DEV).to(torch.bfloat16))
        slots.copy_(torch.randperm(64, generator=gen, device=DEV)[:T])
        results = []
        for run in (call, g.replay):
            for t in (cache.k, cache.v, q):
                t.fill_(5.0)
            run()
            torch.cuda.synchronize()
            results.append([t.clone() for t in (cache.k, cache.v, q)])
        for eager, replayed in zip(*results):
            assert torch.equal(eager.view(torch.int16), replayed.view(torch.int16))
        keys = results[1][0].permute(0, 3, 1, 2, 4).reshape(64, 2, 128)
        values = results[1][1].permute(0, 2, 4, 1, 3).reshape(64, 2, 128)
        assert torch.equal(values[slots], qkv.view(T, 12, 128)[:, 10:]), "the replay did not store the values"
        assert (keys[slots] != 5.0).float().mean() > 0.9, "the replay did not store the keys"
