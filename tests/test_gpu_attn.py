"""GPU parity of the attention operators against the fp64 oracle, with
element-wise bounds (attn_util.py): lengths from none to long ones, pages that
end inside a tile, masks that leave a row empty, poisoned slots and page ids
that no query may touch, caches past 32-bit offsets, other streams, graphs."""
import numpy as np
import pytest
import torch

from attn_util import E, U, assert_within, bf16, make_batch
from oracle import attn_oracle as AO
from routed_expert_mlp_amd import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda"


def config(heads=8, kv=2, dim=128, page=16, rotary=0, style=A.ROPE_HALF, eps=1e-6, window=0, sinks=0, scale=None):
    return A.AttnConfig(n_heads=heads, n_kv_heads=kv, head_dim=dim, page_size=page, rotary_dim=rotary,
                        rope_style=style, norm_eps=eps, scale=dim ** -0.5 if scale is None else scale, window=window,
                        n_sinks=sinks)


def cache_of(b):
    return A.KVCache(b.k.to(DEV), b.v.to(DEV))


def run_decode(b, max_len=None, stream=None):
    B, n = len(b.lens), b.new[0]
    q = b.q.to(DEV).view(B, n, b.cfg.n_heads, b.cfg.head_dim)
    lens = torch.tensor(b.lens, dtype=torch.int32, device=DEV)
    out = torch.full_like(q, float("nan"))
    A.moe_attn_decode(b.cfg, cache_of(b), q, lens, b.table.to(DEV), max(b.lens) if max_len is None else max_len, out,
                      stream=stream)
    return out


def run_prefill(b, pad=0, max_len=None, max_q=None):
    """pad: rows of q before and behind the sequences' (not written)."""
    q = torch.zeros((b.q.shape[0] + 2 * pad,) + tuple(b.q.shape[1:]), dtype=torch.bfloat16)
    q[pad:pad + b.q.shape[0]] = b.q
    q = q.to(DEV)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(b.new)]) + pad, dtype=torch.int32, device=DEV)
    lens = torch.tensor(b.lens, dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 7.0)
    A.moe_attn_prefill(b.cfg, cache_of(b), q, cu, max(b.new) if max_q is None else max_q, lens, b.table.to(DEV),
                       max(b.lens) if max_len is None else max_len, out)
    torch.cuda.synchronize()
    if pad:
        assert torch.all(out[:pad] == 7.0) and torch.all(out[-pad:] == 7.0), "rows of no sequence were written"
    return out[pad:pad + b.q.shape[0]]


def check(b, out, what):
    got = out.double().cpu().numpy().reshape(-1, b.cfg.n_heads, b.cfg.head_dim)
    row = 0
    for i, (want, bound) in enumerate(b.expected()):
        assert_within(got[row:row + want.shape[0]], want, bound, f"{what} sequence {i} of {b.lens[i]}")
        row += want.shape[0]


# ---- decode ---------------------------------------------------------------

DECODE = [
    # heads, kv, dim, page, new, lens, window, sinks
    (8, 2, 128, 16, 1, [1, 2, 15, 16, 17, 31, 32, 33, 0], 0, 0),
    (8, 8, 64, 16, 1, [0, 63, 64, 65, 127, 129], 0, 0),
    (5, 1, 128, 32, 1, [257, 300, 1], 0, 0),
    (32, 2, 256, 64, 1, [70, 511, 1025], 0, 0),
    (20, 1, 64, 128, 1, [129, 700], 0, 0),           # more query heads per key/value head than one tile holds
    (71, 1, 128, 16, 1, [77], 0, 0),
    (6, 2, 128, 256, 1, [256, 257, 1000], 0, 0),
    (8, 2, 128, 16, 4, [0, 1, 3, 4, 5, 36, 100], 0, 0),      # sequences shorter than the new tokens: empty rows
    (4, 4, 64, 32, 8, [8, 7, 263], 0, 0),
    (12, 4, 256, 16, 3, [50, 96], 0, 0),
    (8, 2, 128, 16, 1, [5, 40, 200, 1000], 1, 0),    # a window of one key
    (8, 2, 128, 16, 1, [5, 40, 200, 1000], 33, 0),
    (8, 2, 128, 16, 1, [5, 40, 200, 1000], 33, 1),
    (8, 2, 64, 64, 2, [5, 40, 200, 3000], 100, 4),
    (8, 2, 128, 32, 4, [300, 2000], 64, 70),         # sinks past a tile
    (8, 2, 128, 32, 4, [60, 500], 64, 5000),         # more sinks than keys
    (8, 2, 128, 16, 1, [500], 100000, 3),            # a window longer than the sequence
    (16, 2, 128, 16, 1, [9000, 33, 4097], 0, 0),
    (4, 1, 128, 64, 1, [30001], 0, 0),
    (4, 1, 64, 64, 1, [20000], 9000, 17),
]


@pytest.mark.parametrize("heads,kv,dim,page,new,lens,window,sinks", DECODE)
def test_decode(heads, kv, dim, page, new, lens, window, sinks):
    cfg = config(heads, kv, dim, page, window=window, sinks=sinks)
    b = make_batch(cfg, lens, [new] * len(lens), seed=heads * 1000 + dim + len(lens))
    what = f"decode {heads}/{kv}x{dim} page {page} new {new} window {window}+{sinks}"
    print(f"[case] {what} lens {lens}", flush=True)
    check(b, run_decode(b), what)


@pytest.mark.parametrize("heads,kv,dim,new,window", [(32, 8, 64, 1, 0), (32, 8, 128, 1, 0), (16, 4, 128, 2, 700),
                                                     (32, 4, 256, 1, 0)])
def test_decode_many_rows(heads, kv, dim, new, window):
    """A thousand rows and more, of sequences with no key, one part and several."""
    rng = np.random.default_rng(dim + new)
    lens = [0, 1, 31, 1400, 129] + [int(n) for n in rng.integers(1, 1200, 35)]
    b = make_batch(config(heads, kv, dim, 32, window=window, sinks=2), lens, [new] * len(lens), seed=dim)
    print(f"[case] decode of {len(lens) * new * heads} rows of {dim} dims, window {window}", flush=True)
    check(b, run_decode(b), f"decode, many rows of {dim} dims")


@pytest.mark.parametrize("heads,kv,dim,new,window", [(64, 1, 128, 1, 0), (71, 1, 64, 1, 0), (16, 2, 64, 8, 9000),
                                                     (12, 1, 128, 4, 0)])
def test_decode_wide_groups(heads, kv, dim, new, window):
    """More than 32 rows of a key/value head: several blocks that read the same keys."""
    lens = [16000, 0, 5, 33, 64, 700, 1, 4001, 12, 32, 2050, 8]
    b = make_batch(config(heads, kv, dim, 64, window=window, sinks=3), lens, [new] * len(lens), seed=heads)
    print(f"[case] decode of {new * heads // kv} rows a head of {dim} dims, window {window}", flush=True)
    check(b, run_decode(b), f"decode, wide groups of {dim} dims")


def test_decode_bound_on_length_above_and_below():
    """max_len far above the lengths changes nothing; below, sequences are cut to it."""
    cfg = config(8, 2, 128, 16)
    b = make_batch(cfg, [40, 333], [1, 1], seed=5, poison=False)
    print("[case] decode max_len", flush=True)
    wide = torch.zeros((2, 200), dtype=torch.int32)
    wide[:, :b.table.shape[1]] = b.table
    table, b.table = b.table, wide
    check(b, run_decode(b, max_len=3200), "decode, max_len 3200")
    b.table = table
    b.lens[1], b.keys[1], b.values[1] = 100, b.keys[1][:100], b.values[1][:100]
    q = b.q.to(DEV).view(2, 1, 8, 128)
    out = torch.empty_like(q)
    A.moe_attn_decode(cfg, cache_of(b), q, torch.tensor([40, 333], dtype=torch.int32, device=DEV), table.to(DEV), 100,
                      out)
    check(b, out, "decode, cut to 100")


def test_decode_large_scores_and_equal_scores():
    """Scores of thousands (only the largest counts) and scores that are all equal."""
    cfg = config(8, 2, 128, 16, scale=30.0)
    b = make_batch(cfg, [100, 700], [1, 1], seed=6)
    print("[case] decode large scores", flush=True)
    out = run_decode(b).double().cpu().numpy().reshape(2, 8, 128)
    for i, (want, bound) in enumerate(b.expected()):
        assert_within(out[i:i + 1], want, bound, f"scale 30, sequence {i}")
    cfg = config(8, 2, 128, 16)
    b = make_batch(cfg, [100, 700], [1, 1], seed=7, q_std=0.0, v_mean=3.0)
    check(b, run_decode(b), "equal scores")


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_cache_past_32_bit_offsets(form):
    """Pages at the far end of a cache of more than 4 GiB (2^32 bytes, and 2^31 values) per side."""
    cfg = config(16, 8, 128, 64)
    n_pages = 36000
    print(f"[case] {form} large cache", flush=True)
    cache = A.new_cache(cfg, n_pages)
    assert cache.k.numel() > 2 ** 31 and cache.k.numel() * 2 > 2 ** 32
    b = make_batch(cfg, [200, 130], [1, 1], seed=8)
    used = sorted(set(b.table.flatten().tolist()) & set(range(b.k.shape[0])))
    far = {p: n_pages - 1 - 7 * i for i, p in enumerate(used)}
    for p in used:
        cache.k[far[p]].copy_(b.k[p])
        cache.v[far[p]].copy_(b.v[p])
    table = torch.tensor([[far.get(p, 2 ** 31 - 1) for p in row] for row in b.table.tolist()], dtype=torch.int32)
    q = b.q.to(DEV)
    lens = torch.tensor(b.lens, dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    if form == "decode":
        A.moe_attn_decode(cfg, cache, q.view(2, 1, 16, 128), lens, table.to(DEV), 200, out.view(2, 1, 16, 128))
    else:
        cu = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
        A.moe_attn_prefill(cfg, cache, q, cu, 1, lens, table.to(DEV), 200, out)
    check(b, out, f"{form} large cache")


# ---- prefill --------------------------------------------------------------

PREFILL = [
    # heads, kv, dim, page, new, lens, window, sinks
    (8, 2, 128, 16, [1], [1], 0, 0),
    (8, 2, 128, 16, [37], [37], 0, 0),
    (8, 8, 64, 16, [130, 1, 0, 65], [130, 1, 5, 300], 0, 0),
    (5, 1, 128, 32, [100, 7], [100, 260], 0, 0),
    (9, 3, 256, 64, [70, 33], [70, 150], 0, 0),
    (20, 1, 64, 128, [50], [200], 0, 0),
    (71, 1, 128, 16, [9], [40], 0, 0),
    (6, 2, 128, 256, [300], [513], 0, 0),
    (8, 2, 128, 16, [5, 9], [3, 0], 0, 0),            # positions below zero: empty rows
    (4, 2, 128, 16, [200], [200], 1, 0),
    (4, 2, 128, 16, [200, 50], [200, 400], 33, 0),
    (4, 2, 64, 32, [200, 50], [200, 400], 33, 4),
    (4, 2, 128, 32, [300], [300], 64, 70),
    (4, 2, 256, 16, [100], [500], 40, 1000),
    (2, 1, 128, 64, [700], [1500], 256, 3),
    (2, 2, 128, 16, [1000], [1000], 0, 0),
    (3, 1, 64, 16, [513], [2000], 0, 0),
    # few rows far into long sequences: the keys are taken in parts and joined
    (8, 2, 128, 16, [5, 3, 0, 2], [3000, 40, 0, 1200], 0, 0),
    (4, 2, 128, 16, [40], [4000], 2500, 700),
    (6, 2, 256, 64, [33, 1], [1500, 2047], 0, 0),
    (10, 2, 64, 32, [70], [5001], 0, 0),
    (4, 1, 128, 128, [9], [4097], 1100, 1),
]


@pytest.mark.parametrize("heads,kv,dim,page,new,lens,window,sinks", PREFILL)
def test_prefill(heads, kv, dim, page, new, lens, window, sinks):
    cfg = config(heads, kv, dim, page, window=window, sinks=sinks)
    b = make_batch(cfg, lens, new, seed=heads * 1000 + dim + len(lens))
    what = f"prefill {heads}/{kv}x{dim} page {page} window {window}+{sinks}"
    print(f"[case] {what} new {new} lens {lens}", flush=True)
    check(b, run_prefill(b, pad=2), what)


@pytest.mark.parametrize("heads,kv,dim,new,lens,window,sinks", [
    (32, 8, 64, [256, 3], [4000, 50], 0, 0),
    (32, 8, 128, [300], [5000], 0, 0),
    (32, 8, 128, [250, 1, 20], [1100, 40, 2000], 0, 0),
    (32, 8, 256, [230, 9], [2500, 9], 0, 0),
    (48, 4, 128, [150], [5000], 3000, 40),
])
def test_prefill_many_rows_in_parts(heads, kv, dim, new, lens, window, sinks):
    """Thousands of rows far into their sequences: keys in parts, several rows a wavefront in the join."""
    b = make_batch(config(heads, kv, dim, 32, window=window, sinks=sinks), lens, new, seed=dim + heads)
    what = f"prefill of {sum(new) * heads} rows of {dim} dims, window {window}+{sinks}"
    print(f"[case] {what}", flush=True)
    check(b, run_prefill(b, pad=1), what)


@pytest.mark.parametrize("B", [65, 200])
def test_prefill_many_sequences(B):
    """More sequences than a wavefront has lanes, some without new tokens."""
    rng = np.random.default_rng(B)
    new = [int(n) for n in rng.integers(0, 9, B)]
    new[3], new[-1], new[63] = 40, 0, 0
    lens = [m + int(p) for m, p in zip(new, rng.integers(0, 30, B))]
    b = make_batch(config(4, 2, 64, 16), lens, new, seed=B)
    print(f"[case] prefill of {B} sequences", flush=True)
    check(b, run_prefill(b, pad=1), f"prefill of {B} sequences")


def test_prefill_bounds_above_and_equal_scores():
    cfg = config(8, 2, 128, 16)
    b = make_batch(cfg, [40, 96], [40, 20], seed=9, poison=False, q_std=0.0, v_mean=2.0)
    wide = torch.zeros((2, 64), dtype=torch.int32)
    wide[:, :b.table.shape[1]] = b.table
    b.table = wide
    print("[case] prefill max_len and max_q above", flush=True)
    check(b, run_prefill(b, max_len=1024, max_q=777), "prefill, loose bounds")
    b = make_batch(config(8, 2, 128, 16, scale=30.0), [40, 300], [40, 20], seed=10)
    check(b, run_prefill(b), "prefill, large scores")


def test_prefill_of_one_token_per_sequence_is_decode():
    """Same rows either way, within both bounds, on lengths around the tile sizes."""
    cfg = config(8, 2, 128, 16, window=50, sinks=2)
    lens = [1, 16, 31, 64, 65, 255, 700]
    b = make_batch(cfg, lens, [1] * len(lens), seed=11)
    print("[case] prefill of single tokens", flush=True)
    check(b, run_prefill(b), "prefill of single tokens")
    check(b, run_decode(b), "decode")


# ---- prepare --------------------------------------------------------------

def prepare_case(T, heads, kv, dim, page, rotary, style, norm, slots, n_pages, positions, seed, pad_cols=0):
    cfg = config(heads, kv, dim, page, rotary=rotary, style=style, eps=1e-5)
    rng = np.random.default_rng(seed)
    width = (heads + 2 * kv) * dim
    x, xd = bf16(rng.standard_normal((T, width)) * 0.7)
    if T > 2:
        x[1] = 0                                     # a row whose norm is eps alone
        xd[1] = 0.0
    buf = torch.full((T, width + pad_cols), float("nan"), dtype=torch.bfloat16)
    buf[:, :width] = x
    qkv = buf.to(DEV)[:, :width]
    qw = (1.0 + 0.3 * rng.standard_normal(dim)).astype(np.float32) if norm in ("both", "q") else None
    kw = (1.0 + 0.3 * rng.standard_normal(dim)).astype(np.float32) if norm in ("both", "k") else None
    table = AO.rope_table(max(max(positions, default=0) + 1, 1), rotary)
    dev = lambda t: None if t is None else torch.from_numpy(t).to(DEV)  # noqa: E731
    kc = torch.full(A.cache_shapes(cfg, n_pages)[0], 3.0, dtype=torch.bfloat16, device=DEV)
    vc = torch.full(A.cache_shapes(cfg, n_pages)[1], 3.0, dtype=torch.bfloat16, device=DEV)
    q_out = torch.empty((T, heads, dim), dtype=torch.bfloat16, device=DEV)
    A.moe_attn_prepare(cfg, A.KVCache(kc, vc), qkv, dev(qw), dev(kw), dev(table) if rotary else None,
                       torch.tensor(positions, dtype=torch.int32, device=DEV) if rotary else None,
                       torch.tensor(slots, dtype=torch.int64, device=DEV), q_out)
    torch.cuda.synchronize()
    x3 = xd.reshape(T, heads + 2 * kv, dim)
    rows = table[np.asarray(positions, np.int64)][:, None, :]
    rows = np.broadcast_to(rows, (T, heads + kv, rotary))
    w = np.concatenate([np.broadcast_to(qw if qw is not None else np.ones(dim), (heads, dim)),
                        np.broadcast_to(kw if kw is not None else np.ones(dim), (kv, dim))])
    y = x3[:, :heads + kv].copy()
    for lo, hi, ww in ((0, heads, qw), (heads, heads + kv, kw)):
        if ww is not None:
            y[:, lo:hi] = AO.norm_rope(y[:, lo:hi], ww, cfg.norm_eps, np.zeros((1, 0)), False)
    want = AO.norm_rope(y, None, 0.0, rows, style == A.ROPE_INTERLEAVED)
    # |a| + |b| of the pair that an element is rotated in
    h = rotary // 2
    i = np.arange(h)
    ia, ib = (2 * i, 2 * i + 1) if style == A.ROPE_INTERLEAVED else (i, i + h)
    mag = np.abs(y)
    if rotary:
        both = np.abs(y[..., ia]) + np.abs(y[..., ib])
        mag[..., ia] = both
        mag[..., ib] = both
    bound = U * np.abs(want) + (dim + 16) * E * mag
    what = f"prepare T={T} {heads}/{kv}x{dim} page {page} rotary {rotary} style {style} norm {norm}"
    assert_within(q_out.double().cpu().numpy(), want[:, :heads], bound[:, :heads], what + ", q")
    k_got, v_got = kc.double().cpu().numpy(), vc.double().cpu().numpy()
    touched = np.zeros((n_pages, page), bool)
    for t, s in enumerate(slots):
        if not 0 <= s < n_pages * page:
            continue
        p, at = divmod(s, page)
        touched[p, at] = True
        k_row, v_row = AO.load(k_got, v_got, p, at)
        assert_within(k_row, want[t, heads:], bound[t, heads:], what + f", k of token {t}") if t < 3 else None
        assert np.all(np.abs(k_row - want[t, heads:]) <= bound[t, heads:]), f"{what}: k of token {t}"
        assert np.array_equal(v_row, x3[t, heads + kv:]), f"{what}: v of token {t}"
    for p, at in zip(*np.nonzero(~touched)):
        k_row, v_row = AO.load(k_got, v_got, p, at)
        assert np.all(k_row == 3.0) and np.all(v_row == 3.0), f"{what}: slot {p * page + at} was written"


PREPARE = [
    # T, heads, kv, dim, page, rotary, style, norm, first slot (None: shuffled)
    (1, 8, 2, 128, 16, 128, A.ROPE_HALF, "both", 5),
    (1, 4, 1, 64, 16, 64, A.ROPE_INTERLEAVED, "both", 0),
    (2, 3, 3, 256, 32, 256, A.ROPE_HALF, "both", 31),
    (16, 8, 2, 128, 16, 64, A.ROPE_HALF, "both", 0),
    (37, 8, 2, 128, 16, 128, A.ROPE_INTERLEAVED, "both", 0),
    (37, 8, 2, 128, 16, 128, A.ROPE_HALF, "both", 3),          # not at a multiple of 8
    (75, 5, 1, 64, 64, 16, A.ROPE_HALF, "q", 8),
    (75, 5, 1, 64, 64, 48, A.ROPE_HALF, "k", 1),
    (33, 4, 2, 256, 128, 128, A.ROPE_INTERLEAVED, "both", 100),
    (50, 4, 4, 128, 256, 0, A.ROPE_HALF, "none", 0),
    (50, 4, 4, 128, 256, 0, A.ROPE_HALF, "both", 0),
    (64, 8, 2, 128, 16, 32, A.ROPE_HALF, "both", None),        # a token of each of many sequences
    (130, 2, 1, 64, 32, 64, A.ROPE_HALF, "both", None),
    (9, 128, 8, 64, 16, 64, A.ROPE_HALF, "both", 7),
]


@pytest.mark.parametrize("T,heads,kv,dim,page,rotary,style,norm,first", PREPARE)
def test_prepare(T, heads, kv, dim, page, rotary, style, norm, first):
    rng = np.random.default_rng(T)
    n_pages = -(-(T + (first or 0)) // page) + 2
    if first is None:
        slots = [int(s) for s in rng.permutation(n_pages * page)[:T]]
        positions = [int(p) for p in rng.integers(0, 5000, T)]
    else:
        order = rng.permutation(n_pages)
        slots = [int(order[(first + t) // page]) * page + (first + t) % page for t in range(T)]
        positions = list(range(first, first + T))
    print(f"[case] prepare T={T} {heads}/{kv}x{dim}", flush=True)
    prepare_case(T, heads, kv, dim, page, rotary, style, norm, slots, n_pages, positions, seed=T + dim)


def test_prepare_skips_slots_out_of_range():
    """Padding tokens (negative slots) and slots past the cache store nothing; runs of slots broken inside 8 tokens."""
    print("[case] prepare, slots out of range", flush=True)
    slots = [-1, 0, 1, 2, -5, 4, 5, 6, 7, 8, 9, 10, 11, 64, 2 ** 40, -2 ** 62, 15, 14, 13, 12, 24, 25, 26, 27, 28, 29,
             30, 31]
    prepare_case(len(slots), 4, 2, 128, 16, 128, A.ROPE_HALF, "both", slots, 4, list(range(len(slots))), seed=1)
    prepare_case(len(slots), 4, 2, 64, 32, 64, A.ROPE_INTERLEAVED, "both", slots, 2, list(range(len(slots))), seed=2)


def test_prepare_row_stride():
    print("[case] prepare, rows of a wider buffer", flush=True)
    prepare_case(20, 4, 2, 128, 16, 128, A.ROPE_HALF, "both", list(range(20)), 2, list(range(20)), seed=3, pad_cols=40)


# ---- streams, graphs, repeatability ----------------------------------------

def test_side_stream_and_repeatability():
    cfg = config(16, 4, 128, 16)
    b = make_batch(cfg, [3000, 17, 900], [1, 1, 1], seed=12)
    print("[case] side stream", flush=True)
    first = run_decode(b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    again = run_decode(b, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int16), again.view(torch.int16))
    check(b, again, "decode on a side stream")
    p = make_batch(cfg, [300, 90], [300, 40], seed=13)
    assert torch.equal(run_prefill(p).view(torch.int16), run_prefill(p).view(torch.int16))


def test_graph_replay_follows_the_buffers():
    """prepare, decode and prefill captured together; each replay is compared with eager calls on changed inputs."""
    cfg = config(8, 2, 128, 16, rotary=128)
    b = make_batch(cfg, [700, 40, 33], [1, 1, 1], seed=14, poison=False)
    cache = cache_of(b)
    T, width = 3, 12 * 128
    qkv = torch.zeros((T, width), dtype=torch.bfloat16, device=DEV)
    table = torch.from_numpy(AO.rope_table(1024, 128)).to(DEV)
    w = torch.ones(128, device=DEV)
    lens = torch.tensor(b.lens, dtype=torch.int32, device=DEV)
    pages = b.table.to(DEV)
    pos = (lens - 1).to(torch.int32)
    slots = (pages[torch.arange(3, device=DEV), (lens - 1) // 16].long() * 16 + (lens - 1).long() % 16)
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device=DEV)
    q = torch.empty((T, 8, 128), dtype=torch.bfloat16, device=DEV)
    o1, o2 = torch.empty_like(q), torch.empty_like(q)
    calls = [A.bind_prepare(cfg, cache, qkv, w, w, table, pos, slots, q),
             A.bind_decode(cfg, cache, q.view(3, 1, 8, 128), lens, pages, 700, o1.view(3, 1, 8, 128)),
             A.bind_prefill(cfg, cache, q, cu, 1, lens, pages, 700, o2)]
    print("[case] graph", flush=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        on_side = [A.bind_prepare(cfg, cache, qkv, w, w, table, pos, slots, q, stream=side),
                   A.bind_decode(cfg, cache, q.view(3, 1, 8, 128), lens, pages, 700, o1.view(3, 1, 8, 128),
                                 stream=side),
                   A.bind_prefill(cfg, cache, q, cu, 1, lens, pages, 700, o2, stream=side)]
        for c in on_side:
            c()
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            for c in on_side:
                c()
    torch.cuda.synchronize()
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    for _ in range(4):
        qkv.copy_(torch.randn((T, width), generator=gen, device=DEV).to(torch.bfloat16))
        for c in calls:
            c()
        torch.cuda.synchronize()
        want = [t.clone() for t in (q, o1, o2, cache.k, cache.v)]
        for t in (q, o1, o2):
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for t, u in zip((q, o1, o2, cache.k, cache.v), want):
            assert torch.equal(t.view(torch.int16), u.view(torch.int16))


def test_no_tokens_and_no_sequences():
    cfg = config(8, 2, 128, 16)
    cache = A.new_cache(cfg, 1)
    e = torch.empty((0, 1, 8, 128), dtype=torch.bfloat16, device=DEV)
    i = torch.empty((0,), dtype=torch.int32, device=DEV)
    A.moe_attn_decode(cfg, cache, e, i, torch.empty((0, 1), dtype=torch.int32, device=DEV), 16, e.clone())
    e = e.view(0, 8, 128)
    A.moe_attn_prefill(cfg, cache, e, torch.zeros(1, dtype=torch.int32, device=DEV), 0, i,
                       torch.empty((0, 1), dtype=torch.int32, device=DEV), 0, e.clone())
    A.moe_attn_prepare(cfg, cache, torch.empty((0, 12 * 128), dtype=torch.bfloat16, device=DEV), None, None, None, None,
                       torch.empty(0, dtype=torch.int64, device=DEV), e.clone())
    # sequences without a page: every row is empty
    q = torch.ones((2, 1, 8, 128), dtype=torch.bfloat16, device=DEV)
    out = torch.ones_like(q)
    A.moe_attn_decode(cfg, cache, q, torch.zeros(2, dtype=torch.int32, device=DEV),
                      torch.empty((2, 0), dtype=torch.int32, device=DEV), 0, out)
    torch.cuda.synchronize()
    assert torch.all(out == 0)


def test_tensor_checks():
    cfg = config(8, 2, 128, 16)
    cache = A.new_cache(cfg, 2)
    q = torch.zeros((1, 1, 8, 128), dtype=torch.bfloat16, device=DEV)
    lens = torch.ones(1, dtype=torch.int32, device=DEV)
    table = torch.zeros((1, 2), dtype=torch.int32, device=DEV)
    good = dict(q=q, seq_lens=lens, page_table=table, max_len=32, out=torch.empty_like(q))
    for bad, err in ((dict(q=q.float()), TypeError), (dict(q=q[:, :, :4]), ValueError),
                     (dict(q=q.cpu()), ValueError), (dict(seq_lens=lens.long()), TypeError),
                     (dict(page_table=table.t()), ValueError),
                     (dict(q=q.transpose(2, 3).contiguous().transpose(2, 3)), ValueError),
                     (dict(max_len=33), A.capi.MoeMlpError), (dict(out=torch.empty_like(q[0])), ValueError)):
        with pytest.raises(err):
            A.moe_attn_decode(cfg, cache, **{**good, **bad})
    with pytest.raises(ValueError):
        A.moe_attn_decode(cfg, A.KVCache(cache.v, cache.k), **good)
    with pytest.raises(ValueError):
        A.moe_attn_prepare(cfg, cache, torch.zeros((2, 12 * 128 * 2), dtype=torch.bfloat16, device=DEV)[:, ::2], None,
                           None, None, None, torch.zeros(2, dtype=torch.int64, device=DEV),
                           torch.empty((2, 8, 128), dtype=torch.bfloat16, device=DEV))
