"""GPU tests of decode behind a shared prefix: against the fp64 definition over each sequence's whole keys, and against
plain decode.  Slots that nobody sees hold NaN, page ids of pages without a visible key are far out of range."""
import numpy as np
import pytest
import torch

from attn_util import E, U, assert_within, bf16
from oracle import attn_oracle as AO
from routed_expert_mlp_amd import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda"


def config(heads, kv, dim, page, window=0, sinks=0):
    return A.AttnConfig(n_heads=heads, n_kv_heads=kv, head_dim=dim, page_size=page, rotary_dim=0,
                        rope_style=A.ROPE_HALF, norm_eps=0.0, scale=dim ** -0.5, window=window, n_sinks=sinks)


class Shared:
    """A batch behind a prefix of `shared` tokens; lens: whole lengths, also below the prefix's."""

    def __init__(self, cfg, shared, lens, n_q, seed, q_std=1.5, v_mean=0.0):
        rng = np.random.default_rng(seed)
        H, K, D, P, B = cfg.n_heads, cfg.n_kv_heads, cfg.head_dim, cfg.page_size, len(lens)
        self.cfg, self.shared, self.lens, self.n_q = cfg, shared, list(lens), n_q
        width, first = max(1, -(-max(max(lens), shared) // P)), shared // P
        lead = -(-shared // P)
        need = lead + sum(max(0, -(-n // P) - first) for n in lens) + 2
        order = rng.permutation(need)
        kc, vc = (np.full(s, np.nan, np.float32) for s in A.cache_shapes(cfg, need))
        self.q, qd = bf16(rng.standard_normal((B, n_q, H, D)) * q_std)
        pk, pv = bf16(rng.standard_normal((shared, K, D)))[1], bf16(rng.standard_normal((shared, K, D)) + v_mean)[1]
        table = np.where(np.arange(B * width).reshape(B, width) % 2, 2 ** 31 - 1, -2 ** 31)
        pages = np.full(max(lead, 1), -2 ** 31, np.int64)
        seen_lead, at, self.rows = np.zeros(shared, bool), lead, []
        for b, n in enumerate(lens):
            m = max(0, n - shared)
            ok, ov = bf16(rng.standard_normal((m, K, D)))[1], bf16(rng.standard_normal((m, K, D)) + v_mean)[1]
            seen = AO.visible(n, n_q, cfg.window, cfg.n_sinks).any(axis=0) if n else np.zeros(0, bool)
            seen_lead[:min(n, shared)] |= seen[:shared]
            for j in range(first, -(-n // P)):
                own = np.arange(max(j * P, shared), min((j + 1) * P, n))
                if own.size and seen[own].any():
                    table[b, j] = order[at]
                    at += 1
                    for t in own[seen[own]]:
                        AO.store(kc, vc, table[b, j], t % P, ok[t - shared], ov[t - shared])
            self.rows.append((qd[b], ok, ov))
        self.lead = pk, pv
        for j in range(lead):
            hit = np.nonzero(seen_lead[j * P:(j + 1) * P])[0] + j * P
            if hit.size:
                pages[j] = order[j]
                for t in hit:
                    AO.store(kc, vc, order[j], t % P, pk[t], pv[t])
        self.k, self.v = bf16(kc)[0].to(DEV), bf16(vc)[0].to(DEV)
        self.table = torch.from_numpy(table.astype(np.int32)).to(DEV)
        self.pages = torch.from_numpy(pages.astype(np.int32)).to(DEV)
        self.dq = self.q.to(DEV)
        self.dlens = torch.tensor(lens, dtype=torch.int32, device=DEV)

    def run(self, max_len=None):
        cfg, B = self.cfg, len(self.lens)
        max_len = max(max(self.lens), self.shared) if max_len is None else max_len
        out = torch.full_like(self.dq, float("nan"))
        need = A.moe_attn_shared_workspace_size(cfg, B, self.n_q, max_len, self.shared)
        ws = torch.full((need + 512,), 255, dtype=torch.uint8, device=DEV)
        A.moe_attn_decode_shared(cfg, A.KVCache(self.k, self.v), self.dq, self.dlens, self.table, max_len, self.pages,
                                 self.shared, out, ws[:need])
        torch.cuda.synchronize()
        assert (ws[need:] == 255).all(), "written past the workspace"
        return out

    def check(self, out, what):
        cfg, D = self.cfg, self.cfg.head_dim
        got, want, bound = out.double().cpu().numpy(), np.zeros(tuple(out.shape)), np.zeros(tuple(out.shape))
        for b, (q, k, v) in enumerate(self.rows):
            k, v = (np.concatenate([t[:self.lens[b]], own]) for t, own in zip(self.lead, (k, v)))
            o, mag, big = AO.attend(q, k, v, cfg.scale, cfg.window, cfg.n_sinks)
            want[b] = o
            bound[b] = U * (mag + np.abs(o)) + (2 * (D + 16) * E * big + 2.0 ** -14) * mag
        assert_within(got, want, bound, what)


def case(heads, kv, dim, page, shared, lens, n_q=1, window=0, sinks=0, seed=0, **kw):
    what = f"shared {heads}/{kv}x{dim}, page {page}, {len(lens)} x {n_q} behind {shared}, lens {lens[:6]}, " \
           f"window {window}+{sinks}"
    print(f"[case] {what}", flush=True)
    s = Shared(config(heads, kv, dim, page, window, sinks), shared, lens, n_q, seed, **kw)
    out = s.run()
    s.check(out, what)
    return s, out


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("shared", [0, 1, 15, 16, 31, 32, 33, 100, 256, 777])
def test_prefix_lengths(dim, shared):
    case(8, 2, dim, 16, shared, [shared + n for n in (1, 40, 7)], seed=shared)
    case(8, 2, dim, 32, shared, [shared + n for n in (1, 64, 100, 33)] * 8, seed=shared + 1)


@pytest.mark.parametrize("dim,page", [(64, 256), (128, 128), (256, 64)])
@pytest.mark.parametrize("heads,kv", [(1, 1), (5, 1), (48, 1), (6, 3), (40, 8)])
def test_heads(heads, kv, dim, page):
    for B in (1, 2, 9, 30):
        case(heads, kv, dim, page, 333, [333 + 1 + 13 * (b % 5) for b in range(B)], seed=B)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n_q", [2, 3, 8])
def test_several_new_tokens(dim, n_q):
    case(12, 3, dim, 32, 190, [190 + n_q + n for n in (0, 1, 30, 200)], n_q=n_q, seed=n_q)
    case(12, 3, dim, 32, 190, [190 + n_q + n for n in (0, 1, 30, 200, 66)] * 5, n_q=n_q, seed=n_q + 1)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_sequences_that_end_inside_the_prefix(dim):
    """Padded rows (0), rows with less than the prefix, rows whose first new tokens have no position."""
    lens = [0, 1, 3, 50, 99, 100, 101, 130, 2, 0]
    for shared in (100, 101, 32):
        for n_q in (1, 4):
            case(8, 2, dim, 16, shared, lens, n_q=n_q, seed=shared + n_q)
            case(8, 2, dim, 16, shared, lens * 4, n_q=n_q, seed=shared + n_q)
    case(8, 2, dim, 16, 64, [0, 0, 0], seed=3)
    case(8, 2, dim, 16, 64, [0] * 40, seed=4)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 3), (40, 0), (64, 70), (200, 4), (10000, 0), (7, 10000)])
def test_windows(dim, window, sinks):
    lens = [210, 211, 260, 333, 205, 700, 203]
    for shared in (203, 64):
        for rep in (1, 5):
            case(8, 2, dim, 16, shared, lens * rep, n_q=3, window=window, sinks=sinks, seed=shared + rep)


@pytest.mark.parametrize("dim,heads,kv", [(64, 24, 8), (128, 32, 8), (256, 16, 2)])
def test_long_prefixes(dim, heads, kv):
    case(heads, kv, dim, 64, 4099, [4099 + n for n in (1, 900, 17)], seed=1, v_mean=0.5)
    case(heads, kv, dim, 64, 4099, [4099 + n for n in (1, 900, 17, 5, 300)] * 6, seed=2, v_mean=0.5)


# Sizes whose prefix is taken in wide column blocks (tests below run the same masks in both forms): heads, key/value
# heads, dims, page, prefix, sequences; with 128 dims in blocks of 4 wavefronts and of 8.
WIDE = [(64, 8, 64, 32, 13001, 128), (32, 8, 128, 16, 16379, 64), (64, 4, 128, 64, 9001, 64), (16, 1, 256, 64, 4100, 64)]


def check_on_gpu(s, out, what):
    """Shared.check with the definition in fp64 on the GPU, all sequences of a key/value head at once."""
    cfg, P, B, M = s.cfg, s.shared, len(s.lens), s.n_q
    G, D, top = cfg.n_heads // cfg.n_kv_heads, cfg.head_dim, max(1, max(n - s.shared for n in s.lens))
    q = torch.from_numpy(np.stack([r[0] for r in s.rows])).to(DEV)                      # [B, M, H, D]
    at = torch.tensor(s.lens, device=DEV)[:, None] - M + torch.arange(M, device=DEV)     # [B, M]
    want, bound = torch.zeros_like(q), torch.zeros_like(q)
    for h in range(cfg.n_kv_heads):
        kp, vp = (torch.from_numpy(np.ascontiguousarray(t[:, h])).to(DEV) for t in s.lead)
        ko, vo = torch.zeros((2, B, top, D), dtype=torch.float64, device=DEV)
        for b, (_, k, v) in enumerate(s.rows):
            ko[b, :len(k)], vo[b, :len(k)] = torch.from_numpy(k[:, h]).to(DEV), torch.from_numpy(v[:, h]).to(DEV)
        mine = q[:, :, h * G:(h + 1) * G]

        def over(f):
            return torch.cat([f(mine) @ f(kp).T, torch.matmul(f(mine), f(ko)[:, None].transpose(-1, -2).contiguous())],
                             dim=-1) * cfg.scale
        key = torch.arange(P + top, device=DEV)
        see = key <= at[..., None]
        if cfg.window:
            see &= (at[..., None] - key < cfg.window) | (key < cfg.n_sinks)
        see = see[:, :, None]
        w = over(lambda t: t).masked_fill(~see, -torch.inf)
        w = (w - w.amax(-1, keepdim=True).clamp(min=-1e300)).exp()
        w /= w.sum(-1, keepdim=True).clamp(min=1e-300)
        big = float(over(torch.abs).masked_fill(~see, 0.0).max())
        o, mag = (w[..., :P] @ f(vp) + torch.matmul(w[..., P:], f(vo)[:, None].contiguous())
                  for f in (lambda t: t, torch.abs))
        want[:, :, h * G:(h + 1) * G] = o
        bound[:, :, h * G:(h + 1) * G] = U * (mag + o.abs()) + (2 * (D + 16) * E * big + 2.0 ** -14) * mag
    assert_within(out.double().cpu().numpy(), want.cpu().numpy(), bound.cpu().numpy(), what)


@pytest.mark.parametrize("heads,kv,dim,page,shared,B", WIDE)
@pytest.mark.parametrize("kind", ["behind", "window", "inside", "verify"])
def test_wide_blocks(heads, kv, dim, page, shared, B, kind):
    """All columns see the whole prefix; a window that ends in it, with sinks; sequences that end inside it, or have
    nothing; several new tokens, some without a position."""
    window, sinks, n_q = 0, 0, 1
    if kind == "behind":
        lens = [shared + 1 + 29 * (b % 5) for b in range(B)]
    elif kind == "window":
        window, sinks = 700, 37
        lens = [shared + 1 + 211 * (b % 6) for b in range(B)]
    elif kind == "inside":
        lens = [(0, 1, 31, 32, 129, shared - 1, shared, shared + 1)[b % 8] for b in range(B)]
    else:
        n_q, B = 4, B // 4
        lens = [(2, 70, shared + 4, shared + 90)[b % 4] for b in range(B)]
    what = f"wide: {heads}/{kv}x{dim}, {B} x {n_q} behind {shared}, {kind}"
    print(f"[case] {what}", flush=True)
    s = Shared(config(heads, kv, dim, page, window, sinks), shared, lens, n_q, seed=dim + B)
    check_on_gpu(s, s.run(), what)


@pytest.mark.parametrize("B", [3, 40])
def test_large_scores(B):
    case(8, 2, 128, 16, 300, [300 + 1 + 9 * (b % 7) for b in range(B)], seed=5, q_std=60.0)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_max_len_cuts_sequences_and_wide_bounds_do_not_matter(dim):
    s, out = case(8, 2, dim, 16, 150, [170, 400, 151], seed=9)
    wide = torch.zeros((3, 4096 // 16), dtype=torch.int32, device=DEV)
    wide[:, :s.table.shape[1]] = s.table
    s.table = wide
    s.check(s.run(max_len=4096), "shared, a wide bound")
    t = Shared(s.cfg, 150, [170, 300, 151], 1, 9)
    t.dlens = torch.tensor([170, 9999, 151], dtype=torch.int32, device=DEV)        # cut to 300
    t.check(t.run(max_len=300), "shared, a sequence longer than max_len")


@pytest.mark.parametrize("B", [2, 20])
def test_equals_plain_decode_on_one_cache(B):
    """The same table and pages through moe_attn_decode: the same sums in another order."""
    cfg = config(16, 4, 128, 32)
    s = Shared(cfg, 320, [320 + 5 + 31 * (b % 4) for b in range(B)], 1, 21)
    s.table[:, :10] = s.pages
    out, ref = s.run().double(), torch.empty_like(s.dq)
    A.moe_attn_decode(cfg, A.KVCache(s.k, s.v), s.dq, s.dlens, s.table, max(s.lens), ref)
    assert float((out - ref.double()).abs().max()) <= 2 * U * float(ref.abs().max()) + 2.0 ** -12
    s.check(ref, "plain decode of the same batch")


@pytest.mark.parametrize("B", [3, 40])
def test_captured_and_replayed(B):
    """One bound call in a graph, replayed with eager calls of other sequences in between and new inputs."""
    cfg = config(8, 2, 128, 16)
    s = Shared(cfg, 100, [100 + 1 + 17 * (b % 4) for b in range(B)], 1, 4)
    out = torch.empty_like(s.dq)
    call = A.bind_decode_shared(cfg, A.KVCache(s.k, s.v), s.dq, s.dlens, s.table, max(s.lens), s.pages, 100, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        s.dq.copy_(torch.randn(s.dq.shape, device=DEV) * (1 + i))
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        want = s.run()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), f"replay {i}"


def test_one_workspace_of_two_streams_is_not_shared():
    """Two callables on two streams have workspaces of their own."""
    cfg = config(8, 2, 64, 16)
    a, b = (Shared(cfg, 200, [200 + n for n in (3, 50, 20)], 1, seed) for seed in (1, 2))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for s, stream in zip((a, b), streams):
        with torch.cuda.stream(stream):
            out = torch.empty_like(s.dq)
            call = A.bind_decode_shared(cfg, A.KVCache(s.k, s.v), s.dq, s.dlens, s.table, max(s.lens), s.pages, 200, out)
            for _ in range(20):
                call()
            outs.append((out, call))
    torch.cuda.synchronize()
    for s, (out, _) in zip((a, b), outs):
        s.check(out, "shared, two streams")


def test_refusals():
    cfg = config(8, 2, 64, 16)
    s = Shared(cfg, 100, [120, 130], 1, 0)
    cache, out = A.KVCache(s.k, s.v), torch.empty_like(s.dq)
    good = dict(cfg=cfg, cache=cache, q=s.dq, seq_lens=s.dlens, page_table=s.table, max_len=130, shared_pages=s.pages,
                shared_len=100, out=out)
    A.moe_attn_decode_shared(**good)
    for bad, err in ((dict(shared_pages=s.pages[:3]), ValueError), (dict(shared_pages=s.pages.long()), TypeError),
                     (dict(shared_pages=s.pages.cpu()), ValueError), (dict(q=s.dq.float()), TypeError),
                     (dict(out=out[:1]), ValueError), (dict(seq_lens=s.dlens[:1]), ValueError),
                     (dict(shared_len=131), Exception), (dict(shared_len=-1), Exception),
                     (dict(shared_pages=None), A.capi.MoeMlpError),
                     (dict(ws=torch.empty(64, dtype=torch.uint8, device=DEV)), A.capi.MoeMlpError)):
        with pytest.raises(err):
            A.moe_attn_decode_shared(**{**good, **bad})
