"""GPU tests of the operators around the halves of the layer against their fp64 definitions: norms with the residual
and the E4M3 form, the FP8 projection, the adapters."""
import numpy as np
import pytest
import torch

from oracle import proj_oracle as PO
from proj_util import assert_within, bf16, check_norm, fp8_bound, lora_bound
from routed_expert_mlp_amd import projection as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
GUARD = 64


def guarded(shape, dtype, fill):
    """A tensor with GUARD elements of `fill` behind its end, and a check that they are still there."""
    n = int(np.prod(shape))
    flat = torch.full((n + GUARD,), fill, dtype=dtype, device=DEV)
    return flat[:n].view(shape), lambda: bool((flat[n:] == fill).all())


def norm_case(T, H, residual, weight, outs, seed, pad=0, eps=1e-6, std=1.0):
    rng = np.random.default_rng(seed)
    x, xd = bf16(rng.standard_normal((T, H + pad)) * std * np.exp(0.6 * rng.standard_normal(H + pad)))
    r, rd = bf16(rng.standard_normal((T, H)) * std) if residual else (None, None)
    w = (1.0 + 0.2 * rng.standard_normal(H)).astype(np.float32) if weight else None
    dx = x.to(DEV)[:, :H]
    h, y, q = ("h" in outs), ("y" in outs), ("q" in outs)
    (hb, hok), (yb, yok) = guarded((T, H), torch.bfloat16, 7.0), guarded((T, H), torch.bfloat16, 7.0)
    (qb, qok), (sb, sok) = guarded((T, H), torch.uint8, 77), guarded((T, -(-H // 128)), torch.float32, 7.0)
    what = f"norm {T}x{H} (+{pad}), residual {residual}, weight {weight}, out {outs}"
    print(f"[case] {what}", flush=True)
    P.moe_proj_norm(dx, torch.from_numpy(w).to(DEV) if weight else None, eps, r.to(DEV) if residual else None,
                    hb if h else None, yb if y else None, qb if q else None, sb if q else None)
    torch.cuda.synchronize()
    assert hok() and yok() and qok() and sok(), f"{what}: written past the end"
    for asked, buf, fill in ((h, hb, 7.0), (y, yb, 7.0), (q, qb, 77), (q, sb, 7.0)):
        assert asked or bool((buf == fill).all())
    check_norm(xd[:, :H], rd, w, eps, hb if h else None, yb if y else None, qb if q else None, sb if q else None, what)


@pytest.mark.parametrize("H", [8, 16, 120, 128, 136, 504, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 4104, 8184,
                               8192, 8200, 12296, 16384])
@pytest.mark.parametrize("T", [1, 5])
def test_norm_widths(T, H):
    norm_case(T, H, True, True, "hyq", T + H)


@pytest.mark.parametrize("outs", ["y", "q", "hy", "hq", "yq", "hyq"])
@pytest.mark.parametrize("residual,weight", [(False, False), (True, False), (False, True)])
def test_norm_outputs(outs, residual, weight):
    norm_case(7, 776, residual, weight, outs, 3)
    norm_case(3, 1544, residual, weight, outs, 4, pad=24)


@pytest.mark.parametrize("T", [2, 63, 257, 2049])
def test_norm_rows(T):
    norm_case(T, 1288, True, True, "hyq", T, pad=8)
    norm_case(T, 200, True, True, "hyq", T)


def test_norm_small_and_large_rows():
    norm_case(9, 640, True, True, "hyq", 5, std=2.0 ** 55)
    norm_case(9, 640, True, True, "hyq", 6, std=2.0 ** -40, eps=0.0)
    norm_case(9, 640, True, True, "hyq", 7, std=2.0 ** -40)


def test_norm_ends_of_the_range():
    """Squares whose sum is close to the largest fp32 in the widest row, and the least sum that eps 0 allows."""
    for H, value in ((16384, 2.0 ** 56), (16384, -2.0 ** 56), (128, 2.0 ** -53), (16384, 2.0 ** -56)):
        x = torch.full((2, H), value, dtype=torch.bfloat16)
        x[1, ::3] *= -0.5
        y, q = torch.empty((2, H), dtype=torch.bfloat16, device=DEV), torch.empty((2, H), dtype=torch.uint8, device=DEV)
        s = torch.empty((2, H // 128), dtype=torch.float32, device=DEV)
        P.moe_proj_norm(x.to(DEV), None, 0.0, None, None, y, q, s)
        check_norm(x.double().numpy(), None, None, 0.0, None, y, q, s, f"norm of {H} of {value}")


def test_norm_rows_of_zeros_and_not_finite():
    T, H = 8, 392
    x = torch.randn((T, H), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 300] = float("inf")
    x[4, :128] = 0
    h, y = torch.empty((T, H), dtype=torch.bfloat16, device=DEV), torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    q = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty((T, 4), dtype=torch.float32, device=DEV)
    P.moe_proj_norm(x.to(DEV), None, 1e-6, None, h, y, q, s)
    assert torch.equal(h.cpu().view(torch.int16), x.view(torch.int16))
    fine = [0, 1, 4, 5, 6, 7]
    check_norm(x[fine].double().numpy(), None, None, 1e-6, h[fine], y[fine], q.view(torch.uint8)[fine], s[fine],
               "norm beside rows that are not finite")
    for got in (y.float(), q.float()):
        assert torch.isnan(got[2]).all()
        assert torch.isnan(got[3, 300]) and (got[3, :300] == 0).all() and (got[3, 301:] == 0).all()
        assert (got[1] == 0).all()
    assert torch.isfinite(s).all()


@pytest.mark.parametrize("H", [264, 4096])
def test_norm_in_place(H):
    T = 37
    rng = np.random.default_rng(H)
    (x, xd), (r, rd) = bf16(rng.standard_normal((T, H))), bf16(rng.standard_normal((T, H)))
    for where in ("h in residual", "h in x", "y in x, h in residual", "y in residual"):
        dx, dr = x.to(DEV), r.to(DEV)
        h = dr if "h in residual" in where else dx if "h in x" in where else torch.empty_like(dx)
        y = dx if "y in x" in where else dr if "y in residual" in where else torch.empty_like(dx)
        P.moe_proj_norm(dx, None, 1e-6, dr, h, y)
        check_norm(xd, rd, None, 1e-6, h, y, None, None, f"norm {T}x{H}, {where}")


def fp8_case(T, N, K, seed, what=None, f8=False):
    rng = np.random.default_rng(seed)
    x, xs = PO.quantise(rng.standard_normal((T, K)) * np.exp(0.8 * rng.standard_normal(K)), 1)
    w, ws = PO.quantise(rng.standard_normal((N, K)) * np.exp(0.5 * rng.standard_normal((N, 1))), 128)
    what = what or f"fp8 {T}x{N}x{K}"
    print(f"[case] {what}", flush=True)
    y, ok = guarded((T, N), torch.bfloat16, 7.0)
    d = [torch.from_numpy(t).to(DEV) for t in (x, xs, w, ws)]
    if f8:
        d[0], d[2] = d[0].view(torch.float8_e4m3fn), d[2].view(torch.float8_e4m3fn)
    P.moe_proj_fp8(*d, y)
    torch.cuda.synchronize()
    assert ok(), f"{what}: written past the end"
    want, mag, tops = PO.fp8_product(x, xs, w, ws)
    assert_within(y.double().cpu().numpy(), want, fp8_bound(want, mag, tops, K), what)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 32, 33, 48, 63, 64, 65, 100, 127, 128, 129, 200, 256, 257, 300, 513])
def test_fp8_rows(T):
    fp8_case(T, 272, 640, T)


@pytest.mark.parametrize("N", [16, 32, 112, 128, 144, 240, 256, 272, 400, 528])
def test_fp8_columns(N):
    fp8_case(5, N, 384, N)
    fp8_case(300, N, 384, N)


@pytest.mark.parametrize("K", [128, 256, 384, 896, 1024, 1152, 2048, 4224])
def test_fp8_sums(K):
    fp8_case(3, 48, K, K, f8=True)
    fp8_case(160, 144, K, K)


@pytest.mark.parametrize("K", [128, 256, 384, 512, 640, 896, 1152])
def test_fp8_larger_calls(K):
    """Blocks of every size (32 x 16, 32 x 32, 64 x 32, 64 x 64 and 32 x 32 again, tiles of 128 x 128, fewer and more
    than the GPU has CUs, and of 256 x 256), with rows past their ends, and with numbers of spans that leave a group of
    scales unfilled at the end of the last row."""
    for i, (T, N) in enumerate(((100, 1040), (16, 12304), (200, 1040), (300, 1040), (700, 1040), (1024, 1024),
                                (1100, 1040), (2049, 528), (1500, 1552), (2049, 2960), (3000, 2960), (2305, 3600))):
        fp8_case(T, N, K, i)


def test_fp8_keeps_not_finite_rows_to_themselves():
    T, N, K = 70, 64, 256
    rng = np.random.default_rng(8)
    x, xs = PO.quantise(rng.standard_normal((T, K)), 1)
    w, ws = PO.quantise(rng.standard_normal((N, K)), 128)
    x[3, 7] = 0x7F
    xs[65, 1] = np.inf
    w[9, 200] = 0xFF
    y = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
    P.moe_proj_fp8(*(torch.from_numpy(t).to(DEV) for t in (x, xs, w, ws)), y)
    got = y.float().cpu().numpy()
    assert np.isnan(got[3]).all() and np.isnan(got[:, 9]).all() and not np.isfinite(got[65]).any()
    rows, cols = np.ones(T, bool), np.ones(N, bool)
    rows[[3, 65]] = cols[9] = False
    want, mag, tops = PO.fp8_product(np.where(x == 0x7F, 0, x), np.where(np.isinf(xs), 1, xs), np.where(w == 0xFF, 0, w),
                                     ws)
    assert_within(got[rows][:, cols], want[rows][:, cols], fp8_bound(want, mag, tops, K)[rows][:, cols],
                  "fp8 beside NaN")


def lora_case(T, K, N, R, n, ids, seed, ranks=None, scales=True, in_place=False, pad=(0, 0, 0), what=""):
    rng = np.random.default_rng(seed)
    x, xd = bf16(rng.standard_normal((T, K + pad[0])))
    base, bd = bf16(rng.standard_normal((T, N + pad[1])))
    a, ad = bf16(rng.standard_normal((n, R, K)) * K ** -0.5)
    b, bbd = bf16(rng.standard_normal((n, N, R)) * R ** -0.5)
    s = (0.5 + rng.random(n)).astype(np.float32) if scales else None
    ids = np.asarray(ids, np.int32)
    if ranks is not None:          # nothing past an adapter's rank matters
        for i, r in enumerate(ranks):
            a[i, max(0, min(r, R)):] = float("nan")
            b[i, :, max(0, min(r, R)):] = float("nan")
    what = f"lora {T} tokens, {K} -> {R} -> {N}, {n} adapters {what}"
    print(f"[case] {what}", flush=True)
    live = (ids >= 0) & (ids < n)
    x[torch.from_numpy(~live)] = float("nan")
    dx, dbase = x.to(DEV)[:, :K], base.to(DEV)[:, :N]
    wide = torch.full((T, N + pad[2]), 7.0, dtype=torch.bfloat16, device=DEV)
    out = None if in_place else wide[:, :N]
    ad_ = P.Adapters(a.to(DEV), b.to(DEV), None if ranks is None else torch.tensor(ranks, dtype=torch.int32, device=DEV),
                     None if s is None else torch.from_numpy(s).to(DEV))
    need = P.moe_proj_lora_workspace_size(ad_, T)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)
    P.moe_proj_lora(ad_, dx, torch.from_numpy(ids).to(DEV), dbase, out, ws[:need])
    torch.cuda.synchronize()
    assert (ws[need:] == 255).all(), f"{what}: written past the workspace"
    assert in_place or (wide[:, N:] == 7.0).all(), f"{what}: written past the columns"
    got = dbase if in_place else out
    assert torch.equal(got[torch.from_numpy(~live).to(DEV)].cpu(), base[torch.from_numpy(~live), :N]), \
        f"{what}: a row without an adapter"
    want, mag, deep = PO.lora(xd[:, :K], bd[:, :N], ids, ad, bbd, ranks, s)
    assert_within(got.double().cpu().numpy(), want, lora_bound(want, mag, deep, K, R), what)


def mixed(T, n, seed, none=0.15):
    rng = np.random.default_rng(seed)
    return np.where(rng.random(T) < none, -1, rng.integers(0, n, T))


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 128, 200, 513])
@pytest.mark.parametrize("n", [1, 3, 70])
def test_lora_tokens(T, n):
    lora_case(T, 200, 136, 16, n, mixed(T, n, T), T + n)


@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 72, 128, 256])
def test_lora_ranks(R):
    lora_case(37, 264, 280, R, 4, mixed(37, 4, R), R)
    ranks = [R, max(1, R // 3), 0, R + 5, 1, -3, R - 1]
    lora_case(90, 136, 264, R, 7, mixed(90, 7, R), R, ranks=ranks, what=f"of ranks {ranks}")


@pytest.mark.parametrize("K", [8, 56, 64, 72, 1000, 4096])
@pytest.mark.parametrize("N", [8, 248, 256, 264, 1544])
def test_lora_features(K, N):
    lora_case(21, K, N, 16, 3, mixed(21, 3, K + N), K + N)


@pytest.mark.parametrize("in_place", [False, True])
def test_lora_strides(in_place):
    lora_case(70, 128, 264, 32, 5, mixed(70, 5, 1), 1, in_place=in_place, pad=(8, 40, 24), what="columns of wider tensors")
    lora_case(70, 128, 264, 32, 5, mixed(70, 5, 2), 2, scales=False, in_place=in_place)


@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 72, 128, 200, 256])
def test_lora_ranks_of_sorted_calls(R):
    """Tokens sorted by adapter: tiles of up to 16 and of up to 64 of them, ranks in up to four groups of 64."""
    n = 40
    ids = np.concatenate([np.full(70, 0), np.full(9, 1), mixed(81, n, R)])
    ranks = [R, max(1, R - 3), 1, 0, R // 2 + 1] * 8
    lora_case(160, 264, 280, R, n, ids, R, ranks=ranks, what="sorted")
    lora_case(160, 1096, 72, R, n, ids, R + 1, in_place=True, what="sorted, in place")


@pytest.mark.parametrize("T", [65, 127, 300, 513, 704, 705, 1000])
def test_lora_windows_of_few_adapters(T):
    """Several windows of 64 tokens, and from 705 on the same sorted."""
    lora_case(T, 136, 264, 16, 3, mixed(T, 3, T), T, what="in any order")
    lora_case(T, 72, 520, 72, 3, np.sort(mixed(T, 3, T)), T, ranks=[72, 5, 40], in_place=True, what="in runs")


@pytest.mark.parametrize("n", [511, 512, 700])
@pytest.mark.parametrize("T", [1, 64, 65, 200, 330])
def test_lora_many_adapters(T, n):
    """More adapters than one block sorts by: windows of 64 tokens; and the most that it does."""
    lora_case(T, 72, 136, 8, n, mixed(T, n, T + n), T + n, ranks=[1 + i % 8 for i in range(n)], what="many adapters")


def test_lora_sorts_long_calls():
    """More tokens than a wavefront of the sorting block holds at once, in any order and in runs."""
    lora_case(9000, 64, 72, 8, 5, mixed(9000, 5, 3), 3, what="any order")
    lora_case(8193, 64, 72, 8, 300, np.sort(mixed(8193, 300, 4))[::-1].copy(), 4, what="falling")


def test_lora_runs_and_extremes():
    runs = np.repeat([2, -1, 0, 1, 0, 7, 1 << 30, -(1 << 31)], [130, 3, 70, 1, 250, 64, 5, 9])
    lora_case(len(runs), 320, 520, 32, 3, runs, 11, what="in runs, some of them past the last adapter")
    lora_case(4097, 192, 264, 16, 2, np.repeat([1, 0], [1000, 3097]), 12, what="in two runs")
    lora_case(64, 640, 264, 64, 64, np.arange(64)[::-1].copy(), 13, what="one token of each")
    lora_case(50, 128, 136, 16, 3, np.full(50, -1), 14, what="none has any")
    lora_case(50, 128, 136, 16, 3, np.full(50, -1), 15, in_place=True, what="none has any, in place")
