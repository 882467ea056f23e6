"""GPU tests of decode behind a shared prefix where the sequences of one block of columns see different keys of it:
windows beside sequences that end inside the prefix or have nothing.  Slots that no sequence sees hold NaN (Shared), the
tiles between two windows among them.  Bounds as in attn_util.py."""
import pytest

from test_gpu_attn_shared import Shared, case, check_on_gpu, config

pytestmark = pytest.mark.gpu

# heads, key/value heads, dims, page, prefix, sequences whose prefix is taken in wide column blocks: of 128 columns, and
# with 128 dims and 64 heads of 256
WIDE = [(64, 8, 64, 32, 13001, 128), (32, 8, 128, 16, 16379, 64), (64, 4, 128, 64, 9001, 64), (16, 1, 256, 64, 4100, 64)]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 0), (40, 3), (33, 50), (64, 0)])
def test_windows_beside_padded_rows(dim, window, sinks):
    case(8, 2, dim, 16, 203, [210, 0], window=window, sinks=sinks, seed=1)
    case(8, 2, dim, 16, 203, [0, 0, 333, 0, 211], window=window, sinks=sinks, seed=2)
    case(8, 2, dim, 16, 203, [0, 210, 0, 333] * 6, n_q=3, window=window, sinks=sinks, seed=3)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 0), (20, 5), (33, 70)])
@pytest.mark.parametrize("n_q", [1, 4])
def test_windows_of_sequences_that_end_inside_the_prefix(dim, window, sinks, n_q):
    """Windows with gaps between them, of whole tiles and of parts of one; n_q - 1: the first new tokens of some have
    no position."""
    lens = [500, 30, 0, 250, 399, 2, 251, 120, 401, 700]
    for shared in (400, 384, 97):
        case(8, 2, dim, 16, shared, lens, n_q=n_q, window=window, sinks=sinks, seed=shared)
        case(12, 1, dim, 32, shared, lens[::-1] * 2, n_q=n_q, window=window, sinks=sinks, seed=shared + 1)
    case(8, 2, dim, 16, 400, [60, 340], n_q=n_q, window=window, sinks=sinks, seed=5)


@pytest.mark.parametrize("heads,kv,dim,page,shared,B", WIDE)
@pytest.mark.parametrize("kind", ["padded", "inside", "few inside", "verify"])
def test_wide_blocks_with_windows(heads, kv, dim, page, shared, B, kind):
    n_q, window, sinks = 1, 700, 37
    if kind == "padded":
        lens = [shared + 1 + 211 * (b % 3) if b % 4 else 0 for b in range(B)]
    elif kind == "inside":
        window = 90
        lens = [(shared * (b % 11) // 9 + b) % (shared + 200) for b in range(B)]
    elif kind == "few inside":
        sinks = 0
        lens = [shared // 2 - 5 if b == 3 else 777 if b == B - 2 else shared + 40 + b for b in range(B)]
    else:
        n_q, B = 4, B // 4
        lens = [(2, 70, shared // 3, shared + 90, 0, shared - 1)[b % 6] for b in range(B)]
    what = f"wide: {heads}/{kv}x{dim}, {B} x {n_q} behind {shared}, window {window}+{sinks}, {kind}"
    print(f"[case] {what}", flush=True)
    s = Shared(config(heads, kv, dim, page, window, sinks), shared, lens, n_q, seed=dim + B)
    check_on_gpu(s, s.run(), what)
