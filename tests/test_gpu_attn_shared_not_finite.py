"""GPU tests of decode behind a shared prefix with values that are not finite: a sequence that sees one has it in its
own output, in that dim of the heads of that group, and every other output is what it is with zeros in their places.
Bounds as in attn_util.py."""
import pytest
import torch

from test_gpu_attn_shared import DEV, Shared, check_on_gpu, config

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def not_finite_case(heads, kv, dim, page, shared, lens, n_q, window, sinks, marks, seed):
    """marks: (key of the prefix, key/value head, dim, value), of different dims for one key/value head."""
    what = f"shared {heads}/{kv}x{dim}, {len(lens)} x {n_q} behind {shared}, lens {lens[:6]}, window {window}+{sinks}, " \
           f"not finite: {[m[0] for m in marks]}"
    print(f"[case] {what}", flush=True)
    s = Shared(config(heads, kv, dim, page, window, sinks), shared, lens, n_q, seed)
    s.lead = s.lead[0], s.lead[1].copy()
    pages, group = s.pages.cpu().numpy(), heads // kv
    sees, value = torch.zeros(s.dq.shape, dtype=torch.bool), torch.zeros(s.dq.shape)

    def put(zero):
        for key, h, d, x in marks:
            s.v[int(pages[key // page]), h, key % page // 8, d, key % 8] = 0.0 if zero else x

    for key, h, d, x in marks:
        s.lead[1][key, h, d] = 0.0
        for b, n in enumerate(lens):
            for m in range(n_q):
                p = n - n_q + m
                if key <= p and (not window or p - key < window or key < sinks):
                    sees[b, m, h * group:(h + 1) * group, d] = True
                    value[b, m, h * group:(h + 1) * group, d] = x
    assert sees.flatten(1).any(1).any(), what
    put(zero=True)
    plain = s.run()
    check_on_gpu(s, plain, what + ", with zeros there")
    put(zero=False)
    out, sees, value = s.run(), sees.to(DEV), value.to(DEV)
    got = out.float()[sees]
    same = (got == value[sees]) | (torch.isnan(got) & torch.isnan(value[sees]))
    assert bool(same.all()), f"{what}: {int((~same).sum())} of {same.numel()} outputs of those who see them"
    # all other outputs are those with zeros there (sums in another order); the ones above are taken from there too
    check_on_gpu(s, torch.where(sees, plain, out), what)


def marks_of(keys, kv, dim):
    """+inf, -inf and NaN in turn, each in a dim and a key/value head of its own."""
    return [(k, i % kv, (5 + 11 * i) % dim, (INF, -INF, NAN)[i % 3]) for i, k in enumerate(keys)]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n_q", [1, 3])
def test_sequences_that_end_before_it(dim, n_q):
    lens = [0, 3, 50, 129, 130, 131, 200, 230, 340]
    not_finite_case(8, 2, dim, 16, 203, lens, n_q, 0, 0, marks_of([0, 48, 49, 129, 130, 160, 202], 2, dim), 1)
    not_finite_case(8, 2, dim, 32, 203, lens * 4, n_q, 0, 0, marks_of([2, 127, 128, 199, 201], 2, dim), 2)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("sinks", [0, 9])
def test_windows_that_have_passed_it(dim, sinks):
    lens = [210, 0, 230, 260, 120, 204, 30]
    marks = marks_of([8, 29, 100, 119, 180, 191, 202], 2, dim)
    not_finite_case(8, 2, dim, 16, 203, lens, 1, 40, sinks, marks, 3)
    not_finite_case(8, 2, dim, 16, 203, lens * 5, 2, 41, sinks, marks, 4)


@pytest.mark.parametrize("heads,kv,dim,page,shared,B", [(64, 8, 64, 32, 13001, 128), (32, 8, 128, 16, 16379, 64),
                                                        (64, 4, 128, 64, 9001, 64), (16, 1, 256, 64, 4100, 64)])
@pytest.mark.parametrize("window", [0, 900])
def test_wide_blocks(heads, kv, dim, page, shared, B, window):
    lens = [(shared + 1, 0, 333, shared + 250, shared // 2, shared - 1, shared + 77, 1500)[b % 8] for b in range(B)]
    keys = [0, 332, 333, 500, 1499, shared // 2 - 1, shared - 800, shared - 2] if not window else \
        [332, 1400, shared // 2 - 3, shared - 800, shared - 2]
    not_finite_case(heads, kv, dim, page, shared, lens, 1, window, 0, marks_of(keys, kv, dim), 5)


def test_values_that_everyone_sees():
    """Nothing to keep apart: the same outcome."""
    not_finite_case(8, 2, 128, 16, 203, [210, 260, 204], 1, 0, 0, marks_of([0, 100, 202], 2, 128), 6)
    not_finite_case(32, 8, 128, 16, 16379, [16380 + 9 * (b % 5) for b in range(64)], 1, 0, 0,
                    marks_of([77, 9000, 16378], 8, 128), 7)
