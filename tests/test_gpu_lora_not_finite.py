"""GPU tests of the adapters with infinite and very large values: what the definition gives, infinities with their signs
and NaN in the same places.  Bounds as in proj_util.py."""
import numpy as np
import pytest
import torch

from proj_util import assert_within, bf16, lora_bound
from oracle import proj_oracle as PO
from routed_expert_mlp_amd import projection as P

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run_lora(x, ids, base, a, b, scales=None, ranks=None):
    ad = P.Adapters(a.to(DEV), b.to(DEV), None if ranks is None else torch.tensor(ranks, dtype=torch.int32, device=DEV),
                    None if scales is None else torch.tensor(scales, dtype=torch.float32, device=DEV))
    out = torch.full_like(base, 7.0).to(DEV)
    P.moe_proj_lora(ad, x.to(DEV), torch.tensor(ids, dtype=torch.int32, device=DEV), base.to(DEV), out)
    torch.cuda.synchronize()
    return out


def inputs(T, K, N, R, n, seed):
    rng = np.random.default_rng(seed)
    x, base = rng.standard_normal((T, K)), rng.standard_normal((T, N))
    a, b = rng.standard_normal((n, R, K)) * K ** -0.5, rng.standard_normal((n, N, R)) * R ** -0.5
    return (bf16(t)[0] for t in (x, base, a, b))


# tokens and adapters whose products are taken in windows, and sorted
FORMS = [(37, 4), (300, 200)]


def check(out, x, ids, base, a, b, what):
    """Against the definition in fp64, infinities and NaN in the same places."""
    T, K = x.shape
    with np.errstate(invalid="ignore"):
        want, mag, deep = PO.lora(x.double().numpy(), base.double().numpy(), ids, a.double().numpy(), b.double().numpy(),
                                  None, None)
        got, fine = out.double().cpu().numpy(), np.isfinite(want)
        bad = ~((got == want) | (np.isnan(got) & np.isnan(want))) & ~fine
        assert not bad.any(), f"{what}: {int(bad.sum())} of {int((~fine).sum())} outputs, first {np.argwhere(bad)[0]}: " \
                              f"{got[bad][0]} for {want[bad][0]}"
        assert_within(got[fine], want[fine], lora_bound(want, mag, deep, K, a.shape[1])[fine], what)


@pytest.mark.parametrize("T,n", FORMS)
@pytest.mark.parametrize("R", [8, 40, 136])
def test_lora_of_infinite_inputs(T, n, R):
    """An infinity in a row of x makes all of its inner values infinite, and an output whose weights' signs agree with
    theirs is an infinity; where they do not, inf - inf, NaN."""
    K, N = 136, 72
    x, base, a, b = inputs(T, K, N, R, n, R)
    ids = np.arange(T) % n
    sign = torch.where(torch.arange(R) % 3 == 1, -1.0, 1.0)
    a[:, :, 9] = (0.5 * sign).to(torch.bfloat16)
    for j in range(0, N, 2):
        b[:, j] = (b[:, j].float().abs().clamp(min=0.01) * sign * (-1.0 if j % 4 else 1.0)).to(torch.bfloat16)
    x[3, 9], x[T - 1, 9] = float("inf"), float("-inf")
    out = run_lora(x, ids, base, a, b)
    check(out, x, ids, base, a, b, f"lora, x infinite, {T} tokens of {n} of rank {R}")
    assert torch.isinf(out[3, ::2]).all() and torch.isinf(out[T - 1, ::2]).all()


@pytest.mark.parametrize("T,n", FORMS)
def test_lora_of_rank_one_and_infinite_inputs(T, n):
    """Rank 1: an infinity times a weight is an infinity."""
    K, N, R = 136, 72, 8
    x, base, a, b = inputs(T, K, N, R, n, 3)
    ids = np.arange(T) % n
    x[5, 70], x[T - 2, 0] = float("-inf"), float("inf")
    out = run_lora(x, ids, base, a, b, ranks=[1] * n)
    a1, b1 = a[:, :1], b[:, :, :1]
    assert (a1 != 0).all() and (b1 != 0).all()
    check(out, x, ids, base, a1, b1, f"lora, rank 1, x infinite, {T} tokens")
    assert torch.isinf(out[5]).all() and torch.isinf(out[T - 2]).all()


@pytest.mark.parametrize("T,n", FORMS)
@pytest.mark.parametrize("R", [8, 40, 136])
def test_lora_of_infinite_weights(T, n, R):
    """Infinities in both sides' weights: their outputs alone, those of their adapter."""
    K, N = 72, 264
    x, base, a, b = inputs(T, K, N, R, n, R + 1)
    ids = np.arange(T) % n
    b[1, 7, R - 1] = float("inf")
    b[2, 200, 3] = float("-inf")
    b[0, N - 1, 0], b[0, N - 1, 1] = float("inf"), float("nan")
    check(run_lora(x, ids, base, a, b), x, ids, base, a, b, f"lora, weights infinite, {T} tokens of {n} of rank {R}")


@pytest.mark.parametrize("T,n", FORMS)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_lora_of_inner_values_at_the_end_of_fp32(T, n, sign):
    """An inner value of 2^128 - 2^112, which fp32 has and which would round to an infinity in bf16."""
    K, N, R = 64, 72, 8
    x, base, a, b = inputs(T, K, N, R, n, 5)
    ids = np.arange(T) % n
    x[4] = 0
    x[4, 10], x[4, 11] = 2.0 ** 64, 2.0 ** 64
    a[:, :, 10], a[:, :, 11] = 0, 0
    a[:, 2, 10], a[:, 2, 11] = sign * (2.0 ** 64 - 2.0 ** 56), sign * (2.0 ** 56 - 2.0 ** 48)
    b[:, :, 2] = b[:, :, 2] * 2.0 ** -110
    check(run_lora(x, ids, base, a, b), x, ids, base, a, b, f"lora, inner value at the end of fp32, {T} tokens")
