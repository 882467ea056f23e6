"""The plain definitions of the operators around the halves of the layer, against closed forms and torch (CPU)."""
import numpy as np
import torch

from oracle import proj_oracle as PO


def test_e4m3_tables_agree_with_torch():
    every = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(every).view(torch.float8_e4m3fn).double().numpy()
    got = PO.decode(every)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = ~np.isnan(want)
    assert np.array_equal(got[fine], want[fine])
    assert np.array_equal(PO.encode(got[fine]), every[fine])


def test_e4m3_rounds_to_the_nearest_value():
    table = np.sort(PO.decode(np.arange(127)))
    rng = np.random.default_rng(0)
    v = np.concatenate([table, (table[1:] + table[:-1]) / 2, rng.uniform(0, 448, 4000), 2.0 ** rng.uniform(-14, 8.8, 4000)])
    v = np.concatenate([v, -v])
    got = PO.e4m3(v)
    want = torch.from_numpy(v).to(torch.float32).to(torch.float8_e4m3fn).double().numpy()
    assert np.all(np.abs(got - v) <= np.min(np.abs(table[None, :] - np.abs(v)[:, None]), axis=1) + 1e-15)
    exact = v.astype(np.float32) == v
    assert np.array_equal(got[exact], want[exact])


def test_norm_of_known_rows():
    h, y = PO.norm(np.array([[3.0, 4.0], [0.0, 0.0]]), None, np.array([1.0, 2.0]), 0.5)
    assert np.allclose(y, [[3 / np.sqrt(13.0), 8 / np.sqrt(13.0)], [0, 0]], rtol=1e-15)
    h, _ = PO.norm(np.array([[3.0, 4.0]]), np.array([[-1.0, 1.0]]), None, 0.0)
    assert np.array_equal(h, [[2.0, 5.0]])


def test_quantise_keeps_the_largest_value_of_a_block():
    rng = np.random.default_rng(1)
    v = rng.standard_normal((130, 300)) * np.exp(rng.standard_normal(300))
    v[:, 256:] = 0
    q, s = PO.quantise(v, 128)
    back = PO.decode(q) * PO.spread(s, 128, *v.shape)
    assert q.shape == v.shape and s.shape == (2, 3)
    assert np.all(back[:, 256:] == 0)
    assert np.all(np.abs(back - v) <= 2.0 ** -4 * np.abs(v) + 2.0 ** -10 * PO.spread(s, 128, *v.shape) + 1e-7 * np.abs(v))


def test_products_against_loops():
    rng = np.random.default_rng(2)
    x, xs = PO.quantise(rng.standard_normal((3, 256)), 1)
    w, ws = PO.quantise(rng.standard_normal((144, 256)), 128)
    y, mag, tops = PO.fp8_product(x, xs, w, ws)
    assert np.all(tops >= mag / 8 * (1 - 1e-12)) and np.all(tops >= np.abs(y) / 8 * (1 - 1e-12))
    for t, n in ((0, 0), (2, 127), (1, 128), (2, 143)):
        terms = [PO.decode(x[t, k]) * xs[t, k // 128] * PO.decode(w[n, k]) * ws[n // 128, k // 128] for k in range(256)]
        assert np.isclose(y[t, n], float(np.sum(terms)), rtol=1e-12)
        assert np.isclose(mag[t, n], float(np.sum(np.abs(terms))), rtol=1e-12)


def test_lora_against_whole_matrices():
    rng = np.random.default_rng(3)
    a, b = rng.standard_normal((2, 8, 24)), rng.standard_normal((2, 16, 8))
    x, base = rng.standard_normal((4, 24)), rng.standard_normal((4, 16))
    out, _, _ = PO.lora(x, base, [1, -1, 0, 2], a, b, [8, 3], [2.0, -0.5])
    assert np.array_equal(out[[1, 3]], base[[1, 3]])
    assert np.allclose(out[0], base[0] - 0.5 * (b[1, :, :3] @ a[1, :3]) @ x[0])
    assert np.allclose(out[2], base[2] + 2.0 * (b[0] @ a[0]) @ x[2])
