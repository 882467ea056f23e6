"""Pins of the fp64 attention oracle against closed forms and brute force (CPU)."""
import math

import numpy as np
import pytest

from oracle import attn_oracle as AO


def test_visible_against_the_definition():
    for n, m, w, s in [(7, 3, 0, 0), (7, 7, 2, 1), (9, 4, 1, 0), (3, 6, 0, 0), (12, 5, 4, 20), (10, 2, 3, 2)]:
        got = AO.visible(n, m, w, s)
        for i in range(m):
            p = n - m + i
            for k in range(n):
                want = k <= p and (w == 0 or p - k < w or k < s)
                assert bool(got[i, k]) == want


def test_attend_brute_force():
    rng = np.random.default_rng(0)
    n, m, H, K, D = 11, 4, 6, 2, 8
    q, k, v = rng.standard_normal((m, H, D)), rng.standard_normal((n, K, D)), rng.standard_normal((n, K, D))
    for w, s in [(0, 0), (3, 0), (3, 2)]:
        out, mag, _ = AO.attend(q, k, v, 0.4, w, s)
        for i in range(m):
            for h in range(H):
                p = n - m + i
                ks = [j for j in range(n) if j <= p and (w == 0 or p - j < w or j < s)]
                e = [math.exp(0.4 * float(q[i, h] @ k[j, h // 3])) for j in ks]
                want = sum(x * v[j, h // 3] for x, j in zip(e, ks)) / sum(e)
                assert np.allclose(out[i, h], want, rtol=1e-12, atol=1e-14)
                assert np.all(mag[i, h] >= np.abs(out[i, h]) - 1e-12)


def test_attend_empty_rows_and_equal_scores():
    v = np.arange(12.0).reshape(3, 1, 4)
    out, _, _ = AO.attend(np.zeros((5, 2, 4)), np.ones((3, 1, 4)), v, 1.0, 0, 0)
    assert np.all(out[:2] == 0)                            # positions -2 and -1 see nothing
    for i in range(3):
        assert np.allclose(out[2 + i], np.mean(v[:i + 1, 0], axis=0))
    out, _, _ = AO.attend(np.ones((1, 1, 4)), np.zeros((0, 1, 4)), np.zeros((0, 1, 4)), 1.0, 0, 0)
    assert np.all(out == 0)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_is_a_rotation_that_depends_on_distance(inter):
    rng = np.random.default_rng(1)
    t = AO.rope_table(50, 16)
    a, b = rng.standard_normal(32), rng.standard_normal(32)
    ra, rb = (lambda p: AO.norm_rope(a, None, 0.0, t[p], inter)), (lambda p: AO.norm_rope(b, None, 0.0, t[p], inter))
    assert np.allclose(np.linalg.norm(ra(17)), np.linalg.norm(a))
    assert np.array_equal(ra(17)[16:], a[16:])
    assert np.allclose(ra(9) @ rb(4), ra(39) @ rb(34), atol=1e-5)      # the table is fp32
    assert np.allclose(ra(0), a)


def test_norm():
    x = np.array([[3.0, 4.0]])
    y = AO.norm_rope(x, np.array([1.0, 2.0]), 0.5, np.zeros((1, 0)), False)
    assert np.allclose(y, [[3.0 / math.sqrt(13.0), 8.0 / math.sqrt(13.0)]])


def test_store_and_load():
    K, D, P = 2, 16, 16
    kc, vc = np.zeros((3, K, D // 8, P, 8)), np.zeros((3, K, P // 8, D, 8))
    k, v = np.arange(K * D).reshape(K, D) + 1.0, -np.arange(K * D).reshape(K, D) - 1.0
    AO.store(kc, vc, 1, 11, k, v)
    assert kc[1, 1, 1, 11, 3] == k[1, 11] and vc[1, 0, 1, 5, 3] == v[0, 5]
    assert np.count_nonzero(kc) == K * D and np.count_nonzero(vc) == K * D
    a, b = AO.load(kc, vc, 1, 11)
    assert np.array_equal(a, k) and np.array_equal(b, v)
    assert AO.place(37, [5, 6, 7], 16) == (7, 5)
