"""Inputs and element-wise error bounds of the attention tests.

A batch is built on the host: tokens in bf16, pages in a shuffled order, and a
cache in which every slot that no query sees holds NaN and every page-table
entry without a visible key an id far out of range.

Bounds (u = 2^-8, the rounding of a value to bf16; e = 2^-24, to fp32):
  attention: the weights are rounded to bf16 (u sum w|v|) and the result once
  (u |ref|); a score's fp32 error is at most (D + 16) e times
  scale sum |q||k| and moves every weight by twice that, relatively; the
  fp32 sums over keys add no more than 2^-14 of sum w|v| (exp2, rescaling and
  the sums, each a few e per 32 keys).
  prepare: one rounding to bf16 of a value computed in fp32 from the pair
  (a, b) it is rotated in: u |ref| + (D + 16) e (|a| + |b|).
"""
import dataclasses

import numpy as np
import torch

from oracle import attn_oracle as AO

U, E = 2.0 ** -8, 2.0 ** -24


def bf16(x):
    """fp array -> (torch bf16, its values in fp64)."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)
    return t, t.double().numpy()


@dataclasses.dataclass
class Batch:
    cfg: object
    lens: list
    new: list
    q: torch.Tensor            # [T, H, D] bf16
    k: torch.Tensor            # cache
    v: torch.Tensor
    table: torch.Tensor        # [B, pages] int32
    keys: list                 # per sequence [n, K, D] fp64
    values: list
    qs: list                   # per sequence [m, H, D] fp64

    def expected(self):
        """Per sequence (out, bound)."""
        c, D, res = self.cfg, self.cfg.head_dim, []
        for q, k, v in zip(self.qs, self.keys, self.values):
            out, mag, big = AO.attend(q, k, v, c.scale, c.window, c.n_sinks)
            bound = U * (mag + np.abs(out)) + (2 * (D + 16) * E * big + 2.0 ** -14) * mag
            res.append((out, bound))
        return res


def make_batch(cfg, lens, new, seed, v_mean=0.0, poison=True, extra_pages=2, q_std=1.5):
    rng = np.random.default_rng(seed)
    H, K, D, P = cfg.n_heads, cfg.n_kv_heads, cfg.head_dim, cfg.page_size
    B, T = len(lens), sum(new)
    width = max(1, max(-(-n // P) for n in lens))
    need = sum(-(-n // P) for n in lens) + extra_pages
    order = rng.permutation(need)
    hole = float("nan") if poison else 0.0
    kc = np.full((need, K, D // 8, P, 8), hole, np.float32)
    vc = np.full((need, K, P // 8, D, 8), hole, np.float32)
    table = np.full((B, width), -2 ** 31 if poison else 0, np.int64)
    q, qd = bf16(rng.standard_normal((T, H, D)) * q_std)
    keys, values, qs, at, row = [], [], [], 0, 0
    for b, (n, m) in enumerate(zip(lens, new)):
        _, k = bf16(rng.standard_normal((n, K, D)))
        _, v = bf16(rng.standard_normal((n, K, D)) + v_mean)
        seen = AO.visible(n, m, cfg.window, cfg.n_sinks).any(axis=0) if n and m else np.zeros(n, bool)
        if not poison:
            seen[:] = True
        for j in range(-(-n // P)):
            hit = np.nonzero(seen[j * P:(j + 1) * P])[0] + j * P
            if hit.size:
                table[b, j] = order[at]
                at += 1
                for t in hit:
                    AO.store(kc, vc, table[b, j], t % P, k[t], v[t])
            elif poison:
                table[b, j] = 2 ** 31 - 1 if j % 2 else -2 ** 31
        keys.append(k)
        values.append(v)
        qs.append(qd[row:row + m])
        row += m
    return Batch(cfg, list(lens), list(new), q, bf16(kc)[0], bf16(vc)[0], torch.from_numpy(table.astype(np.int32)),
                 keys, values, qs)


def assert_within(got, want, bound, what):
    got = np.asarray(got, np.float64)
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    over = np.abs(got - want) - bound
    worst = float(np.max(np.abs(got - want) / np.maximum(bound, 1e-300))) if got.size else 0.0
    print(f"[parity] {what}: worst error {worst:.3f} of its bound", flush=True)
    assert over.size == 0 or float(np.max(over)) <= 0.0, f"{what}: {worst} times the bound"
