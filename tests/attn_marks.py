"""Long sequences for the attention tests: values in which no tile of keys can be lost unnoticed, and the
definition in fp64 torch, so that it can run on the GPU for thousands of rows.

With values of mean 0 a row over n keys is a sum of n weighted values that nearly cancel, and 32 keys of 30000
change it by less than its rounding bound.  With marks, the keys of tile j (32 of them) have a value of about 1 in
dim j % D and next to nothing elsewhere: dim d of a row is then what the n / (32 D) tiles of its number
contribute, and a tile that is lost, or counted twice, is a large part of that.
"""
import numpy as np
import torch

from attn_util import E, U, bf16
from oracle import attn_oracle as AO

TILE = 32


def mark_values(b, seed=0):
    """Replaces the values of a batch (attn_util.make_batch, poisoned) by marked ones, in the cache too."""
    rng = np.random.default_rng(seed)
    D, P = b.cfg.head_dim, b.cfg.page_size
    vc = b.v.float().numpy()
    kc = np.zeros(tuple(b.k.shape), np.float32)          # not used: store() writes a key beside each value
    for i, (n, m) in enumerate(zip(b.lens, b.new)):
        v = 0.02 * rng.standard_normal(b.values[i].shape)
        at = np.arange(n)
        v[at, :, at // TILE % D] += 1.0 + 0.2 * rng.standard_normal((n, b.cfg.n_kv_heads))
        b.values[i] = bf16(v)[1]
        seen = AO.visible(n, m, b.cfg.window, b.cfg.n_sinks).any(axis=0) if n and m else np.zeros(n, bool)
        for t in np.nonzero(seen)[0]:
            AO.store(kc, vc, int(b.table[i, t // P]), t % P, np.zeros_like(b.values[i][t]), b.values[i][t])
    b.v = bf16(vc)[0]
    return b


def attend_torch(cfg, q, k, v, device):
    """oracle.attn_oracle.attend and the bound of attn_util, head by head in fp64 on `device`: (out, bound)."""
    q, k, v = (torch.from_numpy(np.ascontiguousarray(t)).double().to(device) for t in (q, k, v))
    m, n, G = q.shape[0], k.shape[0], cfg.n_heads // cfg.n_kv_heads
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    big = 0.0
    p = torch.arange(n - m, n, device=device)[:, None]
    key = torch.arange(n, device=device)[None, :]
    hidden = key > p
    if cfg.window:
        hidden |= (p - key >= cfg.window) & (key >= cfg.n_sinks)
    for h in range(cfg.n_heads):
        kk, vv = k[:, h // G], v[:, h // G]
        s = q[:, h] @ kk.T * cfg.scale
        s[hidden] = -torch.inf
        top = s.amax(dim=1, keepdim=True).clamp(min=-1e300)
        w = (s - top).exp()
        w /= w.sum(dim=1, keepdim=True).clamp(min=1e-300)
        out[:, h], mag[:, h] = w @ vv, w @ vv.abs()
        s = q[:, h].abs() @ kk.abs().T * cfg.scale
        s[hidden] = 0.0
        big = max(big, float(s.max()))
    bound = U * (mag + out.abs()) + (2 * (cfg.head_dim + 16) * E * big + 2.0 ** -14) * mag
    return out.cpu().numpy(), bound.cpu().numpy()
