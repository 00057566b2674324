"""Inputs, layouts and tolerances of the paged-cache and attention tests (no attention arithmetic)."""
from __future__ import annotations

import numpy as np
import torch


def gdn():
    import gated_deltanet_delta_amd as m
    m.lib()
    return m


def half_step(dtype) -> float:
    """The largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def tolerance(ref, mag, q, k, scale, n_keys, dtype):
    """Elementwise bound of |got - ref| for the attention kernels.

    ref: the fp64 result; mag = sum_j p_j |v_j|.  With u = 2^-24 and h the half step of dtype:
      - a logit is a sum of D products and a multiplication, in fp32: off by at most (D + 2) u A, where A is the
        largest scale sum_d |q_d k_d|; the base-2 exponential and its argument's scaling add (2 + |logit|) u at
        most, |logit| <= A; each weight, and the sum of the weights, is off by that factor: 2 (D + 5) u (A + 1);
      - the sums over keys: n u each (of p and of p v), 2 n u; running rescales, one rounding per 32 keys or more, are below that;
      - weights rounded to dtype for the product with V: h of mag (none for fp32);
      - the output's own rounding: h |ref|.
    """
    u, h = 2.0 ** -24, half_step(dtype)
    D = q.shape[-1]
    g = q.shape[-2] // k.shape[-2]
    A = scale * float(np.max(np.sum(np.abs(q).max(axis=tuple(range(q.ndim - 2)))
                                    * np.repeat(np.abs(k).max(axis=tuple(range(k.ndim - 2))), g, axis=0), axis=-1)))
    weights = 2 * (D + 5) * u * (A + 1) + 2 * n_keys * u
    return 1.02 * (h * np.abs(ref) + (weights + (h if dtype != torch.float32 else 0.0)) * mag) + 1e-30


def host(t) -> np.ndarray:
    return t.detach().double().cpu().numpy()


class Paged:
    """Random K and V pages with each row's tokens in pages of its own, in no order; everything that no row owns (spare
    pages, the tails of last pages) holds NaN."""

    def __init__(self, seed, ctx, Hk, D, page, dtype, spare=2, width_extra=1):
        g = torch.Generator().manual_seed(seed)
        need = [-(-c // page) for c in ctx]
        self.n_pages = sum(need) + spare
        self.width = max(need + [0]) + width_extra
        order = torch.randperm(self.n_pages, generator=g).to(torch.int32)
        self.table = torch.full((len(ctx), self.width), -7, dtype=torch.int32)
        nan = float("nan")
        self.k = torch.full((self.n_pages, Hk, page, D), nan, dtype=dtype)
        self.v = torch.full_like(self.k, nan)
        at = 0
        for i, (c, n) in enumerate(zip(ctx, need)):
            self.table[i, :n] = order[at:at + n]
            at += n
            for e in range(n):
                m = min(page, c - e * page)
                self.k[self.table[i, e], :, :m] = torch.randn(Hk, m, D, generator=g).to(dtype)
                self.v[self.table[i, e], :, :m] = torch.randn(Hk, m, D, generator=g).to(dtype)

    def cache(self):
        return gdn().KVCache(self.k.cuda(), self.v.cuda())


def qkv(seed, rows, Hq, Hk, D, dtype, fused):
    """q, k, v rows on the CPU: tensors of their own, or views of one fused row."""
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(rows, Hq + 2 * Hk, D, generator=g).to(dtype)
    parts = t[:, :Hq], t[:, Hq:Hq + Hk], t[:, Hq + Hk:]
    return t, parts if fused else tuple(p.contiguous() for p in parts)


def to_gpu(fused_rows, parts, fused, Hq, Hk):
    """The same rows on the GPU with the same layout."""
    if not fused:
        return tuple(p.cuda() for p in parts)
    t = fused_rows.cuda()
    return t[:, :Hq], t[:, Hq:Hq + Hk], t[:, Hq + Hk:]


def parents(seed, batch, n):
    """Random trees: every node hangs from an earlier one, or from the committed tokens (-1)."""
    rng = np.random.Generator(np.random.PCG64(seed))
    return np.stack([[int(rng.integers(-1, j)) if j else -1 for j in range(n)] for _ in range(batch)]).astype(np.int32)
