"""Inputs and plain 64-bit forms for the tests of nexus_append, nexus_quantize and
nexus_attend. Rows that no slice holds are NaN (in the image: NaN codes and scales)."""
from __future__ import annotations

import math

import numpy as np
import torch

DEV = "cuda:0"


class Case:
    def __init__(self, seqs=1, kv_heads=2, group=2, d=128, dtype=torch.bfloat16, page=0,
                 capacity=64, lens=None, layers=1, seed=0, device=DEV, spare=2):
        """lens: [seqs][kv_heads] (or one number) for every layer."""
        self.rng = np.random.default_rng(seed)
        self.g = torch.Generator().manual_seed(seed)
        self.S, self.H, self.G, self.d, self.dtype, self.page = seqs, kv_heads, group, d, dtype, page
        self.L, self.dev = layers, torch.device(device)
        if page:
            self.per_seq = -(-capacity // page)
            capacity = self.per_seq * page
            self.pages = seqs * self.per_seq + spare
            self.table = torch.as_tensor(
                self.rng.permutation(self.pages)[:seqs * self.per_seq].reshape(seqs, -1)
                .astype(np.int32))
            self.shape = (layers, self.pages, kv_heads, page)
        else:
            self.per_seq = self.pages = 0
            self.table = None
            self.shape = (layers, seqs, kv_heads, capacity)
        self.capacity = capacity
        self.b = min(32, page) if page else 32
        self.lens = np.broadcast_to(np.asarray(0 if lens is None else lens, np.int32),
                                    (layers, seqs, kv_heads)).copy()
        self.k = torch.full((*self.shape, d), math.nan, dtype=dtype)
        self.v = torch.full((*self.shape, d), math.nan, dtype=dtype)
        self.pos = torch.full(self.shape, -7, dtype=torch.int32)
        for l in range(layers):
            for s in range(seqs):
                for h in range(kv_heads):
                    n = int(self.lens[l, s, h])
                    at = self.at(l, s, h, n)
                    self.k[at] = torch.randn(n, d, generator=self.g).to(dtype)
                    self.v[at] = torch.randn(n, d, generator=self.g).to(dtype)
                    self.pos[at] = torch.arange(n, dtype=torch.int32)

    def at(self, l, s, h, n, first=0):
        """Index of slots first .. n - 1 of a slice."""
        j = torch.arange(first, n)
        if self.page:
            return l, self.table[s].long()[j // self.page], h, j % self.page
        return l, s, h, j

    def device_cache(self):
        from streaming_kv_cache_step_gb300 import nexus
        put = lambda t: None if t is None else t.to(self.dev)  # noqa: E731
        return nexus.Cache(k=put(self.k), v=put(self.v), pos=put(self.pos),
                           lens=torch.as_tensor(self.lens, device=self.dev), layers=self.L,
                           seqs=self.S, kv_heads=self.H, group=self.G, head_dim=self.d,
                           capacity=self.capacity, page_size=self.page, num_pages=self.pages,
                           max_pages_per_seq=self.per_seq, block_table=put(self.table))

    def cu(self, n):
        return torch.as_tensor(np.concatenate([[0], np.cumsum(n)]).astype(np.int32))


def rotate64(x, pos, freqs, interleaved):
    """x [tokens, heads, d] float64, each pair turned by pos * freq."""
    x = x.clone()
    r = 2 * len(freqs)
    if not r:
        return x
    i = torch.arange(len(freqs))
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    ang = torch.tensor([[math.fmod(int(p) * f, 2 * math.pi) for f in freqs] for p in pos],
                       dtype=torch.float64).reshape(len(pos), 1, len(freqs))
    xa, xb = x[..., a], x[..., b]
    x[..., a], x[..., b] = (xa * ang.cos() - xb * ang.sin(), xb * ang.cos() + xa * ang.sin())
    return x


def norm64(x, w, eps):
    x = x.double()
    return x if w is None else x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()


def e4m3_grid():
    """The finite values of e4m3 (sign, 4 exponent bits of bias 7, 3 mantissa bits)."""
    mags = [m * 2.0 ** -9 for m in range(8)]
    mags += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)
             if not (e == 15 and m == 7)]
    return np.array(mags)


def quantize64(x):
    """x [rows, d]: (codes' values, scale) of one block, by search in the grid."""
    x = x.double().numpy()
    fin = np.abs(x[np.isfinite(x)])
    most = fin.max() if fin.size else 0.0
    scale = 1.0
    if most > 0:
        e = -100
        while most > 448 * 2.0 ** e and e < 120:
            e += 1
        scale = 2.0 ** e
    grid = e4m3_grid()
    y = np.abs(x / scale)
    yc = np.where(np.isnan(y), 0, np.minimum(y, 448.0))
    hi = np.searchsorted(grid, yc).clip(max=len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = yc - grid[lo], grid[hi] - yc
    # ties to the even code
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    val = np.copysign(grid[pick], x)
    return np.where(np.isnan(x), np.nan, val), scale


def attend64(q, k, v, M, scale):
    """One slice's softmax attention in float64. q [m, d]; k, v [T, d]; M [m] rows seen.
    Returns out, lse, A = sum p |v| / sum p and the largest sum |q_i k_i| of each row."""
    q, k, v = q.double(), k.double(), v.double()
    out = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64)
    A = torch.zeros_like(out)
    lse = torch.full((q.shape[0],), -math.inf, dtype=torch.float64)
    big = torch.zeros(q.shape[0], dtype=torch.float64)
    for i in range(q.shape[0]):
        n = int(M[i])
        if n <= 0:
            continue
        x = (k[:n] @ q[i]) * scale
        top = x.max()
        p = torch.exp(x - top)
        out[i], A[i] = p @ v[:n] / p.sum(), p @ v[:n].abs() / p.sum()
        lse[i] = top + torch.log(p.sum())
        big[i] = (k[:n].abs() @ q[i].abs()).max()
    return out, lse, A, big
