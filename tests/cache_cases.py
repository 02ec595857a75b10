"""Inputs and 64-bit references for the calls on the paged cache.

The references are plain numpy in float64, written from the definitions in
include/treeverify.h, one sequence, head and token at a time.  Inputs are numpy
float32 arrays that hold values of the storage type exactly, so that the
references see what the kernels see.
"""
from __future__ import annotations

import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_STEP = {k: torch.finfo(t).eps / 2 for k, t in TYPES.items()}


def as_type(x: np.ndarray, dtype: str) -> np.ndarray:
    """The nearest values of the storage type, as float32."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(TYPES[dtype]).float().numpy()


def to_gpu(x: np.ndarray, dtype: str | None = None) -> torch.Tensor:
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(TYPES[dtype])


def host(t: torch.Tensor) -> np.ndarray:
    t = t.detach().cpu()
    return t.float().numpy() if t.is_floating_point() else t.numpy()


class Cache:
    """A paged cache with physical blocks in no order; blocks that no table entry names hold NaN."""

    def __init__(self, seed, lens, hkv, d, dtype, block=16, spare=3, width=None):
        rng = np.random.default_rng(seed)
        self.rng, self.dtype, self.block, self.hkv, self.d = rng, dtype, block, hkv, d
        self.lens = np.asarray(lens, np.int32)
        b = len(lens)
        need = max(1, -(-int(max(lens)) // block))
        self.width = width or need
        nb = b * self.width + spare
        ids = rng.permutation(nb).astype(np.int32)
        self.table = ids[:b * self.width].reshape(b, self.width).copy()
        self.spare = ids[b * self.width:].copy()
        self.k = np.full((nb, block, hkv, d), np.nan, np.float32)
        self.v = np.full_like(self.k, np.nan)
        for i, n in enumerate(lens):  # slots past a sequence's end stay NaN
            for t in range(0, int(n), block):
                m = min(block, int(n) - t)
                blk = self.table[i, t // block]
                self.k[blk, :m] = as_type(rng.standard_normal((m, hkv, d)), dtype)
                self.v[blk, :m] = as_type(rng.standard_normal((m, hkv, d)), dtype)

    def rows(self, cache, b, h, n=None, table=None):
        """[n][D] float64: the first n rows of one head of sequence b."""
        n = int(self.lens[b]) if n is None else n
        t = np.arange(n)
        tab = self.table if table is None else table
        return cache[tab[b][t // self.block], t % self.block, h].astype(np.float64)


# ------------------------------------------------------------------ references

def decode_reference(c: Cache, q: np.ndarray, weights=None, scale=None):
    """(out, lse, weights) in float64, and the bounds of their errors (see decode_bounds)."""
    b, hq, d = q.shape
    g = hq // c.hkv
    scale = d ** -0.5 if scale is None else scale
    out = np.zeros((b, hq, d))
    lse = np.full((b, hq), -np.inf)
    w = None if weights is None else weights.astype(np.float64)
    tol_out, tol_lse = np.zeros_like(out), np.zeros_like(lse)
    tol_w = None if w is None else np.zeros_like(w)
    for i in range(b):
        n = int(c.lens[i])
        if n == 0:
            continue
        for h in range(hq):
            k, v = c.rows(c.k, i, h // g), c.rows(c.v, i, h // g)
            s = scale * (k @ q[i, h].astype(np.float64))
            m = s.max()
            e = np.exp(s - m)
            p = e / e.sum()
            out[i, h] = p @ v
            lse[i, h] = m + np.log(e.sum())
            size = scale * (np.abs(k) @ np.abs(q[i, h]).astype(np.float64))
            ds, rel = decode_bounds(size.max(), n, d)
            tol_out[i, h] = rel * (p @ np.abs(v)) + HALF_STEP[c.dtype] * np.abs(out[i, h]) * (1 + rel)
            tol_lse[i, h] = ds + 2 ** -20 + 2 ** -22 * abs(lse[i, h])
            if w is not None:
                w[i, h // g, :n] += p
                tol_w[i, h // g, :n] += rel * p
    if w is not None:
        # one fp32 addition to the old sum
        tol_w += 2 ** -23 * np.abs(w) * (tol_w > 0)
    return (out, lse, w), (tol_out, tol_lse, tol_w)


def decode_bounds(size: float, n: int, d: int):
    """Bounds of the error of a score and, relative, of a weight and of the sum of weights times values.

    A score is d products added in fp32 (each addition off by at most 2^-23 of the sum of the
    magnitudes, `size`, whether it rounds or truncates), scaled (two roundings) and turned into base
    2, so it is off by ds = (d + 8) 2^-23 size.  A weight is an exponential (2^-22) of a score and a
    reference that cancels, over a sum of such: 2 ds + 2^-21, plus the additions of the sum.  Into the
    product with the values it goes as two 16-bit parts (what they leave is under 2^-16 of it for bf16,
    less for fp16).  A warp adds one 16-token tile after the other: at most n / 16 + 64 additions of
    2^-23 in a row, joins among them, for the sum and for the product."""
    ds = (d + 8) * 2 ** -23 * size
    return ds, 2 * ds + 2 ** -21 + 2 ** -16 + 2 * (n / 16 + 64) * 2 ** -23


def evict_reference(c: Cache, weights, budget, sink, recent, dst=None):
    """(k, v, weights_out, kept, new_lens), weights_out starting from a copy of `weights`."""
    k, v, w = c.k.copy(), c.v.copy(), weights.copy()
    b = len(c.lens)
    kept = np.full((b, c.hkv, budget), -1, np.int32)
    new = np.minimum(c.lens, budget).astype(np.int32)
    for i in range(b):
        n = int(c.lens[i])
        for h in range(c.hkv):
            if n <= budget:
                keep = np.arange(n)
            else:
                mid = np.arange(sink, n - recent)
                x = weights[i, h, mid].astype(np.float64)
                # NaN below every number, then by value, then the lower position first
                order = sorted(range(len(mid)), key=lambda j: (not np.isnan(x[j]), x[j] if not np.isnan(x[j]) else 0, -mid[j]),
                               reverse=True)
                best = mid[order[:budget - sink - recent]]
                keep = np.sort(np.concatenate([np.arange(sink), best, np.arange(n - recent, n)])).astype(int)
            kept[i, h, :len(keep)] = keep
            w[i, h, :n] = 0
            w[i, h, :len(keep)] = weights[i, h, keep]
            r = np.arange(len(keep))
            to = c.table if dst is None else dst
            for old, new_cache in ((c.k, k), (c.v, v)):
                rows = old[c.table[i][keep // c.block], keep % c.block, h]
                new_cache[to[i][r // c.block], r % c.block, h] = rows
    return k, v, w, kept, new


def depth_of(parent, j):
    d = 0
    while j > 0:
        j = int(parent[j])
        d += 1
    return d


def rotary_reference(x, pos, inv_freq, axis, interleaved):
    """x [H][D] float64 turned by positions pos[axis]; returns (result, |x| + |y| of each element's pair)."""
    y = x.astype(np.float64).copy()
    size = np.zeros_like(y)
    r = 2 * len(inv_freq)
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        angle = float(pos[axis[i]]) * float(f)
        cs, sn = np.cos(angle), np.sin(angle)
        xa, xb = x[:, a].astype(np.float64), x[:, b].astype(np.float64)
        y[:, a], y[:, b] = xa * cs - xb * sn, xa * sn + xb * cs
        size[:, a] = size[:, b] = np.abs(xa) + np.abs(xb)
    return y, size
