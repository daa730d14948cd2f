"""Plain 64-bit implementations of the serving calls around the paged cache, for the tests: rotary positions
by products of complex numbers, attention of a chunk of new tokens one row at a time.  CPU only; shares
nothing with the library."""
from __future__ import annotations

import math

import numpy as np
import torch


def turned(x, pos, inv, axes=None, interleaved=False, sign=1):
    """x [n,H,d] (float64) turned, and the magnitude |x_a cos| + |x_b sin| that its roundings are measured by."""
    x = x.double()
    half = inv.shape[0]
    pos = pos.double().reshape(x.shape[0], -1)
    at = pos[:, [0] * half] if axes is None else pos[:, axes.long().clamp(0, pos.shape[1] - 1)]
    angle = sign * at * inv.double()
    unit = torch.complex(angle.cos(), angle.sin())[:, None]
    y, mag = x.clone(), x.abs()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    c, s = unit.real, unit.imag
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    mag[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
    mag[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, mag


def frequencies(half, theta=1e4):
    return (theta ** (-torch.arange(half, dtype=torch.float64) / half)).float()


def places(cu, held):
    return torch.tensor([h + j for i, h in enumerate(held) for j in range(cu[i + 1] - cu[i])], dtype=torch.int64)


def chunk(cache, q, cu, ctx, table, scale):
    """o, lse and o's magnitude of the new tokens' rows, over an ``_mixers.Cache``; row r of sequence i sees the
    tokens up to ctx[i] - new + r that lie in a page of the cache.  Rows of no sequence stay NaN."""
    P, pages, Hkv = cache.side["k"].shape[2], cache.side["k"].shape[0], cache.side["k"].shape[1]
    n, Hq, d = q.shape
    o = torch.full((n, Hq, d), math.nan, dtype=torch.float64)
    lse, mag = torch.full((n, Hq), math.nan, dtype=torch.float64), torch.zeros(n, Hq, d, dtype=torch.float64)
    for i in range(len(ctx)):
        rows, new = slice(cu[i], cu[i + 1]), cu[i + 1] - cu[i]
        room = min(max(ctx[i], 0), len(table[i]) * P)
        tok = np.array([p for p in range(room) if 0 <= table[i][p // P] < pages], dtype=np.int64)
        pg = np.array([table[i][p // P] for p in tok], dtype=np.int64)
        seen = torch.from_numpy(tok)[None] <= torch.arange(max(ctx[i], 0) - new, max(ctx[i], 0))[:, None]
        some = seen.any(1)
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            k = torch.from_numpy(cache.side["k"][pg, hk, tok % P] * cache.scale["k"][pg, hk][:, None]).reshape(-1, d)
            v = torch.from_numpy(cache.side["v"][pg, hk, tok % P] * cache.scale["v"][pg, hk][:, None]).reshape(-1, d)
            w = torch.where(seen, q[rows, h] @ k.T * scale, -math.inf)
            lse[rows, h] = torch.logsumexp(w, -1) if tok.size else -math.inf
            p = torch.where(some[:, None], torch.softmax(w, -1), 0.0)
            p = torch.where(seen, p, 0.0)
            # a term that a row does not see is no term, whatever the value
            o[rows, h] = p @ v if bool(v.isfinite().all()) else torch.where(seen[..., None], p[..., None] * v, 0.0).sum(1)
            mag[rows, h] = p @ v.nan_to_num(0, 0, 0).abs()
    return o, lse, mag
