"""Plain 64-bit implementations of the mixers beside the delta rule, for the tests: the token
recurrence of linear attention and its reverse, softmax attention one sequence at a time, and the
8-bit cache as a table of values.  CPU only; shares nothing with the library.

Beside each result comes the magnitude its roundings are measured by: the same sums with the
terms' absolute values, wherever the kernels round a term (to the element type) or add in fp32.
A rounding moves a term by at most half a step, U[dtype] of its value.
"""
from __future__ import annotations

import math

import numpy as np
import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
E4M3 = 2.0 ** -4


def f64(t):
    return None if t is None else t.detach().double().cpu()


def linear(q, k, v, g, S0, scale):
    """o [B,T,H,dv], the final state, and the magnitudes of both: every term (q.k) v and the state's
    own q_c S_cv, absolute."""
    B, T, H, dk = q.shape
    S = torch.zeros(B, H, dk, v.shape[-1], dtype=torch.float64) if S0 is None else S0.clone()
    a = g.expand(B, T, H).exp()
    o, mag = torch.zeros_like(v), torch.zeros_like(v)
    M = S.abs()
    for t in range(T):
        S = S * a[:, t, :, None, None] + k[:, t, :, :, None] * v[:, t, :, None, :]
        M = M * a[:, t, :, None, None] + (k[:, t, :, :, None] * v[:, t, :, None, :]).abs()
        o[:, t] = scale * (q[:, t, :, :, None] * S).sum(-2)
        mag[:, t] = abs(scale) * (q[:, t, :, :, None].abs() * M).sum(-2)
    return o, S, mag, M


def linear_grad(q, k, v, g, S0, do, dS, scale):
    """Gradients by the reverse recurrence, and their magnitudes."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    per_head = g.dim() == 1
    a = g.expand(B, T, H).exp()
    zero = torch.zeros(B, H, dk, dv, dtype=torch.float64)
    S = zero if S0 is None else S0
    states = [S]
    mags = [S.abs()]
    for t in range(T):
        kv = k[:, t, :, :, None] * v[:, t, :, None, :]
        states.append(states[-1] * a[:, t, :, None, None] + kv)
        mags.append(mags[-1] * a[:, t, :, None, None] + kv.abs())
    R = zero if dS is None else dS.clone()
    M = R.abs()
    out = {n: torch.zeros_like(x) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    out["dg"] = torch.zeros(B, T, H, dtype=torch.float64)
    mag = {n: torch.zeros_like(x) for n, x in out.items()}
    for t in range(T - 1, -1, -1):
        qd = scale * q[:, t, :, :, None] * do[:, t, :, None, :]
        R, M = R + qd, M + qd.abs()
        out["dq"][:, t] = scale * (states[t + 1] * do[:, t, :, None, :]).sum(-1)
        mag["dq"][:, t] = abs(scale) * (mags[t + 1] * do[:, t, :, None, :].abs()).sum(-1)
        out["dk"][:, t] = (R * v[:, t, :, None, :]).sum(-1)
        mag["dk"][:, t] = (M * v[:, t, :, None, :].abs()).sum(-1)
        out["dv"][:, t] = (R * k[:, t, :, :, None]).sum(-2)
        mag["dv"][:, t] = (M * k[:, t, :, :, None].abs()).sum(-2)
        R, M = R * a[:, t, :, None, None], M * a[:, t, :, None, None]
        out["dg"][:, t] = (R * states[t]).sum((-1, -2))
        mag["dg"][:, t] = (M * mags[t]).sum((-1, -2))
    out["dS_in"], mag["dS_in"] = R, M
    if per_head:
        out["dg"], mag["dg"] = out["dg"].sum((0, 1)), mag["dg"].sum((0, 1))
    return out, mag


def prompt(q, k, v, cu, scale, do=None):
    """o, lse (and the gradients), with the magnitudes of o and of the gradients; rows behind the last
    sequence stay NaN."""
    n, Hq, d = q.shape
    G = Hq // k.shape[1]
    nan = lambda *s: torch.full(s, math.nan, dtype=torch.float64)  # noqa: E731
    out = {"o": nan(n, Hq, d), "lse": nan(n, Hq)}
    if do is not None:
        out |= {"dq": nan(n, Hq, d), "dk": nan(*k.shape), "dv": nan(*k.shape)}
    mag = {x: torch.zeros_like(y) for x, y in out.items()}
    for a, b in zip(cu, cu[1:]):
        low = torch.ones(b - a, b - a, dtype=torch.bool).tril()
        if do is not None:
            out["dk"][a:b] = 0
            out["dv"][a:b] = 0
        for h in range(Hq):
            kh, vh, qh = k[a:b, h // G], v[a:b, h // G], q[a:b, h]
            s = torch.where(low, qh @ kh.T * scale, -math.inf)
            out["lse"][a:b, h] = torch.logsumexp(s, -1)
            p = torch.softmax(s, -1)
            out["o"][a:b, h] = p @ vh
            mag["o"][a:b, h] = p @ vh.abs()
            if do is not None:
                dh = do[a:b, h]
                dp = dh @ vh.T
                D = (dh * out["o"][a:b, h]).sum(-1, keepdim=True)
                ds = p * (dp - D) * scale
                # D is formed from the rounded o: its error is in units of sum |do| |o|
                dm = p * ((dp - D).abs() + (dh * out["o"][a:b, h]).abs().sum(-1, keepdim=True)) * abs(scale)
                out["dv"][a:b, h // G] += p.T @ dh
                mag["dv"][a:b, h // G] += p.T @ dh.abs()
                out["dq"][a:b, h] = ds @ kh
                mag["dq"][a:b, h] = dm @ kh.abs()
                out["dk"][a:b, h // G] += ds.T @ qh
                mag["dk"][a:b, h // G] += dm.T @ qh.abs()
    return out, mag


def e4m3_values():
    """The 127 non-negative finite values in code order, as float64."""
    c = np.arange(127)
    e, m = c // 8, c % 8
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def e4m3_round(x):
    """Nearest value, ties to the even code; beyond the largest value, the largest."""
    vals = e4m3_values()
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    up = np.clip(np.searchsorted(vals, a), 1, 126)
    lo, hi = vals[up - 1], vals[up]
    take = (a - lo > hi - a) | ((a - lo == hi - a) & (up % 2 == 0))
    r = np.where(take, hi, lo) * np.where(np.signbit(x), -1.0, 1.0)
    return np.where(np.isnan(x), np.nan, r)


def scale_of(x):
    x = np.abs(x[np.isfinite(x)])
    m = float(x.max()) if x.size else 0.0
    if m == 0.0:
        return 2.0 ** -100
    e = math.ceil(math.log2(m / 448.0) - 1e-12)
    while m > 448.0 * 2.0 ** e:
        e += 1
    while m <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    return 2.0 ** max(e, -100)


class Cache:
    """Codes' values and scales, page by page."""

    def __init__(self, kc, vc, ks, vs):
        val = lambda c: c.cpu().view(torch.uint8).view(torch.float8_e4m3fn).float().double().numpy()  # noqa: E731
        self.side = {"k": val(kc).copy(), "v": val(vc).transpose(0, 1, 3, 2).copy()}  # [pages, Hkv, P, d]
        self.scale = {"k": ks.cpu().double().numpy().copy(), "v": vs.cpu().double().numpy().copy()}

    def append(self, k, v, cu, held, table):
        P, pages = self.side["k"].shape[2], self.side["k"].shape[0]
        for name, x in (("k", k), ("v", v)):
            x, c, sc = x.numpy(), self.side[name], self.scale[name]
            for i in range(len(held)):
                pos, end = held[i], held[i] + cu[i + 1] - cu[i]
                while pos < end:
                    r, at = pos % P, pos // P
                    n = min(P - r, end - pos)
                    pg = table[i][at] if at < len(table[i]) else -1
                    rows = x[cu[i] + pos - held[i]:][:n]
                    pos += n
                    if not 0 <= pg < pages:
                        continue
                    for h in range(x.shape[1]):
                        s = scale_of(rows[:, h])
                        if r:
                            s = max(s, sc[pg, h])
                            if s > sc[pg, h]:
                                c[pg, h, :r] = e4m3_round(c[pg, h, :r] * (sc[pg, h] / s))
                        c[pg, h, r:r + n] = e4m3_round(np.clip(rows[:, h] / s, -448, 448))
                        sc[pg, h] = s

    def attend(self, q, ctx, table, scale):
        P, pages, Hkv = self.side["k"].shape[2], self.side["k"].shape[0], self.side["k"].shape[1]
        N, Hq, d = q.shape
        o, lse = torch.zeros(N, Hq, d, dtype=torch.float64), torch.full((N, Hq), -math.inf, dtype=torch.float64)
        mag = torch.zeros_like(o)
        for i in range(N):
            at = [(table[i][p // P], p % P) for p in range(min(ctx[i], len(table[i]) * P))]
            at = [(a, b) for a, b in at if 0 <= a < pages]
            if not at:
                continue
            pg, row = np.array([a for a, _ in at]), np.array([b for _, b in at])
            for h in range(Hq):
                hk = h // (Hq // Hkv)
                k = torch.from_numpy(self.side["k"][pg, hk, row] * self.scale["k"][pg, hk][:, None])
                v = torch.from_numpy(self.side["v"][pg, hk, row] * self.scale["v"][pg, hk][:, None])
                s = (k @ q[i, h]) * scale
                lse[i, h] = torch.logsumexp(s, 0)
                p = torch.softmax(s, 0)
                o[i, h], mag[i, h] = p @ v, p @ v.abs()
        return o, lse, mag


def close(label, got, want, mag, dtype, terms=2.0, fp32_terms=0.0):
    """|got - want| <= terms roundings to ``dtype`` of the magnitude, and ``fp32_terms`` roundings to fp32."""
    got, want, mag = f64(got), f64(want), f64(mag)
    assert got.shape == want.shape, (label, got.shape, want.shape)
    same = (got == want) | (got.isnan() & want.isnan())
    bound = (terms * U[dtype] + fp32_terms * U[torch.float32]) * torch.maximum(mag, want.abs()) + 1e-37
    bad = ~same & ~((got - want).abs() <= bound)
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{label}: {int(bad.sum())} of {bad.numel()} values off, first at {i}: {got[i]} for {want[i]}, "
                             f"bound {bound[i]}")
