"""Gradients of the packed prompts' attention where dP - D cancels, far from a sequence's start: rows
whose weight lies on one key, and values with much in common.  There an o that was rounded to bf16
(or formed from rounded probabilities) gives a D = do . o that is off by more than dS itself.

Bounds, derived from the arithmetic, with S = sum_j |dS_j| of a row, all in 64 bits:
  - dS is rounded to the element type once, and the gradient once: U |dS| |k| and U |dq|;
  - dq may be formed with a D that is off by up to 2^-10 S (bf16 elements; exact to fp32 otherwise), which
    moves it by 2^-10 S sum_j P_j |k_j|; dk always takes the corrected D;
  - dP and D are fp32 sums over the channels of terms |do v| and |do o|, d + 16 roundings at most, and
    P multiplies their difference; sums over n keys (rows) round n times more, relative to |dS| |k|;
  - a score's own rounding moves P, and with it dS, relative to itself: d + 16 roundings of sum |q k|."""
import math

import pytest
import torch

import gated_delta_rule_11_amd as kda
from tests import _mixers as mx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
LENS = [5, 430, 1, 300]


def inputs(kind, Hq, Hkv, d, dtype, lens=LENS, seed=0):
    gen = torch.Generator().manual_seed(seed + d)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    n, G, cu = sum(lens), Hq // Hkv, [0]
    for x in lens:
        cu.append(cu[-1] + x)
    q, k, v, do = rn(n, Hq, d), rn(n, Hkv, d), rn(n, Hkv, d), rn(n, Hq, d)
    if kind == "sink":  # every row of a sequence looks at its first key
        u = rn(Hkv, d)
        u *= math.sqrt(d) / u.norm(dim=-1, keepdim=True)
        k[cu[:-1]] = 1.5 * u
        q = 0.3 * q + u.repeat_interleave(G, 0) * torch.linspace(0.6, 1.4, n)[:, None, None]
    elif kind == "own":  # every row looks at itself
        q = 0.3 * q + k.repeat_interleave(G, 1) * torch.linspace(0.8, 1.6, n)[:, None, None]
    elif kind == "one late":  # a key in the middle, after many that have some weight
        for a, b in zip(cu, cu[1:]):
            k[a + (b - a) // 2] *= 3.0
            q[a:b] += 0.5 * k[a + (b - a) // 2].repeat_interleave(G, 0)
    else:  # the values of a head share a large part
        v += 8.0 * rn(Hkv, d)
    return {"q": q.to(dtype), "k": k.to(dtype), "v": v.to(dtype), "do": do.to(dtype), "cu": cu}


def reference(x, scale):
    """Gradients, and for each the bound's parts: roundings of dS, of D's remainder, of fp32 terms."""
    q, k, v, do = (mx.f64(x[y]) for y in ("q", "k", "v", "do"))
    n, Hq, d = q.shape
    G = Hq // k.shape[1]
    out = {y: torch.zeros_like(z) for y, z in (("dq", q), ("dk", k), ("dv", v))}
    part = {y: [torch.zeros_like(z) for _ in range(3)] for y, z in out.items()}
    for a, b in zip(x["cu"], x["cu"][1:]):
        low = torch.ones(b - a, b - a, dtype=torch.bool).tril()
        for h in range(Hq):
            qh, kh, vh, dh = q[a:b, h], k[a:b, h // G], v[a:b, h // G], do[a:b, h]
            s = torch.where(low, qh @ kh.T * scale, -math.inf)
            p = torch.softmax(s, -1)
            dp = dh @ vh.T
            o = p @ vh
            ds = p * (dp - (dh * o).sum(-1, keepdim=True)) * abs(scale)
            size = ds.abs().sum(-1, keepdim=True)
            f = p * (dh.abs() @ vh.abs().T + (dh * o).abs().sum(-1, keepdim=True)) * abs(scale)
            w = f + ds.abs() * (qh.abs() @ kh.abs().T * abs(scale) + b - a)  # fp32 terms of dS
            sg = math.copysign(1.0, scale)
            out["dq"][a:b, h] = sg * ds @ kh
            out["dk"][a:b, h // G] += sg * ds.T @ qh
            out["dv"][a:b, h // G] += p.T @ dh
            for y, (of, at) in (("dq", (ds.abs(), kh.abs())), ("dk", (ds.abs().T, qh.abs())), ("dv", (p.T, dh.abs()))):
                i = h if y == "dq" else h // G
                part[y][0][a:b, i] += of @ at
            part["dq"][1][a:b, h] = size * (p @ kh.abs())
            part["dq"][2][a:b, h] = w @ kh.abs()
            part["dk"][2][a:b, h // G] += w.T @ qh.abs()
            part["dv"][2][a:b, h // G] += (p * (qh.abs() @ kh.abs().T * abs(scale) + b - a)).T @ dh.abs()
    return out, part


@pytest.mark.parametrize("dtype,o_dtype", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (2, 2, 128)])
@pytest.mark.parametrize("kind", ["sink", "own", "one late", "shared values"])
def test_gradients(kind, Hq, Hkv, d, dtype, o_dtype):
    x = inputs(kind, Hq, Hkv, d, dtype)
    g = {y: (z.to(DEV) if y != "cu" else torch.tensor(z, dtype=torch.int32, device=DEV)) for y, z in x.items()}
    o, lse = kda.attn_prompt_fwd(g["q"], g["k"], g["v"], g["cu"], o_dtype=o_dtype)
    got = kda.attn_prompt_bwd(g["q"], g["k"], g["v"], g["cu"], o, lse, g["do"])
    torch.cuda.synchronize()
    want, part = reference(x, d ** -0.5)
    u = mx.U[dtype]
    for y in want:
        bound = 1.05 * u * part[y][0] + (2.0 ** -10 * part[y][1] if dtype == BF else 0.0) + (d + 16) * 2.0 ** -24 * part[y][2]
        err = (mx.f64(got[y]) - want[y]).abs()
        worst = (err / bound).max()
        assert bool((err <= bound).all()), (y, float(worst), float(err.norm() / want[y].norm()))
