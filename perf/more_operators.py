"""Measured cases of what a serving step over the paged 8-bit cache needs beside it: rotary
positions of one or several axes and their gradient, appending keys and values with the rotation
on the way (the step's queries in the same call), and attention of a chunk of new tokens over the
cache.

With ``own`` false ``run`` computes each operator from elementary torch operations in 32 bits
(angles in 64: a far position times a frequency has to keep its fraction of a turn); with ``own``
true it makes the calls a user makes of the library.  ``exact`` is the definition in 64 bits, written
apart: complex products for the rotation, a table of the 8-bit format's values, the softmax one
sequence and key head at a time.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
E4M3_MAX = 448.0
LEAST_EXPONENT = -100  # of a page's scale: an all-zero page has 2^-100


def listed():
    return [
        # a decode step's queries: eight tokens far into their documents, launch-bound
        dict(name="rope_token", op="rope", n=8, H=32, more=0, d=128, rot=128, axes=1, turns=False, interleaved=False, far=131072, theta=1e6, dtype="bf16"),
        # a packed prompt's queries and keys, where they lie in the projection's output (8 value heads behind them)
        dict(name="rope_prompt", op="rope", n=16270, H=40, more=8, d=128, rot=128, axes=1, turns=False, interleaved=False, far=16270, theta=1e6, dtype="bf16"),
        # a training step over video: time, height and width, half of the channels, output and gradient, in single precision
        dict(name="rope_video", op="rope_train", n=9001, H=24, more=0, d=64, rot=32, axes=3, turns=True, interleaved=True, far=400, theta=1e4, dtype="f32"),
        # prompts go into the cache, some behind a page already begun, with their queries, as views of one projection
        dict(name="append_prompt", op="append", N=5, single=0, new_lo=400, new_hi=6000, held_lo=0, held_hi=777, Hq=32, Hkv=8, d=128, page=64, rot=128, axes=1, turns=False, interleaved=False, theta=1e6, fused=True, dtype="bf16"),
        # a decode step's one token for each sequence
        dict(name="append_token", op="append", N=256, single=256, new_lo=1, new_hi=1, held_lo=0, held_hi=1500, Hq=32, Hkv=8, d=128, page=64, rot=128, axes=1, turns=False, interleaved=False, theta=1e6, fused=True, dtype="bf16"),
        # images between text, positions given for three axes, in single precision
        dict(name="append_image", op="append", N=7, single=1, new_lo=33, new_hi=1100, held_lo=0, held_hi=300, Hq=0, Hkv=4, d=64, page=16, rot=64, axes=3, turns=False, interleaved=True, theta=1e4, fused=False, dtype="f32"),
        # a few tokens for three short sequences: a small model's step, latency
        dict(name="chunk_small", op="chunk", N=3, single=1, new_lo=2, new_hi=5, held_lo=0, held_hi=300, Hq=8, Hkv=2, d=64, page=16, dtype="f32"),
        # a verification step: five drafted tokens for each of 64 sequences
        dict(name="chunk_verify", op="chunk", N=64, single=0, new_lo=5, new_hi=5, held_lo=1, held_hi=8192, Hq=32, Hkv=8, d=128, page=64, dtype="bf16"),
        # a mixed batch: most sequences decode one token, some bring a piece of their prompt
        dict(name="chunk_mixed", op="chunk", N=32, single=26, new_lo=32, new_hi=256, held_lo=0, held_hi=6000, Hq=32, Hkv=8, d=128, page=16, dtype="bf16"),
        # whole prompts attended through the cache
        dict(name="chunk_prompt", op="chunk", N=4, single=0, new_lo=500, new_hi=2048, held_lo=0, held_hi=0, Hq=32, Hkv=8, d=128, page=32, dtype="bf16"),
        # a piece of one long document behind all that came before it
        dict(name="chunk_long", op="chunk", N=1, single=0, new_lo=1024, new_hi=1024, held_lo=64511, held_hi=64511, Hq=32, Hkv=8, d=128, page=64, dtype="bf16"),
        # single precision, odd lengths, six query heads to a key head
        dict(name="chunk_f32", op="chunk", N=4, single=0, new_lo=101, new_hi=700, held_lo=0, held_hi=1501, Hq=24, Hkv=4, d=64, page=32, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_train", "append", "append", "chunk", "chunk", "chunk"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 128])
    turn = dict(rot=rng.choice([d, d, d // 2, 48]), axes=rng.choice([1, 1, 2, 3]), turns=rng.random() < 0.5, interleaved=rng.random() < 0.5,
                theta=rng.choice([1e4, 5e5, 1e6]))
    if op.startswith("rope"):
        H = rng.choice([1, 2, 5, 8, 24, 32, 40])
        most = 16270 * 40 * 128 // (H * d) // (2 if op == "rope_train" else 1) // (2 if dtype == "f32" else 1)
        return dict(op=op, n=_log(rng, 1, min(60000, most)), H=H, more=rng.choice([0, 0, 1, 8]), d=d, far=_log(rng, 100, 1000000), dtype=dtype, **turn)
    Hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64])
    N = _log(rng, 1, 64 if op == "append" else 48)
    single = rng.choice([0, 0, N // 2, N])
    if op == "append":
        hi = _log(rng, 1, 16000 // N)
        G = rng.choice([0, 1, 2, 4])
        return dict(op=op, N=N, single=single, new_lo=rng.randint(1, hi), new_hi=hi, held_lo=0, held_hi=_log(rng, 1, 1500), Hq=G * Hkv, Hkv=Hkv, d=d, page=page,
                    fused=rng.random() < 0.5, dtype=dtype, **turn)
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    pairs = 1024 * 32 * 65536 * 128 // (N * Hq * d) // (8 if dtype == "f32" else 2)
    hi = _log(rng, 1, min(2048, int(pairs ** 0.5)))
    held = _log(rng, 1, max(1, min(65536, pairs // hi - hi, 2000000 // (N * Hkv))))
    return dict(op=op, N=N, single=single, new_lo=rng.randint(1, hi), new_hi=hi, held_lo=rng.randint(0, held), held_hi=held, Hq=Hq, Hkv=Hkv, d=d, page=page, dtype=dtype)


def _spread(n, lo, hi, salt=0):
    """n whole numbers over [lo, hi], the two ends among them, in a fixed mixed order."""
    r = random.Random(n * 1000003 + lo * 1009 + hi * 31 + salt)
    xs = [r.randint(lo, hi) for _ in range(n)]
    if n:
        xs[0] = hi
    if n > 1:
        xs[-1] = lo
    r.shuffle(xs)
    return xs


def _lengths(case):
    """New tokens and held tokens of each sequence."""
    one = case["single"]
    new = [1] * one + _spread(case["N"] - one, case["new_lo"], case["new_hi"])
    random.Random(case["N"]).shuffle(new)
    return new, _spread(case["N"], case["held_lo"], case["held_hi"], 1)


# ----------------------------------------------------------------- inputs

def _normal(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device=DEV) * std


def _int32(x):
    return torch.tensor(x, dtype=torch.int32).to(DEV)


def _plan(case):
    """Frequencies of the rotated pairs, and the axis each goes by: in blocks or in turns."""
    half, A = case["rot"] // 2, case["axes"]
    j = torch.arange(half, dtype=torch.float64)
    inv = (case["theta"] ** (-j / half)).float().to(DEV)
    if A == 1:
        return inv, None
    axes = torch.arange(half) % A if case["turns"] else torch.arange(half) * A // half
    return inv, axes.to(torch.int32).to(DEV)


def _prepare_rope(case, gen):
    n, H, d = case["n"], case["H"], case["d"]
    whole = _normal(gen, n, H + case["more"], d).to(TYPES[case["dtype"]])
    s = {"x": whole[:, :H]}
    s["inv"], s["axes"] = _plan(case)
    s["pos"] = torch.randint(0, case["far"], (n, case["axes"]), generator=gen, device=DEV, dtype=torch.int32)
    if case["axes"] == 1:  # positions that rise, up to the farthest
        s["pos"] = s["pos"][:, 0].sort().values.contiguous()
    if case["op"] == "rope_train":
        s["dy"] = _normal(gen, n, H, d).to(TYPES[case["dtype"]])
    s["interleaved"] = case["interleaved"]
    return s


def _table(case, room, gen):
    """A block table with pages in a mixed order, and how many pages there are."""
    P = case["page"]
    need = [-(-n // P) for n in room]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32).cpu()
    table, at = torch.zeros(len(room), max(1, max(need)), dtype=torch.int32), 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table.to(DEV), pages


def _filled(gen, pages, Hkv, rows, cols):
    """One side of a cache as earlier appends left it, and its scales."""
    x = torch.randn(pages, Hkv, rows, cols, generator=gen, device=DEV)
    x *= torch.exp(_normal(gen, pages, Hkv, 1, 1, std=0.5))
    scale = _scale_for(x.abs().amax((2, 3)))
    x /= scale[:, :, None, None]
    return x.to(torch.float8_e4m3fn), scale


def _prepare_cache(case, gen):
    Hq, Hkv, d, P, t = case["Hq"], case["Hkv"], case["d"], case["page"], TYPES[case["dtype"]]
    new, held = _lengths(case)
    n = sum(new)
    s = {"cu": _int32([0] + new).cumsum(0).to(torch.int32), "most_new": max(new)}
    s["table"], pages = _table(case, [a + b for a, b in zip(new, held)], gen)
    s["kc"], s["ks"] = _filled(gen, pages, Hkv, P, d)
    s["vc"], s["vs"] = _filled(gen, pages, Hkv, d, P)
    if case["op"] == "chunk":  # the new tokens' keys and values are in the cache
        s["ctx"] = _int32([a + b for a, b in zip(new, held)])
        s["q"], s["scale"] = _normal(gen, n, Hq, d).to(t), d ** -0.5
        return s
    s["held"] = _int32(held)
    whole = _normal(gen, n, Hq + 2 * Hkv, d)
    whole[:, Hq:] *= torch.exp(_normal(gen, n, 1, 1, std=0.7))  # some tokens are larger: a page's scale grows
    whole = whole.to(t)
    s["q"] = whole[:, :Hq] if Hq else None
    s["k"], s["v"] = whole[:, Hq:Hq + Hkv], whole[:, Hq + Hkv:]
    if not case["fused"]:
        s["q"], s["k"], s["v"] = (None if x is None else x.contiguous() for x in (s["q"], s["k"], s["v"]))
    s["inv"], s["axes"] = _plan(case)
    s["pos"] = None  # each token's place in its sequence
    if case["axes"] > 1:  # the place plus a patch's offsets
        at = torch.cat([torch.arange(a, a + b) for a, b in zip(held, new)]).to(DEV)
        s["pos"] = (at[:, None] + torch.randint(0, 64, (n, case["axes"]), generator=gen, device=DEV)).to(torch.int32)
    s["interleaved"] = case["interleaved"]
    return s


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(int(seed))
    s = (_prepare_rope if case["op"].startswith("rope") else _prepare_cache)(case, gen)
    s["op"] = case["op"]
    return s


# ------------------------------------------------- plain forms, in 32 bits

def _turned(x, pos, inv, axes, interleaved):
    """x [n,H,d] in fp32 with its pairs of channels turned; angles in 64 bits."""
    at = pos.view(x.shape[0], -1).double()
    at = at[:, :1] if axes is None else at[:, axes.long()]
    angle = at * inv.double()
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    half = inv.shape[0]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        r = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([r, rest], -1)


def _scale_for(amax):
    """The smallest power of two s with amax <= 448 s."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= E4M3_MAX / 512, e - 9, e - 8).clamp_min(LEAST_EXPONENT)
    return torch.ldexp(torch.ones_like(amax), e)


def _to_8bit(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _append_side(x, slot, off, first, touched, cache, scale):
    """x [n,Hkv,d] fp32 into rows `off` of the touched pages numbered `slot`; `first`: how
    many tokens each touched page held before.  cache [pages,Hkv,page,d] is written."""
    n, Hkv, d = x.shape
    need = torch.zeros(len(touched), Hkv, device=x.device)
    need.scatter_reduce_(0, slot[:, None].expand(n, Hkv), x.abs().amax(-1), "amax")
    old = scale[touched]
    begun = (first > 0)[:, None]
    new = torch.where(begun, torch.maximum(old, _scale_for(need)), _scale_for(need))
    page = cache.view(torch.uint8)[touched].view(torch.float8_e4m3fn).float()
    kept = (torch.arange(page.shape[2], device=x.device) < first[:, None])[:, None, :, None]
    page = torch.where(kept, page * (old / new)[..., None, None], page)
    page[slot, :, off] = x / new[slot][..., None]
    cache.view(torch.uint8)[touched] = _to_8bit(page).view(torch.uint8)
    scale[touched] = new


def _append_plain(s):
    cu, held, table = s["cu"].long(), s["held"].long(), s["table"].long()
    P = s["kc"].shape[2]
    at = torch.arange(s["k"].shape[0], device=DEV)
    seq = torch.bucketize(at, cu[1:], right=True)
    place = held[seq] + at - cu[seq]
    turn = [place if s["pos"] is None else s["pos"], s["inv"], s["axes"], s["interleaved"]]
    page = table[seq, place // P]
    touched, slot = torch.unique(page, return_inverse=True)
    first = torch.full_like(touched, P).scatter_reduce_(0, slot, place % P, "amin")
    _append_side(_turned(s["k"].float(), *turn), slot, place % P, first, touched, s["kc"], s["ks"])
    vt = s["vc"].view(torch.uint8).transpose(2, 3).contiguous().view(torch.float8_e4m3fn)
    _append_side(s["v"].float(), slot, place % P, first, touched, vt, s["vs"])
    s["vc"].view(torch.uint8).copy_(vt.view(torch.uint8).transpose(2, 3))
    return None if s["q"] is None else _turned(s["q"].float(), *turn).to(s["q"].dtype)


def _chunk_plain(s):
    """o [n,Hq,d] in fp32 and the log of the softmax' sum [n,Hq]; sequences side by side, filled up to the longest."""
    q, ctx, cu, t = s["q"].float(), s["ctx"].long(), s["cu"].long(), s["table"].long()
    n, Hq, d = q.shape
    N, Hkv, P, M = len(ctx), s["kc"].shape[1], s["kc"].shape[2], s["most_new"]
    G = Hq // Hkv
    new = cu[1:] - cu[:-1]
    i = torch.arange(M, device=DEV)
    row = (cu[:-1, None] + i).clamp_max(n - 1)
    q = (q * s["scale"])[row].view(N, M, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(N, Hkv, G * M, d)
    k = (s["kc"].view(torch.uint8)[t].view(torch.float8_e4m3fn).float() * s["ks"][t][..., None, None]).transpose(1, 2).reshape(N, Hkv, -1, d)
    w = q @ k.transpose(-1, -2)
    del k
    C = w.shape[-1]
    w = w.view(N, Hkv, G, M, C)
    last = (ctx - new)[:, None] + i  # the last token that a row sees: its own
    w.masked_fill_((torch.arange(C, device=DEV) > last[:, :, None])[:, None, None], -math.inf)
    m = w.amax(-1, keepdim=True)
    w = w.sub_(m).exp_()
    z = w.sum(-1, keepdim=True)
    v = (s["vc"].view(torch.uint8)[t].view(torch.float8_e4m3fn).float() * s["vs"][t][..., None, None]).permute(0, 2, 1, 4, 3).reshape(N, Hkv, -1, d)
    o = (w.view(N, Hkv, G * M, C) @ v).view(N, Hkv, G, M, d) / z
    lse = (m + z.log())[..., 0]
    own_rows = i < new[:, None]
    return o.permute(0, 3, 1, 2, 4).reshape(N, M, Hq, d)[own_rows], lse.permute(0, 3, 1, 2).reshape(N, M, Hq)[own_rows]


# --------------------------------------------------------------------- run

def _run_plain(s):
    op = s["op"]
    if op == "append":
        q = _append_plain(s)
        outs = {"k_cache": s["kc"], "v_cache": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}
        return outs if q is None else {**outs, "q": q}
    if op == "chunk":
        o, lse = _chunk_plain(s)
        return {"o": o.to(s["q"].dtype), "lse": lse}
    x, turn = s["x"], (s["pos"], s["inv"], s["axes"], s["interleaved"])
    if op == "rope":
        return {"y": _turned(x.float(), *turn).to(x.dtype)}
    leaf = x.float().detach().requires_grad_()
    with torch.enable_grad():
        y = _turned(leaf, *turn)
        (dx,) = torch.autograd.grad(y, leaf, s["dy"].float())
    return {"y": y.detach().to(x.dtype), "dx": dx.to(x.dtype)}


def _run_own(s):
    import gated_delta_rule_11_amd as kda

    op = s["op"]
    if op == "append":
        q = kda.kv_cache_append_rope(s["k"], s["v"], s["cu"], s["held"], s["table"], s["kc"], s["vc"], s["ks"], s["vs"], s["inv"],
                                     positions=s["pos"], axes=s["axes"], interleaved=s["interleaved"], q=s["q"])
        outs = {"k_cache": s["kc"], "v_cache": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}
        return outs if q is None else {**outs, "q": q}
    if op == "chunk":
        o, lse = kda.attn_chunk_fwd(s["q"], s["cu"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["ctx"], scale=s["scale"],
                                    o_dtype=s["q"].dtype, want_lse=True)
        return {"o": o, "lse": lse}
    y = kda.rope(s["x"], s["pos"], s["inv"], axes=s["axes"], interleaved=s["interleaved"])
    if op == "rope":
        return {"y": y}
    return {"y": y, "dx": kda.rope(s["dy"], s["pos"], s["inv"], axes=s["axes"], interleaved=s["interleaved"], inverse=True)}


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# -------------------------------------------------------------------- work

def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op, d = case["op"], case["d"]
    if op.startswith("rope"):
        n, both = case["n"], 2 if op == "rope_train" else 1
        return {"bytes": both * 2 * n * case["H"] * d * e + 4 * n * case["axes"] + 2 * case["rot"], "flops": both * 3 * n * case["H"] * case["rot"]}
    Hq, Hkv = case["Hq"], case["Hkv"]
    new, held = _lengths(case)
    n = sum(new)
    if op == "append":
        return {"bytes": 2 * n * Hkv * d * (e + 1) + 2 * n * Hq * d * e + 8 * Hkv * (case["N"] + n // case["page"]) + (4 * n * case["axes"] if case["axes"] > 1 else 0),
                "flops": 4 * n * Hkv * d + 3 * n * (Hq + Hkv) * case["rot"]}
    ctx = sum(new) + sum(held)
    pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(new, held)) * Hq
    return {"bytes": 2 * ctx * Hkv * d + 8 * Hkv * (ctx // case["page"]) + 2 * n * Hq * d * e + 4 * n * Hq, "flops": 4 * d * pairs}


# ------------------------------------------------- the definitions, 64 bits

def _exact_turned(x, at, s, sign=1):
    """Channel pairs as complex numbers, times e^(i angle); one axis after the other."""
    x, half = x.double(), s["inv"].shape[0]
    at = at.double().reshape(x.shape[0], -1)
    angle = torch.zeros(x.shape[0], half, dtype=torch.float64, device=DEV)
    for a in range(at.shape[1]):
        mine = torch.ones(half, dtype=torch.float64, device=DEV) if s["axes"] is None else (s["axes"] == a).double()
        angle += at[:, a:a + 1] * (s["inv"].double() * mine)
    unit = torch.polar(torch.ones_like(angle), sign * angle)[:, None]
    out = x.clone()
    if s["interleaved"]:
        z = torch.complex(x[..., 0:2 * half:2].contiguous(), x[..., 1:2 * half:2].contiguous()) * unit
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * unit
        out[..., :half], out[..., half:2 * half] = z.real, z.imag
    return out


def _table_round(x):
    """The nearest of the 8-bit format's values (4 exponent bits, 3 of mantissa), ties to the even code."""
    codes = torch.arange(127, dtype=torch.float64, device=DEV)
    e, m = (codes / 8).floor(), codes % 8
    values = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e - 10))
    up = torch.searchsorted(values, x.abs().contiguous()).clamp(1, 126)
    lo, hi = values[up - 1], values[up]
    far, near = hi - x.abs(), x.abs() - lo
    take = (near > far) | ((near == far) & (up % 2 == 0))
    return torch.where(take, hi, lo) * torch.where(x < 0, -1.0, 1.0)


def _exact_append(s):
    cu, held, table, P = s["cu"].tolist(), s["held"].tolist(), s["table"].tolist(), s["kc"].shape[2]
    out = {"k_cache": s["kc"].double(), "v_cache": s["vc"].double(), "k_scale": s["ks"].double(), "v_scale": s["vs"].double()}
    at = s["pos"]
    if at is None:
        at = torch.cat([torch.arange(h, h + b - a) for h, a, b in zip(held, cu, cu[1:])]).to(DEV)
    if s["q"] is not None:
        out["q"] = _exact_turned(s["q"], at, s)
    for side in ("k", "v"):
        x = _exact_turned(s["k"], at, s) if side == "k" else s["v"].double()
        cache = out[side + "_cache"] if side == "k" else out[side + "_cache"].transpose(2, 3)
        scale = out[side + "_scale"]
        for i in range(len(held)):
            a, end = held[i], held[i] + cu[i + 1] - cu[i]
            while a < end:
                n, r, pg = min(P - a % P, end - a), a % P, table[i][a // P]
                fresh = x[cu[i] + a - held[i]:][:n].transpose(0, 1)  # [Hkv, n, d]
                need = torch.exp2((fresh.abs().amax((1, 2)) / E4M3_MAX).log2().ceil().clamp_min(LEAST_EXPONENT))
                if r:
                    need = torch.maximum(need, scale[pg])
                    cache[pg, :, :r] = _table_round(cache[pg, :, :r] * (scale[pg] / need)[:, None, None])
                cache[pg, :, r:r + n] = _table_round(fresh / need[:, None, None])
                scale[pg] = need
                a += n
    return out


def _exact_chunk(s):
    q, P = s["q"].double(), s["kc"].shape[2]
    n, Hq, d = q.shape
    Hkv = s["kc"].shape[1]
    G = Hq // Hkv
    o, lse = torch.zeros_like(q), torch.empty(n, Hq, dtype=torch.float64, device=DEV)
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    for i, c in enumerate(ctx):
        rows, new = slice(cu[i], cu[i + 1]), cu[i + 1] - cu[i]
        at = s["table"][i, :-(-c // P)].long()
        hidden = torch.arange(c, device=DEV) > torch.arange(c - new, c, device=DEV)[:, None]
        for h in range(Hkv):
            k = (s["kc"].view(torch.uint8)[at, h].view(torch.float8_e4m3fn).double() * s["ks"][at, h].double()[:, None, None]).reshape(-1, d)[:c]
            v = (s["vc"].view(torch.uint8)[at, h].view(torch.float8_e4m3fn).double() * s["vs"][at, h].double()[:, None, None]).transpose(1, 2).reshape(-1, d)[:c]
            for g in range(h * G, h * G + G):
                w = (q[rows, g] @ k.T * s["scale"]).masked_fill_(hidden, -math.inf)
                lse[rows, g] = torch.logsumexp(w, -1)
                o[rows, g] = torch.softmax(w, -1) @ v
    return {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if s["op"] == "append":
            return _exact_append(s)
        if s["op"] == "chunk":
            return _exact_chunk(s)
        out = {"y": _exact_turned(s["x"], s["pos"], s)}
        if s["op"] == "rope_train":
            out["dx"] = _exact_turned(s["dy"], s["pos"], s, -1)
        return out
