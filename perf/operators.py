"""Measured cases of the sequence mixers beside the delta rule: linear attention
with a decay per head, causal attention over packed prompts, and attention over a
paged key-value cache held in 8 bits.

With ``own`` false ``run`` computes each operator from elementary torch operations
in 32 bits (sums of log-decays in 64); with ``own`` true it makes the calls a user
makes of the library.  ``exact`` is the definition in 64 bits, written apart: the
token recurrence, the softmax one sequence and head at a time, a table of the 8-bit
format's values.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
E4M3_MAX = 448.0
LEAST_EXPONENT = -100  # of a page's scale: an all-zero page has 2^-100


def _spread(n, lo, hi, salt=0):
    """n whole numbers over [lo, hi], the two ends among them, in a fixed mixed order."""
    r = random.Random(n * 1000003 + lo * 1009 + hi * 31 + salt)
    xs = [r.randint(lo, hi) for _ in range(n)]
    xs[0] = hi
    if n > 1:
        xs[-1] = lo
    r.shuffle(xs)
    return xs


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def listed():
    return [
        # the smallest prefill of the repository's configurations: one call, launch-bound
        dict(name="linear_tiny", op="linear_prefill", B=1, T=64, H=2, dk=16, dv=16, dtype="f32", decay="token", state=False),
        # the repository's throughput shape, with a state carried in
        dict(name="linear_32k", op="linear_prefill", B=4, T=32768, H=32, dk=128, dv=128, dtype="bf16", decay="token", state=True),
        # one long document on few heads, a fixed decay for each head
        dict(name="linear_long", op="linear_prefill", B=1, T=131072, H=8, dk=128, dv=128, dtype="bf16", decay="head", state=False),
        # a training step's forward and backward, an odd length, the final state in the loss
        dict(name="linear_train", op="linear_train", B=4, T=4001, H=32, dk=128, dv=128, dtype="bf16", decay="token", state=True),
        # the repository's decode batch: one token for each of 256 sequences
        dict(name="linear_step", op="linear_step", B=256, T=1, H=32, dk=128, dv=128, dtype="bf16", decay="token", state=True),
        # short prompts in single precision: a unit test's or a small model's call
        dict(name="prompt_small", op="prompt", lens="1,33,200", Hq=8, Hkv=2, d=64, dtype="f32"),
        # a serving batch of prompts of very different lengths, packed
        dict(name="prompt_packed", op="prompt", lens="8192,5000,1,2300,777", Hq=32, Hkv=8, d=128, dtype="bf16"),
        # a training batch packed to 8K tokens
        dict(name="prompt_train", op="prompt_train", lens="4096,1023,2500,64,509", Hq=16, Hkv=4, d=128, dtype="bf16"),
        # prompts' keys and values go into the cache, some behind a page already begun
        dict(name="append_prompt", op="append", N=5, new_lo=400, new_hi=6000, held_lo=0, held_hi=777, Hkv=8, d=128, page=64, dtype="bf16"),
        # a decode step's one token for each sequence
        dict(name="append_token", op="append", N=256, new_lo=1, new_hi=1, held_lo=0, held_hi=1500, Hkv=8, d=128, page=64, dtype="bf16"),
        # a decode batch with contexts of very different lengths
        dict(name="step_batch", op="step", N=256, ctx_lo=1, ctx_hi=4096, Hq=32, Hkv=8, d=128, page=64, dtype="bf16"),
        # one user with a long document
        dict(name="step_long", op="step", N=1, ctx_lo=131072, ctx_hi=131072, Hq=32, Hkv=8, d=128, page=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["linear_prefill", "linear_train", "linear_step", "prompt", "prompt_train", "append", "step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("linear"):
        dk, dv = rng.choice([16, 32, 64, 128]), rng.choice([16, 32, 64, 128])
        decay, state = rng.choice(["token", "head"]), rng.random() < 0.5
        if op == "linear_step":
            H = rng.choice([1, 4, 8, 16, 32])
            return dict(op=op, B=_log(rng, 1, 8192 // H), T=1, H=H, dk=dk, dv=dv, dtype=dtype, decay=decay, state=True)
        most = 4 * 32768 * 32 if op == "linear_prefill" else 4 * 4001 * 32
        H = rng.choice([1, 2, 5, 8, 16, 32])
        B = _log(rng, 1, 8)
        T = _log(rng, 1, min(131072 if op == "linear_prefill" else 32768, most // (B * H) // (2 if dtype == "f32" else 1)))
        return dict(op=op, B=B, T=T, H=H, dk=dk, dv=dv, dtype=dtype, decay=decay, state=state)
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    if op.startswith("prompt"):
        train = op == "prompt_train"
        total, lens = _log(rng, 1, 4800 if train else 9500), []
        while total > 0:
            n = min(total, _log(rng, 1, total))
            lens.append(n)
            total -= n
            if len(lens) == 40:
                lens.append(total)
                break
        lens = [n for n in lens if n] or [1]
        rng.shuffle(lens)
        G = rng.choice([1, 2, 4]) if train else rng.choice([1, 2, 3, 4, 8])
        Hq = Hkv * G if Hkv * G <= (16 if train else 32) else Hkv
        return dict(op=op, lens=",".join(map(str, lens)), Hq=Hq, Hkv=Hkv, d=d, dtype=dtype)
    page = rng.choice([16, 32, 64])
    if op == "append":
        N = _log(rng, 1, 64)
        hi = _log(rng, 1, 16000 // N)
        return dict(op=op, N=N, new_lo=rng.randint(1, hi), new_hi=hi, held_lo=0, held_hi=_log(rng, 1, 1500), Hkv=Hkv, d=d, page=page, dtype=dtype)
    N = _log(rng, 1, 256)
    hi = _log(rng, 1, min(131072, 500000 // N))
    return dict(op=op, N=N, ctx_lo=rng.randint(0, hi), ctx_hi=hi, Hq=Hkv * rng.choice([1, 2, 4, 7, 8]), Hkv=Hkv, d=d, page=page, dtype=dtype)


# ----------------------------------------------------------------- inputs

def _normal(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device=DEV) * std


def _unit(x):
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)


def _prepare_linear(case, gen):
    B, T, H, dk, dv = (case[x] for x in ("B", "T", "H", "dk", "dv"))
    t = TYPES[case["dtype"]]
    s = {"q": _unit(_normal(gen, B, T, H, dk)).to(t), "k": _unit(_normal(gen, B, T, H, dk)).to(t),
         "v": _normal(gen, B, T, H, dv).to(t), "scale": 1.0}
    if case["decay"] == "head":  # fixed rates, a memory of 2 to 256 tokens over the heads
        h = torch.arange(H, device=DEV, dtype=torch.float32)
        s["g"] = -torch.exp2(-1 - 7 * h / max(1, H - 1)) * torch.exp(_normal(gen, H, std=0.05))
    else:  # rates that the input sets, most between 1/40 and 1/2 for a token
        s["g"] = -0.1 * torch.exp(_normal(gen, B, T, H, std=0.8))
    s["S"] = _normal(gen, B, H, dk, dv, std=0.1) if case["state"] else None
    if case["op"] == "linear_train":
        s["do"] = _normal(gen, B, T, H, dv).to(t)
        s["dS"] = _normal(gen, B, H, dk, dv, std=0.1) if case["state"] else None
    if case["op"] == "linear_step":
        for x in ("q", "k", "v"):
            s[x] = s[x][:, 0].contiguous()
        s["g"] = s["g"][:, 0].contiguous() if case["decay"] == "token" else s["g"]
    return s


def _prepare_prompt(case, gen):
    lens, t = _lens(case), TYPES[case["dtype"]]
    n, Hq, Hkv, d = sum(lens), case["Hq"], case["Hkv"], case["d"]
    s = {"q": _normal(gen, n, Hq, d).to(t), "k": _normal(gen, n, Hkv, d).to(t), "v": _normal(gen, n, Hkv, d).to(t)}
    s["cu"] = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    s["scale"] = d ** -0.5
    if case["op"] == "prompt_train":
        s["do"] = _normal(gen, n, Hq, d).to(t)
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
    Hkv, d, P, t = case["Hkv"], case["d"], case["page"], TYPES[case["dtype"]]
    if case["op"] == "append":
        new = _spread(case["N"], case["new_lo"], case["new_hi"])
        held = _spread(case["N"], case["held_lo"], case["held_hi"], 1)
        table, pages = _table(case, [a + b for a, b in zip(new, held)], gen)
        s = {"k": _normal(gen, sum(new), Hkv, d), "v": _normal(gen, sum(new), Hkv, d)}
        wide = torch.exp(_normal(gen, sum(new), 1, 1, std=0.7))  # some tokens are larger: a page's scale grows
        s["k"], s["v"] = (s["k"] * wide).to(t), (s["v"] * wide).to(t)
        s["cu"] = torch.tensor([0] + new).cumsum(0).to(torch.int32).to(DEV)
        s["held"] = torch.tensor(held, dtype=torch.int32, device=DEV)
    else:
        ctx = _spread(case["N"], case["ctx_lo"], case["ctx_hi"])
        table, pages = _table(case, ctx, gen)
        s = {"q": _normal(gen, case["N"], case["Hq"], d).to(t), "scale": d ** -0.5}
        s["held"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    s["table"] = table
    s["kc"], s["ks"] = _filled(gen, pages, Hkv, P, d)
    s["vc"], s["vs"] = _filled(gen, pages, Hkv, d, P)
    return s


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(int(seed))
    s = (_prepare_linear if case["op"].startswith("linear") else _prepare_prompt if case["op"].startswith("prompt") else _prepare_cache)(case, gen)
    s["op"] = case["op"]
    return s


# ------------------------------------------------- plain forms, in 32 bits

CHUNK = 64


def _linear_plain(q, k, v, g, S_in, scale):
    """o [B,T,H,dv] and the final state, from fp32 inputs, chunk by chunk side by side:
    the states that enter the chunks come from one product with the decays between chunks."""
    B, T, H, dk = q.shape
    dv, C = v.shape[-1], CHUNK
    nc = max(1, -(-T // C))
    pad = lambda x: torch.nn.functional.pad(x, (0, 0, 0, 0, 0, nc * C - T)).view(B, nc, C, H, -1).permute(0, 3, 1, 2, 4)  # noqa: E731
    q, k, v = pad(q), pad(k), pad(v)  # [B,H,nc,C,d]
    g = g.double().expand(B, T, H)[..., None]
    L = pad(g)[..., 0].cumsum(-1)  # log-decay within the chunk, its own token's included
    E = L[..., -1].cumsum(-1)  # to a chunk's end, from the start
    E_in = E - L[..., -1]
    low = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    D = torch.exp((L[..., :, None] - L[..., None, :]).masked_fill(~low, -math.inf)).float()
    o = (q @ k.transpose(-1, -2) * D) @ v
    KV = (k * torch.exp(L[..., -1:] - L).float()[..., None]).transpose(-1, -2) @ v
    before = torch.ones(nc, nc, dtype=torch.bool, device=q.device).tril(-1)
    W = torch.exp((E_in[..., :, None] - E[..., None, :]).masked_fill(~before, -math.inf)).float()
    S = (W @ KV.reshape(B, H, nc, dk * dv)).view(B, H, nc, dk, dv)
    last = torch.exp(E[..., -1:] - E).float()
    S_out = (last[..., None, :] @ KV.reshape(B, H, nc, dk * dv)).view(B, H, dk, dv)
    if S_in is not None:
        S = S + torch.exp(E_in).float()[..., None, None] * S_in[:, :, None]
        S_out = S_out + torch.exp(E[..., -1]).float()[..., None, None] * S_in
    o = scale * (o + torch.exp(L).float()[..., None] * (q @ S))
    return o.permute(0, 2, 3, 1, 4).reshape(B, nc * C, H, dv)[:, :T], S_out


def _linear_step_plain(q, k, v, g, S, scale):
    a = torch.exp(g.expand(q.shape[:2]))
    S = S * a[..., None, None] + k[..., :, None] * v[..., None, :]
    return scale * (S * q[..., :, None]).sum(-2), S


def _prompt_plain(q, k, v, cu, scale):
    """o [n,Hq,d] and the log of the softmax' sum [n,Hq], from fp32 inputs."""
    n, Hq, d = q.shape
    Hkv = k.shape[1]
    at = torch.arange(n, device=q.device)
    doc = torch.bucketize(at, cu[1:].long(), right=True)
    seen = (doc[:, None] == doc[None, :]) & (at[:, None] >= at[None, :])
    q = q.view(n, Hkv, Hq // Hkv, d).permute(1, 2, 0, 3).reshape(Hkv, -1, d)
    s = q @ (k.permute(1, 2, 0) * scale)  # [Hkv, G n, n]
    s = s.view(Hkv, -1, n, n).masked_fill(~seen, -math.inf)
    m = s.detach().amax(-1, keepdim=True)
    s = (s - m).exp() if s.requires_grad else s.sub_(m).exp_()
    z = s.sum(-1, keepdim=True)
    o = (s.view(Hkv, -1, n) @ v.permute(1, 0, 2)).view(Hkv, -1, n, d) / z
    lse = (m + z.log())[..., 0]
    return o.permute(2, 0, 1, 3).reshape(n, Hq, d), lse.permute(2, 0, 1).reshape(n, Hq)


def _scale_for(amax):
    """The smallest power of two s with amax <= 448 s."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= E4M3_MAX / 512, e - 9, e - 8).clamp_min(LEAST_EXPONENT)
    return torch.ldexp(torch.ones_like(amax), e)


def _to_8bit(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _append_plain(x, slot, off, first, touched, cache, scale):
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


def _append(s):
    cu, held, table = s["cu"].long(), s["held"].long(), s["table"].long()
    P = s["kc"].shape[2]
    at = torch.arange(s["k"].shape[0], device=DEV)
    seq = torch.bucketize(at, cu[1:], right=True)
    pos = held[seq] + at - cu[seq]
    page = table[seq, pos // P]
    touched, slot = torch.unique(page, return_inverse=True)
    first = torch.full_like(touched, P).scatter_reduce_(0, slot, pos % P, "amin")
    _append_plain(s["k"].float(), slot, pos % P, first, touched, s["kc"], s["ks"])
    vt = s["vc"].view(torch.uint8).transpose(2, 3).contiguous().view(torch.float8_e4m3fn)
    _append_plain(s["v"].float(), slot, pos % P, first, touched, vt, s["vs"])
    s["vc"].view(torch.uint8).copy_(vt.view(torch.uint8).transpose(2, 3))


def _step_plain(q, kc, vc, ks, vs, table, ctx, scale):
    N, Hq, d = q.shape
    Hkv, P = kc.shape[1], kc.shape[2]
    t = table.long()
    k = (kc.view(torch.uint8)[t].view(torch.float8_e4m3fn).float() * ks[t][..., None, None]).transpose(1, 2).reshape(N, Hkv, -1, d)
    s = q.view(N, Hkv, -1, d) * scale @ k.transpose(-1, -2)
    del k
    dead = torch.arange(s.shape[-1], device=q.device) >= ctx[:, None, None, None]
    s.masked_fill_(dead, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m.clamp_min(-3e38))
    z = p.sum(-1, keepdim=True)
    v = (vc.view(torch.uint8)[t].view(torch.float8_e4m3fn).float() * vs[t][..., None, None]).permute(0, 2, 1, 4, 3).reshape(N, Hkv, -1, d)
    o = (p @ v) / torch.where(z > 0, z, 1.0)
    return o.reshape(N, Hq, d), (m + z.log()).reshape(N, Hq)


# --------------------------------------------------------------------- run

def _run_plain(s):
    op = s["op"]
    if op == "append":
        _append(s)
        return {"k_cache": s["kc"], "v_cache": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}
    f = {x: s[x].float() for x in ("q", "k", "v") if x in s}
    t = s["q"].dtype
    if op == "step":
        o, lse = _step_plain(f["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["held"], s["scale"])
        return {"o": o.to(t), "lse": lse}
    if op == "linear_step":
        o, S = _linear_step_plain(f["q"], f["k"], f["v"], s["g"], s["S"], s["scale"])
        return {"o": o.to(t), "S": S}
    if op == "linear_prefill":
        o, S = _linear_plain(f["q"], f["k"], f["v"], s["g"], s["S"], s["scale"])
        return {"o": o.to(t), "S": S}
    if op == "prompt":
        o, lse = _prompt_plain(f["q"], f["k"], f["v"], s["cu"], s["scale"])
        return {"o": o.to(t), "lse": lse}
    names = ["q", "k", "v"]
    if op == "linear_train":
        names += ["g"] + (["S"] if s["S"] is not None else [])
    leaves = {x: s[x].float().detach().requires_grad_() for x in names}
    with torch.enable_grad():
        if op == "linear_train":
            o, S = _linear_plain(leaves["q"], leaves["k"], leaves["v"], leaves["g"], leaves.get("S"), s["scale"])
            outs, grads, back = {"o": o.detach().to(t), "S": S.detach()}, [s["do"].float()], [o]
            if s["dS"] is not None:
                grads.append(s["dS"])
                back.append(S)
        else:
            o, lse = _prompt_plain(leaves["q"], leaves["k"], leaves["v"], s["cu"], s["scale"])
            outs, grads, back = {"o": o.detach().to(t), "lse": lse.detach()}, [s["do"].float()], [o]
        got = torch.autograd.grad(back, list(leaves.values()), grads)
    for x, y in zip(names, got):
        outs["d" + x] = y.to(t) if x in ("q", "k", "v") else y
    return outs


def _run_own(s):
    import gated_delta_rule_11_amd as kda

    op = s["op"]
    if op == "append":
        kda.kv_cache_append(s["k"], s["v"], s["cu"], s["held"], s["table"], s["kc"], s["vc"], s["ks"], s["vs"])
        return {"k_cache": s["kc"], "v_cache": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}
    t = s["q"].dtype
    if op == "step":
        o, lse = kda.attn_decode_step(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["held"], scale=s["scale"], o_dtype=t, want_lse=True)
        return {"o": o, "lse": lse}
    if op == "linear_step":
        # the state a step starts from is kept (a cached prefix): the step writes another
        o, S = kda.linear_decode_step(s["q"], s["k"], s["v"], s["g"], s["S"], scale=s["scale"], o_dtype=t, S_out=torch.empty_like(s["S"]))
        return {"o": o, "S": S}
    if op in ("prompt", "prompt_train"):
        o, lse = kda.attn_prompt_fwd(s["q"], s["k"], s["v"], s["cu"], scale=s["scale"], o_dtype=t, want_lse=True)
        if op == "prompt":
            return {"o": o, "lse": lse}
        g = kda.attn_prompt_bwd(s["q"], s["k"], s["v"], s["cu"], o, lse, s["do"], scale=s["scale"], grad_dtype=t)
        return {"o": o, "lse": lse, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"]}
    o, S = kda.linear_chunk_fwd(s["q"], s["k"], s["v"], s["g"], S_in=s["S"], scale=s["scale"], o_dtype=t)
    if op == "linear_prefill":
        return {"o": o, "S": S}
    g = kda.linear_chunk_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], dS_out=s["dS"], S_in=s["S"], scale=s["scale"],
                             want_dS_in=s["S"] is not None, grad_dtype=t)
    outs = {"o": o, "S": S, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"], "dg": g["dg"]}
    if s["S"] is not None:
        outs["dS"] = g["dS_in"]
    return outs


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# -------------------------------------------------------------------- work

def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op.startswith("linear"):
        n = case["B"] * case["T"] * case["H"]
        states = case["B"] * case["H"] * case["dk"] * case["dv"] * 4
        dk, dv = case["dk"], case["dv"]
        gate = n * 4 if case["decay"] == "token" else case["H"] * 4
        if op == "linear_step":
            return {"bytes": n * e * (2 * dk + 2 * dv) + gate + 2 * states, "flops": n * 5 * dk * dv}
        held = (2 if case["state"] else 1) * states
        fwd = {"bytes": n * e * (2 * dk + 2 * dv) + gate + held, "flops": n * 4 * dk * dv}
        if op == "linear_prefill":
            return fwd
        # the backward reads q, k, v, do and g, writes three gradients and g's, and moves the states' gradients
        return {"bytes": fwd["bytes"] + n * e * (4 * dk + 3 * dv) + 2 * gate + 2 * held, "flops": n * 4 * dk * dv + n * 10 * dk * dv}
    if op.startswith("prompt"):
        lens, Hq, Hkv, d = _lens(case), case["Hq"], case["Hkv"], case["d"]
        n, pairs = sum(lens), sum(x * (x + 1) // 2 for x in lens) * Hq
        b = n * e * d * (2 * Hq + 2 * Hkv) + 4 * n * Hq
        if op == "prompt":
            return {"bytes": b, "flops": 4 * d * pairs}
        return {"bytes": b + n * e * d * (4 * Hq + 4 * Hkv), "flops": 14 * d * pairs}
    Hkv, d = case["Hkv"], case["d"]
    if op == "append":
        n = sum(_spread(case["N"], case["new_lo"], case["new_hi"]))
        return {"bytes": 2 * n * Hkv * d * (e + 1) + 8 * Hkv * (case["N"] + n // case["page"]), "flops": 4 * n * Hkv * d}
    n = sum(_spread(case["N"], case["ctx_lo"], case["ctx_hi"]))
    return {"bytes": 2 * n * Hkv * d + 8 * Hkv * (n // case["page"]) + case["N"] * case["Hq"] * d * 2 * e, "flops": 4 * n * case["Hq"] * d}


# ------------------------------------------------- the definitions, 64 bits

def _exact_linear(s, train):
    """The recurrence, one token at a time."""
    step = s["op"] == "linear_step"
    q, k, v = (s[x].double()[:, None] if step else s[x].double() for x in ("q", "k", "v"))
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    S0 = torch.zeros(B, H, dk, dv, dtype=torch.float64, device=DEV) if s["S"] is None else s["S"].double()
    g = s["g"].double()
    g = g.expand(B, T, H) if g.dim() == 1 else g.view(B, T, H)
    a = g.exp()
    q, k, v, a = (x.transpose(0, 1).contiguous() for x in (q, k, v, a))  # [T,B,H,..]
    a = a[..., None, None]
    S, o = S0.clone(), torch.empty(T, B, H, dv, dtype=torch.float64, device=DEV)
    dq = torch.empty_like(q) if train else None
    do = s["do"].double().transpose(0, 1).contiguous() if train else None
    for t in range(T):
        S.mul_(a[t]).add_(k[t][..., :, None] * v[t][..., None, :])
        torch.matmul(q[t][..., None, :], S, out=o[t][..., None, :])
        if train:
            torch.matmul(S, do[t][..., :, None], out=dq[t][..., :, None])
    o = (o * s["scale"]).transpose(0, 1)
    out = {"o": o[:, 0] if step else o, "S": S}
    if not train:
        return out
    dS = s["dS"].double() if s["dS"] is not None else torch.zeros_like(S0)
    R, dk_, dv_ = dS.clone(), torch.empty_like(k), torch.empty_like(v)
    for t in range(T - 1, -1, -1):
        R.add_((q[t] * s["scale"])[..., :, None] * do[t][..., None, :])
        torch.matmul(R, v[t][..., :, None], out=dk_[t][..., :, None])
        torch.matmul(k[t][..., None, :], R, out=dv_[t][..., None, :])
        R.mul_(a[t])
    dq *= s["scale"]
    # a decay scales all that crosses it: what later queries read less what later keys wrote, and the final state
    x = (q * dq).sum(-1) - (k * dk_).sum(-1)
    dg = x.flip(0).cumsum(0).flip(0) + (S * dS).sum((-1, -2))
    out |= {"dq": dq.transpose(0, 1), "dk": dk_.transpose(0, 1), "dv": dv_.transpose(0, 1),
            "dg": dg.transpose(0, 1) if s["g"].dim() == 3 else dg.sum((0, 1))}
    if s["S"] is not None:
        out["dS"] = R
    return out


def _exact_prompt(s, train):
    q, k, v = (s[x].double() for x in ("q", "k", "v"))
    n, Hq, d = q.shape
    G = Hq // k.shape[1]
    o, lse = torch.empty_like(q), torch.empty(n, Hq, dtype=torch.float64, device=DEV)
    grads = {"dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v)} if train else {}
    ends = s["cu"].tolist()
    for a, b in zip(ends, ends[1:]):
        low = torch.ones(b - a, b - a, dtype=torch.bool, device=DEV).tril()
        for h in range(Hq):
            kh, vh = k[a:b, h // G], v[a:b, h // G]
            w = torch.where(low, q[a:b, h] @ kh.T * s["scale"], -math.inf)
            lse[a:b, h] = torch.logsumexp(w, -1)
            p = torch.exp(w - lse[a:b, h, None])
            o[a:b, h] = p @ vh
            if train:
                do = s["do"][a:b, h].double()
                grads["dv"][a:b, h // G] += p.T @ do
                w = p * (do @ vh.T - (do * o[a:b, h]).sum(-1, keepdim=True)) * s["scale"]
                grads["dq"][a:b, h] = w @ kh
                grads["dk"][a:b, h // G] += w.T @ q[a:b, h]
    return {"o": o, "lse": lse, **grads}


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
    for side in ("k", "v"):
        x = s[side].double()
        cache = out[side + "_cache"] if side == "k" else out[side + "_cache"].transpose(2, 3)
        scale = out[side + "_scale"]
        for i in range(len(held)):
            at, end = held[i], held[i] + cu[i + 1] - cu[i]
            while at < end:
                n, r, pg = min(P - at % P, end - at), at % P, table[i][at // P]
                new = x[cu[i] + at - held[i]:][:n].transpose(0, 1)  # [Hkv, n, d]
                need = torch.exp2((new.abs().amax((1, 2)) / E4M3_MAX).log2().ceil().clamp_min(LEAST_EXPONENT))
                if r:
                    need = torch.maximum(need, scale[pg])
                    cache[pg, :, :r] = _table_round(cache[pg, :, :r] * (scale[pg] / need)[:, None, None])
                cache[pg, :, r:r + n] = _table_round(new / need[:, None, None])
                scale[pg] = need
                at += n
    return out


def _exact_step(s):
    q, P = s["q"].double(), s["kc"].shape[2]
    N, Hq, d = q.shape
    Hkv = s["kc"].shape[1]
    o, lse = torch.zeros_like(q), torch.full((N, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for i, n in enumerate(s["held"].tolist()):
        if n == 0:
            continue
        pages = s["table"][i, :-(-n // P)].tolist()
        at = torch.tensor(pages, device=DEV)
        k = s["kc"].view(torch.uint8)[at].view(torch.float8_e4m3fn).double() * s["ks"][at].double()[..., None, None]
        v = s["vc"].view(torch.uint8)[at].view(torch.float8_e4m3fn).double() * s["vs"][at].double()[..., None, None]
        k = k.transpose(0, 1).reshape(Hkv, -1, d)[:, :n]
        v = v.permute(1, 0, 3, 2).reshape(Hkv, -1, d)[:, :n]
        w = torch.matmul(q[i].view(Hkv, -1, d), k.transpose(1, 2).contiguous()) * s["scale"]
        lse[i] = torch.logsumexp(w, -1).view(Hq)
        o[i] = torch.matmul(torch.softmax(w, -1), v).view(Hq, d)
    return {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if s["op"].startswith("linear"):
            return _exact_linear(s, s["op"] == "linear_train")
        if s["op"].startswith("prompt"):
            return _exact_prompt(s, s["op"] == "prompt_train")
        return _exact_append(s) if s["op"] == "append" else _exact_step(s)
