"""The serving calls as a layer uses them: prompts in pieces through the turned append and attention over the cache, mixed with
sequences that decode, drafted tokens of which some are taken; and the training path, rotation, packed attention and
both gradients."""
import pytest
import torch

import gated_delta_rule_11_amd as kda
from tests import _mixers as mx
from tests import _serve as sv
from tests.test_gpu_cache import empty_cache, i32, same, table_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def ends(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return out


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pieces_drafts_and_single_tokens(dtype):
    """Every step: [queries, keys, values] of the new tokens as one projection's output.  The cache holds what the exactly
    turned keys give, and the attention is the softmax over it."""
    Hq, Hkv, d, P, N = 8, 2, 128, 32, 3
    gen = torch.Generator().manual_seed(0)
    inv, table = sv.frequencies(64), table_of([400] * N, P, 45)
    c = {x: y.to(DEV) for x, y in empty_cache(45, Hkv, P, d).items()}
    ref, held = mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"]), [0, 0, 0]
    # (new tokens, taken of them): pieces of prompts, mixed with decoding, drafts
    steps = [([100, 7, 0], None), ([60, 1, 130], None), ([1, 1, 1], None), ([5, 5, 5], [2, 5, 1]), ([1, 4, 70], [1, 2, 70]), ([1, 1, 1], None)]
    for new, taken in steps:
        n, cu = sum(new), ends(new)
        x = torch.randn(n, Hq + 2 * Hkv, d, generator=gen).to(dtype)
        q, k, v = x.to(DEV).split([Hq, Hkv, Hkv], 1)
        tab, before, after = i32(table), i32(held), i32([a + b for a, b in zip(held, new)])
        kda.kv_cache_append_rope(k, v, i32(cu), before, tab, c["kc"], c["vc"], c["ks"], c["vs"], inv.to(DEV), q=q, q_out=q)
        o, lse = kda.attn_chunk_fwd(q, i32(cu), c["kc"], c["vc"], c["ks"], c["vs"], tab, after, o_dtype=dtype, want_lse=True)
        at = sv.places(cu, held)
        fq, fk, fv = mx.f64(x).split([Hq, Hkv, Hkv], 1)
        ref.append(sv.turned(fk, at, inv)[0], fv, cu, held, table)
        same(c, ref, Hkv)
        want, mag = sv.turned(fq, at, inv)
        mx.close("q", q, want, mag, dtype, 1.0, 3.0)
        ro, rl, rm = sv.chunk(ref, mx.f64(q), cu, [a + b for a, b in zip(held, new)], table, d ** -0.5)
        mx.close(f"{new}", o, ro, rm, dtype, 2.0, 3 * d + 3 * 400 + 256)
        mx.close(f"{new} lse", lse, rl, torch.full_like(rl, 8.0), F32, 1.0, 3 * d + 3 * 400 + 256)
        held = [a + b for a, b in zip(held, taken or new)]


def test_pieces_equal_the_whole_prompt():
    """A prompt in one piece or in three: the same rows to the cache's own rounding (a page's scale may have been smaller
    while the page was filled, which rounds earlier codes twice) and near the packed attention of the unrounded keys."""
    Hq, Hkv, d, P, n = 4, 2, 64, 16, 300
    gen = torch.Generator().manual_seed(1)
    inv, scale = sv.frequencies(32), d ** -0.5
    x = torch.randn(n, Hq + 2 * Hkv, d, generator=gen)
    table = i32([list(range(20))])
    outs = []
    for pieces in ([n], [100, 1, 150, 49]):
        c = {a: b.to(DEV) for a, b in empty_cache(20, Hkv, P, d).items()}
        done, rows = 0, []
        for m in pieces:
            q, k, v = x[done:done + m].to(DEV).split([Hq, Hkv, Hkv], 1)
            q = kda.kv_cache_append_rope(k, v, i32([0, m]), i32([done]), table, c["kc"], c["vc"], c["ks"], c["vs"], inv.to(DEV), q=q)
            done += m
            rows.append(kda.attn_chunk_fwd(q, i32([0, m]), c["kc"], c["vc"], c["ks"], c["vs"], table, i32([done]))[0])
        outs.append(torch.cat(rows))
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    q, k, v = x.to(DEV).split([Hq, Hkv, Hkv], 1)
    full, _ = kda.attn_prompt_fwd(kda.rope(q, pos, inv.to(DEV)), kda.rope(k, pos, inv.to(DEV)), v.contiguous(), i32([0, n]), scale=scale)
    torch.cuda.synchronize()
    fq, fk, fv = mx.f64(x).split([Hq, Hkv, Hkv], 1)
    at = torch.arange(n)
    (want, mag) = mx.prompt(sv.turned(fq, at, inv)[0], sv.turned(fk, at, inv)[0], fv, [0, n], scale)
    mx.close("packed", full, want["o"], mag["o"] * 8, F32, 1.0, d + n + 200)
    for o in outs:
        # values: 2^-4 of each, 2^-4 again where a page's scale grew.  Scores move by at most 2^-3 sum |q k| scale, on average
        # far less, and a probability by twice its score: the norm of the rows' error against their terms' magnitude
        assert float((o.cpu().double() - want["o"]).norm() / mag["o"].norm()) < 2 ** -3 + 0.3


def test_training_path():
    """Rotation, packed attention and both gradients against autograd of the formulas in 64 bits."""
    Hq, Hkv, d, cu = 4, 2, 64, [0, 50, 51, 131]
    n, inv, gen = cu[-1], sv.frequencies(24), torch.Generator().manual_seed(2)
    x = torch.randn(n, Hq + 2 * Hkv, d, generator=gen)
    do = torch.randn(n, Hq, d, generator=gen)
    pos = torch.stack([torch.arange(n), torch.arange(n) // 7, torch.arange(n) % 7], 1).to(torch.int32)
    axes = (torch.arange(24) % 3).to(torch.int32)
    turn = dict(axes=axes.to(DEV), interleaved=True)
    qk = kda.rope(x.to(DEV)[:, :Hq + Hkv], pos.to(DEV), inv.to(DEV), **turn)
    q, k, v = qk[:, :Hq].contiguous(), qk[:, Hq:].contiguous(), x.to(DEV)[:, Hq + Hkv:].contiguous()
    o, lse = kda.attn_prompt_fwd(q, k, v, i32(cu))
    g = kda.attn_prompt_bwd(q, k, v, i32(cu), o, lse, do.to(DEV))
    dqk = kda.rope(torch.cat([g["dq"], g["dk"]], 1), pos.to(DEV), inv.to(DEV), inverse=True, **turn)
    torch.cuda.synchronize()
    leaf = x.double().requires_grad_()
    tq = sv.turned(leaf[:, :Hq], pos, inv, axes, True)[0]
    tk = sv.turned(leaf[:, Hq:Hq + Hkv], pos, inv, axes, True)[0]
    rows = []
    for a, b in zip(cu, cu[1:]):
        w = torch.einsum("ihd,jhd->hij", tq[a:b], tk[a:b].repeat_interleave(Hq // Hkv, 1)) * d ** -0.5
        w = w.masked_fill(~torch.ones(b - a, b - a, dtype=torch.bool).tril(), float("-inf")).softmax(-1)
        rows.append(torch.einsum("hij,jhd->ihd", w, leaf[a:b, Hq + Hkv:].repeat_interleave(Hq // Hkv, 1)))
    want = torch.cat(rows)
    (grad,) = torch.autograd.grad(want, leaf, do.double())
    # fp32 throughout: sums of at most d + n terms forwards, twice that and both heads of a group backwards
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    eps = 2.0 ** -24 * (d + n)
    assert rel(o, want.detach()) < eps
    assert rel(dqk, grad[:, :Hq + Hkv]) < 4 * eps and rel(g["dv"], grad[:, Hq + Hkv:]) < 4 * eps


def test_a_captured_layer_step():
    """Append with queries, then attention, captured once and replayed while lengths, positions and inputs move on."""
    Hq, Hkv, d, P, N, new = 8, 2, 64, 16, 5, 3
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(N * new, Hq + 2 * Hkv, d, generator=gen).to(BF).to(DEV)
    q, k, v = x.split([Hq, Hkv, Hkv], 1)
    inv, cu, table = sv.frequencies(32).to(DEV), i32([new * i for i in range(N + 1)]), i32(table_of([700] * N, P, 230))
    held = i32([600, 0, 16, 31, 250])
    after = held + new
    c = {a: b.to(DEV) for a, b in empty_cache(230, Hkv, P, d).items()}
    c["kc"].view(torch.uint8).fill_(0x30)
    c["vc"].view(torch.uint8).fill_(0x28)
    twin = {a: b.clone() for a, b in c.items()}

    def step(c):
        t = kda.kv_cache_append_rope(k, v, cu, held, table, c["kc"], c["vc"], c["ks"], c["vs"], inv, q=q)
        return kda.attn_chunk_fwd(t, cu, c["kc"], c["vc"], c["ks"], c["vs"], table, after, o_dtype=BF, want_lse=True)

    step({a: b.clone() for a, b in c.items()})
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step(c)
    for _ in range(5):
        graph.replay()
        eager = step(twin)
        torch.cuda.synchronize()
        assert torch.equal(o, eager[0]) and torch.equal(lse, eager[1])
        assert all(torch.equal(c[a].view(torch.uint8), twin[a].view(torch.uint8)) for a in c)
        held += new
        after += new
        x.mul_(-1.1)
