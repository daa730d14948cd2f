"""The 8-bit paged cache on the GPU: appended codes and scales equal the table's exactly (scales
are powers of two, so the only rounding is the 8-bit one), and single-token attention over them
against softmax in 64 bits on the same codes.

Bounds of the attention: with bf16 queries each probability is rounded once and the output once
(2^-8 each); in fp32 a sum over channels, one over the tokens, and the exponential's |x| 2^-24."""
import math

import numpy as np
import pytest
import torch

import gated_delta_rule_11_amd as kda
from tests import _mixers as mx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
F8 = torch.float8_e4m3fn


def empty_cache(pages, Hkv, P, d, seed=0):
    """A cache full of what earlier use left: random codes, NaN among them, and scales."""
    gen = torch.Generator().manual_seed(seed)
    code = lambda *s: torch.randint(0, 256, s, generator=gen, dtype=torch.uint8).view(F8)  # noqa: E731
    return {"kc": code(pages, Hkv, P, d), "vc": code(pages, Hkv, d, P),
            "ks": torch.exp2(torch.randint(-8, 3, (pages, Hkv), generator=gen).float()),
            "vs": torch.exp2(torch.randint(-8, 3, (pages, Hkv), generator=gen).float())}


def table_of(rooms, P, pages, seed=0, width=None):
    need = [-(-n // P) for n in rooms]
    order = np.random.default_rng(seed).permutation(pages)[: sum(need)].tolist()
    width = width or max(1, *need)
    t, at = [], 0
    for n in need:
        t.append(order[at:at + n] + [0] * (width - n))
        at += n
    return t


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def append(c, k, v, new, held, table):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    kda.kv_cache_append(k.to(DEV), v.to(DEV), i32(cu), i32(held), i32(table), c["kc"], c["vc"], c["ks"], c["vs"])
    return cu


def same(c, ref, Hkv):
    torch.cuda.synchronize()
    got = mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"])
    for x in ("k", "v"):
        assert np.array_equal(got.scale[x], ref.scale[x]), x
        assert np.array_equal(got.side[x], ref.side[x], equal_nan=True), x


def tokens(gen, n, Hkv, d, dtype, wide=1.0):
    x = torch.randn(n, Hkv, d, generator=gen) * torch.exp(wide * torch.randn(n, 1, 1, generator=gen))
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_append_codes_and_scales(d, P, dtype):
    """New pages, begun pages whose scale grows, several calls, odd lengths, untouched pages left alone."""
    gen = torch.Generator().manual_seed(P + d)
    Hkv, pages = 3, 40
    c = {x: y.to(DEV) for x, y in empty_cache(pages, Hkv, P, d).items()}
    ref = mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"])
    steps = [[37, 0, 1, 2 * P], [1, 1, 1, 1], [P, 3, 0, 5], [1, 1, 1, 1], [0, 0, 2, P - 1]]
    table = table_of([sum(s[i] for s in steps) for i in range(4)], P, pages)
    held = [0, 0, 0, 0]
    for new in steps:
        k, v = (tokens(gen, sum(new), Hkv, d, dtype) for _ in range(2))
        cu = append(c, k, v, new, held, table)
        ref.append(mx.f64(k), mx.f64(v), cu, held, table)
        held = [a + b for a, b in zip(held, new)]
        same(c, ref, Hkv)


def test_append_every_length_of_a_page():
    gen = torch.Generator().manual_seed(2)
    for off in (0, 1, 2, 3, 5, 15):
        for n in (1, 2, 3, 4, 7, 14, 17, 33):
            c = {x: y.to(DEV) for x, y in empty_cache(8, 1, 16, 64).items()}
            ref = mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"])
            table = table_of([off + n], 16, 8)
            k, v = (tokens(gen, n, 1, 64, BF) for _ in range(2))
            cu = append(c, k, v, [n], [off], table)
            ref.append(mx.f64(k), mx.f64(v), cu, [off], table)
            same(c, ref, 1)


def test_append_special_values():
    """Zeros, infinities, NaN, denormals, the largest values, and ties of the 8-bit rounding."""
    x = torch.zeros(9, 1, 64)
    x[1, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 1.0])
    x[2] = 1e-41
    x[3] = 3e38
    x[4, 0, :3] = torch.tensor([-3.4e38, 1e-30, -0.0])
    ties = torch.from_numpy(np.concatenate([mx.e4m3_values()[:-1] + np.diff(mx.e4m3_values()) / 2, [448.0]])).float()
    x[5, 0, :] = 448.0
    x[6, 0, :], x[7, 0, :63], x[8, 0, 0] = ties[:64], ties[64:], 448.0
    for lo, hi in ((0, 1), (1, 2), (2, 3), (3, 5), (5, 9), (0, 9)):
        c = {a: b.to(DEV) for a, b in empty_cache(3, 1, 16, 64).items()}
        ref = mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"])
        k = x[lo:hi].contiguous()
        cu = append(c, k, -k, [hi - lo], [0], [[1]])
        ref.append(mx.f64(k), mx.f64(-k), cu, [0], [[1]])
        same(c, ref, 1)


def test_append_drops_what_has_no_place():
    """Past the table's pages, and page ids outside the cache; rows behind the last sequence are not read."""
    gen = torch.Generator().manual_seed(4)
    c = {x: y.to(DEV) for x, y in empty_cache(6, 2, 16, 64).items()}
    ref = mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"])
    table = [[4, -1, 3], [99, 1, 6], [2, 0, 5]]
    new, held = [48, 40, 30], [0, 0, 25]  # the last one ends 7 tokens behind its table
    k, v = (tokens(gen, 130, 2, 64, BF) for _ in range(2))
    k[118:] = math.nan
    cu = append(c, k, v, new, held, table)
    ref.append(mx.f64(k), mx.f64(v), cu, held, table)
    same(c, ref, 2)


def filled(ctx, Hkv, P, d, seed=0, spare=3, width=None):
    """A cache with real codes in the tokens in use and anything elsewhere."""
    gen = torch.Generator().manual_seed(seed)
    pages = sum(-(-n // P) for n in ctx) + spare
    c = {x: y.to(DEV) for x, y in empty_cache(pages, Hkv, P, d, seed).items()}
    table = table_of(ctx, P, pages, seed, width)
    k, v = (tokens(gen, sum(ctx), Hkv, d, BF, 0.3) for _ in range(2))
    append(c, k, v, ctx, [0] * len(ctx), table)
    return c, table


def check_step(label, ctx, Hq, Hkv, P, d, dtype, scale=None, table=None, **kw):
    c, t = filled(ctx, Hkv, P, d, seed=sum(ctx) + Hq, **kw)
    t = table or t
    q = torch.randn(len(ctx), Hq, d, generator=torch.Generator().manual_seed(9)).to(dtype)
    o, lse = kda.attn_decode_step(q.to(DEV), c["kc"], c["vc"], c["ks"], c["vs"], i32(t), i32(ctx), scale=scale,
                                  o_dtype=dtype, want_lse=True)
    torch.cuda.synchronize()
    ref = mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"])
    ro, rl, mag = ref.attend(mx.f64(q), ctx, t, d ** -0.5 if scale is None else scale)
    terms = d + max(ctx) + 3 * 40 + 64
    mx.close(label + " o", o, ro, mag, dtype, 2.0, terms)
    mx.close(label + " lse", lse, rl, torch.full_like(rl, 8.0), F32, 1.0, terms)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_step_contexts(d, P, dtype):
    check_step(f"P={P} d={d}", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 100, 0, 128, 300], 4, 2, P, d, dtype)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (7, 1), (16, 1), (17, 1), (40, 2), (64, 8)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_step_heads(Hq, Hkv, dtype):
    check_step(f"heads {Hq}/{Hkv}", [70, 5], Hq, Hkv, 32, 64, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_step_long_contexts_are_split(dtype):
    assert kda.attn_decode_step_workspace_bytes(2, 8, 2, 128, 16, 512) > 0
    check_step("long", [5000, 37], 8, 2, 16, 128, dtype)
    check_step("one long", [3001], 4, 1, 64, 64, dtype, scale=-0.1)
    check_step("wide table", [700, 0, 65], 4, 2, 64, 64, dtype, width=200)


def test_step_many_sequences_are_not_split():
    assert kda.attn_decode_step_workspace_bytes(300, 8, 8, 64, 64, 4) == 0
    check_step("many", [(37 * i) % 150 for i in range(300)], 8, 8, 64, 64, BF)


def test_step_pages_outside_the_cache_are_left_out():
    ctx, P = [100, 90, 40], 16
    c, t = filled(ctx, 2, P, 64)
    t[0][2], t[1][0], t[1][5], t[2] = -1, 10 ** 6, -5, [-1] * len(t[2])
    q = torch.randn(3, 4, 64)
    o, lse = kda.attn_decode_step(q.to(DEV), c["kc"], c["vc"], c["ks"], c["vs"], i32(t), i32(ctx), want_lse=True)
    torch.cuda.synchronize()
    ro, rl, mag = mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"]).attend(mx.f64(q), ctx, t, 0.125)
    mx.close("o", o, ro, mag, F32, 2.0, 400)
    mx.close("lse", lse, rl, torch.full_like(rl, 8.0), F32, 1.0, 400)
    assert not o[2].any() and bool((lse[2] == -math.inf).all())


def test_step_context_longer_than_the_table():
    ctx = [64, 32]
    c, t = filled(ctx, 1, 32, 64)
    q = torch.randn(2, 1, 64)
    o, _ = kda.attn_decode_step(q.to(DEV), c["kc"], c["vc"], c["ks"], c["vs"], i32(t), i32([1000, 32]))
    p, _ = kda.attn_decode_step(q.to(DEV), c["kc"], c["vc"], c["ks"], c["vs"], i32(t), i32(ctx))
    torch.cuda.synchronize()
    assert torch.equal(o, p)


def test_streams_and_graph():
    """A decode step captured (append, then attention) and replayed while eager calls run between."""
    ctx = [500, 1, 64]
    c, t = filled([x + 1 for x in ctx], 2, 16, 64)
    gen = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(3, h, 64, generator=gen).to(BF).to(DEV) for h in (8, 2, 2))
    cu, held, after, table = i32([0, 1, 2, 3]), i32(ctx), i32([x + 1 for x in ctx]), i32(t)

    def step(**kw):
        kda.kv_cache_append(k, v, cu, held, table, c["kc"], c["vc"], c["ks"], c["vs"], **kw)
        return kda.attn_decode_step(q, c["kc"], c["vc"], c["ks"], c["vs"], table, after, want_lse=True, **kw)

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = step(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held_out = step()
    for _ in range(3):
        for x in held_out:
            x.fill_(float("nan"))
        graph.replay()
        again = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held_out, want)) and all(torch.equal(a, b) for a, b in zip(again, want))
