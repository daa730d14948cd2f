"""Appending to the 8-bit cache with rotary positions on the way: the codes and scales are those of the keys turned in
64 bits, exactly; values as in plain appending; queries within the bounds of the rotation alone."""
import numpy as np
import pytest
import torch

import gated_delta_rule_11_amd as kda
from tests import _mixers as mx
from tests import _serve as sv
from tests.test_gpu_cache import empty_cache, i32, same, table_of, tokens

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def cache(pages, Hkv, P, d, seed=0):
    return {x: y.to(DEV) for x, y in empty_cache(pages, Hkv, P, d, seed).items()}


def ends(new):
    return [0, *np.cumsum(new).tolist()]


def append(c, k, v, cu, held, table, inv, **more):
    return kda.kv_cache_append_rope(k, v, i32(cu), i32(held), i32(table), c["kc"], c["vc"], c["ks"], c["vs"], inv.to(DEV), **more)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("d,rot,interleaved,A", [(64, 64, False, 1), (64, 48, True, 3), (128, 128, False, 1), (128, 64, False, 2),
                                                 (128, 128, True, 3)])
def test_codes_scales_and_queries(d, rot, interleaved, A, P, dtype):
    """Several calls: new pages, begun pages whose scale grows, odd lengths, sequences that bring nothing."""
    gen = torch.Generator().manual_seed(P + d + rot)
    Hq, Hkv, pages = 6, 3, 40
    c = cache(pages, Hkv, P, d)
    ref = mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"])
    steps = [[37, 0, 1, 2 * P], [1, 1, 1, 1], [P, 3, 0, 5], [1, 1, 1, 1], [0, 0, 2, P - 1]]
    table = table_of([sum(s[i] for s in steps) for i in range(4)], P, pages)
    held, inv = [0, 0, 0, 0], sv.frequencies(rot // 2)
    axes = torch.randint(0, A, (rot // 2,), generator=gen, dtype=torch.int32) if A > 1 else None
    for new in steps:
        n, cu = sum(new), ends(new)
        k, v, q = (tokens(gen, n, h, d, dtype) for h in (Hkv, Hkv, Hq))
        pos = torch.randint(0, 100000, (n, A), generator=gen, dtype=torch.int32) if A > 1 else None
        got = append(c, k.to(DEV), v.to(DEV), cu, held, table, inv, q=q.to(DEV), interleaved=interleaved,
                     positions=None if pos is None else pos.to(DEV), axes=None if axes is None else axes.to(DEV))
        at = sv.places(cu, held) if pos is None else pos
        ref.append(sv.turned(mx.f64(k), at, inv, axes, interleaved)[0], mx.f64(v), cu, held, table)
        held = [a + b for a, b in zip(held, new)]
        same(c, ref, Hkv)
        want, mag = sv.turned(mx.f64(q), at, inv, axes, interleaved)
        mx.close("q", got, want, mag, dtype, 1.0, 3.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,rot,interleaved,Hkv", [(64, 64, False, 8), (64, 32, True, 4), (128, 128, True, 8), (128, 96, False, 7)])
def test_so_many_pages_that_heads_share_the_sines(d, rot, interleaved, Hkv, dtype):
    gen = torch.Generator().manual_seed(d + rot)
    P, new, held = 16, [3000, 1, 0, 3300], [5, 16, 3, 0]
    c = cache(500, Hkv, P, d)
    ref = mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"])
    table, cu, inv = table_of([a + b for a, b in zip(new, held)], P, 500), ends(new), sv.frequencies(rot // 2)
    k, v = (tokens(gen, cu[-1], Hkv, d, dtype) for _ in range(2))
    append(c, k.to(DEV), v.to(DEV), cu, held, table, inv, interleaved=interleaved)
    ref.append(sv.turned(mx.f64(k), sv.places(cu, held), inv, None, interleaved)[0], mx.f64(v), cu, held, table)
    same(c, ref, Hkv)


def test_every_length_of_a_page():
    gen = torch.Generator().manual_seed(2)
    inv = sv.frequencies(32)
    for off in (0, 1, 2, 3, 5, 15):
        for n in (1, 2, 3, 4, 7, 14, 17, 33):
            c = cache(8, 1, 16, 64)
            ref = mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"])
            table = table_of([off + n], 16, 8)
            k, v = (tokens(gen, n, 1, 64, BF) for _ in range(2))
            append(c, k.to(DEV), v.to(DEV), [0, n], [off], table, inv)
            ref.append(sv.turned(mx.f64(k), sv.places([0, n], [off]), inv)[0], mx.f64(v), [0, n], [off], table)
            same(c, ref, 1)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_turned_by_nothing_it_is_plain_appending(dtype):
    gen = torch.Generator().manual_seed(5)
    new, held = [40, 1, 0, 19], [7, 100, 3, 0]
    cu, table = ends(new), table_of([47, 101, 3, 19], 32, 12)
    k, v, q = (tokens(gen, 60, h, 128, dtype).to(DEV) for h in (2, 2, 4))
    a, b = cache(12, 2, 32, 128), cache(12, 2, 32, 128)
    got = append(a, k, v, cu, held, table, sv.frequencies(64), positions=torch.zeros(60, dtype=torch.int32, device=DEV), q=q)
    kda.kv_cache_append(k, v, i32(cu), i32(held), i32(table), b["kc"], b["vc"], b["ks"], b["vs"])
    torch.cuda.synchronize()
    assert all(torch.equal(a[x].view(torch.uint8), b[x].view(torch.uint8)) for x in a) and torch.equal(got, q)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_views_of_one_projection_and_queries_in_place(dtype):
    gen = torch.Generator().manual_seed(6)
    n, Hq, Hkv, d = 50, 5, 1, 64
    whole = tokens(gen, n, Hq + 2 * Hkv, d, dtype)
    held, cu, table, inv = [9, 20], [0, 13, 50], table_of([22, 57], 16, 9), sv.frequencies(32)
    apart, there = cache(9, Hkv, 16, d), cache(9, Hkv, 16, d)
    q, k, v = (x.contiguous().to(DEV) for x in whole.split([Hq, Hkv, Hkv], 1))
    want = append(apart, k, v, cu, held, table, inv, q=q)
    buf = whole.to(DEV)
    q, k, v = buf.split([Hq, Hkv, Hkv], 1)
    got = append(there, k, v, cu, held, table, inv, q=q, q_out=q)
    torch.cuda.synchronize()
    assert got.data_ptr() == buf.data_ptr() and torch.equal(got, want)
    assert torch.equal(buf[:, Hq:].cpu(), whole[:, Hq:])
    assert all(torch.equal(apart[x].view(torch.uint8), there[x].view(torch.uint8)) for x in apart)
    with pytest.raises(kda.KDAError):  # the turned queries would lie over the keys
        append(there, k, v, cu, held, table, inv, q=q, q_out=buf[:, 1:1 + Hq])


def test_rows_behind_the_last_sequence():
    gen = torch.Generator().manual_seed(7)
    n, Hq, d = 30, 3, 64
    k, v, q = (tokens(gen, n, h, d, F32).to(DEV) for h in (1, 1, Hq))
    k[21:], v[21:] = float("nan"), float("inf")
    inv, cu, held, table = sv.frequencies(32), [0, 4, 4, 21], [3, 5, 0], [[0, 0], [1, 0], [2, 3]]
    c = cache(4, 1, 16, d)
    ref = mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"])
    new = append(c, k, v, cu, held, table, inv, q=q)
    kept = append(c, k, v, cu, held, table, inv, q=q, q_out=torch.full_like(q, 7.0))
    torch.cuda.synchronize()
    assert torch.equal(new[:21], kept[:21]) and not new[21:].any() and bool((kept[21:] == 7).all())
    at = sv.places(cu, held)
    ref.append(sv.turned(mx.f64(k[:21]), at, inv)[0], mx.f64(v[:21]), cu, held, table)
    same(c, ref, 1)
    none = torch.zeros(0, 2, dtype=torch.int32, device=DEV)  # no sequences at all
    got = kda.kv_cache_append_rope(k, v, i32([0]), none[:, 0], none, c["kc"], c["vc"], c["ks"], c["vs"], inv.to(DEV), q=q)
    torch.cuda.synchronize()
    assert got.shape == q.shape and not got.any()
    same(c, ref, 1)


def test_dropped_tokens_still_have_their_queries_turned():
    """Past the table's pages, page ids outside the cache, and a cache without pages."""
    gen = torch.Generator().manual_seed(8)
    d, P = 64, 16
    inv, held, cu = sv.frequencies(32), [10, 0], [0, 40, 60]
    k, v, q = (tokens(gen, 60, h, d, BF).to(DEV) for h in (2, 2, 4))
    for pages, table in ((5, [[1, 2], [9, -1]]), (5, [[0, 3], [4, 1]])):
        c = cache(pages, 2, P, d)
        ref = mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"])
        got = append(c, k, v, cu, held, table, inv, q=q)
        ref.append(sv.turned(mx.f64(k), sv.places(cu, held), inv)[0], mx.f64(v), cu, held, table)
        same(c, ref, 2)
        want, mag = sv.turned(mx.f64(q), sv.places(cu, held), inv)
        mx.close("q", got, want, mag, BF, 1.0, 3.0)
    c = cache(1, 2, P, d)
    c = {x: y[:0] for x, y in c.items()}
    none = append(c, k, v, cu, held, [[0, 0], [0, 0]], inv, q=q)
    torch.cuda.synchronize()
    assert torch.equal(none, got)


def test_many_sequences():
    """More sequences than one look at them holds, most with nothing or one token."""
    gen = torch.Generator().manual_seed(9)
    rng = np.random.default_rng(3)
    N, P, d = 5000, 16, 64
    new, held = rng.choice([0, 0, 1, 1, 2, 19], N).tolist(), rng.integers(0, 30, N).tolist()
    cu, table = ends(new), table_of([a + b for a, b in zip(new, held)], P, 3 * N)
    n, inv = cu[-1], sv.frequencies(32)
    k, v, q = (tokens(gen, n, 1, d, BF) for _ in range(3))
    c = cache(3 * N, 1, P, d)
    ref = mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"])
    got = append(c, k.to(DEV), v.to(DEV), cu, held, table, inv, q=q.to(DEV))
    at = sv.places(cu, held)
    ref.append(sv.turned(mx.f64(k), at, inv)[0], mx.f64(v), cu, held, table)
    same(c, ref, 1)
    want, mag = sv.turned(mx.f64(q), at, inv)
    mx.close("q", got, want, mag, BF, 1.0, 3.0)


def test_a_cache_beyond_32_bits_of_offsets():
    """The last pages of a cache of more than 4 GiB a side, by both forms."""
    gen = torch.Generator().manual_seed(11)
    P, d, inv = 64, 128, sv.frequencies(64).to(DEV)
    far = 2 ** 32 // (P * d) + 5
    big = {x: torch.zeros(far + 6, 1, *s, dtype=t, device=DEV) for x, s, t in (("kc", (P, d), torch.uint8), ("vc", (d, P), torch.uint8), ("ks", (), F32), ("vs", (), F32))}
    for new, held in (([3, 1], [70, 0]), ([150, 90], [5, 60])):
        c = cache(6, 1, P, d)
        for x in c:
            big[x][far:] = c[x].view(big[x].dtype)
        at = {x: y.view(c[x].dtype) for x, y in big.items()}
        table = [[0, 3, 1], [5, 2, 4]]
        k, v = (tokens(gen, sum(new), 1, d, BF).to(DEV) for _ in range(2))
        append(c, k, v, ends(new), held, table, inv)
        append(at, k, v, ends(new), held, [[p + far for p in x] for x in table], inv)
        torch.cuda.synchronize()
        for x in c:
            assert torch.equal(big[x][far:], c[x].view(big[x].dtype)), x


def test_more_pages_than_the_larger_workgroups_fit_a_launch():
    """480000 sequences of eight tokens and more, seven heads: the last ones' pages are as if they came alone."""
    N, Hkv, P, d, inv = 480000, 7, 16, 128, sv.frequencies(64).to(DEV)
    new = torch.full((N,), 8, dtype=torch.int64)
    new[-3:] = torch.tensor([21, 1, 16])
    n = int(new.sum())
    assert (n // P + 2 * N) * Hkv * 512 > 2 ** 32 and n > 8 * N
    cu = torch.zeros(N + 1, dtype=torch.int32)
    cu[1:] = new.cumsum(0)
    x = torch.zeros(n, Hkv, d, dtype=BF, device=DEV)
    last = n - 38
    x[last:] = torch.randn(38, Hkv, d, device=DEV).to(BF)
    table = torch.full((N, 2), -1, dtype=torch.int32)
    table[-3:] = torch.tensor([[0, 3], [2, -1], [1, -1]])
    got, want = cache(4, Hkv, P, d), cache(4, Hkv, P, d)
    kda.kv_cache_append_rope(x, x, cu.to(DEV), torch.zeros(N, dtype=torch.int32, device=DEV), table.to(DEV), got["kc"], got["vc"], got["ks"], got["vs"], inv)
    append(want, x[last:], x[last:], [0, 21, 22, 38], [0, 0, 0], [[0, 3], [2, -1], [1, -1]], inv)
    torch.cuda.synchronize()
    for y in got:
        assert torch.equal(got[y].view(torch.uint8 if y[1] == "c" else F32), want[y].view(torch.uint8 if y[1] == "c" else F32)), y


def test_special_values():
    """Infinities and NaN among the turned channels do not enter the scale; the largest values overflow to it."""
    inv, pos = sv.frequencies(32), torch.zeros(4, dtype=torch.int32)
    x = torch.randn(4, 1, 64)
    x[1, 0, 3], x[2, 0, 9], x[3, 0, :] = float("nan"), float("inf"), 0.0
    pos[:] = torch.tensor([5, 0, 3, 100])
    c = cache(2, 1, 16, 64)
    ref = mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"])
    append(c, x.to(DEV), -x.to(DEV), [0, 4], [0], [[1]], inv, positions=pos.to(DEV))
    ref.append(sv.turned(mx.f64(x), pos, inv)[0], mx.f64(-x), [0, 4], [0], [[1]])
    same(c, ref, 1)


def test_stream_and_replays():
    """Captured, with positions that move on between replays."""
    gen = torch.Generator().manual_seed(10)
    N, P, d = 6, 16, 64
    k, v, q = (tokens(gen, N, h, d, BF).to(DEV) for h in (2, 2, 4))
    held, inv = i32([0, 5, 15, 16, 31, 3]), sv.frequencies(32).to(DEV)
    table = i32(table_of([64] * N, P, 24))
    cu = i32(list(range(N + 1)))
    c = cache(24, 2, P, d)
    out, g = torch.zeros_like(q), torch.cuda.CUDAGraph()
    call = lambda c, o, **m: kda.kv_cache_append_rope(k, v, cu, held, table, c["kc"], c["vc"], c["ks"], c["vs"], inv, q=q, q_out=o, **m)  # noqa: E731
    eager = {x: y.clone() for x, y in c.items()}
    with torch.cuda.graph(g):
        call(c, out)
    side = torch.cuda.Stream()
    for t in range(4):
        want = torch.zeros_like(q)
        side.wait_stream(torch.cuda.current_stream())
        call(eager, want, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and all(torch.equal(c[x].view(torch.uint8), eager[x].view(torch.uint8)) for x in c)
        held += 1
        k.mul_(1.5)


def test_refused_by_the_binding():
    c = cache(4, 2, 16, 64)
    k, inv = torch.zeros(5, 2, 64, device=DEV), sv.frequencies(32)
    ok = dict(cu=[0, 5], held=[0], table=[[0]])
    append(c, k, k.clone(), **ok, inv=inv)
    q = torch.zeros(5, 4, 64, device=DEV)
    for bad in (dict(q_out=q), dict(q=q.to(BF)), dict(q=q[:4]), dict(q=q[..., :32]), dict(q=q, q_out=q.half()), dict(q=q, q_out_dtype=torch.float16),
                dict(positions=torch.zeros(5, device=DEV)), dict(positions=torch.zeros(4, dtype=torch.int32, device=DEV)),
                dict(axes=torch.zeros(5, dtype=torch.int32, device=DEV)), dict(q=q[:, :3].contiguous()),
                dict(q=q.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(kda.KDAError):
            append(c, k, k, **ok, inv=inv, **bad)
    for args in (dict(cu=[0, 5, 5]), dict(held=[0, 0]), dict(inv=sv.frequencies(20)), dict(inv=sv.frequencies(40))):
        with pytest.raises(kda.KDAError):
            append(c, k, k, **{**ok, "inv": inv, **args})
    with pytest.raises(kda.KDAError):
        append(c, k, k.to(BF), **ok, inv=inv)
