"""Attention of a chunk of new tokens over the 8-bit cache on the GPU, against the softmax in 64 bits on the same codes.

Bounds: with bf16 queries each probability and the output are rounded once (2^-8 each).  In fp32: a sum over the channels and
one over the tokens (three exact products to a term with fp32 queries), the exponent's own |x| 2^-24 for |x| up to 48, the
joins.  Two forms divide the work: one workgroup to a tile of rows, and where the table has room for many tokens all rows'
keys in even shares.  Every test runs with the table as it is and with one that has room for more (``wider``)."""
import math

import numpy as np
import pytest
import torch

import gated_delta_rule_11_amd as kda
from tests import _mixers as mx
from tests import _serve as sv
from tests.test_gpu_cache import filled, i32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
F8 = torch.float8_e4m3fn


MORE = 0


@pytest.fixture(params=[0, 4500], autouse=True)
def more(request):
    global MORE
    MORE = request.param


def wider(t, P):
    """The table with room for MORE tokens: columns of no page."""
    return [list(x) + [-1] * max(0, MORE // P - len(x)) for x in t]


def ends(new):
    return [0, *np.cumsum(new).tolist()]


def run(c, t, q, new, ctx, **kw):
    kw = {"o_dtype": q.dtype, "want_lse": True, **kw}
    return kda.attn_chunk_fwd(q.to(DEV), i32(ends(new)), c["kc"], c["vc"], c["ks"], c["vs"], i32(wider(t, c["kc"].shape[2])), i32(ctx), **kw)


def compare(label, got, c, t, q, new, ctx, scale=None):
    torch.cuda.synchronize()
    d, dtype = q.shape[-1], q.dtype
    n = sum(new)
    o, lse, mag = sv.chunk(mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"]), mx.f64(q)[:n], ends(new), ctx, t, d ** -0.5 if scale is None else scale)
    terms = 3 * d + 3 * max(1, *ctx) + 4 * 48 + 64
    mx.close(label + " o", got[0][:n], o, mag, BF if got[0].dtype == BF or dtype == BF else F32, 2.0, terms)
    mx.close(label + " lse", got[1][:n], lse, torch.full_like(lse, 8.0), F32, 1.0, terms)


def check(label, new, ctx, Hq, Hkv, P, d, dtype, scale=None, seed=0, **kw):
    c, t = filled(ctx, Hkv, P, d, seed=sum(ctx) + Hq + seed, **kw)
    q = torch.randn(sum(new), Hq, d, generator=torch.Generator().manual_seed(9 + seed)).to(dtype)
    got = run(c, t, q, new, ctx, scale=scale)
    compare(label, got, c, t, q, new, ctx, scale)
    return c, t, q, got


NEW = [1, 2, 0, 15, 16, 17, 33, 64, 7, 1, 40, 5]
CTX = [1, 300, 70, 15, 64, 129, 33, 65, 250, 64, 41, 16]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("width", [None, 64])
def test_lengths(width, d, P, dtype):
    more = {} if width is None else {"width": width * 16 // P * 4}
    assert (kda.attn_chunk_fwd_workspace_bytes(sum(NEW), 12, 4, 2, d, P, more.get("width", -(-300 // P)), dtype) > 0) == (width is not None)
    check(f"P={P} d={d}", NEW, CTX, 4, 2, P, d, dtype, **more)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (7, 1), (16, 1), (17, 1), (40, 2), (64, 8), (130, 1)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("width", [None, 40])
def test_heads(Hq, Hkv, dtype, width):
    check(f"heads {Hq}/{Hkv}", [3, 1, 30, 9], [70, 5, 90, 200], Hq, Hkv, 32, 64, dtype, **({} if width is None else {"width": width}))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,P", [(128, 16), (64, 64), (128, 64)])
def test_long_contexts_are_divided(d, P, dtype):
    check("one row", [1], [4001], 4, 1, P, d, dtype)
    check("drafts", [5, 3], [3000, 1111], 8, 2, P, d, dtype)
    check("chunk", [130], [2500], 4, 2, P, d, dtype)
    check("whole prompts", [700, 1, 333], [700, 1, 333], 2, 1, P, d, dtype)
    check("uneven", [1, 200, 1, 1, 17], [10, 2200, 1700, 1, 600], 4, 2, P, d, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scales(dtype):
    for scale in (-0.3, 0.0, 1e-30, 2.0):
        for new, ctx in (([3, 60], [200, 65]), ([2, 50], [700, 300])):
            check(f"scale {scale}", new, ctx, 2, 1, 32, 64, dtype, scale=scale)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_that_see_nothing(dtype):
    """More new tokens than the sequence holds: the first rows lie before its start."""
    for new, ctx in (([5, 40, 3], [2, 7, 0]), ([5, 200, 3, 70], [2, 9, 0, 900]), ([300], [1])):
        c, t, q, (o, lse) = check("before the start", new, ctx, 4, 2, 16, 64, dtype)
        for a, b, x in zip(ends(new), ends(new)[1:], ctx):
            none = slice(a, max(a, b - x))
            assert not o[none].any() and bool((lse[none] == -math.inf).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pages_outside_the_cache_are_left_out(dtype):
    new, ctx, P = [2, 40, 33, 3, 40], [100, 90, 40, 900, 200], 16
    c, t = filled(ctx, 2, P, 64)
    t[0][2], t[1][0], t[1][5], t[2] = -1, 10 ** 6, -5, [-1] * len(t[2])
    t[3][7], t[3][-8], t[4][1], t[4][12] = -1, 2 ** 31 - 1, -1, 10 ** 5
    q = torch.randn(sum(new), 4, 64).to(dtype)
    got = run(c, t, q, new, ctx)
    compare("left out", got, c, t, q, new, ctx)
    assert not got[0][42:75].any() and bool((got[1][42:75] == -math.inf).all())
    short = [x[:12] for x in t[:3]]
    got = run(c, short, q[:75], new[:3], ctx[:3])
    compare("left out, one workgroup to a tile", got, c, short, q[:75], new[:3], ctx[:3])


def test_context_longer_than_the_table():
    for new, ctx, P in (([3, 70], [1000, 128], 32), ([3, 70], [2000, 128], 32)):
        c, t = filled([128, 128], 1, P, 64)
        if ctx[0] == 2000:
            t = [x + x[:0] + [-1] * 20 for x in t]
        q = torch.randn(73, 2, 64)
        compare("short table", run(c, t, q, new, ctx), c, t, q, new, ctx)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("width", [None, 70])
def test_nan_and_infinity_reach_the_rows_that_see_them(width, dtype):
    """NaN codes behind the last token are not used; one in a new token's values reaches its own row and those behind it;
    one in its key likewise; so do values that the page's scale takes beyond fp32."""
    for new, ctx in (([6, 1], [70, 40]), ([9, 60], [30, 130]), ([20, 100], [100, 100])):
        c, t = filled(ctx, 1, 16, 64, **({} if width is None else {"width": width}))
        q = torch.randn(sum(new), 3, 64).to(dtype)
        clean = run(c, t, q, new, ctx)
        code = {x: c[x].view(torch.uint8) for x in ("kc", "vc")}
        for i in range(2):  # what lies behind the last token
            if ctx[i] % 16:
                code["kc"][t[i][ctx[i] // 16], 0, ctx[i] % 16:] = 0x7F
                code["vc"][t[i][ctx[i] // 16], 0, :, ctx[i] % 16:] = 0xFF
        got = run(c, t, q, new, ctx)
        torch.cuda.synchronize()
        assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
        at = ctx[1] - new[1] // 2 - 1  # a token among the second sequence's new ones
        page, off = t[1][at // 16], at % 16
        row = new[0] + (at - (ctx[1] - new[1]))
        kept = code["vc"][page, 0, 5, off].item(), code["kc"][page, 0, off, 7].item()
        code["vc"][page, 0, 5, off] = 0x7F
        o = run(c, t, q, new, ctx)[0]
        torch.cuda.synchronize()
        assert bool(o[row:, :, 5].isnan().all())
        o[row:, :, 5] = clean[0][row:, :, 5]
        assert torch.equal(o, clean[0])
        code["vc"][page, 0, 5, off], code["kc"][page, 0, off, 7] = kept[0], 0xFF
        o, lse = run(c, t, q, new, ctx)
        torch.cuda.synchronize()
        assert bool(o[row:].isnan().all()) and bool(lse[row:].isnan().all())
        assert torch.equal(o[:row], clean[0][:row]) and torch.equal(lse[:row], clean[1][:row])
        code["kc"][page, 0, off, 7] = kept[1]
        before = c["vs"][page, 0].item()
        code["vc"][page, 0, :, :] = 0
        code["vc"][page, 0, 3, off] = 0x7E  # 448 * 2^120
        c["vs"][page, 0] = 2.0 ** 120
        o = run(c, t, q, new, ctx)[0]
        torch.cuda.synchronize()
        # infinite, or NaN: fp32 queries' probabilities go in as three parts, and a last part of zero (a probability of
        # up to 16 significant bits) times infinity is NaN
        assert not o[row:, :, 3].isfinite().any() and bool(o[:row].isfinite().all())
        o[row:, :, 3] = 0
        assert bool(o.isfinite().all()) and before > 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P,d", [(16, 64), (32, 128), (64, 128)])
def test_scales_of_pages_not_in_use_do_not_matter(P, d, dtype):
    """Page 0 among them, NaN and infinite: with lengths that end inside a step, and with pages left out."""
    new, ctx = [3, 40, 90, 20], [70, 90, 150, 700]
    for width in (None, 70 * 64 // P):
        c, t = filled(ctx, 1, P, d, **({} if width is None else {"width": width}))
        held = [t[i][:-(-x // P)] for i, x in enumerate(ctx)]
        free = min(set(range(c["kc"].shape[0])) - {p for x in held for p in x})
        swap = {0: free, free: 0}
        for x in c:
            both = c[x].view(torch.uint8) if x[1] == "c" else c[x]
            both[[0, free]] = both[[free, 0]]
        t = [[swap.get(p, p) for p in held[i]] + [0] * (len(t[i]) - len(held[i])) for i in range(4)]
        t[1][0] = t[2][1] = t[3][-1] = -1
        q = torch.randn(sum(new), 2, d).to(dtype)
        want = run(c, t, q, new, ctx)
        compare("before", want, c, t, q, new, ctx)
        unused = sorted(set(range(c["kc"].shape[0])) - {p for i, x in enumerate(ctx) for p in t[i][:-(-x // P)]})
        assert 0 in unused
        for word in (math.nan, math.inf, -math.inf):
            c["ks"][unused], c["vs"][unused] = word, word
            got = run(c, t, q, new, ctx)
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P,d", [(16, 64), (64, 128)])
def test_nan_among_values_that_every_row_sees(P, d, dtype):
    """In the first steps of a long context, for every number of a tile's rows, also beside tokens that lie in no page."""
    for width in (None, 70 * 64 // P):
        for new in (1, 9, 20, 40, 70, 128):  # two heads of a group: up to 128 rows to a tile, whole tiles behind it
            ctx = [new + 200]
            c, t = filled(ctx, 1, P, d, **({} if width is None else {"width": width}))
            q = torch.randn(new, 2, d).to(dtype)
            for gone in (None, 0 if P == 64 else 2):
                if gone is not None:
                    t[0][gone] = -1
                clean = run(c, t, q, [new], ctx)
                code = c["vc"].view(torch.uint8)
                at = [1, 70, 130, 199] if gone is None else [65, 70, 199]
                kept = [code[t[0][x // P], 0, 5 + i, x % P].item() for i, x in enumerate(at)]
                for i, x in enumerate(at):
                    code[t[0][x // P], 0, 5 + i, x % P] = 0x7F
                got = run(c, t, q, [new], ctx)
                torch.cuda.synchronize()
                for i, x in enumerate(at):
                    assert bool(got[0][..., 5 + i].isnan().all()), (width, new, gone, x)
                    code[t[0][x // P], 0, 5 + i, x % P] = kept[i]
                got[0][..., 5:5 + len(at)] = clean[0][..., 5:5 + len(at)]
                assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
                if gone == 2:  # the missing page's neighbours in its step
                    code[t[0][1], 0, 9, 3] = 0x7F
                    got = run(c, t, q, [new], ctx)
                    torch.cuda.synchronize()
                    assert bool(got[0][..., 9].isnan().all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_cache_beyond_32_bits_of_offsets(dtype):
    """The last pages of a cache of more than 4 GiB a side give what the first pages of a small one give."""
    new, ctx, P, d = [40, 3], [700, 50], 64, 128
    c, t = filled(ctx, 1, P, d)
    pages = c["kc"].shape[0]
    far = 2 ** 32 // (P * d) + 5
    big = {x: torch.zeros((far + pages, *c[x].shape[1:]), dtype=torch.uint8 if x[1] == "c" else F32, device=DEV) for x in c}
    for x in c:
        big[x][far:] = c[x].view(big[x].dtype)
        big[x] = big[x].view(c[x].dtype)
    q = torch.randn(43, 4, d).to(dtype)
    want = run(c, t, q, new, ctx)
    got = run(big, [[p + far for p in x] for x in t], q, new, ctx)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_workspace_of_any_contents():
    """Words of one, which would mark every part as one that goes on, and words of a large number."""
    new, ctx = [5, 150, 1], [3000, 700, 90]
    c, t = filled(ctx, 2, 16, 64)
    q = torch.randn(156, 4, 64).to(BF)
    want = run(c, t, q, new, ctx)
    for word in (1, 2, 0x7F7F7F7F, -1):
        ws = torch.full((kda.attn_chunk_fwd_workspace_bytes(156, 3, 4, 2, 64, 16, len(wider(t, 16)[0]), BF) // 4,), word, dtype=torch.int32, device=DEV)
        got = run(c, t, q, new, ctx, workspace=ws.view(torch.uint8))
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_largest_values(dtype):
    """Values near the end of fp32 and probabilities summed without overflow on the way."""
    new, ctx = [4, 50], [600, 90]
    c, t = filled(ctx, 1, 16, 64)
    c["vs"].fill_(2.0 ** 119)
    c["vc"].view(torch.uint8).fill_(0x78)  # 256: 2^127
    q = torch.randn(54, 2, 64).to(dtype)
    o, _ = run(c, t, q, new, ctx)
    torch.cuda.synchronize()
    mx.close("2^127", o, torch.full((54, 2, 64), 2.0 ** 127, dtype=torch.float64), torch.full((54, 2, 64), 2.0 ** 127, dtype=torch.float64), dtype, 2.0, 2500)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_peaked_rows(dtype):
    """Scores of hundreds: one token has all the weight, wherever among the steps it lies."""
    new, ctx = [3, 90], [700, 400]
    c, t = filled(ctx, 1, 32, 64)
    q = (torch.randn(93, 2, 64) * 30).to(dtype)
    got = run(c, t, q, new, ctx, scale=1.0)
    torch.cuda.synchronize()
    o, lse, mag = sv.chunk(mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"]), mx.f64(q), ends(new), ctx, t, 1.0)
    # a score's rounding: |s| log2(e) 2^-24 and its sum's, in units of the channels' magnitude (below 30 * 64 * 30)
    top = 2.0 ** 16
    terms = 3 * 64 + 3 * 700
    mx.close("o", got[0], o, mag, dtype, 2.0, terms + 2 * top * 64 * 3)
    mx.close("lse", got[1], lse, torch.full_like(lse, top), F32, 1.0, 3 * 64 + 8)


@pytest.mark.parametrize("out", [BF, F32])
def test_types_mix(out):
    c, t = filled([90, 700], 2, 16, 128)
    q = torch.randn(80, 4, 128).to(F32 if out == BF else BF)
    got = run(c, t, q, [40, 40], [90, 700], o_dtype=out)
    assert got[0].dtype == out
    compare("mixed", got, c, t, q, [40, 40], [90, 700])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_single_tokens_agree_with_the_step(dtype):
    ctx = [1, 17, 500, 64, 2000]
    c, t, q, got = check("singles", [1] * 5, ctx, 8, 2, 64, 128, dtype)
    o, lse = kda.attn_decode_step(q.to(DEV), c["kc"], c["vc"], c["ks"], c["vs"], i32(t), i32(ctx), o_dtype=dtype, want_lse=True)
    compare("the step", (o, lse), c, t, q, [1] * 5, ctx)


def test_many_sequences():
    rng = np.random.default_rng(1)
    N = 700
    new = rng.choice([0, 0, 1, 1, 1, 2, 9, 40], N).tolist()
    ctx = [a + int(b) for a, b in zip(new, rng.integers(0, 60, N))]
    check("many", new, ctx, 2, 1, 16, 64, BF)
    check("many, wide table", new, ctx, 2, 1, 16, 64, BF, width=100)


def test_random_configurations():
    rng = np.random.default_rng(7)
    for case in range(40):
        N, Hkv = int(rng.integers(1, 7)), int(rng.choice([1, 2, 3]))
        Hq, P, d = Hkv * int(rng.choice([1, 2, 3, 4, 5, 8])), int(rng.choice([16, 32, 64])), int(rng.choice([64, 128]))
        new = [int(x) for x in rng.choice([0, 1, 1, 3, 8, 21, 70, 150], N)]
        ctx = [a + int(rng.choice([0, 1, 17, 64, 300, 900])) for a in new]
        if sum(new) == 0:
            continue
        check(f"case {case}: {new} {ctx} {Hq}/{Hkv} P={P} d={d}", new, ctx, Hq, Hkv, P, d, BF if case % 3 else F32, seed=case)


def guarded(shape, dtype):
    n, pad = math.prod(shape), 4096
    buf = torch.full((n + 2 * pad,), 7.0, dtype=dtype, device=DEV)
    return buf[pad:pad + n].view(shape), lambda: bool((buf[:pad] == 7).all()) and bool((buf[pad + n:] == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_views_guards_tail_and_workspace(dtype):
    """Queries as a view of a projection's output; outputs between guards; rows behind the last sequence; a workspace of NaN."""
    for new, ctx, Hq, P, d in (([3, 50, 1], [40, 70, 1], 6, 16, 64), ([3, 50, 1], [900, 70, 1], 4, 64, 128)):
        c, t = filled(ctx, 2, P, d)
        n, rows = sum(new), sum(new) + 9
        whole = torch.randn(rows, Hq + 4, d).to(dtype)
        whole[n:] = float("nan")
        q = whole.to(DEV)[:, 1:1 + Hq]
        want = run(c, t, q.contiguous(), new, ctx)
        torch.cuda.synchronize()
        assert not want[0][n:].any() and not want[1][n:].any()
        compare("tail", want, c, t, whole[:n, 1:1 + Hq], new, ctx)
        (o, fine), (lse, fine_l) = guarded((rows, Hq, d), dtype), guarded((rows, Hq), F32)
        ws = torch.full((max(16, kda.attn_chunk_fwd_workspace_bytes(rows, 3, Hq, 2, d, P, len(wider(t, P)[0]), dtype)),), 255, dtype=torch.uint8, device=DEV)
        run(c, t, q, new, ctx, o=o, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        assert fine() and fine_l() and torch.equal(o[:n], want[0][:n]) and torch.equal(lse[:n], want[1][:n])
        assert bool((o[n:] == 7).all()) and bool((lse[n:] == 7).all())


def test_entries_out_of_order_touch_nothing_outside():
    """Meaningless offsets and lengths give meaningless rows, within the outputs."""
    c, t = filled([600, 90], 2, 16, 64)
    for cu in ([0, 50, 20], [30, 10, 5], [-7, 10, 10 ** 6], [0, 2 ** 31 - 1, 3], [60, 0, 0]):
        for ctx in ([600, 90], [-5, 2 ** 31 - 1], [2 ** 31 - 1, -2 ** 31]):
            for tab in (wider(t, 16), [x[:20] for x in t]):
                (o, fine), (lse, fine_l) = guarded((60, 4, 64), F32), guarded((60, 4), F32)
                kda.attn_chunk_fwd(torch.randn(60, 4, 64, device=DEV), i32(cu), c["kc"], c["vc"], c["ks"], c["vs"], i32(tab), i32(ctx), o=o, lse=lse)
                torch.cuda.synchronize()
                assert fine() and fine_l()


def test_streams_replays_and_the_same_bits():
    new, ctx = [5, 1, 90, 33], [900, 40, 400, 64]
    c, t = filled([x + 3 for x in ctx], 2, 16, 128)
    q = torch.randn(sum(new), 8, 128, device=DEV).to(BF)
    cu, held, table = i32(ends(new)), i32(ctx), i32(wider(t, 16))
    call = lambda **kw: kda.attn_chunk_fwd(q, cu, c["kc"], c["vc"], c["ks"], c["vs"], table, held, want_lse=True, o_dtype=BF, **kw)  # noqa: E731
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = call(stream=side)
    mine = call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, m) for a, b, m in zip(want, other, mine))
    a, b = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(a):
        first = call()
    with torch.cuda.graph(b):
        second = call()
    for i in range(4):
        a.replay()
        b.replay()
        eager = call()
        torch.cuda.synchronize()
        assert all(torch.equal(x, e) and torch.equal(y, e) for x, y, e in zip(first, second, eager))
        q.mul_(1.25)
        held.add_(1 if i < 3 else 0)


def test_two_graphs_on_one_workspace():
    """Of different sizes, replayed in turn, with eager calls on it in between."""
    c, t = filled([3000, 700, 90], 2, 16, 64)
    q = torch.randn(160, 4, 64, device=DEV).to(BF)
    table = i32(wider(t, 16))
    most = kda.attn_chunk_fwd_workspace_bytes(160, 3, 4, 2, 64, 16, table.shape[1], BF)
    ws = torch.full((most,), 255, dtype=torch.uint8, device=DEV)
    cu = [i32(ends(new)) for new in ([5, 150, 1], [2, 0, 7])]
    ctx = i32([3000, 700, 90])
    call = lambda i, w: kda.attn_chunk_fwd(q[:(160, 9)[i]], cu[i], c["kc"], c["vc"], c["ks"], c["vs"], table, ctx, want_lse=True, workspace=w)  # noqa: E731
    want = [call(i, None) for i in range(2)]
    graphs, got = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            got.append(call(i, ws))
    for i in (0, 1, 1, 0, 0, 1, 0):
        for x in got[i]:
            x.fill_(7)
        graphs[i].replay()
        eager = call(1 - i, ws)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i])) and all(torch.equal(a, b) for a, b in zip(eager, want[1 - i]))


def test_nothing_to_do_and_no_pages():
    c, t = filled([40], 2, 16, 64)
    q = torch.randn(5, 4, 64, device=DEV)
    args = lambda cu, tab, ctx: (i32(cu), c["kc"], c["vc"], c["ks"], c["vs"], tab, ctx)  # noqa: E731
    none = torch.zeros(0, 3, dtype=torch.int32, device=DEV)
    o, lse = kda.attn_chunk_fwd(q, *args([0], none, none[:, 0]), want_lse=True)
    assert not o.any() and not lse.any()
    o, _ = kda.attn_chunk_fwd(q[:0], *args([0, 0], i32(t), i32([40])))
    assert o.shape == (0, 4, 64)
    for tab in (i32(t), i32([[]]).view(1, 0)):
        empty = {x: (y if tab.numel() == 0 else y[:0]) for x, y in c.items()}
        o, lse = kda.attn_chunk_fwd(q, i32([0, 3]), empty["kc"], empty["vc"], empty["ks"], empty["vs"], tab, i32([40]), want_lse=True)
        torch.cuda.synchronize()
        assert not o.any() and bool((lse[:3] == -math.inf).all()) and not lse[3:].any()


def test_refused_by_the_binding():
    c, t = filled([20], 2, 16, 64)
    q = torch.zeros(3, 4, 64, device=DEV)
    ok = dict(q=q, cu_seqlens=i32([0, 3]), k_cache=c["kc"], v_cache=c["vc"], k_scale=c["ks"], v_scale=c["vs"], block_table=i32(t), context_len=i32([20]))
    kda.attn_chunk_fwd(**ok)
    for bad in (dict(q=q[0]), dict(q=q.half()), dict(q=q[..., :32]), dict(q=q[:, :3].contiguous()), dict(q=q.transpose(0, 1)), dict(cu_seqlens=i32([0, 1, 3])),
                dict(cu_seqlens=torch.tensor([0, 3], device=DEV)), dict(k_cache=c["kc"].view(torch.uint8)), dict(v_cache=c["kc"]), dict(k_scale=c["ks"].double()),
                dict(block_table=i32(t + t)), dict(context_len=i32([20, 3])), dict(o=torch.zeros(3, 4, 32, device=DEV)), dict(o=q), dict(lse=torch.zeros(3, 4, 1, device=DEV)),
                dict(scale=math.nan), dict(o_dtype=torch.float16), dict(workspace=torch.zeros(16)), dict(context_len=i32([20]).cpu())):
        with pytest.raises(kda.KDAError):
            kda.attn_chunk_fwd(**{**ok, **bad})
    long = i32([[0] * 100])
    with pytest.raises(kda.KDAError):
        kda.attn_chunk_fwd(**{**ok, "block_table": long, "workspace": torch.zeros(16, dtype=torch.uint8, device=DEV)})
