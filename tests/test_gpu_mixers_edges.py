"""Calls of the linear, prompt and cache entry points that their documentation allows at the ends of
its ranges: a cache without pages, many heads in one call, NaN and infinities."""
import ctypes
import math

import pytest
import torch

import gated_delta_rule_11_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("N,max_pages", [(3, 4), (1, 600)])
def test_step_over_a_cache_without_pages(N, max_pages):
    """Every token lies in a page outside the cache: o = 0, lse = -inf, and the table, which may be NULL,
    is not read.  Through the C ABI with NULL, whole and in parts, and through the binding."""
    Hq, Hkv, d, P = 4, 2, 64, 16
    q = torch.randn(N, Hq, d, device=DEV)
    ctx = torch.tensor([max_pages * P] * N, dtype=torch.int32, device=DEV)
    o, lse = torch.full((N, Hq, d), 7.0, device=DEV), torch.full((N, Hq), 7.0, device=DEV)
    need = kda.attn_decode_step_workspace_bytes(N, Hq, Hkv, d, P, max_pages)
    assert (need > 0) == (max_pages > 4)
    ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device=DEV)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    st = kda.lib().kda_attn_decode_step(p(q), 0, None, None, None, None, None, p(ctx), p(o), 0, p(lse), N, Hq, Hkv, d, P, 0,
                                        max_pages, 0.125, p(ws), need, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert st == 0 and not o.any() and bool((lse == -math.inf).all())
    code = torch.zeros(0, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    none = torch.zeros(0, Hkv, device=DEV)
    table = torch.zeros(N, max_pages, dtype=torch.int32, device=DEV)
    o, lse = kda.attn_decode_step(q, code.view(0, Hkv, P, d), code.view(0, Hkv, d, P), none, none, table, ctx, want_lse=True)
    torch.cuda.synchronize()
    assert not o.any() and bool((lse == -math.inf).all())


def test_linear_many_heads_of_one_call():
    """B * H = 2^18 heads of two tokens, forward and backward: the same bits as those entries alone."""
    B, T, H, d, n = 8192, 2, 32, 16, 4
    gen = torch.Generator(DEV).manual_seed(0)
    rn = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    q, k, v, do = (rn(B, T, H, d).to(BF) for _ in range(4))
    g, S, dS = -rn(B, T, H).abs(), rn(B, H, d, d), rn(B, H, d, d)
    o, So = kda.linear_chunk_fwd(q, k, v, g, S_in=S)
    got = kda.linear_chunk_bwd(q, k, v, g, do, dS_out=dS, S_in=S)
    for b in (0, B // 2 - 3, B - n):
        x = [t[b:b + n].contiguous() for t in (q, k, v, g, do, dS, S)]
        o1, S1 = kda.linear_chunk_fwd(*x[:4], S_in=x[6])
        want = kda.linear_chunk_bwd(*x[:5], dS_out=x[5], S_in=x[6])
        torch.cuda.synchronize()
        assert torch.equal(o[b:b + n], o1) and torch.equal(So[b:b + n], S1)
        assert all(torch.equal(got[y][b:b + n], want[y]) for y in want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,d", [([30, 45, 20], 64), ([190, 260, 1, 69], 128)])
def test_prompt_gradients_of_non_finite_rows(lens, d, dtype):
    """A NaN or infinity in a row of one sequence reaches the gradients that depend on it, and no others: those
    are the same bits as without it.  What depends on row r of its sequence: through q, dq of r, dk and dv of
    keys up to r; through do, dq of r, dk up to r, one channel of dv up to r; through k, dq from r on, and all
    of the sequence's dk and dv; through v, dq from r on, and dk."""
    Hq, Hkv, ch = 4, 2, 3
    gen = torch.Generator().manual_seed(len(lens))
    n, cu = sum(lens), [0]
    for x in lens:
        cu.append(cu[-1] + x)
    clean = {x: torch.randn(n, h, d, generator=gen).to(dtype) for x, h in (("q", Hq), ("k", Hkv), ("v", Hkv), ("do", Hq))}
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)

    def grads(x):
        g = {y: z.to(DEV) for y, z in x.items()}
        o, lse = kda.attn_prompt_fwd(g["q"], g["k"], g["v"], c, o_dtype=dtype)
        r = kda.attn_prompt_bwd(g["q"], g["k"], g["v"], c, o, lse, g["do"], grad_dtype=dtype)
        torch.cuda.synchronize()
        return {y: z.cpu() for y, z in r.items()}

    want = grads(clean)
    a, b = cu[1], cu[2]
    for r in (a, a + lens[1] // 2, b - 1):
        for name, val in (("q", math.nan), ("do", math.nan), ("do", math.inf), ("k", math.nan), ("v", math.nan), ("v", -math.inf)):
            x = dict(clean, **{name: clean[name].clone()})
            x[name][r, :, ch] = val
            got = grads(x)
            hit = {"dq": range(r, r + 1) if name in ("q", "do") else range(r, b),
                   "dk": range(a, r + 1) if name in ("q", "do") else range(a, b),
                   "dv": range(a, r + 1) if name in ("q", "do") else range(a, b) if name == "k" else range(0)}
            for y, rows in hit.items():
                same = [i for i in range(n) if i not in rows]
                assert torch.equal(got[y][same], want[y][same]), (name, val, r, y)
                if name == "do" and y == "dv":
                    rest = [i for i in range(d) if i != ch]
                    assert torch.equal(got[y][..., rest], want[y][..., rest]), (val, r)
                    assert not torch.isfinite(got[y][list(rows), :, ch]).any(), (val, r)
                elif len(rows):
                    assert not torch.isfinite(got[y][list(rows)]).any(), (name, val, r, y)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H,dk,dv", [(150, 2, 128, 128), (90, 2, 16, 64), (70, 1, 64, 16), (900, 1, 32, 32)])
def test_linear_non_finite_values(T, H, dk, dv, dtype):
    """A NaN or infinity in token s reaches what depends on it, and nothing else changes by a bit: through q
    its own output, dk (one channel) and dv up to s; through k outputs and dq (one channel) from s on, and
    its own dv; through v one channel of the outputs from s on, dq from s on, and its own dk; through do its own
    dq, dk and dv (one channel) up to s; through g outputs from s on."""
    B, ch = 2, 3
    gen = torch.Generator().manual_seed(T)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    clean = {"q": unit(rn(B, T, H, dk)).to(dtype), "k": unit(rn(B, T, H, dk)).to(dtype), "v": rn(B, T, H, dv).to(dtype),
             "g": -0.1 * torch.rand(B, T, H, generator=gen), "do": rn(B, T, H, dv).to(dtype)}

    def run(x):
        g = [x[n].to(DEV) for n in ("q", "k", "v", "g")]
        o, S = kda.linear_chunk_fwd(*g, o_dtype=dtype)
        r = kda.linear_chunk_bwd(*g, x["do"].to(DEV), grad_dtype=dtype)
        torch.cuda.synchronize()
        return {"o": o.cpu(), **{n: r[n].cpu() for n in ("dq", "dk", "dv")}}

    want = run(clean)
    none, one = range(0), slice(ch, ch + 1)
    for s in (0, 20, 63, T - 5, T - 1):
        own, back, on = range(s, s + 1), range(0, s + 1), range(s, T)
        hits = {"q": {"o": (own, None), "dq": (none, None), "dk": (back, one), "dv": (back, None)},
                "k": {"o": (on, None), "dq": (on, one), "dk": (none, None), "dv": (own, None)},
                "v": {"o": (on, one), "dq": (on, None), "dk": (own, None), "dv": (none, None)},
                "do": {"o": (none, None), "dq": (own, None), "dk": (back, None), "dv": (back, one)},
                "g": {"o": (on, None)}}
        for name, hit in hits.items():
            for val in (math.nan, math.inf) if name in ("v", "do") else (math.nan,):
                x = dict(clean, **{name: clean[name].clone()})
                x[name][(1, s, 0) if name == "g" else (1, s, 0, ch)] = val
                got = run(x)
                for y, (rows, chan) in hit.items():
                    mark = torch.zeros(got[y].shape, dtype=torch.bool)
                    if len(rows):
                        mark[1, rows[0]:rows[-1] + 1, 0, chan if chan else slice(None)] = True
                    assert torch.equal(got[y][~mark], want[y][~mark]), (name, val, s, y)
                    assert not torch.isfinite(got[y][mark]).any(), (name, val, s, y)


def test_what_is_no_tensor_is_refused():
    """A missing or foreign argument is the binding's own error, whichever it is."""
    q = torch.zeros(1, 4, 2, 64, device=DEV)
    g, cu, S = q[..., 0].contiguous(), torch.tensor([0, 4], dtype=torch.int32, device=DEV), torch.zeros(4, 2, 64, 64, device=DEV)
    c = torch.zeros(1, 2, 16, 64, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    ct, s, s2, one = c.clone().view(1, 2, 64, 16), torch.ones(1, 2, device=DEV), torch.ones(1, 2, device=DEV), cu[:1]
    table = one.view(1, 1)
    calls = [(kda.linear_chunk_fwd, [q, q, q, g]), (kda.linear_chunk_bwd, [q, q, q, g, q]),
             (kda.linear_decode_step, [q[0], q[0], q[0], g[0], S]), (kda.attn_prompt_fwd, [q[0], q[0], q[0], cu]),
             (kda.attn_prompt_bwd, [q[0], q[0], q[0], cu, q[0], g[0], q[0]]),
             (kda.kv_cache_append, [q[0], q[0], cu, one, table, c, ct, s, s2]),
             (kda.attn_decode_step, [q[0, :1], c, ct, s, s2, table, one])]
    for call, args in calls:
        call(*args)
        for i in range(1, len(args)):
            for bad in (None, [0.0], 3):
                with pytest.raises(kda.KDAError):
                    call(*args[:i], bad, *args[i + 1:])
    torch.cuda.synchronize()
