"""The linear, prompt and cache entry points on the CPU: what they refuse, before anything is
launched (fake device addresses; every call below fails validation or has nothing to do), what the
binding refuses, and the 64-bit references against differences."""
import ctypes
import math

import pytest
import torch

import gated_delta_rule_11_amd as kda
from tests import _mixers as mx
from tests.test_abi import BF16, ERR_ALIAS, ERR_ALIGN, ERR_DTYPE, ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, ERR_WORKSPACE, F32, L, OK  # noqa: F401


def P(i, off=0):
    return ctypes.c_void_p(0x100000000 * (i + 1) + off)


HUGE = 1 << 40


def lin_fwd(L, q=P(0), k=P(1), v=P(2), it=BF16, g=P(3), ph=0, S_in=P(4), o=P(5), ot=BF16, S_out=P(6), B=2, T=100, H=3,  # noqa: F811
            dk=64, dv=64, scale=1.0, ws=P(7), wsb=HUGE):
    return L.kda_linear_chunk_fwd(q, k, v, it, g, ph, S_in, o, ot, S_out, B, T, H, dk, dv, scale, ws, wsb, None)


def lin_bwd(L, q=P(0), k=P(1), v=P(2), it=BF16, g=P(3), ph=0, S_in=P(4), do=P(5), dS=P(6), dq=P(8), dk=P(9), dv=P(10),  # noqa: F811
            gt=F32, dg=P(11), dSi=P(12), B=2, T=100, H=3, dkd=64, dvd=64, scale=1.0, ws=P(13), wsb=HUGE):
    return L.kda_linear_chunk_bwd(q, k, v, it, g, ph, S_in, do, dS, dq, dk, dv, gt, dg, dSi, B, T, H, dkd, dvd, scale, ws,
                                  wsb, None)


def lin_step(L, q=P(0), k=P(1), v=P(2), it=BF16, g=P(3), ph=0, S_in=P(4), S_out=P(4), o=P(5), ot=F32, N=4, H=3, dk=64,  # noqa: F811
             dv=64, scale=1.0):
    return L.kda_linear_decode_step(q, k, v, it, g, ph, S_in, S_out, o, ot, N, H, dk, dv, scale, None)


def prompt_fwd(L, q=P(0), k=P(1), v=P(2), it=BF16, cu=P(3), o=P(4), ot=F32, lse=P(5), n=100, ns=2, Hq=4, Hkv=2, d=64,  # noqa: F811
               scale=1.0, tail=0):
    return L.kda_attn_prompt_fwd(q, k, v, it, cu, o, ot, lse, n, ns, Hq, Hkv, d, scale, tail, None)


def prompt_bwd(L, q=P(0), k=P(1), v=P(2), it=BF16, cu=P(3), o=P(4), ot=F32, lse=P(5), do=P(6), dq=P(7), dk=P(8), dv=P(9),  # noqa: F811
               gt=F32, n=100, ns=2, Hq=4, Hkv=2, d=64, scale=1.0, tail=0, ws=P(10), wsb=HUGE):
    return L.kda_attn_prompt_bwd(q, k, v, it, cu, o, ot, lse, do, dq, dk, dv, gt, n, ns, Hq, Hkv, d, scale, tail, ws, wsb,
                                 None)


def append(L, k=P(0), v=P(1), it=BF16, cu=P(2), ctx=P(3), table=P(4), kc=P(5), vc=P(6), ks=P(7), vs=P(8), n=10, N=2, Hkv=2,  # noqa: F811
           d=64, page=16, pages=8, mp=4):
    return L.kda_kv_cache_append(k, v, it, cu, ctx, table, kc, vc, ks, vs, n, N, Hkv, d, page, pages, mp, None)


def step(L, q=P(0), it=BF16, kc=P(1), vc=P(2), ks=P(3), vs=P(4), table=P(5), ctx=P(6), o=P(7), ot=F32, lse=P(8), N=2, Hq=4,  # noqa: F811
         Hkv=2, d=64, page=16, pages=8, mp=400, scale=1.0, ws=P(9), wsb=HUGE):
    return L.kda_attn_decode_step(q, it, kc, vc, ks, vs, table, ctx, o, ot, lse, N, Hq, Hkv, d, page, pages, mp, scale, ws,
                                  wsb, None)


@pytest.mark.parametrize("call", [lin_fwd, lin_bwd, lin_step])
def test_linear_refusals(L, call):  # noqa: F811
    assert call(L, it=2) == ERR_DTYPE and call(L, it=-1) == ERR_DTYPE
    assert call(L, **{"gt" if call is lin_bwd else "ot": 3}) == ERR_DTYPE
    B = "N" if call is lin_step else "B"
    dk, dv = ("dkd", "dvd") if call is lin_bwd else ("dk", "dv")
    assert call(L, **{B: -1}) == ERR_SHAPE and call(L, H=0) == ERR_SHAPE and call(L, **{dk: 0}) == ERR_SHAPE
    assert call(L, **{B: 1 << 20, "H": 1 << 10}) == ERR_SHAPE
    assert call(L, **{dk: 48}) == ERR_UNSUPPORTED and call(L, **{dv: 256}) == ERR_UNSUPPORTED
    assert call(L, ph=2) == ERR_UNSUPPORTED and call(L, scale=math.nan) == ERR_UNSUPPORTED
    assert call(L, scale=math.inf) == ERR_UNSUPPORTED
    for x in ("q", "k", "v", "g"):
        assert call(L, **{x: None}) == ERR_NULL
        assert call(L, **{x: P(20, 2)}) == ERR_ALIGN
    assert call(L, **{B: 0}) == OK


def test_linear_forward_refusals(L):  # noqa: F811
    assert lin_fwd(L, T=-1) == ERR_SHAPE and lin_fwd(L, T=(1 << 31) - 1) == ERR_SHAPE
    assert lin_fwd(L, o=None) == ERR_NULL
    assert lin_fwd(L, o=P(0)) == ERR_ALIAS and lin_fwd(L, S_out=P(3)) == ERR_ALIAS and lin_fwd(L, o=P(4)) == ERR_ALIAS
    assert lin_fwd(L, S_in=P(4), S_out=P(4, 64)) == ERR_ALIAS and lin_fwd(L, o=P(6)) == ERR_ALIAS
    need = L.kda_linear_chunk_fwd_workspace_bytes(1, 4096, 8, 64, 64, BF16)
    assert need > 0 and L.kda_linear_chunk_fwd_workspace_bytes(4, 4096, 64, 64, 64, BF16) == 0
    few = dict(B=1, T=4096, H=8)
    assert lin_fwd(L, ws=None, **few) == ERR_NULL and lin_fwd(L, wsb=need - 1, **few) == ERR_WORKSPACE
    assert lin_fwd(L, ws=P(7, 4), **few) == ERR_ALIGN and lin_fwd(L, ws=P(0), **few) == ERR_ALIAS
    assert lin_fwd(L, ws=P(6), **few) == ERR_ALIAS
    assert L.kda_linear_chunk_fwd_workspace_bytes(1, 4096, 8, 64, 48, BF16) == 0
    assert L.kda_linear_chunk_fwd_workspace_bytes(-1, 4096, 8, 64, 64, BF16) == 0


def test_linear_backward_refusals(L):  # noqa: F811
    for x in ("do", "dq", "dk", "dv", "dg"):
        assert lin_bwd(L, **{x: None}) == ERR_NULL
    for x in ("dq", "dk", "dv", "dg", "dSi", "ws"):
        for at in (P(0), P(3), P(5), P(6)):
            assert lin_bwd(L, **{x: at}) == ERR_ALIAS, x
    assert lin_bwd(L, dq=P(9)) == ERR_ALIAS and lin_bwd(L, ws=P(12)) == ERR_ALIAS
    need = L.kda_linear_chunk_bwd_workspace_bytes(2, 100, 3, 64, 64, BF16, 0)
    assert lin_bwd(L, wsb=need - 1) == ERR_WORKSPACE and lin_bwd(L, ws=None) == ERR_NULL
    assert L.kda_linear_chunk_bwd_workspace_bytes(2, 100, 3, 64, 64, BF16, 1) > need
    assert lin_bwd(L, B=1 << 12, T=1 << 12, H=1 << 7) == ERR_SHAPE  # more chunks than a launch holds
    assert L.kda_linear_chunk_bwd_workspace_bytes(1 << 12, 1 << 12, 1 << 7, 64, 64, BF16, 0) == 0


def test_linear_step_refusals(L):  # noqa: F811
    assert lin_step(L, S_in=None) == ERR_NULL and lin_step(L, S_out=None) == ERR_NULL and lin_step(L, o=None) == ERR_NULL
    assert lin_step(L, S_out=P(4, 256)) == ERR_ALIAS and lin_step(L, o=P(4)) == ERR_ALIAS and lin_step(L, S_out=P(0)) == ERR_ALIAS


@pytest.mark.parametrize("call", [prompt_fwd, prompt_bwd])
def test_prompt_refusals(L, call):  # noqa: F811
    assert call(L, it=5) == ERR_DTYPE and call(L, ot=5) == ERR_DTYPE
    assert call(L, n=-1) == ERR_SHAPE and call(L, ns=-1) == ERR_SHAPE and call(L, Hkv=0) == ERR_SHAPE and call(L, Hq=0) == ERR_SHAPE
    assert call(L, n=(1 << 31) - 1, Hq=1, Hkv=1) == ERR_SHAPE
    assert call(L, d=32) == ERR_UNSUPPORTED and call(L, d=96) == ERR_UNSUPPORTED and call(L, Hq=5) == ERR_UNSUPPORTED
    assert call(L, Hq=2, Hkv=4) == ERR_UNSUPPORTED and call(L, scale=math.inf) == ERR_UNSUPPORTED
    assert call(L, tail=2) == ERR_UNSUPPORTED
    for x in ("q", "k", "v", "cu", "o"):
        assert call(L, **{x: None}) == ERR_NULL
        assert call(L, **{x: P(20, 2)}) == ERR_ALIGN
    assert call(L, n=0) == OK and call(L, ns=0) == OK


def test_prompt_aliases_and_workspace(L):  # noqa: F811
    assert prompt_fwd(L, o=P(0)) == ERR_ALIAS and prompt_fwd(L, lse=P(3)) == ERR_ALIAS and prompt_fwd(L, lse=P(4)) == ERR_ALIAS
    for x in ("lse", "do", "dq", "dk", "dv", "ws"):
        assert prompt_bwd(L, **{x: None}) == ERR_NULL
    for x in ("dq", "dk", "dv", "ws"):
        for at in (P(0), P(4), P(5), P(6)):
            assert prompt_bwd(L, **{x: at}) == ERR_ALIAS
    assert prompt_bwd(L, dk=P(9)) == ERR_ALIAS and prompt_bwd(L, wsb=L.kda_attn_prompt_bwd_workspace_bytes(100, 4, 2, 64) - 1) == ERR_WORKSPACE
    assert L.kda_attn_prompt_bwd_workspace_bytes(100, 5, 2, 64) == 0
    assert prompt_bwd(L, gt=2) == ERR_DTYPE


def test_cache_refusals(L):  # noqa: F811
    for call in (append, step):
        assert call(L, it=9) == ERR_DTYPE
        assert call(L, N=-1) == ERR_SHAPE and call(L, pages=-1) == ERR_SHAPE and call(L, mp=-1) == ERR_SHAPE and call(L, page=0) == ERR_SHAPE
        assert call(L, page=48) == ERR_UNSUPPORTED and call(L, d=32) == ERR_UNSUPPORTED
        for x in ("kc", "vc", "ks", "vs", "table", "ctx"):
            assert call(L, **{x: None}) == ERR_NULL
            assert call(L, **{x: P(20, 2)}) == ERR_ALIGN
        assert call(L, N=0) == OK
    for x in ("k", "v", "cu"):
        assert append(L, **{x: None}) == ERR_NULL
    assert append(L, n=0) == OK and append(L, pages=0) == OK and append(L, mp=0) == OK and append(L, n=-1) == ERR_SHAPE
    assert append(L, kc=P(0)) == ERR_ALIAS and append(L, ks=P(8)) == ERR_ALIAS and append(L, vs=P(3)) == ERR_ALIAS
    assert step(L, Hq=5) == ERR_UNSUPPORTED and step(L, scale=math.nan) == ERR_UNSUPPORTED and step(L, ot=4) == ERR_DTYPE
    assert step(L, q=None) == ERR_NULL and step(L, o=None) == ERR_NULL and step(L, ws=None) == ERR_NULL
    assert step(L, o=P(1)) == ERR_ALIAS and step(L, lse=P(7)) == ERR_ALIAS and step(L, ws=P(2)) == ERR_ALIAS
    need = L.kda_attn_decode_step_workspace_bytes(2, 4, 2, 64, 16, 400)
    assert need > 0 and step(L, wsb=need - 1) == ERR_WORKSPACE


def test_binding_refusals():
    """Before any pointer is passed: tensors on the CPU, and what is no tensor."""
    q = torch.zeros(1, 4, 2, 64)
    for call in (lambda: kda.linear_chunk_fwd(q, q, q, q[..., 0]), lambda: kda.linear_chunk_bwd(q, q, q, q[..., 0], q),
                 lambda: kda.linear_decode_step(q[0], q[0], q[0], q[0, ..., 0], q),
                 lambda: kda.attn_prompt_fwd(q[0], q[0], q[0], torch.tensor([0, 4], dtype=torch.int32)),
                 lambda: kda.attn_decode_step(q[0], q, q, q, q, q, q), lambda: kda.kv_cache_append(q, q, q, q, q, q, q, q, q),
                 lambda: kda.linear_chunk_fwd(None, None, None, None)):
        with pytest.raises(kda.KDAError):
            call()


def test_linear_reference_against_differences():
    gen = torch.Generator().manual_seed(0)
    rn = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x = {"q": rn(1, 7, 2, 3), "k": rn(1, 7, 2, 3), "v": rn(1, 7, 2, 4), "g": -rn(1, 7, 2).exp() * 0.2, "S": rn(1, 2, 3, 4)}
    do, dS = rn(1, 7, 2, 4), rn(1, 2, 3, 4)
    got, _ = mx.linear_grad(*x.values(), do, dS, 0.7)
    loss = lambda *a: (lambda r: (r[0] * do).sum() + (r[1] * dS).sum())(mx.linear(*a, 0.7))  # noqa: E731
    for name in x:
        u = rn(*x[name].shape)
        at = lambda s: loss(*[y + s * 1e-5 * u if n == name else y for n, y in x.items()])  # noqa: E731,B023
        diff = (at(1) - at(-1)) / 2e-5
        assert abs(diff - (got[{"S": "dS_in"}.get(name, "d" + name)] * u).sum()) < 1e-7, name


def test_prompt_reference_against_differences():
    gen = torch.Generator().manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, cu = {"q": rn(9, 4, 5), "k": rn(9, 2, 5), "v": rn(9, 2, 5)}, [0, 3, 3, 9]
    do = rn(9, 4, 5)
    got, _ = mx.prompt(*x.values(), cu, 0.4, do)
    for name in x:
        u = rn(*x[name].shape)
        at = lambda s: (mx.prompt(*[y + s * 1e-5 * u if n == name else y for n, y in x.items()], cu, 0.4)[0]["o"] * do).sum()  # noqa: E731,B023
        assert abs((at(1) - at(-1)) / 2e-5 - (got["d" + name] * u).sum()) < 1e-7, name


def test_table_of_the_8bit_format():
    """The reference's values are torch's for the format, and its rounding torch's conversion."""
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double().numpy()
    assert (mx.e4m3_values() == codes).all()
    x = torch.randn(20000, generator=torch.Generator().manual_seed(2)) * torch.exp(2 * torch.randn(20000, generator=torch.Generator().manual_seed(3)))
    x = x.clamp(-448, 448)
    assert (mx.e4m3_round(x.double().numpy()) == x.to(torch.float8_e4m3fn).float().double().numpy()).all()
    assert mx.scale_of(torch.tensor([448.0]).numpy()) == 1.0 and mx.scale_of(torch.tensor([448.5]).numpy()) == 2.0
    assert mx.scale_of(torch.tensor([224.0, math.inf]).numpy()) == 0.5 and mx.scale_of(torch.zeros(1).numpy()) == 2.0 ** -100
