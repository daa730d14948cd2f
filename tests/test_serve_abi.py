"""The serving calls around the paged cache on the CPU: what they refuse, before anything is launched (fake device
addresses; every call below fails validation or has nothing to do), the sizes at which they begin to refuse, and the
64-bit references against closed forms."""
import math

import pytest
import torch

import gated_delta_rule_11_amd as kda
from tests import _serve as sv
from tests.test_abi import BF16, ERR_ALIAS, ERR_ALIGN, ERR_DTYPE, ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, ERR_WORKSPACE, F32, L, OK  # noqa: F401
from tests.test_mixers_abi import HUGE, P


def rope(L, x=P(0), it=BF16, xs=256, pos=P(1), A=1, inv=P(2), ax=None, rot=64, inter=0, back=0, y=P(3), yt=BF16, ys=256, n=10, H=4, d=64):  # noqa: F811
    return L.kda_rope(x, it, xs, pos, A, inv, ax, rot, inter, back, y, yt, ys, n, H, d, None)


def append(L, k=P(0), ks=128, v=P(1), vs=128, it=BF16, q=P(2), qs=256, qo=P(3), qt=BF16, qos=256, pos=None, A=1, inv=P(4), ax=None, rot=64,  # noqa: F811
           inter=0, cu=P(5), ctx=P(6), table=P(7), kc=P(8), vc=P(9), ksc=P(10), vsc=P(11), n=10, N=2, Hq=4, Hkv=2, d=64, page=16, pages=8, mp=4,
           tail=0):
    return L.kda_kv_cache_append_rope(k, ks, v, vs, it, q, qs, qo, qt, qos, pos, A, inv, ax, rot, inter, cu, ctx, table, kc, vc, ksc, vsc, n, N, Hq,
                                      Hkv, d, page, pages, mp, tail, None)


def chunk(L, q=P(0), qs=256, it=BF16, cu=P(1), kc=P(2), vc=P(3), ks=P(4), vs=P(5), table=P(6), ctx=P(7), o=P(8), ot=F32, lse=P(9), n=10, N=2, Hq=4,  # noqa: F811
          Hkv=2, d=64, page=16, pages=8, mp=400, scale=1.0, tail=0, ws=P(10), wsb=HUGE):
    return L.kda_attn_chunk_fwd(q, qs, it, cu, kc, vc, ks, vs, table, ctx, o, ot, lse, n, N, Hq, Hkv, d, page, pages, mp, scale, tail, ws, wsb, None)


def test_rope_refusals(L):  # noqa: F811
    assert rope(L, it=2) == ERR_DTYPE and rope(L, yt=-1) == ERR_DTYPE
    assert rope(L, n=-1) == ERR_SHAPE and rope(L, H=0) == ERR_SHAPE and rope(L, d=0) == ERR_SHAPE and rope(L, n=1 << 20, H=1 << 12, xs=1 << 18, ys=1 << 18) == ERR_SHAPE
    for bad in (dict(d=24, xs=96, ys=96, rot=16), dict(d=272, xs=1088, ys=1088), dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=80), dict(A=0), dict(A=9),
                dict(inter=2), dict(back=-1)):
        assert rope(L, **bad) == ERR_UNSUPPORTED, bad
    assert rope(L, xs=255) == ERR_SHAPE and rope(L, ys=248) == ERR_SHAPE and rope(L, xs=1 << 29) == ERR_SHAPE
    assert rope(L, xs=260) == ERR_ALIGN and rope(L, ys=257) == ERR_ALIGN and rope(L, it=F32, xs=258) == ERR_ALIGN
    for x in ("x", "pos", "inv", "y"):
        assert rope(L, **{x: None}) == ERR_NULL
        assert rope(L, **{x: P(20, 2)}) == ERR_ALIGN
    assert rope(L, ax=P(20, 2)) == ERR_ALIGN
    assert rope(L, n=0, x=None) == OK


def test_rope_overlaps(L):  # noqa: F811
    for at in (P(1), P(2)):
        assert rope(L, y=at) == ERR_ALIAS
    assert rope(L, ax=P(3)) == ERR_ALIAS
    assert rope(L, y=P(0, 16)) == ERR_ALIAS and rope(L, y=P(0), yt=F32) == ERR_ALIAS and rope(L, y=P(0), ys=512) == ERR_ALIAS
    # rows of 4 heads of 64 (512 bytes) in a buffer of 1280 bytes a row: apart by a row's width or meeting
    wide = dict(xs=640, ys=640, x=P(0), pos=None)  # (pos is missing: refused for that once the sizes and strides are taken)
    assert rope(L, **wide) == ERR_NULL
    wide["pos"] = P(1)
    for off, meets in ((16, True), (496, True), (784, True), (1264, True), (1280 * 3 + 256, True)):
        assert (rope(L, y=P(0, off), **wide) == ERR_ALIAS) == meets, off


def test_append_refusals(L):  # noqa: F811
    assert append(L, it=2) == ERR_DTYPE and append(L, qt=5) == ERR_DTYPE
    for x in ("n", "N", "pages", "mp"):
        assert append(L, **{x: -1}) == ERR_SHAPE
    assert append(L, page=0) == ERR_SHAPE and append(L, Hkv=0) == ERR_SHAPE
    for bad in (dict(page=48), dict(d=32), dict(Hq=3), dict(rot=72), dict(rot=8), dict(A=0), dict(A=9), dict(inter=3), dict(tail=2)):
        assert append(L, **bad) == ERR_UNSUPPORTED, bad
    for x, w in (("ks", 128), ("vs", 128), ("qs", 256), ("qos", 256)):
        assert append(L, **{x: w - 8}) == ERR_SHAPE and append(L, **{x: w + 4}) == ERR_ALIGN
    for x in ("k", "v", "qo", "inv", "cu", "ctx", "table", "kc", "vc", "ksc", "vsc"):
        assert append(L, **{x: None}) == ERR_NULL, x
        assert append(L, **{x: P(20, 2)}) == ERR_ALIGN, x
    assert append(L, q=P(20, 8)) == ERR_ALIGN and append(L, pos=P(20, 2)) == ERR_ALIGN and append(L, ax=P(20, 1)) == ERR_ALIGN
    assert append(L, A=2) == ERR_NULL  # two axes and no positions
    for x in ("kc", "vc", "ksc", "vsc"):
        for at in (P(0), P(1), P(2), P(3), P(4), P(5), P(6), P(7)):
            assert append(L, **{x: at}) == ERR_ALIAS, x
    assert append(L, kc=P(9)) == ERR_ALIAS and append(L, ksc=P(11)) == ERR_ALIAS
    for at in (P(0), P(1), P(4), P(5), P(6), P(7), P(2, 16)):
        assert append(L, qo=at) == ERR_ALIAS
    assert append(L, qo=P(2), qt=F32) == ERR_ALIAS and append(L, pos=P(3)) == ERR_ALIAS
    assert append(L, n=0) == OK and append(L, N=0) == OK and append(L, pages=0, q=None) == OK and append(L, mp=0, q=None) == OK
    assert append(L, pages=0, k=None, v=None, table=None, kc=None, vc=None, ksc=None, vsc=None, inv=None) == ERR_NULL  # queries to turn
    assert append(L, n=1 << 28, Hq=1 << 6, Hkv=1 << 6, q=None) == ERR_SHAPE


def test_chunk_refusals(L):  # noqa: F811
    assert chunk(L, it=2) == ERR_DTYPE and chunk(L, ot=-1) == ERR_DTYPE
    for x in ("n", "N", "pages", "mp"):
        assert chunk(L, **{x: -1}) == ERR_SHAPE
    assert chunk(L, page=0) == ERR_SHAPE and chunk(L, Hq=0) == ERR_SHAPE and chunk(L, Hkv=0) == ERR_SHAPE
    for bad in (dict(page=48), dict(d=32), dict(Hq=3), dict(scale=math.nan), dict(scale=math.inf), dict(tail=-1), dict(Hq=2048, qs=2048 * 64, Hkv=1)):
        assert chunk(L, **bad) == ERR_UNSUPPORTED, bad
    assert chunk(L, qs=255) == ERR_SHAPE and chunk(L, qs=260) == ERR_ALIGN
    for x in ("q", "cu", "kc", "vc", "ks", "vs", "table", "ctx", "o", "ws"):
        assert chunk(L, **{x: None}) == ERR_NULL, x
        assert chunk(L, **{x: P(20, 2)}) == ERR_ALIGN, x
    assert chunk(L, lse=P(20, 2)) == ERR_ALIGN
    need = L.kda_attn_chunk_fwd_workspace_bytes(10, 2, 4, 2, 64, 16, 400, BF16)
    assert need > 0 and chunk(L, wsb=need - 1) == ERR_WORKSPACE
    for x in ("o", "lse", "ws"):
        for i in range(8):
            assert chunk(L, **{x: P(i)}) == ERR_ALIAS, (x, i)
    assert chunk(L, lse=P(8)) == ERR_ALIAS and chunk(L, ws=P(8)) == ERR_ALIAS and chunk(L, ws=P(9)) == ERR_ALIAS
    assert chunk(L, n=0) == OK and chunk(L, N=0) == OK
    assert chunk(L, n=1, N=(1 << 24) - 1, Hq=4, Hkv=2) == ERR_SHAPE  # more tiles than a launch holds
    assert chunk(L, n=1, N=(1 << 23) - 1, Hq=4, Hkv=2, q=None) == ERR_NULL


def test_chunk_workspace(L):  # noqa: F811
    size = L.kda_attn_chunk_fwd_workspace_bytes
    assert size(10, 2, 4, 2, 64, 16, 64, BF16) == 0 and size(10, 2, 4, 2, 64, 16, 65, BF16) > 0  # 1024 tokens
    assert size(0, 2, 4, 2, 64, 16, 400, BF16) == 0 and size(10, 0, 4, 2, 64, 16, 400, BF16) == 0
    for bad in (dict(d=32), dict(page=48), dict(Hq=3), dict(it=7), dict(n=-1)):
        a = dict(n=10, N=2, Hq=4, Hkv=2, d=64, page=16, mp=400, it=BF16) | bad
        assert size(*a.values()) == 0, bad
    assert size(1 << 20, 4096, 32, 8, 128, 64, 1 << 20, BF16) == size(1000, 256, 32, 8, 128, 64, 4096, BF16)  # goes by the GPU, not by the call
    for page, mp in ((16, 100), (64, 30), (64, 60), (32, 2000)):  # what is enough for a call is enough for smaller ones
        sizes = [size(n, N, 16, 4, 64, page, mp, BF16) for n, N in ((1, 1), (3, 2), (40, 7), (900, 64), (40000, 700))]
        assert sizes == sorted(sizes) and sizes[0] > 0
        for n, N in ((1, 1), (40, 7), (40000, 700)):
            ok = dict(n=n, N=N, Hq=16, Hkv=4, qs=1024, page=page, mp=mp, ws=P(20), wsb=size(n, N, 16, 4, 64, page, mp, BF16))
            assert chunk(L, **ok, o=None) == ERR_NULL and chunk(L, **ok, q=P(20, 2)) == ERR_ALIGN


def test_binding_refuses_cpu_tensors(L):  # noqa: F811
    x, i = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32)
    c = torch.zeros(2, 2, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s, t = torch.zeros(2, 2), torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(kda.KDAError):
        kda.rope(x, i, torch.zeros(32))
    with pytest.raises(kda.KDAError):
        kda.kv_cache_append_rope(x, x, i[:2], i[:1], t, c, c.view(2, 2, 64, 16), s, s, torch.zeros(32))
    with pytest.raises(kda.KDAError):
        kda.attn_chunk_fwd(x, i[:2], c, c.view(2, 2, 64, 16), s, s, t, i[:1])


def test_reference_rotation():
    """A quarter turn exchanges the pair, turns add, and lengths stay."""
    inv = torch.tensor([1.0, 0.5])
    x = torch.randn(5, 2, 6, dtype=torch.float64)
    for inter in (False, True):
        y, _ = sv.turned(x, torch.tensor([3, 1, 4, 1, 5]), inv, None, inter)
        z, _ = sv.turned(y, torch.tensor([2, 7, -4, 0, 1]), inv, None, inter)
        w, _ = sv.turned(x, torch.tensor([5, 8, 0, 1, 6]), inv, None, inter)
        assert torch.allclose(z, w, atol=1e-14) and torch.equal(z[..., 4:], x[..., 4:])
        assert torch.allclose(y[..., :4].norm(dim=-1), x[..., :4].norm(dim=-1))
    quarter = torch.tensor([math.pi / 2], dtype=torch.float64)
    y, _ = sv.turned(torch.tensor([[[1.0, 2.0]]]), torch.tensor([1]), quarter)
    assert torch.allclose(y, torch.tensor([[[-2.0, 1.0]]], dtype=torch.float64))
    two, _ = sv.turned(x[..., :4], torch.tensor([[1, 10]] * 5), inv, torch.tensor([1, 0]))
    ten, _ = sv.turned(x[..., :4], torch.tensor([10] * 5), inv)
    one, _ = sv.turned(x[..., :4], torch.tensor([1] * 5), inv)
    assert torch.allclose(two[..., 0::2], ten[..., 0::2]) and torch.allclose(two[..., 1::2], one[..., 1::2])
