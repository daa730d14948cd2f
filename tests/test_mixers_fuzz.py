"""Property-based checks of the host validation of the linear, prompt and cache entry points (CPU only),
in the manner and with the helpers of test_abi_fuzz: arguments from mixes of valid, boundary and
invalid values, fake device addresses; every call returns a documented status, a bad dtype code is
KDA_ERR_DTYPE, KDA_OK never comes back for a negative size, and a workspace smaller than what the
query asks for is never accepted.  (A call that passes validation fails at its first HIP call here.)"""
import math

import pytest

pytest.importorskip("hypothesis")
from hypothesis import given  # noqa: E402
from hypothesis import strategies as st  # noqa: E402

from tests.test_abi_fuzz import (DIMS, DTYPES, ERR_HIP, FUZZ, OK, SCALES, SIZES, WSB, L, _check,  # noqa: E402,F401
                                 pointers, pytestmark)

FLAGS = st.sampled_from([0, 0, 1, 1, 2, -1])
HEADS = st.sampled_from([-1, 0, 1, 2, 3, 4, 8, 24, 64, 1 << 16])
PAGES = st.sampled_from([-16, 0, 1, 16, 32, 48, 64, 128])
ATTN = st.sampled_from([-64, 0, 32, 64, 64, 128, 128, 256])


def _accepted(s, wsb, need, *floats):
    if s == ERR_HIP:  # validation is behind it
        assert wsb >= need and all(math.isfinite(x) for x in floats)


@FUZZ
@given(p=pointers(8), it=DTYPES, ot=DTYPES, ph=FLAGS, scale=SCALES, B=SIZES, T=SIZES, H=SIZES, dk=DIMS, dv=DIMS, wsb=WSB)
def test_fuzz_linear_fwd(L, p, it, ot, ph, scale, B, T, H, dk, dv, wsb):  # noqa: F811
    need = L.kda_linear_chunk_fwd_workspace_bytes(B, T, H, dk, dv, it)
    s = L.kda_linear_chunk_fwd(p[0], p[1], p[2], it, p[3], ph, p[4], p[5], ot, p[6], B, T, H, dk, dv, scale, p[7], wsb, None)
    _check(s, [it, ot], [B, T, H])
    _accepted(s, wsb, need, scale)


@FUZZ
@given(p=pointers(14), it=DTYPES, gt=DTYPES, ph=FLAGS, scale=SCALES, B=SIZES, T=SIZES, H=SIZES, dk=DIMS, dv=DIMS, wsb=WSB)
def test_fuzz_linear_bwd(L, p, it, gt, ph, scale, B, T, H, dk, dv, wsb):  # noqa: F811
    need = L.kda_linear_chunk_bwd_workspace_bytes(B, T, H, dk, dv, it, ph)
    s = L.kda_linear_chunk_bwd(p[0], p[1], p[2], it, p[3], ph, p[4], p[5], p[6], p[7], p[8], p[9], gt, p[10], p[11], B, T, H,
                               dk, dv, scale, p[12], wsb, None)
    _check(s, [it, gt], [B, T, H])
    _accepted(s, wsb, need, scale)


@FUZZ
@given(p=pointers(7), it=DTYPES, ot=DTYPES, ph=FLAGS, scale=SCALES, N=SIZES, H=SIZES, dk=DIMS, dv=DIMS)
def test_fuzz_linear_step(L, p, it, ot, ph, scale, N, H, dk, dv):  # noqa: F811
    s = L.kda_linear_decode_step(p[0], p[1], p[2], it, p[3], ph, p[4], p[5], p[6], ot, N, H, dk, dv, scale, None)
    _check(s, [it, ot], [N, H])
    _accepted(s, 0, 0, scale)


@FUZZ
@given(p=pointers(12), it=DTYPES, ot=DTYPES, gt=DTYPES, tail=FLAGS, scale=SCALES, n=SIZES, ns=SIZES, Hq=HEADS, Hkv=HEADS, d=ATTN,
       wsb=WSB, backward=st.booleans())
def test_fuzz_prompt(L, p, it, ot, gt, tail, scale, n, ns, Hq, Hkv, d, wsb, backward):  # noqa: F811
    if backward:
        need = L.kda_attn_prompt_bwd_workspace_bytes(n, Hq, Hkv, d)
        s = L.kda_attn_prompt_bwd(p[0], p[1], p[2], it, p[3], p[4], ot, p[5], p[6], p[7], p[8], p[9], gt, n, ns, Hq, Hkv, d,
                                  scale, tail, p[10], wsb, None)
        _check(s, [it, ot, gt], [n, ns, Hq, Hkv])
        _accepted(s, wsb, need, scale)
    else:
        s = L.kda_attn_prompt_fwd(p[0], p[1], p[2], it, p[3], p[4], ot, p[5], n, ns, Hq, Hkv, d, scale, tail, None)
        _check(s, [it, ot], [n, ns, Hq, Hkv])
        _accepted(s, 0, 0, scale)
    if s in (OK, ERR_HIP):
        assert d in (64, 128) and Hq % Hkv == 0 and tail in (0, 1)


@FUZZ
@given(p=pointers(9), it=DTYPES, n=SIZES, N=SIZES, Hkv=HEADS, d=ATTN, page=PAGES, pages=SIZES, mp=SIZES)
def test_fuzz_append(L, p, it, n, N, Hkv, d, page, pages, mp):  # noqa: F811
    s = L.kda_kv_cache_append(p[0], p[1], it, p[2], p[3], p[4], p[5], p[6], p[7], p[8], n, N, Hkv, d, page, pages, mp, None)
    _check(s, [it], [n, N, Hkv, pages, mp])
    if s in (OK, ERR_HIP):
        assert d in (64, 128) and page in (16, 32, 64)


@FUZZ
@given(p=pointers(10), it=DTYPES, ot=DTYPES, scale=SCALES, N=SIZES, Hq=HEADS, Hkv=HEADS, d=ATTN, page=PAGES, pages=SIZES,
       mp=SIZES, wsb=WSB)
def test_fuzz_step(L, p, it, ot, scale, N, Hq, Hkv, d, page, pages, mp, wsb):  # noqa: F811
    need = L.kda_attn_decode_step_workspace_bytes(N, Hq, Hkv, d, page, mp)
    s = L.kda_attn_decode_step(p[0], it, p[1], p[2], p[3], p[4], p[5], p[6], p[7], ot, p[8], N, Hq, Hkv, d, page, pages, mp,
                               scale, p[9], wsb, None)
    _check(s, [it, ot], [N, Hq, Hkv, pages, mp])
    _accepted(s, wsb, need, scale)
    if s in (OK, ERR_HIP):
        assert d in (64, 128) and page in (16, 32, 64) and Hq % Hkv == 0
