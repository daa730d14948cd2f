"""Property-based checks of the host validation of the serving calls (CPU only), in the manner and with the helpers of
test_abi_fuzz and test_mixers_fuzz."""
import pytest

pytest.importorskip("hypothesis")
from hypothesis import given  # noqa: E402
from hypothesis import strategies as st  # noqa: E402

from tests.test_abi_fuzz import DTYPES, ERR_HIP, FUZZ, OK, SCALES, SIZES, WSB, L, _check, pointers, pytestmark  # noqa: E402,F401
from tests.test_mixers_fuzz import ATTN, FLAGS, HEADS, PAGES, _accepted  # noqa: E402

STRIDES = st.sampled_from([-64, 0, 64, 128, 256, 512, 520, 1024, 4096, 1 << 22, 1 << 28, 1 << 62])
ROTS = st.sampled_from([-16, 0, 8, 16, 32, 48, 64, 64, 128, 256])
AXES = st.sampled_from([-1, 0, 1, 1, 1, 2, 3, 8, 9])


@FUZZ
@given(p=pointers(5), it=DTYPES, ot=DTYPES, xs=STRIDES, ys=STRIDES, A=AXES, rot=ROTS, inter=FLAGS, back=FLAGS, n=SIZES, H=HEADS, d=ATTN)
def test_fuzz_rope(L, p, it, ot, xs, ys, A, rot, inter, back, n, H, d):  # noqa: F811
    s = L.kda_rope(p[0], it, xs, p[1], A, p[2], p[3], rot, inter, back, p[4], ot, ys, n, H, d, None)
    _check(s, [it, ot], [n, H])
    if s in (OK, ERR_HIP):
        assert 16 <= rot <= d <= 256 and 1 <= A <= 8 and inter in (0, 1) and back in (0, 1) and min(xs, ys) >= H * d


@FUZZ
@given(p=pointers(14), it=DTYPES, ot=DTYPES, st_=st.tuples(STRIDES, STRIDES, STRIDES, STRIDES), A=AXES, rot=ROTS, inter=FLAGS, tail=FLAGS, n=SIZES, N=SIZES,
       Hq=HEADS, Hkv=HEADS, d=ATTN, page=PAGES, pages=SIZES, mp=SIZES)
def test_fuzz_append(L, p, it, ot, st_, A, rot, inter, tail, n, N, Hq, Hkv, d, page, pages, mp):  # noqa: F811
    s = L.kda_kv_cache_append_rope(p[0], st_[0], p[1], st_[1], it, p[2], st_[2], p[3], ot, st_[3], p[4], A, p[5], p[6], rot, inter, p[7], p[8], p[9],
                                   p[10], p[11], p[12], p[13], n, N, Hq, Hkv, d, page, pages, mp, tail, None)
    _check(s, [it], [n, N, Hkv, pages, mp])
    if s in (OK, ERR_HIP):
        assert d in (64, 128) and page in (16, 32, 64) and 16 <= rot <= d and 1 <= A <= 8 and inter in (0, 1)


@FUZZ
@given(p=pointers(11), it=DTYPES, ot=DTYPES, qs=STRIDES, scale=SCALES, n=SIZES, N=SIZES, Hq=HEADS, Hkv=HEADS, d=ATTN, page=PAGES, pages=SIZES, mp=SIZES,
       tail=FLAGS, wsb=WSB)
def test_fuzz_chunk(L, p, it, ot, qs, scale, n, N, Hq, Hkv, d, page, pages, mp, tail, wsb):  # noqa: F811
    need = L.kda_attn_chunk_fwd_workspace_bytes(n, N, Hq, Hkv, d, page, mp, it) if pages > 0 else 0
    s = L.kda_attn_chunk_fwd(p[0], qs, it, p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], ot, p[9], n, N, Hq, Hkv, d, page, pages, mp, scale, tail,
                             p[10], wsb, None)
    _check(s, [it, ot], [n, N, Hq, Hkv, pages, mp])
    _accepted(s, wsb, need, scale)
    if s in (OK, ERR_HIP):
        assert d in (64, 128) and page in (16, 32, 64) and Hq % Hkv == 0 and tail in (0, 1) and qs >= Hq * d
