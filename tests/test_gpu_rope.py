"""Rotary positions on the GPU against products of complex numbers in 64 bits.

Bound of an element, in units of |x_a cos| + |x_b sin|: the sine's and cosine's rounding to fp32, one product's and the
sum's, 2^-24 each (the first two never meet in one term), and the output's own rounding."""
import math

import pytest
import torch

import gated_delta_rule_11_amd as kda
from tests import _mixers as mx
from tests import _serve as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def check(label, got, x, pos, inv, axes=None, interleaved=False, sign=1):
    want, mag = sv.turned(mx.f64(x), pos, inv, axes, interleaved, sign)
    mx.close(label, got, want, mag, got.dtype, 1.0, 3.0)


def case(n, H, d, rot, A, dtype, seed=0, far=5000, lo=0):
    gen = torch.Generator().manual_seed(seed + n * 31 + H * 7 + d + rot)
    x = torch.randn(n, H, d, generator=gen).to(dtype)
    pos = torch.randint(lo, far, (n, A) if A > 1 else (n,), generator=gen, dtype=torch.int32)
    axes = torch.randint(0, A, (rot // 2,), generator=gen, dtype=torch.int32) if A > 1 else None
    return x, pos, sv.frequencies(rot // 2), axes


def dev(t):
    return None if t is None else t.to(DEV)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(16, 16), (32, 16), (48, 48), (64, 64), (64, 32), (80, 48), (128, 128), (128, 64), (192, 176),
                                   (256, 256)])
def test_forward_and_backward(d, rot, interleaved, dtype):
    for n, H, A in ((1, 1, 1), (1, 40, 3), (7, 3, 2), (133, 5, 1), (2, 9, 8)):
        x, pos, inv, axes = case(n, H, d, rot, A, dtype)
        args = dev(pos), dev(inv)
        for inverse in (False, True):
            y = kda.rope(dev(x), *args, axes=dev(axes), interleaved=interleaved, inverse=inverse)
            torch.cuda.synchronize()
            assert y.dtype == dtype
            check((n, H, A, inverse), y, x, pos, inv, axes, interleaved, -1 if inverse else 1)


def test_many_rows_and_every_split_of_the_heads():
    for n, H in ((9000, 2), (4000, 40), (1000, 33), (300, 41), (20, 200), (1, 300)):
        x, pos, inv, _ = case(n, H, 64, 64, 1, BF)
        y = kda.rope(dev(x), dev(pos), dev(inv))
        torch.cuda.synchronize()
        check((n, H), y, x, pos, inv)


@pytest.mark.parametrize("out", [BF, F32])
def test_types_mix(out):
    x, pos, inv, _ = case(11, 3, 64, 64, 1, F32 if out == BF else BF)
    y = kda.rope(dev(x), dev(pos), dev(inv), out_dtype=out)
    torch.cuda.synchronize()
    assert y.dtype == out
    check("mixed", y, x, pos, inv)


def test_far_and_negative_positions():
    """A frequency of one at the ends of 32 bits: an angle's fraction needs the 64 bits it is reduced in."""
    x, _, inv, _ = case(6, 2, 128, 128, 1, F32)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, -1, 0, 131071], dtype=torch.int32)
    y = kda.rope(dev(x), dev(pos), dev(inv))
    torch.cuda.synchronize()
    # the definition's own angle (53 bits of 2^31) is off by 2^-22 where 24-bit frequencies meet 31-bit positions
    want, mag = sv.turned(mx.f64(x), pos, inv)
    both = mx.f64(x).abs() + torch.cat([mx.f64(x)[..., 64:], mx.f64(x)[..., :64]], -1).abs()
    mx.close("far", y, want, both, F32, 1.0, 3.0 + 2 * 2.0 ** (24 - 22))
    assert torch.equal(y[4].cpu(), x[4])


def test_position_zero_and_channels_that_do_not_turn_are_copies():
    x, _, inv, _ = case(5, 3, 128, 48, 1, BF)
    pos = torch.zeros(5, dtype=torch.int32)
    assert torch.equal(kda.rope(dev(x), dev(pos), dev(inv)).cpu(), x)
    pos += 77
    assert torch.equal(kda.rope(dev(x), dev(pos), dev(inv))[..., 48:].cpu(), x[..., 48:])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_views_and_in_place(dtype):
    """Rows of a projection's output: queries and keys turned where they lie, what lies between them kept."""
    n, H, more, d = 37, 6, 3, 64
    whole, pos, inv, _ = case(n, H + more, d, d, 1, dtype)
    buf = dev(whole)
    y = kda.rope(buf[:, 1:1 + H], dev(pos), dev(inv))
    torch.cuda.synchronize()
    assert torch.equal(buf.cpu(), whole)
    check("view", y, whole[:, 1:1 + H], pos, inv)
    out = torch.full((n, H + 2, d), 7.0, dtype=dtype, device=DEV)
    assert kda.rope(buf[:, 1:1 + H], dev(pos), dev(inv), out=out[:, 1:1 + H]).data_ptr() == out[:, 1:].data_ptr()
    torch.cuda.synchronize()
    assert torch.equal(out[:, 1:1 + H], y) and bool((out[:, 0] == 7).all()) and bool((out[:, 1 + H:] == 7).all())
    kda.rope(buf[:, 1:1 + H], dev(pos), dev(inv), out=buf[:, 1:1 + H])
    torch.cuda.synchronize()
    assert torch.equal(buf[:, 1:1 + H], y)
    assert torch.equal(buf[:, 0].cpu(), whole[:, 0]) and torch.equal(buf[:, 1 + H:].cpu(), whole[:, 1 + H:])
    kda.rope(buf[:, 1:1 + H], dev(pos), dev(inv), out=buf[:, 1:1 + H], inverse=True)
    torch.cuda.synchronize()
    back, mag = mx.f64(whole[:, 1:1 + H]), sv.turned(mx.f64(whole[:, 1:1 + H]), pos, inv)[1]
    other = torch.cat([mag[..., d // 2:], mag[..., :d // 2]], -1)
    mx.close("there and back", buf[:, 1:1 + H], back, mag + other, dtype, 2.0, 8.0)


def test_views_that_alternate_are_taken_and_views_that_meet_refused():
    buf = torch.randn(9, 6, 64, device=DEV)
    pos, inv = torch.arange(9, dtype=torch.int32, device=DEV), dev(sv.frequencies(32))
    y = kda.rope(buf[:, :3], pos, inv, out=buf[:, 3:])
    torch.cuda.synchronize()
    assert torch.equal(y, kda.rope(buf[:, :3], pos, inv))
    with pytest.raises(kda.KDAError):
        kda.rope(buf[:, :3], pos, inv, out=buf[:, 2:5])
    with pytest.raises(kda.KDAError):
        kda.rope(buf[1:], pos[1:], inv, out=buf[:-1])


def test_gradient_is_the_formulas():
    """<dy, rope(x)> = <rope(dy, inverse), x>, and autograd of the plain form."""
    x, pos, inv, axes = case(17, 3, 64, 48, 3, F32)
    dy = torch.randn(17, 3, 64)
    dx = kda.rope(dev(dy), dev(pos), dev(inv), axes=dev(axes), interleaved=True, inverse=True)
    y = kda.rope(dev(x), dev(pos), dev(inv), axes=dev(axes), interleaved=True)
    torch.cuda.synchronize()
    leaf = x.double().requires_grad_()
    (want,) = torch.autograd.grad(sv.turned(leaf, pos, inv, axes, True)[0], leaf, dy.double())
    mag = sv.turned(dy.double(), pos, inv, axes, True, -1)[1]
    mx.close("dx", dx, want, mag, F32, 1.0, 3.0)
    # the difference quotient of sum(dy * rope(x)) along one direction, exact for a linear map
    z = torch.randn(17, 3, 64)
    z1 = kda.rope(dev(x + z), dev(pos), dev(inv), axes=dev(axes), interleaved=True)
    diff = (mx.f64(dy) * (mx.f64(z1) - mx.f64(y))).sum()
    # x + z rounds once, each turned element four times, each at most 2^-24 of the magnitudes
    slack = 5 * 2.0 ** -24 * (mx.f64(dy).abs() * (sv.turned(mx.f64(x + z), pos, inv, axes, True)[1] + sv.turned(mx.f64(x), pos, inv, axes, True)[1])).sum()
    slack += 5 * 2.0 ** -24 * (mag * mx.f64(z).abs()).sum()
    assert abs(float(diff - (mx.f64(dx) * mx.f64(z)).sum())) <= float(slack)


def test_nan_and_infinity_stay_in_their_pair():
    x, pos, inv, _ = case(4, 2, 64, 64, 1, F32)
    pos += 1
    clean = kda.rope(dev(x), dev(pos), dev(inv)).cpu()
    x[1, 0, 5], x[2, 1, 40] = math.nan, math.inf
    y = kda.rope(dev(x), dev(pos), dev(inv)).cpu()
    bad = torch.zeros(4, 2, 64, dtype=torch.bool)
    bad[1, 0, 5] = bad[1, 0, 37] = bad[2, 1, 8] = bad[2, 1, 40] = True
    assert torch.equal(y[~bad], clean[~bad]) and not y[bad].isfinite().any()


def test_axes_out_of_range_are_clamped():
    x, pos, inv, _ = case(5, 2, 64, 32, 3, F32)
    axes = torch.tensor([-5, 7, 0, 1, 2, 2 ** 31 - 1, -2 ** 31, 1] * 2, dtype=torch.int32)
    y = kda.rope(dev(x), dev(pos), dev(inv), axes=dev(axes))
    torch.cuda.synchronize()
    check("axes", y, x, pos, inv, axes)


def test_no_rows_and_no_writes_outside():
    inv = dev(sv.frequencies(32))
    assert kda.rope(torch.zeros(0, 3, 64, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV), inv).shape == (0, 3, 64)
    for n, H in ((1, 1), (3, 5), (65, 2)):
        buf = torch.full((n * H * 64 + 8192,), 7.0, device=DEV)
        out = buf[4096:4096 + n * H * 64].view(n, H, 64)
        kda.rope(torch.randn(n, H, 64, device=DEV), torch.arange(n, dtype=torch.int32, device=DEV), inv, out=out)
        torch.cuda.synchronize()
        assert bool((buf[:4096] == 7).all()) and bool((buf[4096 + n * H * 64:] == 7).all())


def test_streams_and_replays():
    x, pos, inv, _ = case(700, 8, 128, 128, 1, BF)
    x, pos, inv = dev(x), dev(pos), dev(inv)
    want = kda.rope(x, pos, inv)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kda.rope(x, pos, inv, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    out, g = torch.zeros_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.rope(x, pos, inv, out=out)
    for _ in range(3):
        out.zero_()
        x.mul_(-1)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, kda.rope(x, pos, inv))


def test_refused_by_the_binding():
    x = torch.zeros(4, 2, 64, device=DEV)
    pos, inv = torch.zeros(4, dtype=torch.int32, device=DEV), dev(sv.frequencies(32))
    ok = dict(x=x, positions=pos, inv_freq=inv)
    kda.rope(**ok)
    for bad in (dict(x=x[0]), dict(x=x.transpose(0, 1)), dict(x=x.half()), dict(positions=pos.long()), dict(positions=pos[:3]),
                dict(positions=None), dict(inv_freq=inv.double()), dict(inv_freq=inv[:12].contiguous()),
                dict(inv_freq=dev(sv.frequencies(40))), dict(inv_freq=inv[:0]), dict(axes=torch.zeros(31, dtype=torch.int32, device=DEV)),
                dict(axes=torch.zeros(32, device=DEV)), dict(out=torch.zeros(4, 2, 32, device=DEV)), dict(out_dtype=torch.float16),
                dict(x=torch.zeros(4, 2, 24, device=DEV)), dict(x=torch.zeros(4, 2, 272, device=DEV)), dict(out=x[:, :, ::1].cpu()),
                dict(positions=pos.cpu()), dict(x=torch.zeros(4, 130, device=DEV)[:, :128].view(4, 2, 64)),
                dict(positions=torch.zeros(4, 9, dtype=torch.int32, device=DEV))):
        with pytest.raises(kda.KDAError):
            kda.rope(**{**ok, **bad})
