"""Rotary positions at the ends of 32 bits: the product of a 31-bit position and a 24-bit frequency has up to 55 bits, all of
which count.  The reference reduces the exact product by pi to 50 digits."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import gated_delta_rule_11_amd as kda
from tests.test_gpu_cache import i32

DEV = "cuda:0"
FAR = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, 2 ** 30 + 1, -2 ** 30 - 77, 2 ** 29 + 54321, 2 ** 29 - 1, 131071]


def pi():
    """16 atan(1/5) - 4 atan(1/239)."""
    def atan(n):
        term = total = Decimal(1) / n
        for k in range(3, 200, 2):
            term /= -n * n
            total += term / k
        return total
    return 16 * atan(5) - 4 * atan(239)


def units(pos, inv):
    """Cosine and sine of every product, [len(pos), len(inv)]."""
    getcontext().prec = 60
    turn = 2 * pi()
    r = [[float(Decimal(int(p)) * Decimal(float(f)) % turn) for f in inv] for p in pos]
    return np.cos(np.array(r)), np.sin(np.array(r))


def frequencies(n):
    """24 significant bits each, from one down."""
    return torch.from_numpy(np.nextafter(np.float32(1.0) / (1 + np.arange(n, dtype=np.float32) / 7), np.float32(0)))


def test_the_reference():
    assert float(pi()) == math.pi
    c, s = units([1, 3], [0.5, 1.0])
    assert np.abs(c - np.cos([[0.5, 1.0], [1.5, 3.0]])).max() < 1e-15 and np.abs(s - np.sin([[0.5, 1.0], [1.5, 3.0]])).max() < 1e-15


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_sines_and_cosines(interleaved):
    """(1, 0) turned is (cos, sin), each rounded once; the rest is the sums' 2^-48."""
    inv = frequencies(32)
    x = torch.zeros(len(FAR), 1, 64)
    a, b = (slice(0, 64, 2), slice(1, 64, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    x[..., a] = 1
    c, s = units(FAR, inv)
    for inverse in (False, True):
        y = kda.rope(x.to(DEV), i32(FAR), inv.to(DEV), interleaved=interleaved, inverse=inverse).cpu().double().numpy()[:, 0]
        for got, want in ((y[:, a], c), (y[:, b], -s if inverse else s)):
            assert (np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -48).all()


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 2])
def test_codes_are_those_of_the_exactly_turned_keys(new):
    """Keys that turn to either side of the border between two codes, by less than 2^-22 of it.  (Eight tokens of a
    sequence, and sixteen: wavefronts, and workgroups of a page.)"""
    pos, inv, d = FAR * new, frequencies(32), 128
    c, _ = units(pos, inv)
    border, scale = 17 / 32, 2.0 ** -8  # between 1/2 and 9/16, where the largest is 448 scale
    k = np.zeros((len(pos), 1, d), np.float32)
    k[:, 0, 100] = 1.75  # 448 * 2^-8, in a channel that does not turn
    want = np.zeros((len(pos), 32))
    for i in range(len(pos)):
        for j in range(32):
            if abs(c[i, j]) < 0.4:
                continue
            v = np.float32(border / c[i, j])
            for _ in range(4):  # the nearest fp32 number above or below
                if (abs(float(v) * c[i, j]) > border) == bool((i + j) % 2) and abs(abs(float(v) * c[i, j]) / border - 1) > 1e-11:
                    break
                v = np.nextafter(v, np.float32(math.copysign(9, v) if (i + j) % 2 else 0))
            y = float(v) * c[i, j]
            assert 1e-11 < abs(y / border - 1) < 2.0 ** -22
            k[i, 0, j] = v
            want[i, j] = 9 / 16 if y > border else 1 / 2
    n, P = len(pos), 16
    kc, vc = (torch.zeros(1, 1, *s, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for s in ((P, d), (d, P)))
    ks, vs = (torch.zeros(1, 1, device=DEV) for _ in range(2))
    key = torch.from_numpy(k).to(DEV)
    kda.kv_cache_append_rope(key, key, i32([0, n]), i32([0]), i32([[0]]), kc, vc, ks, vs, inv.to(DEV), positions=i32(pos))
    torch.cuda.synchronize()
    assert float(ks) == scale
    got = kc.view(torch.uint8).view(torch.float8_e4m3fn).float().cpu().double().numpy()[0, 0, :n, :32] * scale
    assert (got == want)[want != 0].all() and (want != 0).sum() > 16 * new


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [3, 16])
def test_keys_that_turn_beyond_fp32_count_as_infinite(n, dtype):
    """An eighth of a turn of two equal channels of 3e38: one becomes 4.2e38, the largest code and not in the scale.  The
    other, 3e38 (cos t - sin t) with t = pi/4 + 2.2e-8 in fp32, is -9.3e30: 448 times the scale is at least that, 2^95."""
    P, d, inv = 16, 64, torch.full((8,), math.pi / 4)
    key = torch.zeros(n, 1, d)
    key[1, 0, 0], key[1, 0, 8] = 3e38, 3e38
    key[:, 0, 40] = 1.75
    key = key.to(dtype).to(DEV)
    kc, vc = (torch.zeros(1, 1, *s, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for s in ((P, d), (d, P)))
    ks, vs = (torch.zeros(1, 1, device=DEV) for _ in range(2))
    pos = i32([1] * n)
    kda.kv_cache_append_rope(key, torch.zeros_like(key), i32([0, n]), i32([0]), i32([[0]]), kc, vc, ks, vs, inv.to(DEV), positions=pos)
    torch.cuda.synchronize()
    codes = kc.float()[0, 0]
    assert float(ks) == 2.0 ** 95 and float(codes[1, 8]) == 448 and -448 <= float(codes[1, 0]) < -224
    assert not codes[:n, 40].any()
