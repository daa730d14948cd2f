"""Attention of a chunk over the 8-bit cache where a bound in units of the terms says little: values whose sums leave fp32."""
import math

import pytest
import torch

import gated_delta_rule_11_amd as kda
from tests import _serve as sv
from tests.test_gpu_cache import filled, i32
from tests.test_gpu_cache_chunk import compare, more, run  # noqa: F401  (more: every test runs with both tables)

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# rows of a tile, two heads of a group: up to 16, up to 32, more, several tiles
SHAPES = [([1], [3000]), ([12, 1], [700, 2000]), ([40], [2900]), ([200, 3], [5000, 600])]


def large(new, ctx, P, d):
    """Pages of 2^127 (256 * 2^119) and their tokens' places."""
    c, t = filled(ctx, 1, P, d)
    c["vs"].fill_(2.0 ** 119)
    c["vc"].view(torch.uint8).fill_(0x78)
    return c, t, c["vc"].view(torch.uint8)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P,d", [(16, 64), (64, 128)])
def test_sums_beyond_fp32(P, d, dtype):
    """Means of finite values are finite, however many of them there are: equal ones, ones that cancel, and small
    values of a channel whose large ones are zero."""
    for new, ctx in SHAPES:
        c, t, code = large(new, ctx, P, d)
        q = torch.randn(sum(new), 2, d, generator=torch.Generator().manual_seed(3)).to(dtype)
        for scale in (0.0, d ** -0.5):
            got = run(c, t, q, new, ctx, scale=scale)
            assert bool(got[0].isfinite().all()), (new, ctx, scale)
            compare(f"{new} {ctx} {scale}", got, c, t, q, new, ctx, scale)
        for i, x in enumerate(ctx):
            for p in t[i][x // P // 2:]:  # the later half turned
                code[p, 0, 1::3] = 0xF8
            for p in t[i]:
                code[p, 0, 2] = 0
            last = t[i][x // P // 3]
            c["vs"][last, 0] = 0.5
        got = run(c, t, q, new, ctx)
        compare(f"{new} {ctx} signs", got, c, t, q, new, ctx)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_value_beyond_fp32_among_sums_beyond_fp32(dtype):
    """It stays one that is not finite, in its channel alone."""
    for new, ctx in SHAPES:
        c, t, code = large(new, ctx, 16, 64)
        page = t[0][1]
        c["vs"][page, 0] = 2.0 ** 120
        code[page, 0] = 0x70  # 2^127
        code[page, 0, 5, 3] = 0x7E  # 448 * 2^120
        o, _ = run(c, t, torch.randn(sum(new), 2, 64).to(dtype), new, ctx)
        torch.cuda.synchronize()
        assert not o[:new[0], :, 5].isfinite().any()
        o[:new[0], :, 5] = 2.0 ** 127
        slack = 2.0 ** -7 if dtype == BF else 2.0 ** -24 * 3 * (64 + ctx[0] + 200)
        assert bool(((o.double() / 2.0 ** 127 - 1).abs() <= slack).all())
