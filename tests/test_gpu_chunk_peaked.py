"""Attention of a chunk over the 8-bit cache where one token has all of a row's weight.

Queries and keys are small whole numbers: scores are exact, and the next lower one is e^-64 of the highest.  A row's
output is then the highest token's value (the mean of several that share the score), off by the rounding of its
probability and of the output alone, 2^-8 each in bf16; in fp32 by the three parts of its probability, the sum of the
tokens', the division: 16 roundings of 2^-24.  What is wrong by more than that, zeros or another token's value among them,
is outside the bound, which the first test looks at without a GPU."""
import math

import pytest
import torch

import gated_delta_rule_11_amd as kda
from tests import _mixers as mx
from tests import _serve as sv
from tests.test_gpu_cache import i32, table_of

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
F8 = torch.float8_e4m3fn
SCALE = 64.0

# (new tokens, tokens held with them): single and drafted tokens, up to 32 rows of a tile, more, several tiles
SHAPES = [([1, 5, 1], [900, 333, 64]), ([12, 16], [700, 129]), ([3, 90], [700, 400]), ([200], [1500])]


def ends(new):
    return [0, *torch.tensor(new).cumsum(0).tolist()]


def peaked(new, ctx, P, d, dtype, seed=0):
    """A cache (on the CPU), its table, queries, and the definition's outputs."""
    gen = torch.Generator().manual_seed(seed + sum(ctx) + P)
    pages = sum(-(-n // P) for n in ctx) + 2
    whole = lambda *s: torch.randint(-3, 4, s, generator=gen).float()  # noqa: E731
    c = {"kc": whole(pages, 1, P, d).to(F8), "vc": torch.randn(pages, 1, d, P, generator=gen).to(F8), "ks": torch.ones(pages, 1),
         "vs": torch.exp2(torch.randint(-3, 3, (pages, 1), generator=gen).float())}
    t = table_of(ctx, P, pages, seed)
    q = whole(sum(new), 2, d).to(dtype)
    return c, t, q, sv.chunk(mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"]), mx.f64(q), ends(new), ctx, t, SCALE)


def close(label, got, want, mag, dtype):
    mx.close(label, got, want, mag, dtype, 2.0, 16.0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_wrong_outputs_are_outside_the_bound(dtype):
    slack = 2 * mx.U[dtype] + 16 * 2.0 ** -24
    for new, ctx in SHAPES:
        _, _, _, (o, lse, mag) = peaked(new, ctx, 16, 64, dtype)
        close("right", o, o, mag, dtype)
        for wrong in (torch.zeros_like(o), -o, 0.5 * o, o.roll(1, 0) if sum(new) > 1 else o.flip(1), o * (1 + 2 * slack)):
            off = ~((wrong - o).abs() <= slack * torch.maximum(mag, o.abs()))
            assert float(off.double().mean()) > 0.5
            with pytest.raises(AssertionError):
                close("wrong", wrong, o, mag, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("room", [0, 4500])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P,d", [(16, 64), (32, 128), (64, 64)])
def test_one_token_has_the_weight(P, d, dtype, room):
    """Wherever among the steps it lies, with the table as it is and with one that has room for more."""
    for seed, (new, ctx) in enumerate(SHAPES):
        c, t, q, (o, lse, mag) = peaked(new, ctx, P, d, dtype, seed)
        t = [x + [-1] * max(0, room // P - len(x)) for x in t]
        got = kda.attn_chunk_fwd(q.to(DEV), i32(ends(new)), *(c[x].to(DEV) for x in ("kc", "vc", "ks", "vs")), i32(t), i32(ctx), scale=SCALE,
                                 o_dtype=dtype, want_lse=True)
        torch.cuda.synchronize()
        close(f"{new} {ctx} o", got[0], o, mag, dtype)
        # the scale in base two (the constant, the product), times the score, the reference 8 above it, the sum with the
        # logarithm, back (the constant, the product): seven roundings
        assert not bool(lse.isinf().any())
        mx.close(f"{new} {ctx} lse", got[1], lse, lse.abs() + 8 * math.log(2), F32, 1.0, 6.0)
