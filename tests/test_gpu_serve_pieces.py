"""A prompt in one piece or in several through the turned append and attention over the cache, row by row against the softmax
over the codes that the cache holds at each call, and both runs against the definition of the unrounded prompt.

Against the unrounded prompt each value of the cache is off by at most 2^-4 of itself at a rounding, and a sum of values
that are off either way by less: the norm of the error stays below 2^-4 of the terms' magnitude, of which a rotation left
out, or of the queries alone, scores that do not matter or zeros are more than twice as far off (the first test)."""
import pytest
import torch

import gated_delta_rule_11_amd as kda
from tests import _mixers as mx
from tests import _serve as sv
from tests.test_gpu_cache import empty_cache, i32

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
HQ, HKV, D, P, ROWS = 4, 2, 64, 16, 300
SCALE, BOUND = D ** -0.5, 2.0 ** -4
PIECES = ([ROWS], [100, 1, 150, 49], [5] * 60)
TABLE = [list(range(19))]


def inputs(dtype=F32):
    return torch.randn(ROWS, HQ + 2 * HKV, D, generator=torch.Generator().manual_seed(1)).to(dtype)


def unrounded(x, turn_q=True, turn_k=True, factor=1.0):
    q, k, v = mx.f64(x).split([HQ, HKV, HKV], 1)
    turn = lambda y, do: sv.turned(y, torch.arange(ROWS), sv.frequencies(D // 2))[0] if do else y  # noqa: E731
    out, mag = mx.prompt(turn(q, turn_q), turn(k, turn_k), v, [0, ROWS], SCALE * factor)
    return out["o"], mag["o"]


def distance(o, want, mag):
    return float((mx.f64(o) - want).norm() / mag.norm())


def attend(cache, q, done, new):
    """The definition over the cache's codes."""
    return sv.chunk(cache, mx.f64(q), [0, new], [done + new], TABLE, SCALE)


def test_what_the_bound_tells_apart():
    x = inputs()
    want, mag = unrounded(x)
    wrong = dict(zeros=0 * want, neither=unrounded(x, False, False)[0], queries=unrounded(x, True, False)[0],
                 keys=unrounded(x, False, True)[0], uniform=unrounded(x, factor=0.0)[0], later=want.roll(1, 0))
    assert all(distance(o, want, mag) > 2 * BOUND for o in wrong.values())
    q, k, v = mx.f64(x).split([HQ, HKV, HKV], 1)
    for pieces in PIECES[:2]:
        c = empty_cache(19, HKV, P, D)
        ref, done, rows = mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"]), 0, []
        for m in pieces:
            at, these = torch.arange(done, done + m), slice(done, done + m)
            tq, tk = (sv.turned(y[these], at, sv.frequencies(D // 2))[0] for y in (q, k))
            ref.append(tk, v[these], [0, m], [done], TABLE)
            rows.append(attend(ref, tq, done, m)[0])
            done += m
        assert distance(torch.cat(rows), want, mag) < BOUND


@pytest.mark.gpu
@pytest.mark.parametrize("room", [0, 4500])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_pieces_and_the_whole_prompt(dtype, room):
    x, inv = inputs(dtype), sv.frequencies(D // 2).to(DEV)
    table = i32([TABLE[0] + [-1] * max(0, room // P - len(TABLE[0]))])
    want, mag = unrounded(x)
    for pieces in PIECES:
        c = {a: b.to(DEV) for a, b in empty_cache(19, HKV, P, D).items()}
        done, rows = 0, []
        for m in pieces:
            q, k, v = x[done:done + m].to(DEV).split([HQ, HKV, HKV], 1)
            q = kda.kv_cache_append_rope(k, v, i32([0, m]), i32([done]), table, c["kc"], c["vc"], c["ks"], c["vs"], inv, q=q)
            o, lse = kda.attn_chunk_fwd(q, i32([0, m]), c["kc"], c["vc"], c["ks"], c["vs"], table, i32([done + m]), o_dtype=dtype, want_lse=True)
            torch.cuda.synchronize()
            ro, rl, rm = attend(mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"]), q, done, m)
            terms = 3 * D + 3 * (done + m) + 4 * 48 + 64
            mx.close(f"{done}+{m} o", o, ro, rm, dtype, 2.0, terms)
            mx.close(f"{done}+{m} lse", lse, rl, torch.full_like(rl, 8.0), F32, 1.0, terms)
            rows.append(o)
            done += m
        assert distance(torch.cat(rows), want, mag) < BOUND
