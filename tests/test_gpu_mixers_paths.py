"""The kernels' forms that small calls do not reach, each against the 64-bit references: several query heads
to a workgroup, tiles of 128 rows and sequences cut into segments at 128 channels, one long context
among many; and the three exact parts of the linear state.

Bounds as in the operators' own tests, and for what is fp32-accurate in linear attention (the state, its
gradient, dg; bf16 values enter as three parts, exact): a token's term is rounded for its weight (an
exponential, off by two half steps and its argument's rounding, and a product), then once for every
addition on its way: a chunk's tokens, and two per chunk for the carried state."""
import math

import pytest
import torch

import gated_delta_rule_11_amd as kda
from tests import _mixers as mx
from tests.test_gpu_cache import check_step
from tests.test_gpu_linear import dev, inputs
from tests.test_gpu_prompt import check
from tests.test_gpu_prompt import inputs as prompt_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


# ---- prompts

LENS = [300, 1, 517, 64, 200, 430, 3, 128]


def prompt_parts(n, Hq, Hkv, d):
    """Parts that the gradients' workspace holds for each group of heads (1: none beside D)."""
    floats = kda.attn_prompt_bwd_workspace_bytes(n, Hq, Hkv, d) // 4 - (n * Hq + 3) // 4 * 4
    return max(1, floats // (2 * n * Hkv * d))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv,d,repeat,parts", [(32, 16, 64, 5, 1), (64, 16, 64, 3, 2), (16, 8, 128, 10, 1)])
def test_gradients_with_several_heads_to_a_workgroup(Hq, Hkv, d, repeat, parts, dtype):
    lens = LENS * repeat
    assert prompt_parts(sum(lens), Hq, Hkv, d) == parts and Hq // Hkv // parts > 1
    check(f"{Hq} heads on {Hkv}", prompt_inputs(lens, Hq, Hkv, d, dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tiles_of_128_rows_with_128_channels(dtype):
    """Enough rows and heads that no wavefronts share keys (352 tiles and more), forward and backward."""
    lens = [700, 1, 480, 130, 90]
    assert -(-sum(lens) // 128) * 36 >= 352
    check("whole tiles", prompt_inputs(lens, 36, 6, 128, dtype))


# ---- linear attention

def state_terms(T, dtype):
    chunk = 64 if dtype == BF else 32
    return chunk + 2 * math.ceil(T / chunk) + 40


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [2, 3, 5])
def test_state_takes_every_bit_of_its_terms(T, dtype):
    """A few tokens: two exponentials of small arguments (four half steps, two for the arguments), two products
    and at most T + 4 additions to a term, where a dropped third part would cost up to 2^8 of them."""
    d = inputs(2, T, 2, 64, 64, dtype, rate=0.3)
    o, S = kda.linear_chunk_fwd(*(dev(d[x]) for x in ("q", "k", "v", "g")), S_in=dev(d["S"]))
    g = kda.linear_chunk_bwd(*(dev(d[x]) for x in ("q", "k", "v", "g", "do")), dS_out=dev(d["dS"]), S_in=dev(d["S"]))
    torch.cuda.synchronize()
    f = {x: mx.f64(d[x]) for x in d}
    _, rS, _, mS = mx.linear(f["q"], f["k"], f["v"], f["g"], f["S"], 1.0)
    want, mag = mx.linear_grad(f["q"], f["k"], f["v"], f["g"], f["S"], f["do"], f["dS"], 1.0)
    mx.close("S", S, rS, mS, F32, 0.0, 8 + T + 4)
    mx.close("dS_in", g["dS_in"], want["dS_in"], mag["dS_in"], F32, 0.0, 8 + T + 4)


def dg_magnitude(f, mag, T, dtype):
    """What dg's roundings are relative to: it is formed as the products <R, S> at the end of a block of four
    chunks, and the difference of sums q dq - k dk from the token to there."""
    block = 4 * (64 if dtype == BF else 32)
    x = (f["q"].abs() * mag["dq"]).sum(-1) + (f["k"].abs() * mag["dk"]).sum(-1)  # [B,T,H]
    out = torch.zeros_like(x)
    for a in range(0, T, block):
        b = min(a + block, T)
        # mag["dg"] of a token: sum |R| |S| across it, its own decay in both; at the block's end those of the next
        edge = mag["dg"][:, b] if b < T else (mag["edge"])
        out[:, a:b] = x[:, a:b].flip(1).cumsum(1).flip(1) + edge[:, None]
    return out


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("rate", [0.02, 0.5])
def test_cut_sequences_of_two_slices(rate, decay, dtype):
    """128 x 128 states, a sequence cut into segments, several blocks of dg: outputs, states and every gradient."""
    chunk = 64 if dtype == BF else 32
    T = 13 * chunk + 7
    d = inputs(1, T, 2, 128, 128, dtype, decay=decay, rate=rate)
    assert kda.linear_chunk_fwd_workspace_bytes(1, T, 2, 128, 128, dtype) > 0
    o, S = kda.linear_chunk_fwd(*(dev(d[x]) for x in ("q", "k", "v", "g")), S_in=dev(d["S"]), o_dtype=dtype)
    got = kda.linear_chunk_bwd(*(dev(d[x]) for x in ("q", "k", "v", "g", "do")), dS_out=dev(d["dS"]), S_in=dev(d["S"]), grad_dtype=dtype)
    torch.cuda.synchronize()
    f = {x: mx.f64(d[x]) for x in d}
    ro, rS, mo, mS = mx.linear(f["q"], f["k"], f["v"], f["g"], f["S"], 1.0)
    full = f["g"].expand(1, T, 2)
    want, mag = mx.linear_grad(f["q"], f["k"], f["v"], full, f["S"], f["do"], f["dS"], 1.0)
    n = state_terms(T, dtype)
    mx.close("S", S, rS, mS, F32, 0.0, n)
    mx.close("dS_in", got["dS_in"], want["dS_in"], mag["dS_in"], F32, 0.0, n)
    mx.close("o", o, ro, mo, dtype, 2.0, n + 128)
    for x in ("dq", "dk", "dv"):
        mx.close(x, got[x], want[x], mag[x], dtype, 2.0, n + 128)
    mag["edge"] = (mS * f["dS"].abs()).sum((-1, -2))
    near = dg_magnitude(f, mag, T, dtype)
    if decay == "head":
        want["dg"], near = want["dg"].sum((0, 1)), near.sum((0, 1))
    # dq and dk to their n + 128 roundings, and a dot product over 128 channels each
    mx.close("dg", got["dg"], want["dg"], near, F32, 1.0, n + 256)


def test_cut_sequences_same_bits_streams_and_graph():
    """Walks, scan and workspace of cut sequences: on another stream, captured and replayed between eager
    calls, twice at once; always the bits of the first call."""
    d = {x: dev(y) for x, y in inputs(1, 64 * 14 + 9, 4, 128, 128, BF).items()}
    assert kda.linear_chunk_fwd_workspace_bytes(1, 64 * 14 + 9, 4, 128, 128, BF) > 0

    def run(**kw):
        o, S = kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], S_in=d["S"], **kw)
        g = kda.linear_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], dS_out=d["dS"], S_in=d["S"], **kw)
        return (o, S, *g.values())

    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    both = [run(stream=s) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in both for a, b in zip(r, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for _ in range(3):
        for t in held:
            t.fill_(float("nan"))
        graph.replay()
        again = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)) and all(torch.equal(a, b) for a, b in zip(again, want))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_cut_sequences_write_their_outputs_only(dtype):
    from tests.test_gpu_mixers_guards import dirty, guarded
    T, dk, dv = 64 * 13, 16, 32
    d = {x: dev(y) for x, y in inputs(1, T, 2, dk, dv, dtype).items()}
    need = kda.linear_chunk_fwd_workspace_bytes(1, T, 2, dk, dv, dtype)
    assert need > 0
    want_o, want_S = kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], S_in=d["S"], o_dtype=dtype)
    o, ok_o = guarded(want_o.shape, dtype)
    S, ok_S = guarded(want_S.shape, F32)
    ws, ok_w = guarded((need // 4,), F32)
    ws.view(torch.uint8).copy_(dirty(need))
    kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], S_in=d["S"], o=o, S_out=S, workspace=ws)
    for ok in (ok_o, ok_S, ok_w):
        ok()
    assert torch.equal(o, want_o) and torch.equal(S, want_S)


# ---- cache

@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_long_context_among_many(dtype):
    """Enough sequences that no context is divided, one of them long."""
    ctx = [(29 * i) % 90 for i in range(130)]
    ctx[77] = 3001
    assert kda.attn_decode_step_workspace_bytes(130, 8, 8, 64, 64, 47) == 0
    check_step("one long", ctx, 8, 8, 64, 64, dtype)


def test_appended_and_attended_without_reading_the_cache_back():
    """Prompts appended, tokens appended and attended one at a time: equal to softmax over keys and values that
    were rounded on the host, from the tokens alone; an output of zeros would be off by far more than allowed."""
    Hq, Hkv, d, P, extra, prompts = 8, 2, 64, 16, 4, [70, 1, 133]
    gen = torch.Generator().manual_seed(3)
    full = [n + extra for n in prompts]
    rn = lambda h: [torch.randn(n, h, d, generator=gen).to(BF) for n in full]  # noqa: E731
    q, k, v = rn(Hq), rn(Hkv), rn(Hkv)
    pages, width = sum(-(-n // P) for n in full), max(-(-n // P) for n in full)
    order, table = torch.randperm(pages, generator=gen).tolist(), []
    for n in full:
        m = -(-n // P)
        table.append(order[:m] + [0] * (width - m))
        order = order[m:]
    code = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)  # noqa: E731
    c = {"kc": code(pages, Hkv, P, d), "vc": code(pages, Hkv, d, P), "ks": torch.zeros(pages, Hkv, device=DEV),
         "vs": torch.zeros(pages, Hkv, device=DEV)}
    ref = mx.Cache(c["kc"], c["vc"], c["ks"], c["vs"])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731

    def append(rows, held):
        cu = [0]
        for x in rows[0]:
            cu.append(cu[-1] + len(x))
        kk, vv = (torch.cat(x) for x in rows)
        kda.kv_cache_append(kk.to(DEV), vv.to(DEV), i32(cu), i32(held), i32(table), c["kc"], c["vc"], c["ks"], c["vs"])
        ref.append(mx.f64(kk), mx.f64(vv), cu, held, table)

    append([[x[:n] for x, n in zip(y, prompts)] for y in (k, v)], [0, 0, 0])
    for t in range(extra):
        held = [n + t for n in prompts]
        append([[x[n:n + 1] for x, n in zip(y, held)] for y in (k, v)], held)
        now = torch.stack([x[n] for x, n in zip(q, held)])
        ctx = [n + 1 for n in held]
        o, _ = kda.attn_decode_step(now.to(DEV), c["kc"], c["vc"], c["ks"], c["vs"], i32(table), i32(ctx), o_dtype=BF)
        torch.cuda.synchronize()
        ro, _, mag = ref.attend(mx.f64(now), ctx, table, d ** -0.5)
        mx.close(f"token {t}", o, ro, mag, BF, 2.0, d + max(ctx) + 184)
        assert float(((mx.f64(o) - ro).norm() / ro.norm())) < 2 ** -6
