"""Causal attention over packed prompts on the GPU against softmax in 64 bits, one sequence at a time.

Bounds, derived from the arithmetic.  With bf16 elements the probabilities are rounded once (2^-8 of
each term p v) and the output once.  In the backward, dv: p once, the sum once; dq and dk: dS once
and the sum once, and D, from the rounded output, moves by 2^-8 of sum |do o| (a term of the
magnitude).  In fp32: a sum over channels, over keys, and the exponential of a score x, whose
relative error is |x| 2^-24 for a few units; scores here stay below 40."""
import math

import pytest
import torch

import gated_delta_rule_11_amd as kda
from tests import _mixers as mx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def inputs(lens, Hq, Hkv, d, dtype, seed=0, extra=0):
    gen = torch.Generator().manual_seed(seed + sum(lens))
    n = sum(lens) + extra
    rn = lambda *s: torch.randn(*s, generator=gen).to(dtype)  # noqa: E731
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return {"q": rn(n, Hq, d), "k": rn(n, Hkv, d), "v": rn(n, Hkv, d), "do": rn(n, Hq, d), "cu": cu}


def on(d):
    return {x: (y.to(DEV) if x != "cu" else torch.tensor(y, dtype=torch.int32, device=DEV)) for x, y in d.items()}


def check(label, d, scale=None, backward=True):
    dtype = d["q"].dtype
    g = on(d)
    hd = d["q"].shape[-1]
    sc = hd ** -0.5 if scale is None else scale
    want, mag = mx.prompt(*(mx.f64(d[x]) for x in ("q", "k", "v")), d["cu"], sc, mx.f64(d["do"]) if backward else None)
    n, longest = d["cu"][-1], max([b - a for a, b in zip(d["cu"], d["cu"][1:])] or [0])
    terms = hd + longest + 3 * 40 + 32
    o, lse = kda.attn_prompt_fwd(g["q"], g["k"], g["v"], g["cu"], scale=scale, o_dtype=dtype)
    torch.cuda.synchronize()
    mx.close(label + " o", o[:n], want["o"][:n], mag["o"][:n], dtype, 2.0, terms)
    mx.close(label + " lse", lse[:n], want["lse"][:n], torch.full_like(want["lse"][:n], 8.0), F32, 1.0, terms)
    assert not o[n:].any() and not lse[n:].any()
    if backward:
        got = kda.attn_prompt_bwd(g["q"], g["k"], g["v"], g["cu"], o, lse, g["do"], scale=scale, grad_dtype=dtype)
        torch.cuda.synchronize()
        for x in ("dq", "dk", "dv"):
            mx.close(f"{label} {x}", got[x][:n], want[x][:n], mag[x][:n], dtype, 2.5, 3 * terms)
            assert not got[x][n:].any()
    return o, lse


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[1], [2], [31], [33], [64], [65], [127], [128], [129], [200], [1, 1, 1], [5, 1, 40, 3, 90],
                                  [0, 7, 0, 0, 130, 0], [1] * 140, [257, 64]])
def test_lengths(lens, dtype):
    check(f"lens={lens[:6]}", inputs(lens, 4, 2, 64, dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (4, 1), (6, 2), (10, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_heads(Hq, Hkv, d, dtype):
    check(f"heads={Hq}/{Hkv} d={d}", inputs([70, 3, 101], Hq, Hkv, d, dtype))


@pytest.mark.parametrize("scale", [0.3, -0.2, 0.0])
def test_scales(scale):
    check(f"scale={scale}", inputs([90, 40], 2, 1, 64, F32), scale=scale)
    check(f"scale={scale}", inputs([90, 40], 2, 1, 64, BF), scale=scale)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_behind_the_last_sequence(dtype):
    """They are not read (NaN there stays there) and not written."""
    d = inputs([50, 61], 4, 2, 64, dtype, extra=100)
    for x in ("q", "k", "v", "do"):
        d[x][111:] = math.nan
    check("tail", d)
    g = on(d)
    o = torch.full((211, 4, 64), 7.0, dtype=dtype, device=DEV)
    lse = torch.full((211, 4), 7.0, device=DEV)
    kda.attn_prompt_fwd(g["q"], g["k"], g["v"], g["cu"], o=o, lse=lse)
    torch.cuda.synchronize()
    assert bool((o[111:] == 7.0).all()) and bool((lse[111:] == 7.0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_non_finite_values_stay_in_their_sequence_and_later_rows(dtype):
    """A NaN or infinity in one sequence's row reaches that row and the later ones of the sequence only."""
    d = inputs([30, 45, 20], 2, 1, 64, dtype)
    clean = on(d)
    want, _ = kda.attn_prompt_fwd(clean["q"], clean["k"], clean["v"], clean["cu"], o_dtype=dtype)
    for name, val in (("v", math.nan), ("v", math.inf), ("k", math.nan)):
        e = {x: (y.clone() if x != "cu" else y) for x, y in d.items()}
        e[name][50, :, 3] = val
        g = on(e)
        o, lse = kda.attn_prompt_fwd(g["q"], g["k"], g["v"], g["cu"], o_dtype=dtype)
        torch.cuda.synchronize()
        same = [*range(0, 50), *range(75, 95)]
        assert torch.equal(o[same], want[same]), name
        assert not torch.isfinite(o[50:75, :, 3]).any(), name


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv", [(6, 2), (96, 8)])
def test_few_and_many_workgroups(Hq, Hkv, dtype):
    """Launches that fill the device and such that do not divide the keys differently."""
    d = inputs([190, 260, 1, 69], Hq, Hkv, 64, dtype, seed=5)
    o, _ = check(f"{Hq}", d, backward=False)
    for name, row, val in (("v", 300, math.nan), ("v", 191, math.inf), ("v", 449, -math.inf), ("k", 333, math.nan)):
        e = {x: (y.clone() if x != "cu" else y) for x, y in d.items()}
        e[name][row, :, 3] = val
        g = on(e)
        got, _ = kda.attn_prompt_fwd(g["q"], g["k"], g["v"], g["cu"], o_dtype=dtype)
        torch.cuda.synchronize()
        same = [*range(0, row), *range(450, 520)]
        assert torch.equal(got[same], o[same]), (name, row)
        assert not torch.isfinite(got[row:450, :, 3]).any(), (name, row)
        if name == "v":
            assert torch.equal(got[..., 4:], o[..., 4:]), (name, row)


@pytest.mark.parametrize("Hq", [2, 96])
def test_large_scores_over_many_keys(Hq):
    """Maxima that differ widely between the parts of a row's keys."""
    d = inputs([500], Hq, Hq // 2, 64, F32)
    d["q"] *= torch.linspace(0.1, 12, 500)[:, None, None]
    d["k"] *= torch.linspace(12, 0.1, 500)[:, None, None] ** 0.5
    g = on(d)
    want, mag = mx.prompt(*(mx.f64(d[x]) for x in ("q", "k", "v")), d["cu"], 0.5)
    o, lse = kda.attn_prompt_fwd(g["q"], g["k"], g["v"], g["cu"], scale=0.5)
    torch.cuda.synchronize()
    # a score x is off by |x| 2^-24 for each of its roundings, and p by as much relative to itself
    big = float((d["q"].abs().max() * d["k"].abs().max()) * 0.5 * 64)
    mx.close("o", o, want["o"], mag["o"], F32, 2.0, 16 * big)
    mx.close("lse", lse, want["lse"], want["lse"].abs() + 8, F32, 1.0, 256)


def test_large_scores():
    """Scores in the hundreds: the running maximum moves often, and far."""
    d = inputs([150], 2, 1, 64, F32)
    d["q"] *= torch.linspace(0.1, 12, 150)[:, None, None]
    d["k"] *= torch.linspace(12, 0.1, 150)[:, None, None] ** 0.5
    g = on(d)
    want, mag = mx.prompt(*(mx.f64(d[x]) for x in ("q", "k", "v")), d["cu"], 0.5)
    o, lse = kda.attn_prompt_fwd(g["q"], g["k"], g["v"], g["cu"], scale=0.5)
    torch.cuda.synchronize()
    # a score x is off by |x| 2^-24 for each of its roundings, and p by as much relative to itself
    big = float((d["q"].abs().max() * d["k"].abs().max()) * 0.5 * 64)
    mx.close("o", o, want["o"], mag["o"], F32, 2.0, 16 * big)
    mx.close("lse", lse, want["lse"], want["lse"].abs() + 8, F32, 1.0, 256)


@pytest.mark.parametrize("o_dtype,grad_dtype", [(F32, F32), (BF, F32), (F32, BF)])
def test_output_types(o_dtype, grad_dtype):
    d = inputs([80, 50], 4, 2, 128, BF)
    g = on(d)
    o, lse = kda.attn_prompt_fwd(g["q"], g["k"], g["v"], g["cu"], o_dtype=o_dtype)
    got = kda.attn_prompt_bwd(g["q"], g["k"], g["v"], g["cu"], o, lse, g["do"], grad_dtype=grad_dtype)
    torch.cuda.synchronize()
    want, mag = mx.prompt(*(mx.f64(d[x]) for x in ("q", "k", "v")), d["cu"], 128 ** -0.5, mx.f64(d["do"]))
    assert o.dtype == o_dtype and got["dq"].dtype == grad_dtype
    mx.close("o", o, want["o"], mag["o"], BF, 2.0, 400)
    for x in ("dq", "dk", "dv"):
        mx.close(x, got[x], want[x], mag[x], BF, 2.5, 1200)


def test_gradient_against_differences():
    d = inputs([20, 37], 4, 2, 64, F32)
    f = {x: (mx.f64(d[x]) if x != "cu" else d[x]) for x in d}
    g = on(d)
    o, lse = kda.attn_prompt_fwd(g["q"], g["k"], g["v"], g["cu"])
    got = kda.attn_prompt_bwd(g["q"], g["k"], g["v"], g["cu"], o, lse, g["do"])
    torch.cuda.synchronize()
    loss = lambda q, k, v: (mx.prompt(q, k, v, d["cu"], 64 ** -0.5)[0]["o"] * f["do"]).sum()  # noqa: E731
    gen = torch.Generator().manual_seed(5)
    for name in ("q", "k", "v"):
        u = torch.randn(f[name].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        at = lambda s: loss(*[f[x] + s * h * u if x == name else f[x] for x in ("q", "k", "v")])  # noqa: E731,B023
        diff = (at(1) - at(-1)) / (2 * h)
        dot = (mx.f64(got["d" + name]) * u).sum()
        assert abs(dot - diff) <= 1e-4 * (mx.f64(got["d" + name]).norm() * u.norm()), (name, float(dot), float(diff))


def test_same_bits_streams_and_graph():
    d = inputs([300, 5, 211], 8, 2, 128, BF)
    g = on(d)
    run = lambda **kw: (lambda r: (*r, *kda.attn_prompt_bwd(g["q"], g["k"], g["v"], g["cu"], *r, g["do"], **kw).values()))(  # noqa: E731
        kda.attn_prompt_fwd(g["q"], g["k"], g["v"], g["cu"], o_dtype=BF, **kw))
    want = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = run(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))
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


def test_no_sequences():
    q = torch.randn(5, 4, 64, device=DEV)
    k = torch.randn(5, 2, 64, device=DEV)
    for cu in ([0], [0, 0, 0]):
        c = torch.tensor(cu, dtype=torch.int32, device=DEV)
        o, lse = kda.attn_prompt_fwd(q, k, k, c)
        got = kda.attn_prompt_bwd(q, k, k, c, o, lse, q)
        torch.cuda.synchronize()
        assert not o.any() and not any(x.any() for x in got.values())
    o, _ = kda.attn_prompt_fwd(q[:0], k[:0], k[:0], c)
    assert o.shape == (0, 4, 64)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients_at_a_sequences_start(dtype):
    """A sequence of one row has probability one, whatever its score: dq and dk are zero but for fp32
    roundings of do . v (64 terms and a few), also where o comes rounded to bf16; and short sequences'
    dq and dk have the relative error of dS' rounding and their own, 2^-8 each at most."""
    d = inputs([1] * 40, 4, 2, 64, dtype)
    g = on(d)
    o, lse = kda.attn_prompt_fwd(g["q"], g["k"], g["v"], g["cu"], o_dtype=dtype)
    got = kda.attn_prompt_bwd(g["q"], g["k"], g["v"], g["cu"], o, lse, g["do"])
    torch.cuda.synchronize()
    f = {x: mx.f64(d[x]).abs() for x in ("q", "k", "v", "do")}
    dov = (f["do"].view(40, 2, 2, 64) * f["v"][:, :, None]).sum(-1)  # [n, Hkv, group]
    bound = 128 * 2.0 ** -24 * 64 ** -0.5
    assert bool((mx.f64(got["dq"]).view(40, 2, 2, 64).abs() <= bound * dov[..., None] * f["k"][:, :, None] + 1e-30).all())
    dk_mag = (dov[..., None] * f["q"].view(40, 2, 2, 64)).sum(2)
    assert bool((mx.f64(got["dk"]).abs() <= bound * dk_mag + 1e-30).all())
    d = inputs([3, 9, 2, 17, 30, 4], 4, 2, 64, dtype)
    g = on(d)
    o, lse = kda.attn_prompt_fwd(g["q"], g["k"], g["v"], g["cu"], o_dtype=dtype)
    got = kda.attn_prompt_bwd(g["q"], g["k"], g["v"], g["cu"], o, lse, g["do"], grad_dtype=dtype)
    torch.cuda.synchronize()
    want, _ = mx.prompt(*(mx.f64(d[x]) for x in ("q", "k", "v")), d["cu"], 64 ** -0.5, mx.f64(d["do"]))
    for x in ("dq", "dk", "dv"):
        assert float((mx.f64(got[x]) - want[x]).norm() / want[x].norm()) <= 2 * (mx.U[dtype] if dtype == BF else 64 * mx.U[F32]), x
