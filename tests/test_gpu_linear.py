"""Linear attention with a decay per head on the GPU against the 64-bit token recurrence.

Bounds, derived from the arithmetic.  With bf16 elements an output term is rounded once as the
decayed score (or the state's copy) and the sum once as the output: two roundings of the sum of
the terms' magnitudes.  Gradients likewise.  The state, its gradient and dg are fp32: weighted
values enter as two bf16 parts (2^-17 of each term, 2^7 fp32 roundings; dg has two such factors),
and everything else rounds to fp32 once for every addition: a dot product over the head's channels,
a chunk's tokens, one per chunk for the carried state, and the decay factors."""
import math

import pytest
import torch

import gated_delta_rule_11_amd as kda
from tests import _mixers as mx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def inputs(B, T, H, dk, dv, dtype, decay="token", state=True, seed=0, rate=0.1):
    gen = torch.Generator().manual_seed(seed * 1000 + T)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / (x.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
    d = {"q": unit(rn(B, T, H, dk)).to(dtype), "k": unit(rn(B, T, H, dk)).to(dtype), "v": rn(B, T, H, dv).to(dtype)}
    d["g"] = -rate * torch.exp(0.8 * rn(H) if decay == "head" else 0.8 * rn(B, T, H))
    d["S"] = rn(B, H, dk, dv) if state else None
    d["do"] = rn(B, T, H, dv).to(dtype)
    d["dS"] = rn(B, H, dk, dv) if state else None
    return d


def dev(x):
    return None if x is None else x.to(DEV)


def fp32_terms(T, d, dtype):
    """Roundings to fp32 on the longest path: a channel sum, a chunk's tokens, a carried state's chunks, decays."""
    return d + 64 + math.ceil(T / 32) + 32 + (2 ** 8 if dtype == BF else 0)


def check_forward(label, d, scale=1.0, o_dtype=None, **kw):
    dtype = d["q"].dtype
    o, S = kda.linear_chunk_fwd(dev(d["q"]), dev(d["k"]), dev(d["v"]), dev(d["g"]), S_in=dev(d["S"]), scale=scale,
                                o_dtype=o_dtype or dtype, **kw)
    torch.cuda.synchronize()
    f = {x: mx.f64(d[x]) for x in d}
    ro, rS, mo, mS = mx.linear(f["q"], f["k"], f["v"], f["g"], f["S"], scale)
    n = fp32_terms(d["q"].shape[1], max(d["q"].shape[-1], 64), dtype)
    mx.close(label + " o", o, ro, mo, dtype, 2.0, n)
    mx.close(label + " S", S, rS, mS, F32, 1.0, n)
    return o, S


LENGTHS = [1, 2, 31, 32, 33, 63, 64, 65, 127, 200]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", LENGTHS)
def test_lengths(T, dtype):
    check_forward(f"T={T}", inputs(2, T, 3, 64, 128, dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk", [16, 32, 64, 128])
@pytest.mark.parametrize("dv", [16, 32, 64, 128])
def test_head_sizes(dk, dv, dtype):
    d = inputs(1, 97, 2, dk, dv, dtype, decay="head" if dk == dv else "token", state=dk != dv)
    check_forward(f"dk={dk} dv={dv}", d, scale=0.5 if dv == 64 else 1.0)
    check_backward(f"dk={dk} dv={dv}", d, scale=0.5 if dv == 64 else 1.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rate", [0.001, 0.05, 2.0])
def test_segments(rate, dtype):
    """One sequence of few heads is cut into segments and joined; long and short memories."""
    d = inputs(1, 64 * 13 + 7, 2, 32, 64, dtype, rate=rate)
    B, T, H, dk = d["q"].shape
    assert kda.linear_chunk_fwd_workspace_bytes(B, T, H, dk, 64, dtype) > 0
    check_forward(f"segments rate={rate}", d)
    check_backward(f"segments rate={rate}", d)


def test_many_heads_run_in_one_walk():
    assert kda.linear_chunk_fwd_workspace_bytes(8, 1000, 32, 64, 64, BF) == 0
    check_forward("one walk", inputs(4, 70, 64, 16, 16, BF, state=False))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strong_and_no_decay(dtype):
    """Resets (-inf), decays that are zero in fp32, and none at all, within and at the ends of chunks."""
    d = inputs(1, 150, 2, 32, 32, dtype)
    g = d["g"]
    g[:, 5::17] = -math.inf
    g[:, 20::31] = -300.0
    g[:, 63:66] = -20000.0
    g[:, 70:90] = 0.0
    check_forward("resets", d)
    check_backward("resets", d)
    d["g"] = torch.zeros_like(g)
    check_forward("no decay", d)
    check_backward("no decay", d)


def check_backward(label, d, scale=1.0, grad_dtype=None, **kw):
    dtype = d["q"].dtype
    gd = grad_dtype or dtype
    got = kda.linear_chunk_bwd(dev(d["q"]), dev(d["k"]), dev(d["v"]), dev(d["g"]), dev(d["do"]), dS_out=dev(d["dS"]),
                               S_in=dev(d["S"]), scale=scale, grad_dtype=gd, **kw)
    torch.cuda.synchronize()
    f = {x: mx.f64(d[x]) for x in d}
    want, mag = mx.linear_grad(f["q"], f["k"], f["v"], f["g"], f["S"], f["do"], f["dS"], scale)
    B, T, H, dk = d["q"].shape
    n = fp32_terms(T, max(dk, d["v"].shape[-1]), dtype)
    for x in ("dq", "dk", "dv"):
        mx.close(f"{label} {x}", got[x], want[x], mag[x], dtype, 2.0, 2 * n)
    # dg sums over a chunk's tokens what crosses a token, and its magnitude is that of the products
    near = mag["dg"] if d["g"].dim() == 1 else around(mag["dg"])
    mx.close(f"{label} dg", got["dg"], want["dg"], near, F32, 1.0, 2 * n)
    mx.close(f"{label} dS_in", got["dS_in"], want["dS_in"], mag["dS_in"], F32, 1.0, n)
    assert got["dq"].dtype == gd and got["dg"].shape == d["g"].shape
    return got


def around(m):
    """The largest magnitude within 64 tokens: the in-chunk part of dg is a difference of sums over the chunk,
    so its error is that of the chunk's terms, not of the one token's."""
    B, T, H = m.shape
    return torch.nn.functional.max_pool1d(m.permute(0, 2, 1), 129, 1, 64).permute(0, 2, 1) * 64


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 2, 31, 33, 64, 65, 129])
def test_backward_lengths(T, dtype):
    check_backward(f"T={T}", inputs(2, T, 3, 64, 32, dtype))


def test_backward_without_states_and_fp32_gradients():
    d = inputs(2, 70, 2, 64, 64, BF, state=False)
    check_backward("no states", d, grad_dtype=F32)
    assert kda.linear_chunk_bwd(*(dev(d[x]) for x in ("q", "k", "v", "g", "do")), want_dS_in=False)["dS_in"] is None


@pytest.mark.parametrize("decay", ["token", "head"])
def test_gradient_against_differences(decay):
    """The kernel's gradient along random directions against central differences of the 64-bit loss."""
    d = inputs(1, 45, 2, 32, 16, F32, decay=decay)
    f = {x: mx.f64(d[x]) for x in d}
    got = check_backward("differences", d)
    loss = lambda q, k, v, g, S: (lambda r: (r[0] * f["do"]).sum() + (r[1] * f["dS"]).sum())(mx.linear(q, k, v, g, S, 1.0))  # noqa: E731
    names = ["q", "k", "v", "g", "S"]
    gen = torch.Generator().manual_seed(3)
    for i, name in enumerate(names):
        u = torch.randn(f[name].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        at = lambda s: loss(*[f[x] + s * h * u if x == name else f[x] for x in names])  # noqa: E731,B023
        diff = (at(1) - at(-1)) / (2 * h)
        key = {"S": "dS_in"}.get(name, "d" + name)
        dot = (mx.f64(got[key]) * u).sum()
        # 1e-4: fp32 gradients (2^-24 of each of some 10^3 terms) and the differences' own h^2
        assert abs(dot - diff) <= 1e-4 * (mx.f64(got[key]).norm() * u.norm()), (name, float(dot), float(diff))


def test_same_bits_every_time():
    d = {x: dev(y) for x, y in inputs(1, 700, 4, 128, 128, BF).items()}
    runs = [kda.linear_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], dS_out=d["dS"], S_in=d["S"]) for _ in range(3)]
    fwd = [kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], S_in=d["S"]) for _ in range(3)]
    torch.cuda.synchronize()
    for r in runs[1:]:
        assert all(torch.equal(r[x], runs[0][x]) for x in r)
    for r in fwd[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, fwd[0]))


def test_zero_sizes():
    d = inputs(2, 0, 3, 32, 64, BF)
    o, S = kda.linear_chunk_fwd(*(dev(d[x]) for x in ("q", "k", "v", "g")), S_in=dev(d["S"]))
    g = kda.linear_chunk_bwd(*(dev(d[x]) for x in ("q", "k", "v", "g", "do")), dS_out=dev(d["dS"]), S_in=dev(d["S"]))
    torch.cuda.synchronize()
    assert o.shape == (2, 0, 3, 64) and torch.equal(S.cpu(), d["S"]) and torch.equal(g["dS_in"].cpu(), d["dS"])
    h = inputs(0, 5, 3, 32, 64, BF, decay="head")
    o, S = kda.linear_chunk_fwd(*(dev(h[x]) for x in ("q", "k", "v", "g")))
    g = kda.linear_chunk_bwd(*(dev(h[x]) for x in ("q", "k", "v", "g", "do")))
    torch.cuda.synchronize()
    assert o.numel() == 0 and S.numel() == 0 and torch.equal(g["dg"].cpu(), torch.zeros(3))


def test_state_in_place_and_carried():
    """Two halves with the state carried in place equal the whole."""
    d = inputs(1, 130, 2, 64, 64, BF)
    o, S = check_forward("whole", d)
    S2 = dev(d["S"]).clone()
    parts = []
    for a, b in ((0, 77), (77, 130)):
        x = {n: dev(d[n][:, a:b].contiguous()) for n in ("q", "k", "v", "g")}
        parts.append(kda.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S_in=S2, S_out=S2, o_dtype=BF)[0])
    f = {x: mx.f64(d[x]) for x in d}
    ro, rS, mo, mS = mx.linear(f["q"], f["k"], f["v"], f["g"], f["S"], 1.0)
    mx.close("carried o", torch.cat(parts, 1), ro, mo, BF, 2.0, 600)
    mx.close("carried S", S2, rS, mS, F32, 1.0, 600)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(16, 16), (16, 128), (128, 16), (64, 32), (128, 128)])
def test_step(dk, dv, dtype):
    """Steps from a prefill's state: in place, and kept."""
    d = inputs(3, 9, 2, dk, dv, dtype, decay="head" if dk == 64 else "token")
    S = dev(d["S"]).clone()
    outs = []
    for t in range(9):
        g = dev(d["g"] if d["g"].dim() == 1 else d["g"][:, t].contiguous())
        x = [dev(d[n][:, t].contiguous()) for n in ("q", "k", "v")]
        keep = S.clone()
        o2, S2 = kda.linear_decode_step(*x, g, S, S_out=torch.empty_like(S), scale=0.7, o_dtype=dtype)
        assert torch.equal(S, keep)
        o, S1 = kda.linear_decode_step(*x, g, S, scale=0.7, o_dtype=dtype)
        assert S1.data_ptr() == S.data_ptr() and torch.equal(S1, S2) and torch.equal(o, o2)
        outs.append(o)
    f = {x: mx.f64(d[x]) for x in d}
    ro, rS, mo, mS = mx.linear(f["q"], f["k"], f["v"], f["g"], f["S"], 0.7)
    mx.close("steps o", torch.stack(outs, 1), ro, mo, dtype, 1.0, dk + 64)
    mx.close("steps S", S, rS, mS, F32, 1.0, 64)


def test_other_stream_and_graph():
    """A call on a given stream, and forward with backward captured and replayed beside eager calls."""
    d = {x: dev(y) for x, y in inputs(1, 600, 4, 64, 64, BF).items()}
    want = kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], S_in=d["S"])
    wantg = kda.linear_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], dS_out=d["dS"], S_in=d["S"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], S_in=d["S"], stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, S = kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], S_in=d["S"])
        g = kda.linear_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], dS_out=d["dS"], S_in=d["S"])
    for _ in range(3):
        for t in (o, S, *g.values()):
            t.fill_(float("nan"))
        graph.replay()
        again = kda.linear_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], dS_out=d["dS"], S_in=d["S"])
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(S, want[1])
        assert all(torch.equal(g[x], wantg[x]) and torch.equal(again[x], wantg[x]) for x in g)
