"""The linear, prompt and cache calls against what surrounds them: memory before and behind every output
stays as it was, a workspace's contents do not matter, calls on two streams do not meet, element types
mix, and a backward of several blocks and segments agrees with the recurrence."""
import pytest
import torch

import gated_delta_rule_11_amd as kda
from tests import _mixers as mx
from tests.test_gpu_cache import filled, i32
from tests.test_gpu_linear import check_backward, check_forward, dev, fp32_terms, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def guarded(shape, dtype):
    """A contiguous tensor inside a larger buffer of a known pattern, and a check that the rest kept it."""
    n = 1
    for s in shape:
        n *= s
    pad = 4096
    buf = torch.full((n + 2 * pad,), 7.0, dtype=dtype, device=DEV)
    def intact():
        torch.cuda.synchronize()
        assert bool((buf[:pad] == 7.0).all()) and bool((buf[pad + n:] == 7.0).all())
    return buf[pad:pad + n].view(shape), intact


def dirty(nbytes):
    return torch.full((max(nbytes, 16),), 0xFF, dtype=torch.uint8, device=DEV)  # NaN in every type


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,dk,dv", [(33, 16, 16), (70, 128, 128), (65, 32, 64), (600, 16, 32), (1, 64, 128)])
def test_linear_outputs_and_workspace(T, dk, dv, dtype):
    d = inputs(1, T, 2, dk, dv, dtype)
    g = {x: dev(y) for x, y in d.items()}
    want_o, want_S = kda.linear_chunk_fwd(g["q"], g["k"], g["v"], g["g"], S_in=g["S"], o_dtype=dtype)
    o, ok_o = guarded(want_o.shape, dtype)
    S, ok_S = guarded(want_S.shape, F32)
    ws = dirty(kda.linear_chunk_fwd_workspace_bytes(1, T, 2, dk, dv, dtype))
    kda.linear_chunk_fwd(g["q"], g["k"], g["v"], g["g"], S_in=g["S"], o=o, S_out=S, workspace=ws)
    ok_o()
    ok_S()
    assert torch.equal(o, want_o) and torch.equal(S, want_S)
    want = kda.linear_chunk_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], dS_out=g["dS"], S_in=g["S"], grad_dtype=dtype)
    ws = dirty(kda.linear_chunk_bwd_workspace_bytes(1, T, 2, dk, dv, dtype))
    got = kda.linear_chunk_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], dS_out=g["dS"], S_in=g["S"], grad_dtype=dtype,
                               workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(got[x], want[x]) for x in want)


def test_linear_backward_stays_in_its_gradients():
    """The gradients through the C ABI, each between guards."""
    import ctypes
    B, T, H, dk, dv = 2, 77, 3, 16, 32
    for dtype, code in ((BF, 1), (F32, 0)):
        d = {x: dev(y) for x, y in inputs(B, T, H, dk, dv, dtype).items()}
        outs = {n: guarded(s, t) for n, s, t in (("dq", (B, T, H, dk), dtype), ("dk", (B, T, H, dk), dtype),
                                                 ("dv", (B, T, H, dv), dtype), ("dg", (B, T, H), F32),
                                                 ("dS_in", (B, H, dk, dv), F32))}
        need = kda.linear_chunk_bwd_workspace_bytes(B, T, H, dk, dv, dtype)
        ws, ok_ws = guarded((need // 4,), F32)
        p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
        st = kda.lib().kda_linear_chunk_bwd(
            p(d["q"]), p(d["k"]), p(d["v"]), code, p(d["g"]), 0, p(d["S"]), p(d["do"]), p(d["dS"]), p(outs["dq"][0]),
            p(outs["dk"][0]), p(outs["dv"][0]), code, p(outs["dg"][0]), p(outs["dS_in"][0]), B, T, H, dk, dv, 1.0, p(ws), need,
            ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert st == 0
        want = kda.linear_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], dS_out=d["dS"], S_in=d["S"], grad_dtype=dtype)
        ok_ws()
        for n, (t, ok) in outs.items():
            ok()
            assert torch.equal(t, want[n]), n


@pytest.mark.parametrize("out", [BF, F32])
def test_linear_mixed_types(out):
    d = inputs(2, 75, 2, 32, 64, F32 if out == BF else BF)
    g = {x: dev(y) for x, y in d.items()}
    f = {x: mx.f64(y) for x, y in d.items()}
    o, S = kda.linear_chunk_fwd(g["q"], g["k"], g["v"], g["g"], S_in=g["S"], o_dtype=out)
    got = kda.linear_chunk_bwd(g["q"], g["k"], g["v"], g["g"], g["do"], dS_out=g["dS"], S_in=g["S"], grad_dtype=out)
    torch.cuda.synchronize()
    ro, rS, mo, mS = mx.linear(f["q"], f["k"], f["v"], f["g"], f["S"], 1.0)
    n = fp32_terms(75, 64, BF)
    mx.close("o", o, ro, mo, BF, 2.0, n)
    mx.close("S", S, rS, mS, F32, 1.0, n)
    want, mag = mx.linear_grad(f["q"], f["k"], f["v"], f["g"], f["S"], f["do"], f["dS"], 1.0)
    for x in ("dq", "dk", "dv"):
        assert got[x].dtype == out
        mx.close(x, got[x], want[x], mag[x], BF, 2.0, 2 * n)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear_several_blocks_batches_and_segments(dtype):
    d = inputs(2, 1100, 1, 16, 32, dtype, rate=0.02)
    check_forward("blocks", d)
    check_backward("blocks", d)
    d = inputs(3, 1030, 2, 32, 16, dtype, decay="head")
    check_backward("blocks, per head", d)


def test_linear_without_decay_far_from_one_over_many_tokens():
    """dg far from the sequence's ends, where nearly everything crosses a token."""
    d = inputs(1, 700, 2, 64, 64, F32, rate=1e-4)
    check_backward("no decay", d)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_outputs(d, dtype):
    gen = torch.Generator().manual_seed(d)
    n, Hq, Hkv = 171, 6, 2
    q, k, v, do = (torch.randn(n, h, d, generator=gen).to(dtype).to(DEV) for h in (Hq, Hkv, Hkv, Hq))
    cu = i32([0, 40, 41, 160])
    o, ok_o = guarded((n, Hq, d), dtype)
    lse, ok_l = guarded((n, Hq), F32)
    kda.attn_prompt_fwd(q, k, v, cu, o=o, lse=lse)
    ok_o()
    ok_l()
    want, wl = kda.attn_prompt_fwd(q, k, v, cu, o_dtype=dtype)
    assert torch.equal(o[:160], want[:160]) and torch.equal(lse[:160], wl[:160])
    assert bool((o[160:] == 7.0).all()) and not want[160:].any()
    a = kda.attn_prompt_bwd(q, k, v, cu, want, wl, do, grad_dtype=dtype)
    ws = dirty(kda.attn_prompt_bwd_workspace_bytes(n, Hq, Hkv, d))
    b = kda.attn_prompt_bwd(q, k, v, cu, want, wl, do, grad_dtype=dtype, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a[x], b[x]) for x in a) and all(not a[x][160:].any() for x in a)


def test_prompt_entries_out_of_order_touch_nothing_outside():
    """Meaningless offsets give meaningless rows, within the outputs."""
    n, H, d = 300, 2, 64
    q, k, v, do = (torch.randn(n, H, d, device=DEV).to(BF) for _ in range(4))
    for cu in ([0, 200, 100, 300], [5, 4, 3, 2], [-7, 50, 1000000], [300, 0], [0, 2 ** 31 - 1]):
        o, ok_o = guarded((n, H, d), F32)
        lse, ok_l = guarded((n, H), F32)
        kda.attn_prompt_fwd(q, k, v, i32(cu), o=o, lse=lse)
        kda.attn_prompt_bwd(q, k, v, i32(cu), o, lse, do)
        ok_o()
        ok_l()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_cache_step_outputs_and_workspace(dtype):
    for ctx, Hq, Hkv, P, d in (([700, 3], 6, 2, 16, 64), ([90], 17, 1, 64, 128), ([5] * 300, 8, 8, 32, 64)):
        c, t = filled(ctx, Hkv, P, d)
        N = len(ctx)
        q = torch.randn(N, Hq, d, device=DEV).to(dtype)
        o, ok_o = guarded((N, Hq, d), dtype)
        lse, ok_l = guarded((N, Hq), F32)
        ws = dirty(kda.attn_decode_step_workspace_bytes(N, Hq, Hkv, d, P, len(t[0])))
        args = (q, c["kc"], c["vc"], c["ks"], c["vs"], i32(t), i32(ctx))
        kda.attn_decode_step(*args, o=o, lse=lse, workspace=ws)
        ok_o()
        ok_l()
        want, wl = kda.attn_decode_step(*args, o_dtype=dtype, want_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(lse, wl)


def test_two_streams_at_once():
    """The same calls on two streams, on inputs of their own, give what they give alone."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets, alone = [], []
    for i in range(2):
        x = {n: dev(y) for n, y in inputs(1, 900, 4, 128, 128, BF, seed=i).items()}
        sets.append(x)
        alone.append((kda.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S_in=x["S"])[0],
                      kda.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"])["dk"]))
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for i in range(2):
            x = sets[i]
            got.append((kda.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S_in=x["S"], stream=streams[i])[0],
                        kda.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], stream=streams[i])["dk"]))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, alone) for a, b in zip(g, w))


def test_refused_by_the_binding():
    q = torch.zeros(2, 8, 2, 64, device=DEV)
    g = torch.zeros(2, 8, 2, device=DEV)
    k3, cu = q[0], i32([0, 8])
    with pytest.raises(kda.KDAError):
        kda.linear_chunk_fwd(q, q, q, g[..., :1])
    with pytest.raises(kda.KDAError):
        kda.linear_chunk_fwd(q, q.transpose(1, 2).contiguous().transpose(1, 2), q, g)
    with pytest.raises(kda.KDAError):
        kda.linear_chunk_fwd(q, q, q, g.to(BF))
    with pytest.raises(kda.KDAError):
        kda.linear_chunk_fwd(q, q.to(BF), q, g)
    with pytest.raises(kda.KDAError):
        kda.linear_chunk_fwd(q, q, q, g, o_dtype=torch.float16)
    with pytest.raises(kda.KDAError):
        kda.linear_chunk_fwd(q, q, q, g, workspace=torch.zeros(16))
    with pytest.raises(kda.KDAError):
        kda.linear_chunk_bwd(q, q, q, g, q.to(BF))
    with pytest.raises(kda.KDAError):
        kda.linear_decode_step(q[0], q[0], q[0], g[0], q)
    with pytest.raises(kda.KDAError):
        kda.attn_prompt_fwd(k3, k3, k3, cu.long())
    with pytest.raises(kda.KDAError):
        kda.attn_prompt_fwd(k3, k3[:4], k3, cu)
    with pytest.raises(kda.KDAError):
        kda.attn_prompt_fwd(k3, k3, k3, cu[:0])
    with pytest.raises(kda.KDAError):
        kda.attn_prompt_fwd(k3[..., :32].contiguous(), k3[..., :32].contiguous(), k3[..., :32].contiguous(), cu)
    c, t = filled([20], 2, 16, 64)
    one = torch.zeros(1, 4, 64, device=DEV)
    with pytest.raises(kda.KDAError):
        kda.attn_decode_step(one, c["kc"].view(torch.uint8), c["vc"], c["ks"], c["vs"], i32(t), i32([20]))
    with pytest.raises(kda.KDAError):
        kda.attn_decode_step(one, c["kc"], c["vc"], c["ks"], c["vs"], i32(t), i32([20, 1]))
    with pytest.raises(kda.KDAError):
        kda.kv_cache_append(one[:, :2].contiguous(), one[:, :2].contiguous(), i32([0]), i32([20]), i32(t), c["kc"], c["vc"], c["ks"], c["vs"])
    with pytest.raises(kda.KDAError):
        kda.attn_prompt_bwd(k3, k3, k3, cu, k3, g[0], k3, workspace=dirty(16))
