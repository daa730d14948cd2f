"""The mixers as a hybrid model's layer stack uses them: a prompt through packed attention, its keys
and values into the 8-bit cache, then tokens one at a time through append and attention, beside
linear attention's prefill and its single-token steps."""
import pytest
import torch

import gated_delta_rule_11_amd as kda
from tests import _mixers as mx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_prompt_cache_and_steps():
    """A step's attention over the cache is the prompt attention's last row, but for the rounding of keys
    and values to 8 bits; over the very values the cache holds it is the same to the outputs' type."""
    Hq, Hkv, d, P, extra = 8, 2, 128, 32, 3
    prompts = [70, 1, 133]
    gen = torch.Generator().manual_seed(0)
    full = [n + extra for n in prompts]
    rn = lambda h: [torch.randn(n, h, d, generator=gen).to(BF) for n in full]  # noqa: E731
    q, k, v = rn(Hq), rn(Hkv), rn(Hkv)
    pages = sum(-(-n // P) for n in full)
    width = max(-(-n // P) for n in full)
    order, table = torch.randperm(pages, generator=gen).tolist(), []
    for n in full:
        m = -(-n // P)
        table.append(order[:m] + [0] * (width - m))
        order = order[m:]
    kc = torch.zeros(pages, Hkv, P, d, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    vc = torch.zeros(pages, Hkv, d, P, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    ks, vs = torch.zeros(pages, Hkv, device=DEV), torch.zeros(pages, Hkv, device=DEV)
    tab, held = i32(table), i32([0, 0, 0])
    cu = i32([0, 70, 71, 204])
    pk = lambda x: torch.cat([y[:n] for y, n in zip(x, prompts)]).to(DEV)  # noqa: E731
    o, _ = kda.attn_prompt_fwd(pk(q), pk(k), pk(v), cu, o_dtype=BF)
    kda.kv_cache_append(pk(k), pk(v), cu, held, tab, kc, vc, ks, vs)
    want = [mx.prompt(*(mx.f64(x[i]) for x in (q, k, v)), [0, full[i]], d ** -0.5) for i in range(3)]
    mx.close("prompt", o, torch.cat([w["o"][:n] for (w, _), n in zip(want, prompts)]),
             torch.cat([m["o"][:n] for (_, m), n in zip(want, prompts)]), BF, 2.0, 600)
    one, held = i32([0, 1, 2, 3]), i32(prompts)
    for t in range(extra):
        now = lambda x: torch.stack([y[n + t] for y, n in zip(x, prompts)]).to(DEV)  # noqa: E731,B023
        kda.kv_cache_append(now(k), now(v), one, held, tab, kc, vc, ks, vs)
        held = held + 1
        o, _ = kda.attn_decode_step(now(q), kc, vc, ks, vs, tab, held, o_dtype=BF)
        torch.cuda.synchronize()
        ro, _, mag = mx.Cache(kc, vc, ks, vs).attend(mx.f64(now(q)), held.tolist(), table, d ** -0.5)
        mx.close(f"step {t}", o, ro, mag, BF, 2.0, 600)
        for i, n in enumerate(prompts):
            w, m = want[i]
            # values: 2^-4 of each (and 2^-4 again where a page's scale grew).  Scores: sum |q k| 2^-3, at most
            # |q|.|k| scale 2^-3, seldom above 0.3 in sum; a probability moves by twice that of itself.
            assert float((o[i].cpu().double() - w["o"][n + t]).norm() / m["o"][n + t].norm()) < 2 ** -3 + 0.6


def test_linear_prefill_and_steps():
    """A prefill's state continued token by token equals the longer prefill."""
    B, T, H, dk, dv, more = 2, 150, 4, 128, 128, 5
    gen = torch.Generator().manual_seed(1)
    rn = lambda d: torch.randn(B, T + more, H, d, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    x = {"q": unit(rn(dk)).to(BF), "k": unit(rn(dk)).to(BF), "v": rn(dv).to(BF),
         "g": -0.1 * torch.rand(B, T + more, H, generator=gen)}
    first = [x[n][:, :T].contiguous().to(DEV) for n in ("q", "k", "v", "g")]
    o, S = kda.linear_chunk_fwd(*first, o_dtype=BF)
    outs = [o]
    for t in range(T, T + more):
        outs.append(kda.linear_decode_step(*(x[n][:, t].contiguous().to(DEV) for n in ("q", "k", "v", "g")), S, o_dtype=BF)[0][:, None])
    torch.cuda.synchronize()
    f = {n: mx.f64(y) for n, y in x.items()}
    ro, rS, mo, mS = mx.linear(f["q"], f["k"], f["v"], f["g"], None, 1.0)
    mx.close("o", torch.cat(outs, 1), ro, mo, BF, 2.0, 600)
    mx.close("S", S, rS, mS, F32, 1.0, 600)
