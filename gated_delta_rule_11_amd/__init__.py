"""Python binding of libkda.so -- the MI355X (gfx950) Kimi Delta Attention
forward library.

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI (include/kda.h).  PyTorch supplies device memory and
the current stream.  There is no CPU fallback: the functions raise when the
library is not built or when a tensor is not on a GPU.

Entry points (same names as the C ABI):
  gate(z, A, g_min, chunk)                        -> G           (kda_gate)
  chunk_fwd_workspace_bytes(B, T, H, dk, dv, chunk) -> bytes     (kda_chunk_fwd_workspace_bytes)
  chunk_fwd(q, k, v, beta, G, chunk, ...)         -> (o, S_out)  (kda_chunk_fwd)
  chunk_fwd_z(q, k, v, beta, z, A, g_min, chunk)  -> (o, S_out)  (kda_chunk_fwd_z)
  decode_step(q, k, v, z, beta, A, S, g_min)      -> o           (kda_decode_step; S updated in place)

Beside the delta rule, on the same layouts:
  linear_chunk_fwd(q, k, v, g)                    -> (o, S_out)  linear attention with a decay per head
  linear_chunk_bwd(q, k, v, g, d_o)               -> gradients
  linear_decode_step(q, k, v, g, S)               -> (o, S)      (S updated in place unless S_out is given)
  attn_prompt_fwd(q, k, v, cu_seqlens)            -> (o, lse)    causal attention over packed prompts
  attn_prompt_bwd(q, k, v, cu_seqlens, o, lse, d_o) -> gradients
  rope(x, positions, inv_freq)                    -> y           rotary positions, or (inverse) their gradient
  kv_cache_append(k, v, cu_seqlens, ...)          -> None        paged cache in 8 bits, written in place
  kv_cache_append_rope(k, v, cu_seqlens, ...)     -> q turned    the same with rotary positions on the way
  attn_decode_step(q, k_cache, v_cache, ...)      -> (o, lse)    attention of one token over it
  attn_chunk_fwd(q, cu_seqlens, k_cache, ...)     -> (o, lse)    attention of several new tokens a sequence over it
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Tuple

import torch

__all__ = ["gate", "chunk_fwd", "chunk_fwd_z", "chunk_fwd_workspace_bytes", "decode_step", "chunk_uses_mfma", "lib",
           "linear_chunk_fwd", "linear_chunk_fwd_workspace_bytes", "linear_chunk_bwd",
           "linear_chunk_bwd_workspace_bytes", "linear_decode_step", "attn_prompt_fwd", "attn_prompt_bwd",
           "attn_prompt_bwd_workspace_bytes", "rope", "kv_cache_append", "kv_cache_append_rope", "attn_decode_step",
           "attn_decode_step_workspace_bytes", "attn_chunk_fwd", "attn_chunk_fwd_workspace_bytes", "KDAError", "LIB_PATH", "G_MIN"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkda.so")
G_MIN = -5.0
KDA_F32, KDA_BF16 = 0, 1

_lib = None


class KDAError(RuntimeError):
    pass


def lib() -> ctypes.CDLL:
    """Load libkda.so (raises when it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise KDAError(f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(LIB_PATH)
    P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    L.kda_status_string.argtypes = [I]
    L.kda_status_string.restype = ctypes.c_char_p
    L.kda_version.argtypes = []
    L.kda_version.restype = I
    L.kda_chunk_uses_mfma.argtypes = [I, I, I, I]
    L.kda_chunk_uses_mfma.restype = I
    L.kda_gate.argtypes = [P, I, P, F, I, I, I, I, I, P, P]
    L.kda_gate.restype = I
    Z = ctypes.c_size_t
    L.kda_chunk_fwd_workspace_bytes.argtypes = [I, I, I, I, I, I]
    L.kda_chunk_fwd_workspace_bytes.restype = Z
    L.kda_chunk_fwd.argtypes = [P, P, P, P, I, P, P, P, I, P, I, I, I, I, I, I, F, P, Z, P]
    L.kda_chunk_fwd.restype = I
    L.kda_chunk_fwd_z.argtypes = [P, P, P, P, P, I, P, F, P, P, I, P, I, I, I, I, I, I, F, P, Z, P]
    L.kda_chunk_fwd_z.restype = I
    L.kda_decode_step.argtypes = [P, P, P, P, P, I, P, F, P, P, I, I, I, I, I, F, P]
    L.kda_decode_step.restype = I
    L.kda_decode_replay.argtypes = [P, P, P, P, P, I, P, F, P, P, P, I, P, I, I, I, I, I, F, P]
    L.kda_decode_replay.restype = I
    L.kda_chunk_fwd_z_noalloc.argtypes = [P, P, P, P, P, I, P, F, P, P, I, P, I, I, I, I, I, I, F, P]
    L.kda_chunk_fwd_z_noalloc.restype = I
    L.kda_chunk_fwd_z_prologue.argtypes = L.kda_chunk_fwd_z.argtypes
    L.kda_chunk_fwd_z_prologue.restype = I
    L.kda_decode_step_prologue.argtypes = L.kda_decode_step.argtypes
    L.kda_decode_step_prologue.restype = I
    L.kda_chunk_bwd_z_workspace_bytes.argtypes = [I, I, I, I, I]
    L.kda_chunk_bwd_z_workspace_bytes.restype = ctypes.c_size_t
    L.kda_chunk_bwd_z.argtypes = [P, P, P, P, P, I, P, F, P, P, I, P, P, P, P, P, P, P, P, I, I, I, I, I, F, P,
                                  ctypes.c_size_t, P]
    L.kda_chunk_bwd_z.restype = I
    L.kda_chunk_fwd_z_segmented_workspace_bytes.argtypes = [I, I, I, I, I]
    L.kda_chunk_fwd_z_segmented_workspace_bytes.restype = ctypes.c_size_t
    L.kda_chunk_fwd_z_segmented.argtypes = [P, P, P, P, P, I, P, F, P, P, I, P, I, I, I, I, I, I, F, I, P,
                                            ctypes.c_size_t, P]
    L.kda_chunk_fwd_z_segmented.restype = I
    L.kda_linear_chunk_fwd_workspace_bytes.argtypes = [I] * 6
    L.kda_linear_chunk_fwd_workspace_bytes.restype = Z
    L.kda_linear_chunk_fwd.argtypes = [P, P, P, I, P, I, P, P, I, P, I, I, I, I, I, F, P, Z, P]
    L.kda_linear_chunk_fwd.restype = I
    L.kda_linear_chunk_bwd_workspace_bytes.argtypes = [I] * 7
    L.kda_linear_chunk_bwd_workspace_bytes.restype = Z
    L.kda_linear_chunk_bwd.argtypes = [P, P, P, I, P, I, P, P, P, P, P, P, I, P, P, I, I, I, I, I, F, P, Z, P]
    L.kda_linear_chunk_bwd.restype = I
    L.kda_linear_decode_step.argtypes = [P, P, P, I, P, I, P, P, P, I, I, I, I, I, F, P]
    L.kda_linear_decode_step.restype = I
    L.kda_attn_prompt_fwd.argtypes = [P, P, P, I, P, P, I, P, I, I, I, I, I, F, I, P]
    L.kda_attn_prompt_fwd.restype = I
    L.kda_attn_prompt_bwd_workspace_bytes.argtypes = [I] * 4
    L.kda_attn_prompt_bwd_workspace_bytes.restype = Z
    L.kda_attn_prompt_bwd.argtypes = [P, P, P, I, P, P, I, P, P, P, P, P, I, I, I, I, I, I, F, I, P, Z, P]
    L.kda_attn_prompt_bwd.restype = I
    L.kda_kv_cache_append.argtypes = [P, P, I, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P]
    L.kda_kv_cache_append.restype = I
    W = ctypes.c_int64
    L.kda_rope.argtypes = [P, I, W, P, I, P, P, I, I, I, P, I, W, I, I, I, P]
    L.kda_rope.restype = I
    L.kda_kv_cache_append_rope.argtypes = [P, W, P, W, I, P, W, P, I, W, P, I, P, P, I, I, P, P, P, P, P, P, P, I, I, I, I, I, I,
                                           I, I, I, P]
    L.kda_kv_cache_append_rope.restype = I
    L.kda_attn_chunk_fwd_workspace_bytes.argtypes = [I] * 8
    L.kda_attn_chunk_fwd_workspace_bytes.restype = Z
    L.kda_attn_chunk_fwd.argtypes = [P, W, I, P, P, P, P, P, P, P, P, I, P, I, I, I, I, I, I, I, I, F, I, P, Z, P]
    L.kda_attn_chunk_fwd.restype = I
    L.kda_attn_decode_step_workspace_bytes.argtypes = [I] * 6
    L.kda_attn_decode_step_workspace_bytes.restype = Z
    L.kda_attn_decode_step.argtypes = [P, I, P, P, P, P, P, P, P, I, P, I, I, I, I, I, I, I, F, P, Z, P]
    L.kda_attn_decode_step.restype = I
    _lib = L
    return L


def chunk_uses_mfma(dtype: torch.dtype, dk: int, dv: int, chunk: int) -> bool:
    """True when the chunked prefill runs the MFMA kernel for these arguments."""
    code = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return bool(lib().kda_chunk_uses_mfma(code, dk, dv, chunk))


def _check(status: int, what: str):
    if status != 0:
        msg = lib().kda_status_string(status).decode()
        raise KDAError(f"{what}: {msg}")


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return KDA_F32
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _dev(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise KDAError("libkda runs on the GPU only: tensor is on the CPU")
        if not t.is_contiguous():
            raise KDAError("tensors must be contiguous")


_F32 = (torch.float32,)
_IO = (torch.float32, torch.bfloat16)


def _shapes(what: str, *specs):
    """The C ABI takes raw pointers and trusts the sizes it is given, so every
    tensor's shape and dtype are checked here, before any pointer is passed:
    specs are (name, tensor or None, expected shape, allowed dtypes)."""
    dev = None
    for name, t, shape, dtypes in specs:
        if t is None:
            continue
        if tuple(t.shape) != tuple(shape):
            raise KDAError(f"{what}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.dtype not in dtypes:
            raise KDAError(f"{what}: {name} has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise KDAError(f"{what}: {name} is on {t.device}, the other tensors on {dev}")


def _on_tensor_device(fn):
    """Run a call with the device of its first tensor argument current: the library
    launches on the current device, on that device's current stream."""
    @functools.wraps(fn)
    def wrapper(*args, **kwargs):
        t = next((a for a in args if isinstance(a, torch.Tensor)), None)
        if t is None or not t.is_cuda:
            return fn(*args, **kwargs)
        with torch.cuda.device(t.device):
            return fn(*args, **kwargs)
    return wrapper


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


@_on_tensor_device
def gate(z: torch.Tensor, A: torch.Tensor, g_min: float = G_MIN, chunk: int = 1,
         out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """G [B,T,H,dk] fp32: chunk-local sums of g = g_min*sigmoid(exp(A) z)."""
    B, T, H, dk = z.shape
    if out is None:
        out = torch.empty((B, T, H, dk), dtype=torch.float32, device=z.device)
    _shapes("kda_gate", ("z", z, (B, T, H, dk), _IO), ("A", A, (H, dk), _F32), ("out", out, (B, T, H, dk), _F32))
    _dev(z, A, out)
    _check(lib().kda_gate(_p(z), _dtype_code(z), _p(A), float(g_min), B, T, H, dk, int(chunk), _p(out),
                          _stream(stream)), "kda_gate")
    return out


def _chunk_shapes(what, q, k, v, beta, z=None, A=None, G=None, S_in=None, o=None, S_out=None):
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    io = (q.dtype,) if q.dtype in _IO else _IO
    _shapes(what, ("q", q, (B, T, H, dk), _IO), ("k", k, (B, T, H, dk), io), ("v", v, (B, T, H, dv), io),
            ("beta", beta, (B, T, H), io), ("z", z, (B, T, H, dk), io), ("A", A, (H, dk), _F32),
            ("G", G, (B, T, H, dk), _F32), ("S_in", S_in, (B, H, dk, dv), _F32), ("o", o, (B, T, H, dv), _IO),
            ("S_out", S_out, (B, H, dk, dv), _F32))


def chunk_fwd_workspace_bytes(B: int, T: int, H: int, dk: int, dv: int, chunk: int) -> int:
    """Device bytes kda_chunk_fwd / kda_chunk_fwd_z / kda_chunk_fwd_z_prologue need
    as workspace for these sizes (0: none)."""
    return int(lib().kda_chunk_fwd_workspace_bytes(int(B), int(T), int(H), int(dk), int(dv), int(chunk)))


def _workspace(workspace, q, v, chunk):
    """(pointer, bytes) of the caller's workspace, or of a new one of the queried
    size (None, 0 when the call needs none)."""
    B, T, H, dk = q.shape
    if workspace is None:
        need = chunk_fwd_workspace_bytes(B, T, H, dk, v.shape[-1], chunk)
        if need == 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _dev(workspace)
    return _p(workspace), workspace.numel() * workspace.element_size(), workspace


def _outs(q, v, o, S_out, o_dtype, want_state):
    B, T, H, _ = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=o_dtype or torch.float32, device=q.device)
    if S_out is None and want_state:
        S_out = torch.empty((B, H, q.shape[-1], dv), dtype=torch.float32, device=q.device)
    return o, S_out


@_on_tensor_device
def chunk_fwd(q, k, v, beta, G, chunk: int = 64, S_in=None, o=None, S_out=None, o_dtype=None,
              scale: float = 1.0, want_state: bool = True, workspace=None,
              stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Chunked prefill from the chunk-local sums G of kda_gate (same chunk).
    ``workspace``: a device tensor of at least ``chunk_fwd_workspace_bytes``
    bytes, or None (one is allocated when the call needs it).
    Returns (o [B,T,H,dv], S_out [B,H,dk,dv] or None)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    o, S_out = _outs(q, v, o, S_out, o_dtype, want_state)
    _chunk_shapes("kda_chunk_fwd", q, k, v, beta, G=G, S_in=S_in, o=o, S_out=S_out)
    _dev(q, k, v, beta, G, S_in, o, S_out)
    wp, wb, _keep = _workspace(workspace, q, v, chunk)
    _check(lib().kda_chunk_fwd(_p(q), _p(k), _p(v), _p(beta), _dtype_code(q), _p(G), _p(S_in), _p(o),
                               _dtype_code(o), _p(S_out), B, T, H, dk, dv, int(chunk), float(scale), wp, wb,
                               _stream(stream)), "kda_chunk_fwd")
    return o, S_out


@_on_tensor_device
def chunk_fwd_z(q, k, v, beta, z, A, g_min: float = G_MIN, chunk: int = 64, S_in=None, o=None, S_out=None,
                o_dtype=None, scale: float = 1.0, want_state: bool = True, workspace=None,
                stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Chunked prefill with the gate fused (decay logits z, A, g_min).
    ``workspace``: as ``chunk_fwd``.
    Returns (o [B,T,H,dv], S_out [B,H,dk,dv] or None)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    o, S_out = _outs(q, v, o, S_out, o_dtype, want_state)
    _chunk_shapes("kda_chunk_fwd_z", q, k, v, beta, z=z, A=A, S_in=S_in, o=o, S_out=S_out)
    _dev(q, k, v, beta, z, A, S_in, o, S_out)
    wp, wb, _keep = _workspace(workspace, q, v, chunk)
    _check(lib().kda_chunk_fwd_z(_p(q), _p(k), _p(v), _p(beta), _p(z), _dtype_code(q), _p(A), float(g_min),
                                 _p(S_in), _p(o), _dtype_code(o), _p(S_out), B, T, H, dk, dv, int(chunk),
                                 float(scale), wp, wb, _stream(stream)), "kda_chunk_fwd_z")
    return o, S_out


@_on_tensor_device
def chunk_fwd_z_noalloc(q, k, v, beta, z, A, g_min: float = G_MIN, chunk: int = 64, S_in=None, o=None, S_out=None,
                        o_dtype=None, scale: float = 1.0, want_state: bool = True,
                        stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``chunk_fwd_z`` whose scratch memory is the library's static device array
    (kda_chunk_fwd_z_noalloc): no workspace is allocated for the call.  Calls that
    overlap in time on one device share that array and must not be issued."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    o, S_out = _outs(q, v, o, S_out, o_dtype, want_state)
    _chunk_shapes("kda_chunk_fwd_z_noalloc", q, k, v, beta, z=z, A=A, S_in=S_in, o=o, S_out=S_out)
    _dev(q, k, v, beta, z, A, S_in, o, S_out)
    _check(lib().kda_chunk_fwd_z_noalloc(_p(q), _p(k), _p(v), _p(beta), _p(z), _dtype_code(q), _p(A), float(g_min),
                                         _p(S_in), _p(o), _dtype_code(o), _p(S_out), B, T, H, dk, dv, int(chunk),
                                         float(scale), _stream(stream)), "kda_chunk_fwd_z_noalloc")
    return o, S_out


@_on_tensor_device
def chunk_fwd_z_prologue(q_raw, k_raw, v, beta_logit, z, A, g_min: float = G_MIN, chunk: int = 64, S_in=None,
                         o=None, S_out=None, o_dtype=None, scale: float = 1.0, want_state: bool = True,
                         workspace=None, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``chunk_fwd_z`` with the prologue fused: q, k un-normalised, beta as a logit."""
    B, T, H, dk = q_raw.shape
    dv = v.shape[-1]
    o, S_out = _outs(q_raw, v, o, S_out, o_dtype, want_state)
    _chunk_shapes("kda_chunk_fwd_z_prologue", q_raw, k_raw, v, beta_logit, z=z, A=A, S_in=S_in, o=o, S_out=S_out)
    _dev(q_raw, k_raw, v, beta_logit, z, A, S_in, o, S_out)
    wp, wb, _keep = _workspace(workspace, q_raw, v, chunk)
    _check(lib().kda_chunk_fwd_z_prologue(_p(q_raw), _p(k_raw), _p(v), _p(beta_logit), _p(z), _dtype_code(q_raw),
                                          _p(A), float(g_min), _p(S_in), _p(o), _dtype_code(o), _p(S_out), B, T, H,
                                          dk, dv, int(chunk), float(scale), wp, wb, _stream(stream)),
           "kda_chunk_fwd_z_prologue")
    return o, S_out


@_on_tensor_device
def decode_step_prologue(q_raw, k_raw, v, z, beta_logit, A, S, g_min: float = G_MIN, o=None, o_dtype=None,
                         scale: float = 1.0, stream=None) -> torch.Tensor:
    """``decode_step`` with the prologue fused: q, k un-normalised, beta as a logit."""
    N, H, dk = q_raw.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty((N, H, dv), dtype=o_dtype or torch.float32, device=q_raw.device)
    _decode_shapes("kda_decode_step_prologue", q_raw, k_raw, v, z, beta_logit, A, S, o)
    _dev(q_raw, k_raw, v, z, beta_logit, A, S, o)
    _check(lib().kda_decode_step_prologue(_p(q_raw), _p(k_raw), _p(v), _p(z), _p(beta_logit), _dtype_code(q_raw),
                                          _p(A), float(g_min), _p(S), _p(o), _dtype_code(o), N, H, dk, dv,
                                          float(scale), _stream(stream)), "kda_decode_step_prologue")
    return o


@_on_tensor_device
def chunk_bwd_z(q, k, v, beta, z, A, d_o, dS_out=None, g_min: float = G_MIN, S_in=None, scale: float = 1.0,
                want_dS_in: bool = True, workspace=None, stream=None) -> dict:
    """Backward of ``chunk_fwd_z``: gradients (fp32) of a loss given dL/do (``d_o``)
    and optionally dL/dS_out.  Returns a dict with dq, dk, dv, dbeta, dz, dA and
    dS_in (None unless ``want_dS_in``)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    f32 = torch.float32
    out = {"dq": torch.empty((B, T, H, dk), dtype=f32, device=dev),
           "dk": torch.empty((B, T, H, dk), dtype=f32, device=dev),
           "dv": torch.empty((B, T, H, dv), dtype=f32, device=dev),
           "dbeta": torch.empty((B, T, H), dtype=f32, device=dev),
           "dz": torch.empty((B, T, H, dk), dtype=f32, device=dev),
           "dA": torch.empty((H, dk), dtype=f32, device=dev),
           "dS_in": torch.empty((B, H, dk, dv), dtype=f32, device=dev) if want_dS_in else None}
    need = int(lib().kda_chunk_bwd_z_workspace_bytes(B, T, H, dk, dv))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    _chunk_shapes("kda_chunk_bwd_z", q, k, v, beta, z=z, A=A, S_in=S_in)
    _shapes("kda_chunk_bwd_z", ("q", q, q.shape, _IO), ("d_o", d_o, (B, T, H, dv), _IO),
            ("dS_out", dS_out, (B, H, dk, dv), _F32))
    _dev(q, k, v, beta, z, A, d_o, dS_out, S_in, workspace, *[t for t in out.values() if t is not None])
    _check(lib().kda_chunk_bwd_z(_p(q), _p(k), _p(v), _p(beta), _p(z), _dtype_code(q), _p(A), float(g_min), _p(S_in),
                                 _p(d_o), _dtype_code(d_o), _p(dS_out), _p(out["dq"]), _p(out["dk"]), _p(out["dv"]),
                                 _p(out["dbeta"]), _p(out["dz"]), _p(out["dA"]), _p(out["dS_in"]), B, T, H, dk, dv,
                                 float(scale), _p(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream)), "kda_chunk_bwd_z")
    return out


def chunk_fwd_z_segmented_workspace_bytes(B: int, H: int, dk: int, dv: int, segments: int) -> int:
    """Device bytes the segment-parallel prefill needs for ``segments`` segments."""
    return int(lib().kda_chunk_fwd_z_segmented_workspace_bytes(B, H, dk, dv, int(segments)))


@_on_tensor_device
def chunk_fwd_z_segmented(q, k, v, beta, z, A, segments: int, g_min: float = G_MIN, chunk: int = 64, S_in=None,
                          o=None, S_out=None, o_dtype=None, scale: float = 1.0, want_state: bool = True,
                          workspace=None, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``chunk_fwd_z`` with the sequence cut into ``segments`` chunk-aligned
    segments run in parallel (for small B*H and long T).  ``workspace`` is a
    device tensor of at least ``chunk_fwd_z_segmented_workspace_bytes`` bytes;
    one is allocated when it is None.  Returns (o, S_out or None)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    o, S_out = _outs(q, v, o, S_out, o_dtype, want_state)
    need = chunk_fwd_z_segmented_workspace_bytes(B, H, dk, dv, segments)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _chunk_shapes("kda_chunk_fwd_z_segmented", q, k, v, beta, z=z, A=A, S_in=S_in, o=o, S_out=S_out)
    _dev(q, k, v, beta, z, A, S_in, o, S_out, workspace)
    _check(lib().kda_chunk_fwd_z_segmented(_p(q), _p(k), _p(v), _p(beta), _p(z), _dtype_code(q), _p(A),
                                           float(g_min), _p(S_in), _p(o), _dtype_code(o), _p(S_out), B, T, H, dk,
                                           dv, int(chunk), float(scale), int(segments), _p(workspace),
                                           workspace.numel() * workspace.element_size(), _stream(stream)),
           "kda_chunk_fwd_z_segmented")
    return o, S_out


def _decode_shapes(what, q, k, v, z, beta, A, S, o):
    N, H, dk = q.shape
    dv = v.shape[-1]
    io = (q.dtype,) if q.dtype in _IO else _IO
    _shapes(what, ("q", q, (N, H, dk), _IO), ("k", k, (N, H, dk), io), ("v", v, (N, H, dv), io),
            ("z", z, (N, H, dk), io), ("beta", beta, (N, H), io), ("A", A, (H, dk), _F32),
            ("S", S, (N, H, dk, dv), _F32), ("o", o, (N, H, dv), _IO))


@_on_tensor_device
def decode_step(q, k, v, z, beta, A, S, g_min: float = G_MIN, o=None, o_dtype=None, scale: float = 1.0,
                stream=None) -> torch.Tensor:
    """One token per sequence; S [N,H,dk,dv] fp32 is updated in place.
    Returns o [N,H,dv]."""
    N, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty((N, H, dv), dtype=o_dtype or torch.float32, device=q.device)
    _decode_shapes("kda_decode_step", q, k, v, z, beta, A, S, o)
    _dev(q, k, v, z, beta, A, S, o)
    _check(lib().kda_decode_step(_p(q), _p(k), _p(v), _p(z), _p(beta), _dtype_code(q), _p(A), float(g_min),
                                 _p(S), _p(o), _dtype_code(o), N, H, dk, dv, float(scale), _stream(stream)),
           "kda_decode_step")
    return o


@_on_tensor_device
def decode_replay(q, k, v, z, beta, A, S_snapshot, accepted, g_min: float = G_MIN, o=None, o_dtype=None,
                  S_commit=None, scale: float = 1.0, stream=None):
    """Speculative-decoding replay: the drafted tokens q, k, z [n_draft,N,H,dk],
    v [n_draft,N,H,dv], beta [n_draft,N,H] run from S_snapshot [N,H,dk,dv] fp32
    (left unchanged); accepted [N] int32 holds each sequence's accepted prefix
    length.  Returns (o [n_draft,N,H,dv] for every drafted token, S_commit
    [N,H,dk,dv], the state after the accepted prefix)."""
    n_draft, N, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty((n_draft, N, H, dv), dtype=o_dtype or torch.float32, device=q.device)
    if S_commit is None:
        S_commit = torch.empty_like(S_snapshot)
    io = (q.dtype,) if q.dtype in _IO else _IO
    _shapes("kda_decode_replay", ("q", q, (n_draft, N, H, dk), _IO), ("k", k, (n_draft, N, H, dk), io),
            ("v", v, (n_draft, N, H, dv), io), ("z", z, (n_draft, N, H, dk), io), ("beta", beta, (n_draft, N, H), io),
            ("A", A, (H, dk), _F32), ("S_snapshot", S_snapshot, (N, H, dk, dv), _F32),
            ("accepted", accepted, (N,), (torch.int32,)), ("o", o, (n_draft, N, H, dv), _IO),
            ("S_commit", S_commit, (N, H, dk, dv), _F32))
    _dev(q, k, v, z, beta, A, S_snapshot, accepted, o, S_commit)
    _check(lib().kda_decode_replay(_p(q), _p(k), _p(v), _p(z), _p(beta), _dtype_code(q), _p(A), float(g_min),
                                   _p(S_snapshot), _p(accepted), _p(o), _dtype_code(o), _p(S_commit), n_draft, N,
                                   H, dk, dv, float(scale), _stream(stream)),
           "kda_decode_replay")
    return o, S_commit


# --------------------------------------------------------------------------
# Linear attention with a decay per head, attention over packed prompts and over
# a paged cache in 8 bits.

def _run_on_stream(fn):
    """As ``_on_tensor_device``, and with a ``stream`` argument made current for the call, so that
    outputs and workspaces allocated here belong to the stream that uses them (the allocator
    would otherwise hand their memory on while the call still runs there)."""
    @functools.wraps(fn)
    def wrapper(*args, stream=None, **kwargs):
        t = args[0] if args and isinstance(args[0], torch.Tensor) else next(
            (a for a in (*args, *kwargs.values()) if isinstance(a, torch.Tensor)), None)
        if t is None:
            raise KDAError(f"{fn.__name__}: no tensor given")
        if not t.is_cuda:
            raise KDAError("libkda runs on the GPU only: tensor is on the CPU")
        if stream is None:
            if t.get_device() == torch.cuda.current_device():
                return fn(*args, **kwargs)
            with torch.cuda.device(t.device):
                return fn(*args, **kwargs)
        if stream.device != t.device:
            raise KDAError(f"{fn.__name__}: the stream is on {stream.device}, the tensors on {t.device}")
        with torch.cuda.device(t.device), torch.cuda.stream(stream):
            return fn(*args, **kwargs)
    return wrapper


def _dims(what: str, *specs):
    """specs are (name, tensor, number of dimensions): checked before any shape is unpacked."""
    for name, t, n in specs:
        if not isinstance(t, torch.Tensor) or t.dim() != n:
            raise KDAError(f"{what}: {name} must be a tensor of {n} dimensions")


_MAY_BE_NONE = ("S_in", "S_out", "dS_out", "lse")  # (where one of them is required, the C ABI says so)


def _match(what: str, *specs, like=None):
    """One pass over (name, tensor, shape, allowed dtypes): what ``_shapes`` and ``_dev`` check.  The device is that of
    ``like``, else of the first tensor."""
    dev = None if like is None else like.get_device()
    for name, t, shape, dtypes in specs:
        if not isinstance(t, torch.Tensor):
            if t is None and name in _MAY_BE_NONE:
                continue
            raise KDAError(f"{what}: {name} must be a tensor")
        at = t.get_device()  # (-1: on the CPU)
        if dev is None:
            dev = at
        if at == dev and t.shape == shape and t.dtype in dtypes and at >= 0 and t.is_contiguous():
            continue
        if t.shape != shape:
            raise KDAError(f"{what}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.dtype not in dtypes:
            raise KDAError(f"{what}: {name} has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
        if not t.is_cuda:
            raise KDAError("libkda runs on the GPU only: tensor is on the CPU")
        if not t.is_contiguous():
            raise KDAError(f"{what}: {name} must be contiguous")
        raise KDAError(f"{what}: {name} is on {t.device}, the other tensors on cuda:{dev}")


def _a(t: Optional[torch.Tensor]):
    """A tensor's address, for a call's c_void_p argument."""
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _here(t: torch.Tensor) -> int:
    """The current stream of t's device (current during a call)."""
    if _raw_stream is not None:  # a few times cheaper than building a Stream
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _need(workspace, need: int, device):
    """(address, bytes, tensor) of the caller's workspace, or of a new one of ``need`` bytes."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        _dev(workspace)
        if workspace.device != device:
            raise KDAError(f"the workspace is on {workspace.device}, the tensors on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _out_dtype(dtype, what: str, name: str) -> torch.dtype:
    dtype = dtype or torch.float32
    if dtype not in _IO:
        raise KDAError(f"{what}: {name} is {dtype}, expected {' or '.join(map(str, _IO))}")
    return dtype


def _io_of(t) -> tuple:
    return (t.dtype,) if t.dtype in _IO else _IO


def _linear_shapes(what, q, k, v, g, **more):
    """(B, T, H, dk, dv, g is per head) after every tensor's check; ``more`` maps a name to
    (tensor or None, "o" / "k" / "S" layout, dtypes)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    per_head = isinstance(g, torch.Tensor) and g.dim() == 1
    layouts = {"o": (B, T, H, dv), "k": (B, T, H, dk), "S": (B, H, dk, dv)}
    io = _io_of(q)
    _match(what, ("q", q, (B, T, H, dk), _IO), ("k", k, (B, T, H, dk), io), ("v", v, (B, T, H, dv), io),
           ("g", g, (H,) if per_head else (B, T, H), _F32), *[(n, t, layouts[at], dt) for n, (t, at, dt) in more.items()])
    return B, T, H, dk, dv, per_head


def linear_chunk_fwd_workspace_bytes(B: int, T: int, H: int, dk: int, dv: int, dtype: torch.dtype) -> int:
    """Device bytes ``linear_chunk_fwd`` needs as workspace (0: none) for inputs of ``dtype``."""
    code = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return int(lib().kda_linear_chunk_fwd_workspace_bytes(int(B), int(T), int(H), int(dk), int(dv), code))


@_run_on_stream
def linear_chunk_fwd(q, k, v, g, S_in=None, o=None, S_out=None, o_dtype=None, scale: float = 1.0,
                     want_state: bool = True, workspace=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Linear attention with a decay per head: S_t = e^g S_{t-1} + k v^T, o_t = scale S_t^T q.
    q, k [B,T,H,dk], v [B,T,H,dv]; g fp32 log-decays (at most 0), [B,T,H] or [H].
    Returns (o [B,T,H,dv], S_out [B,H,dk,dv] or None).  bf16 inputs are multiplied in bf16, with an fp32 o
    (the default) too; the state is fp32-accurate.  ``stream``: as everywhere."""
    what = "kda_linear_chunk_fwd"
    _dims(what, ("q", q, 4), ("v", v, 4))
    o, S_out = _outs(q, v, o, S_out, _out_dtype(o_dtype, what, "o_dtype"), want_state)
    B, T, H, dk, dv, ph = _linear_shapes(what, q, k, v, g, S_in=(S_in, "S", _F32), o=(o, "o", _IO),
                                         S_out=(S_out, "S", _F32))
    wp, wb, _keep = _need(workspace, linear_chunk_fwd_workspace_bytes(B, T, H, dk, dv, q.dtype), q.device)
    _check(lib().kda_linear_chunk_fwd(_a(q), _a(k), _a(v), _dtype_code(q), _a(g), int(ph), _a(S_in), _a(o),
                                      _dtype_code(o), _a(S_out), B, T, H, dk, dv, float(scale), wp, wb,
                                      _here(q)), what)
    return o, S_out


def linear_chunk_bwd_workspace_bytes(B: int, T: int, H: int, dk: int, dv: int, dtype: torch.dtype,
                                     g_per_head: bool = False) -> int:
    """Device bytes ``linear_chunk_bwd`` needs as workspace for inputs of ``dtype``."""
    code = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return int(lib().kda_linear_chunk_bwd_workspace_bytes(int(B), int(T), int(H), int(dk), int(dv), code,
                                                          int(bool(g_per_head))))


@_run_on_stream
def linear_chunk_bwd(q, k, v, g, d_o, dS_out=None, S_in=None, scale: float = 1.0, want_dS_in: bool = True,
                     grad_dtype=None, workspace=None) -> dict:
    """Backward of ``linear_chunk_fwd``, given dL/do (``d_o``, the inputs' dtype) and optionally
    dL/dS_out.  Returns a dict with dq, dk, dv (``grad_dtype``, default fp32), dg (fp32, g's shape)
    and dS_in (fp32, None unless ``want_dS_in``)."""
    what = "kda_linear_chunk_bwd"
    grad_dtype = _out_dtype(grad_dtype, what, "grad_dtype")
    _dims(what, ("q", q, 4), ("v", v, 4))
    B, T, H, dk, dv, ph = _linear_shapes(what, q, k, v, g, d_o=(d_o, "o", _io_of(q)), dS_out=(dS_out, "S", _F32),
                                         S_in=(S_in, "S", _F32))
    new = lambda dtype, *shape: torch.empty(shape, dtype=dtype, device=q.device)  # noqa: E731
    out = {"dq": new(grad_dtype, B, T, H, dk), "dk": new(grad_dtype, B, T, H, dk), "dv": new(grad_dtype, B, T, H, dv),
           "dg": torch.empty_like(g), "dS_in": new(torch.float32, B, H, dk, dv) if want_dS_in else None}
    wp, wb, _keep = _need(workspace, linear_chunk_bwd_workspace_bytes(B, T, H, dk, dv, q.dtype, ph), q.device)
    _check(lib().kda_linear_chunk_bwd(_a(q), _a(k), _a(v), _dtype_code(q), _a(g), int(ph), _a(S_in), _a(d_o),
                                      _a(dS_out), _a(out["dq"]), _a(out["dk"]), _a(out["dv"]), _dtype_code(out["dq"]),
                                      _a(out["dg"]), _a(out["dS_in"]), B, T, H, dk, dv, float(scale), wp, wb,
                                      _here(q)), what)
    return out


@_run_on_stream
def linear_decode_step(q, k, v, g, S, o=None, o_dtype=None, scale: float = 1.0,
                       S_out=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """One token per sequence of linear attention with a decay per head: q, k [N,H,dk], v [N,H,dv],
    g [N,H] or [H] fp32.  S [N,H,dk,dv] fp32 is updated in place, or kept when another
    ``S_out`` is given.  Returns (o [N,H,dv], the new state)."""
    what = "kda_linear_decode_step"
    _dims(what, ("q", q, 3), ("v", v, 3), ("S", S, 4))
    N, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty((N, H, dv), dtype=_out_dtype(o_dtype, what, "o_dtype"), device=q.device)
    if S_out is None:
        S_out = S
    ph = isinstance(g, torch.Tensor) and g.dim() == 1
    io = _io_of(q)
    _match(what, ("q", q, (N, H, dk), _IO), ("k", k, (N, H, dk), io), ("v", v, (N, H, dv), io),
           ("g", g, (H,) if ph else (N, H), _F32), ("S", S, (N, H, dk, dv), _F32), ("S_out", S_out, (N, H, dk, dv), _F32),
           ("o", o, (N, H, dv), _IO))
    _check(lib().kda_linear_decode_step(_a(q), _a(k), _a(v), _dtype_code(q), _a(g), int(ph), _a(S), _a(S_out), _a(o),
                                        _dtype_code(o), N, H, dk, dv, float(scale), _here(q)), what)
    return o, S_out


_I32 = (torch.int32,)


def _prompt_shapes(what, q, k, v, cu_seqlens, *more):
    _dims(what, ("q", q, 3), ("k", k, 3), ("cu_seqlens", cu_seqlens, 1))
    n, Hq, d = q.shape
    Hkv = k.shape[1]
    if cu_seqlens.shape[0] < 1:
        raise KDAError(f"{what}: cu_seqlens has no entry (n_seqs + 1 are needed)")
    io = _io_of(q)
    at = {"q": (n, Hq, d), "k": (n, Hkv, d), "l": (n, Hq)}
    _match(what, ("q", q, (n, Hq, d), _IO), ("k", k, (n, Hkv, d), io), ("v", v, (n, Hkv, d), io),
           ("cu_seqlens", cu_seqlens, cu_seqlens.shape, _I32), *[(m, t, at[s], dt) for m, t, s, dt in more])
    return n, cu_seqlens.shape[0] - 1, Hq, Hkv, d


def _softmax_scale(scale, d: int) -> float:
    return float(d) ** -0.5 if scale is None else float(scale)


@_run_on_stream
def attn_prompt_fwd(q, k, v, cu_seqlens, scale: Optional[float] = None, o=None, lse=None, o_dtype=None,
                    want_lse: bool = True) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Causal attention over packed prompts: q [n,Hq,d], k, v [n,Hkv,d], sequence s in rows
    cu_seqlens[s] .. cu_seqlens[s+1] - 1 (int32, on the device).  ``scale`` defaults to 1 / sqrt(d).
    With bf16 inputs probabilities are rounded to bf16, with an fp32 o (the default) too.
    Returns (o [n,Hq,d], lse [n,Hq] fp32 or None).  Rows behind the last sequence are not written:
    given ``o`` and ``lse`` keep what they hold there, new ones are zero there."""
    what = "kda_attn_prompt_fwd"
    _dims(what, ("q", q, 3))
    n, Hq, d = q.shape
    given = o is not None or lse is not None
    if o is None:
        o = (torch.zeros if given else torch.empty)((n, Hq, d), dtype=_out_dtype(o_dtype, what, "o_dtype"), device=q.device)
    if lse is None and want_lse:
        lse = (torch.zeros if given else torch.empty)((n, Hq), dtype=torch.float32, device=q.device)
    n, ns, Hq, Hkv, d = _prompt_shapes(what, q, k, v, cu_seqlens, ("o", o, "q", _IO), ("lse", lse, "l", _F32))
    _check(lib().kda_attn_prompt_fwd(_a(q), _a(k), _a(v), _dtype_code(q), _a(cu_seqlens), _a(o), _dtype_code(o), _a(lse),
                                     n, ns, Hq, Hkv, d, _softmax_scale(scale, d), int(not given), _here(q)), what)
    return o, lse


def attn_prompt_bwd_workspace_bytes(n: int, Hq: int, Hkv: int, d: int) -> int:
    """Device bytes ``attn_prompt_bwd`` needs as workspace for n rows."""
    return int(lib().kda_attn_prompt_bwd_workspace_bytes(int(n), int(Hq), int(Hkv), int(d)))


@_run_on_stream
def attn_prompt_bwd(q, k, v, cu_seqlens, o, lse, d_o, scale: Optional[float] = None, grad_dtype=None,
                    workspace=None) -> dict:
    """Backward of ``attn_prompt_fwd``, from its o and lse and dL/do (``d_o``, the inputs' dtype).
    Returns a dict with dq [n,Hq,d], dk and dv [n,Hkv,d] (``grad_dtype``, default fp32), zero
    in rows behind the last sequence."""
    what = "kda_attn_prompt_bwd"
    grad_dtype = _out_dtype(grad_dtype, what, "grad_dtype")
    n, ns, Hq, Hkv, d = _prompt_shapes(what, q, k, v, cu_seqlens, ("o", o, "q", _IO), ("lse", lse, "l", _F32),
                                       ("d_o", d_o, "q", _io_of(q)))
    out = {"dq": torch.empty((n, Hq, d), dtype=grad_dtype, device=q.device),
           "dk": torch.empty((n, Hkv, d), dtype=grad_dtype, device=q.device),
           "dv": torch.empty((n, Hkv, d), dtype=grad_dtype, device=q.device)}
    wp, wb, _keep = _need(workspace, attn_prompt_bwd_workspace_bytes(n, Hq, Hkv, d), q.device)
    _check(lib().kda_attn_prompt_bwd(_a(q), _a(k), _a(v), _dtype_code(q), _a(cu_seqlens), _a(o), _dtype_code(o), _a(lse),
                                     _a(d_o), _a(out["dq"]), _a(out["dk"]), _a(out["dv"]), _dtype_code(out["dq"]), n, ns,
                                     Hq, Hkv, d, _softmax_scale(scale, d), 1, wp, wb, _here(q)), what)
    return out


def _rows(what: str, name: str, t, shape, dtypes, like) -> int:
    """Checks a tensor [n, H, d] whose rows may lie apart (a view of a projection's output), each
    row's heads together, on ``like``'s device; its row stride in elements."""
    if not isinstance(t, torch.Tensor) or t.shape != shape:
        raise KDAError(f"{what}: {name} must be a tensor of shape {tuple(shape)}")
    if t.dtype not in dtypes:
        raise KDAError(f"{what}: {name} has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    at = t.get_device()
    if at < 0:
        raise KDAError("libkda runs on the GPU only: tensor is on the CPU")
    if at != like.get_device():
        raise KDAError(f"{what}: {name} is on {t.device}, the other tensors on {like.device}")
    n, H, d = shape
    row, head, one = t.stride()
    if n <= 1 or H * d == 0:
        row = H * d
    if (one != 1 and d > 1) or (head != d and H > 1) or row < H * d:
        if t.numel():
            raise KDAError(f"{what}: {name} has strides {t.stride()}: a row's {H} heads of {d} must lie together")
    return row


def _turn(what: str, n: int, positions, inv_freq, axes):
    """A rotation's number of axes, its pairs, and the specs of its tensors for ``_match``."""
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise KDAError(f"{what}: inv_freq must be a tensor of 1 dimensions")
    half, A = inv_freq.shape[0], 1
    specs = [("inv_freq", inv_freq, (half,), _F32)]
    if positions is not None:
        if not isinstance(positions, torch.Tensor) or positions.dim() not in (1, 2):
            raise KDAError(f"{what}: positions must be a tensor [n] or [n, axes]")
        if positions.dim() == 1:
            specs.append(("positions", positions, (n,), _I32))
        else:
            A = positions.shape[1]
            specs.append(("positions", positions, (n, A), _I32))
    if axes is not None:
        specs.append(("axes", axes, (half,), _I32))
    return A, half, specs


@_run_on_stream
def rope(x, positions, inv_freq, axes=None, interleaved: bool = False, inverse: bool = False, out=None,
         out_dtype=None) -> torch.Tensor:
    """Rotary positions: pair j of every head's channels of x [n,H,d] turns by
    positions[row, axes[j]] * inv_freq[j].  positions [n] or [n,axes] int32, inv_freq [rot/2] fp32 (channels from
    rot on are copied), axes [rot/2] int32 or None (all of axis 0); pairs are (j, j + rot/2), or (2j, 2j + 1) where
    ``interleaved``.  ``inverse`` turns backwards: the gradient, dx from dy.  x may be a view whose rows lie apart; so may
    ``out``, which may be x itself.  Returns y [n,H,d] (``out_dtype``, default x's)."""
    what = "kda_rope"
    _dims(what, ("x", x, 3))
    n, H, d = x.shape
    xs = _rows(what, "x", x, (n, H, d), _IO, x)
    if out is None:
        out = torch.empty((n, H, d), dtype=_out_dtype(out_dtype or x.dtype, what, "out_dtype"), device=x.device)
        ys = H * d
    else:
        ys = _rows(what, "out", out, (n, H, d), _IO, x)
    if positions is None:
        raise KDAError(f"{what}: positions must be a tensor [n] or [n, axes]")
    A, half, specs = _turn(what, n, positions, inv_freq, axes)
    _match(what, *specs, like=x)
    _check(lib().kda_rope(x.data_ptr(), _dtype_code(x), xs, positions.data_ptr(), A, inv_freq.data_ptr(), _a(axes), 2 * half,
                          int(bool(interleaved)), int(bool(inverse)), out.data_ptr(), _dtype_code(out), ys, n, H, d, _here(x)), what)
    return out


_F8 = (torch.float8_e4m3fn,)


def _cache_shapes(what, Hkv, d, k_cache, v_cache, k_scale, v_scale, block_table, context_len, *more, like=None):
    _dims(what, ("k_cache", k_cache, 4), ("block_table", block_table, 2))
    pages, _, page, _ = k_cache.shape
    N, max_pages = block_table.shape
    _match(what, *more, ("k_cache", k_cache, (pages, Hkv, page, d), _F8), ("v_cache", v_cache, (pages, Hkv, d, page), _F8),
           ("k_scale", k_scale, (pages, Hkv), _F32), ("v_scale", v_scale, (pages, Hkv), _F32),
           ("block_table", block_table, (N, max_pages), _I32), ("context_len", context_len, (N,), _I32), like=like)
    return N, page, pages, max_pages


@_run_on_stream
def kv_cache_append(k, v, cu_seqlens, context_len, block_table, k_cache, v_cache, k_scale, v_scale) -> None:
    """Quantise new tokens into a paged cache, in place: k, v [n,Hkv,d], rows
    cu_seqlens[i] .. cu_seqlens[i+1] - 1 behind the context_len[i] tokens that sequence i holds.
    k_cache [pages,Hkv,page,d] and v_cache [pages,Hkv,d,page] float8_e4m3fn, k_scale and v_scale
    [pages,Hkv] fp32, block_table [N,max_pages] int32.  context_len is not changed."""
    what = "kda_kv_cache_append"
    _dims(what, ("k", k, 3), ("cu_seqlens", cu_seqlens, 1), ("context_len", context_len, 1))
    n, Hkv, d = k.shape
    N, page, pages, mp = _cache_shapes(what, Hkv, d, k_cache, v_cache, k_scale, v_scale, block_table, context_len,
                                       ("k", k, (n, Hkv, d), _IO), ("v", v, (n, Hkv, d), _io_of(k)),
                                       ("cu_seqlens", cu_seqlens, (context_len.shape[0] + 1,), _I32))
    _check(lib().kda_kv_cache_append(_a(k), _a(v), _dtype_code(k), _a(cu_seqlens), _a(context_len), _a(block_table),
                                     _a(k_cache), _a(v_cache), _a(k_scale), _a(v_scale), n, N, Hkv, d, page, pages, mp,
                                     _here(k)), what)


@_run_on_stream
def kv_cache_append_rope(k, v, cu_seqlens, context_len, block_table, k_cache, v_cache, k_scale, v_scale, inv_freq,
                         positions=None, axes=None, interleaved: bool = False, q=None, q_out=None,
                         q_out_dtype=None) -> Optional[torch.Tensor]:
    """``kv_cache_append`` with rotary positions (``rope``) applied to k on the way, and to the same tokens'
    queries q [n,Hq,d] if given, in one launch.  ``positions`` [n] or [n,axes] int32; None: each token's place in its
    sequence.  k, v and q may be views whose rows lie apart (of one projection's output); ``q_out`` too, and it may be q.
    Returns the turned queries (``q_out_dtype``, default q's), or None without q.  Rows behind the last
    sequence: a given ``q_out`` keeps what it holds there, a new one is zero there."""
    what = "kda_kv_cache_append_rope"
    _dims(what, ("k", k, 3), ("context_len", context_len, 1))
    n, Hkv, d = k.shape
    k_row, v_row = _rows(what, "k", k, (n, Hkv, d), _IO, k), _rows(what, "v", v, (n, Hkv, d), _io_of(k), k)
    given, Hq, q_row, o_row, o_code = q_out is not None, Hkv, Hkv * d, Hkv * d, _dtype_code(k)
    if q is not None:
        _dims(what, ("q", q, 3))
        Hq = q.shape[1]
        q_row = _rows(what, "q", q, (n, Hq, d), _io_of(k), k)
        if given:
            o_row = _rows(what, "q_out", q_out, (n, Hq, d), _IO, k)
        else:
            q_out = torch.empty((n, Hq, d), dtype=_out_dtype(q_out_dtype or q.dtype, what, "q_out_dtype"), device=q.device)
            o_row = Hq * d
        o_code = _dtype_code(q_out)
    elif given:
        raise KDAError(f"{what}: q_out without q")
    A, half, specs = _turn(what, n, positions, inv_freq, axes)
    N, page, pages, mp = _cache_shapes(what, Hkv, d, k_cache, v_cache, k_scale, v_scale, block_table, context_len, *specs,
                                       ("cu_seqlens", cu_seqlens, (context_len.shape[0] + 1,), _I32), like=k)
    _check(lib().kda_kv_cache_append_rope(k.data_ptr(), k_row, v.data_ptr(), v_row, _dtype_code(k), _a(q), q_row, _a(q_out),
                                          o_code, o_row, _a(positions), A, inv_freq.data_ptr(), _a(axes), 2 * half,
                                          int(bool(interleaved)), cu_seqlens.data_ptr(), context_len.data_ptr(),
                                          block_table.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                                          v_scale.data_ptr(), n, N, Hq, Hkv, d, page, pages, mp, int(not given), _here(k)), what)
    return q_out


def attn_decode_step_workspace_bytes(N: int, Hq: int, Hkv: int, d: int, page: int, max_pages: int) -> int:
    """Device bytes ``attn_decode_step`` needs as workspace (0: none)."""
    return int(lib().kda_attn_decode_step_workspace_bytes(int(N), int(Hq), int(Hkv), int(d), int(page), int(max_pages)))


@_run_on_stream
def attn_decode_step(q, k_cache, v_cache, k_scale, v_scale, block_table, context_len, scale: Optional[float] = None,
                     o=None, lse=None, o_dtype=None, want_lse: bool = False,
                     workspace=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Attention of one token per sequence over a paged cache in 8 bits (``kv_cache_append``):
    q [N,Hq,d].  ``scale`` defaults to 1 / sqrt(d).  bf16 queries' probabilities are rounded to bf16.  Returns (o [N,Hq,d], lse [N,Hq] fp32 or
    None); a sequence with no tokens gets o = 0, lse = -inf."""
    what = "kda_attn_decode_step"
    _dims(what, ("q", q, 3), ("k_cache", k_cache, 4))
    N, Hq, d = q.shape
    Hkv = k_cache.shape[1]
    if o is None:
        o = torch.empty((N, Hq, d), dtype=_out_dtype(o_dtype, what, "o_dtype"), device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((N, Hq), dtype=torch.float32, device=q.device)
    Nt, page, pages, mp = _cache_shapes(what, Hkv, d, k_cache, v_cache, k_scale, v_scale, block_table, context_len,
                                        ("q", q, (N, Hq, d), _IO), ("o", o, (N, Hq, d), _IO),
                                        ("lse", lse, (N, Hq), _F32))
    if Nt != N:
        raise KDAError(f"{what}: block_table has {Nt} rows, q {N}")
    wp, wb, _keep = _need(workspace, attn_decode_step_workspace_bytes(N, Hq, Hkv, d, page, mp), q.device)
    _check(lib().kda_attn_decode_step(_a(q), _dtype_code(q), _a(k_cache), _a(v_cache), _a(k_scale), _a(v_scale),
                                      _a(block_table), _a(context_len), _a(o), _dtype_code(o), _a(lse), N, Hq, Hkv, d,
                                      page, pages, mp, _softmax_scale(scale, d), wp, wb, _here(q)), what)
    return o, lse


def attn_chunk_fwd_workspace_bytes(n: int, N: int, Hq: int, Hkv: int, d: int, page: int, max_pages: int,
                                   dtype: torch.dtype) -> int:
    """Device bytes ``attn_chunk_fwd`` needs as workspace (0: none) for queries of ``dtype``."""
    code = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return int(lib().kda_attn_chunk_fwd_workspace_bytes(int(n), int(N), int(Hq), int(Hkv), int(d), int(page), int(max_pages),
                                                        code))


@_run_on_stream
def attn_chunk_fwd(q, cu_seqlens, k_cache, v_cache, k_scale, v_scale, block_table, context_len,
                   scale: Optional[float] = None, o=None, lse=None, o_dtype=None, want_lse: bool = False,
                   workspace=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Attention of each sequence's new tokens over a paged cache in 8 bits that holds them already
    (``kv_cache_append``): rows cu_seqlens[i] .. cu_seqlens[i+1] - 1 of q [n,Hq,d] are the last of sequence i's
    context_len[i] tokens, each sees itself and what lies before it.  q may be a view whose rows lie apart.  ``scale``
    defaults to 1 / sqrt(d).  bf16 queries' probabilities are rounded to bf16.  Returns (o [n,Hq,d], lse [n,Hq]
    fp32 or None); a row that sees no token gets o = 0, lse = -inf.  Rows behind the last sequence: given
    ``o`` and ``lse`` keep what they hold there, new ones are zero there."""
    what = "kda_attn_chunk_fwd"
    _dims(what, ("q", q, 3), ("context_len", context_len, 1), ("k_cache", k_cache, 4))
    n, Hq, d = q.shape
    Hkv = k_cache.shape[1]
    q_row = _rows(what, "q", q, (n, Hq, d), _IO, q)
    given, specs = o is not None or lse is not None, []
    if o is not None:
        specs.append(("o", o, (n, Hq, d), _IO))
    else:
        o = (torch.zeros if given else torch.empty)((n, Hq, d), dtype=_out_dtype(o_dtype, what, "o_dtype"), device=q.device)
    if lse is not None:
        specs.append(("lse", lse, (n, Hq), _F32))
    elif want_lse:
        lse = (torch.zeros if given else torch.empty)((n, Hq), dtype=torch.float32, device=q.device)
    N, page, pages, mp = _cache_shapes(what, Hkv, d, k_cache, v_cache, k_scale, v_scale, block_table, context_len, *specs,
                                       ("cu_seqlens", cu_seqlens, (context_len.shape[0] + 1,), _I32), like=q)
    need = lib().kda_attn_chunk_fwd_workspace_bytes(n, N, Hq, Hkv, d, page, mp, _dtype_code(q)) if pages and Hkv else 0
    wp, wb, _keep = _need(workspace, need, q.device)
    _check(lib().kda_attn_chunk_fwd(q.data_ptr(), q_row, _dtype_code(q), cu_seqlens.data_ptr(), k_cache.data_ptr(),
                                    v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(),
                                    context_len.data_ptr(), o.data_ptr(), _dtype_code(o), _a(lse), n, N, Hq, Hkv, d, page,
                                    pages, mp, _softmax_scale(scale, d), int(not given), wp, wb, _here(q)), what)
    return o, lse
