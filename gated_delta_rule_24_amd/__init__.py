"""gated_delta_rule_24_amd — Python binding of libgdr (gated delta rule on MI355X).

Thin ctypes marshalling over the C ABI declared in ``include/gdr.h``: every
step of the computation runs in the HIP kernels of ``libgdr.so``; PyTorch is
used only for device memory and the current stream.  There is no CPU or
PyTorch fallback: if the library is missing or the device is not a gfx950,
calls raise.

The entry points keep the C names:

* :func:`gdr_chunk_fwd`   — chunkwise-parallel forward
* :func:`gdr_decode_step` — one recurrent decode step, state updated in place
* :func:`gdr_chunk_bwd`   — gate-aware backward
* :func:`gdr_chunk_fwd_varlen`, :func:`gdr_chunk_bwd_varlen` — the forward
  and backward over packed variable-length sequences

* :func:`gdr_rope`, :func:`gdr_attn_fwd`, :func:`gdr_attn_bwd` (and their
  packed forms) — the attention layers a hybrid stack puts between recurrent
  ones: rotary positions, causal attention over a window or the whole past
* :func:`gdr_kv_append`, :func:`gdr_attn_decode` — that layer's 8-bit paged
  cache and its attention for one token

and :func:`chunk_fwd`, :func:`decode_step`, :func:`chunk_bwd`,
:func:`chunk_fwd_varlen`, :func:`chunk_bwd_varlen`, :func:`rope`,
:func:`attn_fwd`, :func:`attn_bwd`, :func:`attn_fwd_varlen`,
:func:`attn_bwd_varlen`, :func:`kv_append`, :func:`attn_decode` are the same
calls with outputs allocated for the caller.

Tensors are contiguous and start at a multiple of 16 bytes, int32 ones as well
(a slice of a longer tensor may not).
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import math
import os
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdr.so")

GDR_ACT_BF16 = 0x0
GDR_ACT_F32 = 0x1
GDR_OUT_BF16 = 0x2
GDR_ALPHA_SCALAR = 0x4
GDR_B_SCALAR = 0x8
GDR_W_SCALAR = 0x10
GDR_FWD_GENERIC = 0x20
GDR_GATE_LOGITS = 0x40
GDR_FWD_SPLIT = 0x80
GDR_TOKEN_MAJOR = 0x1000
GDR_ROPE_INTERLEAVED = 0x2000
GDR_ROPE_INVERSE = 0x4000

# tokens of a cache page
GDR_KV_PAGE = 64

_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "workspace", 4: "launch", 5: "device"}

_lib = None


class GdrError(RuntimeError):
    def __init__(self, fn: str, status: int, why: str = ""):
        self.status = status
        msg = _load().gdr_status_string(status).decode() if _lib is not None else _STATUS.get(status)
        super().__init__(f"{fn} failed with status {status} ({msg}{why and ': ' + why})")


def _load():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libgdr.so not found at {LIB_PATH}; build it with "
                "`python -m gated_delta_rule_24_amd.build` (no fallback path exists)")
        lib = ctypes.CDLL(LIB_PATH)
        P, I, U, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint32, ctypes.c_size_t
        lib.gdr_abi_version.restype = I
        lib.gdr_status_string.argtypes = [I]
        lib.gdr_status_string.restype = ctypes.c_char_p
        lib.gdr_chunk_fwd_workspace_bytes.argtypes = [I] * 6 + [U]
        lib.gdr_chunk_fwd_workspace_bytes.restype = S
        lib.gdr_chunk_fwd.argtypes = [P] * 9 + [I] * 6 + [U, P, S, P]
        lib.gdr_chunk_fwd.restype = I
        lib.gdr_chunk_fwd_noalloc.argtypes = [P] * 9 + [I] * 6 + [U, P]
        lib.gdr_chunk_fwd_noalloc.restype = I
        lib.gdr_chunk_fwd_varlen_workspace_bytes.argtypes = [I] * 5 + [U]
        lib.gdr_chunk_fwd_varlen_workspace_bytes.restype = S
        lib.gdr_chunk_fwd_varlen.argtypes = [P] * 10 + [I] * 5 + [U, P, S, P]
        lib.gdr_chunk_fwd_varlen.restype = I
        lib.gdr_decode_step.argtypes = [P] * 8 + [I] * 4 + [U, P]
        lib.gdr_decode_step.restype = I
        lib.gdr_chunk_bwd_workspace_bytes.argtypes = [I] * 6 + [U]
        lib.gdr_chunk_bwd_workspace_bytes.restype = S
        lib.gdr_chunk_bwd.argtypes = [P] * 16 + [I] * 6 + [U, P, S, P]
        lib.gdr_chunk_bwd.restype = I
        lib.gdr_chunk_bwd_varlen_workspace_bytes.argtypes = [I] * 5 + [U]
        lib.gdr_chunk_bwd_varlen_workspace_bytes.restype = S
        lib.gdr_chunk_bwd_varlen.argtypes = [P] * 17 + [I] * 5 + [U, P, S, P]
        lib.gdr_chunk_bwd_varlen.restype = I
        lib.gdr_mixer_prologue.argtypes = [P] * 15 + [I] * 5 + [U, P]
        lib.gdr_mixer_prologue.restype = I
        lib.gdr_mixer_epilogue.argtypes = [P] * 4 + [I] * 4 + [U, P]
        lib.gdr_mixer_epilogue.restype = I
        lib.gdr_mixer_bwd_workspace_bytes.argtypes = [I] * 5
        lib.gdr_mixer_bwd_workspace_bytes.restype = S
        lib.gdr_mixer_prologue_bwd.argtypes = [P] * 15 + [I] * 5 + [U, P, S, P]
        lib.gdr_mixer_prologue_bwd.restype = I
        lib.gdr_mixer_epilogue_bwd.argtypes = [P] * 7 + [I] * 4 + [U, P, S, P]
        lib.gdr_mixer_epilogue_bwd.restype = I
        F = ctypes.c_float
        lib.gdr_rope.argtypes = [P] * 6 + [I] * 7 + [F, U, P]
        lib.gdr_rope.restype = I
        lib.gdr_attn_fwd.argtypes = [P] * 5 + [I] * 7 + [F, U, P]
        lib.gdr_attn_fwd.restype = I
        lib.gdr_attn_fwd_varlen.argtypes = [P] * 6 + [I] * 6 + [F, U, P]
        lib.gdr_attn_fwd_varlen.restype = I
        lib.gdr_attn_bwd_workspace_bytes.argtypes = [I] * 6
        lib.gdr_attn_bwd_workspace_bytes.restype = S
        lib.gdr_attn_bwd.argtypes = [P] * 9 + [I] * 7 + [F, U, P, S, P]
        lib.gdr_attn_bwd.restype = I
        lib.gdr_attn_bwd_varlen.argtypes = [P] * 10 + [I] * 6 + [F, U, P, S, P]
        lib.gdr_attn_bwd_varlen.restype = I
        lib.gdr_kv_append.argtypes = [P] * 9 + [I] * 6 + [U, P]
        lib.gdr_kv_append.restype = I
        lib.gdr_attn_decode_workspace_bytes.argtypes = [I] * 6
        lib.gdr_attn_decode_workspace_bytes.restype = S
        lib.gdr_attn_decode.argtypes = [P] * 8 + [I] * 7 + [F, U, P, S, P]
        lib.gdr_attn_decode.restype = I
        _lib = lib
    return _lib


def lib():
    """The loaded ctypes library (raises if it is not built)."""
    return _load()


EXPORTED_SYMBOLS = ("gdr_abi_version", "gdr_status_string", "gdr_chunk_fwd_workspace_bytes",
                    "gdr_chunk_fwd", "gdr_chunk_fwd_noalloc", "gdr_chunk_fwd_varlen_workspace_bytes", "gdr_chunk_fwd_varlen",
                    "gdr_decode_step", "gdr_chunk_bwd_workspace_bytes", "gdr_chunk_bwd",
                    "gdr_chunk_bwd_varlen_workspace_bytes", "gdr_chunk_bwd_varlen",
                    "gdr_mixer_prologue", "gdr_mixer_epilogue", "gdr_mixer_bwd_workspace_bytes",
                    "gdr_mixer_prologue_bwd", "gdr_mixer_epilogue_bwd", "gdr_rope", "gdr_attn_fwd",
                    "gdr_attn_fwd_varlen", "gdr_attn_bwd_workspace_bytes", "gdr_attn_bwd", "gdr_attn_bwd_varlen",
                    "gdr_kv_append", "gdr_attn_decode_workspace_bytes", "gdr_attn_decode")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _act_flag(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GDR_ACT_BF16
    if t.dtype == torch.float32:
        return GDR_ACT_F32
    raise ValueError(f"activation dtype must be bfloat16 or float32, got {t.dtype}")


def gate_flags(q, log_alpha, b, w, gate_logits: bool = False) -> int:
    """Flags for the dtype and gate modes implied by tensor ranks (gate_logits:
    log_alpha, b and w hold logits, see GDR_GATE_LOGITS)."""
    f = _act_flag(q) | (GDR_GATE_LOGITS if gate_logits else 0)
    if log_alpha.dim() == q.dim() - 1:
        f |= GDR_ALPHA_SCALAR
    if b.dim() == q.dim() - 1:
        f |= GDR_B_SCALAR
    if w.dim() == q.dim() - 1:
        f |= GDR_W_SCALAR
    return f


def _check(fn, st):
    if st != 0:
        raise GdrError(fn, st)


def _window(window):
    """A window as the library counts it, in 32 bits (ctypes would keep the low ones without
    a word): one past every length is none, one below 0 stays invalid."""
    return window if -1 < window < 1 << 31 else 0 if window > 0 else -1


def _position(position0):
    if not -(1 << 31) <= position0 < 1 << 31:
        raise ValueError(f"position0 must fit 32 bits, got {position0}")
    return position0


# ---------------------------------------------------------------------------
# C-named entry points (outputs provided by the caller)
# ---------------------------------------------------------------------------


def gdr_chunk_fwd_workspace_bytes(B, H, T, d_k, d_v, chunk, flags) -> int:
    return int(_load().gdr_chunk_fwd_workspace_bytes(B, H, T, d_k, d_v, chunk, flags))


def gdr_chunk_fwd(q, k, v, log_alpha, b, w, S0, o, S_final, B, H, T, d_k, d_v, chunk,
                  flags, workspace=None, workspace_bytes=0, stream=None):
    st = _load().gdr_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w),
                               _ptr(S0), _ptr(o), _ptr(S_final), B, H, T, d_k, d_v, chunk,
                               flags, _ptr(workspace), workspace_bytes, _stream(stream))
    _check("gdr_chunk_fwd", st)


# bytes of the library-owned device array gdr_chunk_fwd_noalloc uses per GPU
GDR_NOALLOC_SCRATCH_BYTES = 64 << 20


def gdr_chunk_fwd_noalloc(q, k, v, log_alpha, b, w, S0, o, S_final, B, H, T, d_k, d_v, chunk,
                          flags, stream=None):
    st = _load().gdr_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b),
                                       _ptr(w), _ptr(S0), _ptr(o), _ptr(S_final), B, H, T, d_k, d_v,
                                       chunk, flags, _stream(stream))
    _check("gdr_chunk_fwd_noalloc", st)


def gdr_chunk_fwd_varlen_workspace_bytes(nseq, H, T, d_k, d_v, flags) -> int:
    return int(_load().gdr_chunk_fwd_varlen_workspace_bytes(nseq, H, T, d_k, d_v, flags))


def gdr_chunk_fwd_varlen(q, k, v, log_alpha, b, w, S0, o, S_final, cu_seqlens, nseq, H, T, d_k,
                         d_v, flags, workspace, workspace_bytes, stream=None):
    st = _load().gdr_chunk_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b),
                                      _ptr(w), _ptr(S0), _ptr(o), _ptr(S_final),
                                      _ptr(cu_seqlens), nseq, H, T, d_k, d_v, flags,
                                      _ptr(workspace), workspace_bytes, _stream(stream))
    _check("gdr_chunk_fwd_varlen", st)


def gdr_decode_step(q, k, v, log_alpha, b, w, S, o, N, H, d_k, d_v, flags, stream=None):
    st = _load().gdr_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w),
                                 _ptr(S), _ptr(o), N, H, d_k, d_v, flags, _stream(stream))
    _check("gdr_decode_step", st)


def gdr_chunk_bwd_workspace_bytes(B, H, T, d_k, d_v, chunk, flags) -> int:
    return int(_load().gdr_chunk_bwd_workspace_bytes(B, H, T, d_k, d_v, chunk, flags))


def gdr_chunk_bwd(q, k, v, log_alpha, b, w, S0, dO, dS_final, dq, dk, dv, dlog_alpha, db, dw,
                  dS0, B, H, T, d_k, d_v, chunk, flags, workspace, workspace_bytes,
                  stream=None):
    st = _load().gdr_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w),
                               _ptr(S0), _ptr(dO), _ptr(dS_final), _ptr(dq), _ptr(dk), _ptr(dv),
                               _ptr(dlog_alpha), _ptr(db), _ptr(dw), _ptr(dS0), B, H, T, d_k,
                               d_v, chunk, flags, _ptr(workspace), workspace_bytes,
                               _stream(stream))
    _check("gdr_chunk_bwd", st)


def gdr_chunk_bwd_varlen_workspace_bytes(nseq, H, T, d_k, d_v, flags) -> int:
    return int(_load().gdr_chunk_bwd_varlen_workspace_bytes(nseq, H, T, d_k, d_v, flags))


def gdr_chunk_bwd_varlen(q, k, v, log_alpha, b, w, S0, dO, dS_final, dq, dk, dv, dlog_alpha, db,
                         dw, dS0, cu_seqlens, nseq, H, T, d_k, d_v, flags, workspace,
                         workspace_bytes, stream=None):
    st = _load().gdr_chunk_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b),
                                      _ptr(w), _ptr(S0), _ptr(dO), _ptr(dS_final), _ptr(dq),
                                      _ptr(dk), _ptr(dv), _ptr(dlog_alpha), _ptr(db), _ptr(dw),
                                      _ptr(dS0), _ptr(cu_seqlens), nseq, H, T, d_k, d_v, flags,
                                      _ptr(workspace), workspace_bytes, _stream(stream))
    _check("gdr_chunk_bwd_varlen", st)


def gdr_mixer_prologue(q_pre, k_pre, v_pre, conv_q, conv_k, conv_v, a_pre, b_pre, w_pre, q, k, v,
                       log_alpha, b, w, B, H, T, d_k, d_v, flags, stream=None):
    st = _load().gdr_mixer_prologue(_ptr(q_pre), _ptr(k_pre), _ptr(v_pre), _ptr(conv_q),
                                    _ptr(conv_k), _ptr(conv_v), _ptr(a_pre), _ptr(b_pre),
                                    _ptr(w_pre), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                    _ptr(b), _ptr(w), B, H, T, d_k, d_v, flags, _stream(stream))
    _check("gdr_mixer_prologue", st)


def gdr_mixer_epilogue(o, g, norm_weight, y, B, H, T, d_v, flags=0, stream=None):
    st = _load().gdr_mixer_epilogue(_ptr(o), _ptr(g), _ptr(norm_weight), _ptr(y), B, H, T, d_v,
                                    flags, _stream(stream))
    _check("gdr_mixer_epilogue", st)


def gdr_mixer_bwd_workspace_bytes(B, H, T, d_k, d_v) -> int:
    return int(_load().gdr_mixer_bwd_workspace_bytes(B, H, T, d_k, d_v))


def gdr_mixer_prologue_bwd(q_pre, k_pre, v_pre, conv_q, conv_k, conv_v, dq, dk, dv, dq_pre, dk_pre,
                           dv_pre, dconv_q, dconv_k, dconv_v, B, H, T, d_k, d_v, flags, workspace,
                           workspace_bytes, stream=None):
    st = _load().gdr_mixer_prologue_bwd(*[_ptr(x) for x in (q_pre, k_pre, v_pre, conv_q, conv_k,
                                                            conv_v, dq, dk, dv, dq_pre, dk_pre,
                                                            dv_pre, dconv_q, dconv_k, dconv_v)],
                                        B, H, T, d_k, d_v, flags, _ptr(workspace), workspace_bytes,
                                        _stream(stream))
    _check("gdr_mixer_prologue_bwd", st)


def gdr_mixer_epilogue_bwd(o, g, norm_weight, dy, d_o, dg, dnorm_weight, B, H, T, d_v, flags,
                           workspace, workspace_bytes, stream=None):
    st = _load().gdr_mixer_epilogue_bwd(_ptr(o), _ptr(g), _ptr(norm_weight), _ptr(dy), _ptr(d_o),
                                        _ptr(dg), _ptr(dnorm_weight), B, H, T, d_v, flags,
                                        _ptr(workspace), workspace_bytes, _stream(stream))
    _check("gdr_mixer_epilogue_bwd", st)


def gdr_rope(q, k, q_out, k_out, inv_freq, positions, position0, B, Hq, Hk, T, d, rot_dim, scale, flags,
             stream=None):
    st = _load().gdr_rope(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), _ptr(inv_freq), _ptr(positions),
                          _position(position0), B, Hq, Hk, T, d, rot_dim, scale, flags, _stream(stream))
    _check("gdr_rope", st)


def gdr_attn_fwd(q, k, v, o, lse, B, Hq, Hkv, Tq, Tk, d, window, scale, flags, stream=None):
    st = _load().gdr_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Tq, Tk, d,
                              _window(window), scale, flags, _stream(stream))
    _check("gdr_attn_fwd", st)


def gdr_attn_fwd_varlen(q, k, v, o, lse, cu_seqlens, nseq, Hq, Hkv, T, d, window, scale, flags, stream=None):
    st = _load().gdr_attn_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_seqlens), nseq, Hq,
                                     Hkv, T, d, _window(window), scale, flags, _stream(stream))
    _check("gdr_attn_fwd_varlen", st)


def gdr_attn_bwd_workspace_bytes(B, Hq, Hkv, Tq, Tk, d) -> int:
    return int(_load().gdr_attn_bwd_workspace_bytes(B, Hq, Hkv, Tq, Tk, d))


def gdr_attn_bwd(q, k, v, o, lse, dO, dq, dk, dv, B, Hq, Hkv, Tq, Tk, d, window, scale, flags, workspace,
                 workspace_bytes, stream=None):
    st = _load().gdr_attn_bwd(*[_ptr(x) for x in (q, k, v, o, lse, dO, dq, dk, dv)], B, Hq, Hkv, Tq, Tk, d,
                              _window(window), scale, flags, _ptr(workspace), workspace_bytes, _stream(stream))
    _check("gdr_attn_bwd", st)


def gdr_attn_bwd_varlen(q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens, nseq, Hq, Hkv, T, d, window, scale, flags,
                        workspace, workspace_bytes, stream=None):
    st = _load().gdr_attn_bwd_varlen(*[_ptr(x) for x in (q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens)], nseq, Hq,
                                     Hkv, T, d, _window(window), scale, flags, _ptr(workspace), workspace_bytes,
                                     _stream(stream))
    _check("gdr_attn_bwd_varlen", st)


def gdr_kv_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, cache_len, cu_seqlens, nseq, Hkv, T, d,
                  n_pages, max_pages, flags=0, stream=None):
    st = _load().gdr_kv_append(*[_ptr(x) for x in (k, v, k_cache, v_cache, k_scale, v_scale, block_table, cache_len,
                                                   cu_seqlens)], nseq, Hkv, T, d, n_pages, max_pages, flags,
                               _stream(stream))
    _check("gdr_kv_append", st)


def gdr_attn_decode_workspace_bytes(N, Hq, Hkv, d, max_pages, window) -> int:
    return int(_load().gdr_attn_decode_workspace_bytes(N, Hq, Hkv, d, max_pages, _window(window)))


def gdr_attn_decode(q, k_cache, v_cache, k_scale, v_scale, block_table, cache_len, o, N, Hq, Hkv, d, n_pages,
                    max_pages, window, scale, flags, workspace=None, workspace_bytes=0, stream=None):
    st = _load().gdr_attn_decode(*[_ptr(x) for x in (q, k_cache, v_cache, k_scale, v_scale, block_table, cache_len,
                                                     o)], N, Hq, Hkv, d, n_pages, max_pages, _window(window), scale, flags,
                                 _ptr(workspace), workspace_bytes, _stream(stream))
    _check("gdr_attn_decode", st)


# ---------------------------------------------------------------------------
# convenience wrappers (allocate outputs with torch)
# ---------------------------------------------------------------------------


def _on_its_stream(fn):
    """A call given a `stream` that is not the current one runs with it current, so that
    its outputs and workspaces are allocated there: the allocator hands memory out in
    the order of the stream it is asked on, and another one may still be writing it.
    What is returned is kept for the caller's stream as well, which goes on with it.  That
    the inputs are ready on `stream`, and the results before they are used elsewhere, is
    the caller's to see to."""
    at = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def call(*args, **kw):
        stream = kw.get("stream") if len(args) <= at else args[at]
        if stream is None:
            return fn(*args, **kw)
        caller = torch.cuda.current_stream(stream.device)
        if stream == caller:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            out = fn(*args, **kw)
        for t in (out,) if isinstance(out, torch.Tensor) else out.values() if isinstance(out, dict) else out:
            if t is not None:
                t.record_stream(caller)
        return out
    return call


@_on_its_stream
def chunk_fwd(q, k, v, log_alpha, b, w, S0=None, chunk: int = 64,
              out_dtype=torch.float32, return_state: bool = True, stream=None,
              generic: bool = False, path: str = "auto", gate_logits: bool = False):
    """q, k: [B,H,T,dk]; v: [B,H,T,dv]; log_alpha, b: [B,H,T,dk] or [B,H,T];
    w: [B,H,T,dv] or [B,H,T]; S0: [B,H,dk,dv] fp32 or None.
    path "auto" passes a workspace (the chunk producer and the state chains in
    one persistent kernel where they apply), "split" the same with the two
    roles as two kernels one after the other (GDR_FWD_SPLIT), "fused" passes
    no workspace (single-kernel path).
    Returns (o [B,H,T,dv], S_final [B,H,dk,dv] or None)."""
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    flags = gate_flags(q, log_alpha, b, w, gate_logits)
    if out_dtype == torch.bfloat16:
        flags |= GDR_OUT_BF16
    if generic:
        flags |= GDR_FWD_GENERIC
    o = torch.empty((B, H, T, dv), dtype=out_dtype, device=q.device)
    Sf = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device) if return_state else None
    ws, nbytes = None, 0
    if path == "split":
        flags |= GDR_FWD_SPLIT
    if path in ("auto", "split"):
        nbytes = gdr_chunk_fwd_workspace_bytes(B, H, T, dk, dv, chunk, flags)
        if nbytes > 0:
            ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    elif path != "fused":
        raise ValueError(f"unknown path {path!r}")
    gdr_chunk_fwd(q, k, v, log_alpha, b, w, S0, o, Sf, B, H, T, dk, dv, chunk, flags, ws, nbytes,
                  stream)
    return o, Sf


@_on_its_stream
def chunk_fwd_varlen(q, k, v, log_alpha, b, w, cu_seqlens, S0=None, out_dtype=torch.float32,
                     return_state: bool = True, stream=None, gate_logits: bool = False):
    """Packed sequences: q, k: [H,T,dk]; v: [H,T,dv]; log_alpha, b: [H,T,dk] or
    [H,T]; w: [H,T,dv] or [H,T]; cu_seqlens: int32 [nseq+1] on the GPU; S0:
    [nseq,H,dk,dv] fp32 or None.  Returns (o [H,T,dv], S_final [nseq,H,dk,dv] or None)."""
    H, T, dk = q.shape
    dv = v.shape[-1]
    if cu_seqlens.dtype != torch.int32:
        raise ValueError("cu_seqlens must be int32")
    nseq = cu_seqlens.numel() - 1
    flags = gate_flags(q, log_alpha, b, w, gate_logits)
    if out_dtype == torch.bfloat16:
        flags |= GDR_OUT_BF16
    o = torch.empty((H, T, dv), dtype=out_dtype, device=q.device)
    Sf = torch.empty((nseq, H, dk, dv), dtype=torch.float32, device=q.device) if return_state else None
    nbytes = gdr_chunk_fwd_varlen_workspace_bytes(nseq, H, T, dk, dv, flags)
    if nbytes == 0:
        raise GdrError("gdr_chunk_fwd_varlen_workspace_bytes", 2)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    gdr_chunk_fwd_varlen(q, k, v, log_alpha, b, w, S0, o, Sf, cu_seqlens, nseq, H, T, dk, dv,
                         flags, ws, nbytes, stream)
    return o, Sf


@_on_its_stream
def decode_step(q, k, v, log_alpha, b, w, S, out_dtype=torch.float32, o=None, stream=None,
                gate_logits: bool = False):
    """One token per (n, h): q, k: [N,H,dk]; v: [N,H,dv]; gates channel or
    scalar ([N,H]); S: [N,H,dk,dv] fp32, updated in place.  Returns o."""
    N, H, dk = q.shape
    dv = v.shape[-1]
    flags = gate_flags(q, log_alpha, b, w, gate_logits)
    if out_dtype == torch.bfloat16:
        flags |= GDR_OUT_BF16
    if o is None:
        o = torch.empty((N, H, dv), dtype=out_dtype, device=q.device)
    gdr_decode_step(q, k, v, log_alpha, b, w, S, o, N, H, dk, dv, flags, stream)
    return o


@_on_its_stream
def chunk_bwd(q, k, v, log_alpha, b, w, S0, dO, dS_final=None, chunk: int = 64, stream=None,
              gate_logits: bool = False):
    """Gradients of L = <dO, o> + <dS_final, S_final>.  Returns a dict of fp32
    tensors dq, dk, dv, dlog_alpha, db, dw (scalar gates keep their scalar
    shape) and dS0."""
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    flags = gate_flags(q, log_alpha, b, w, gate_logits)
    dev = q.device
    f32 = torch.float32
    out = dict(dq=torch.empty((B, H, T, dk), dtype=f32, device=dev),
               dk=torch.empty((B, H, T, dk), dtype=f32, device=dev),
               dv=torch.empty((B, H, T, dv), dtype=f32, device=dev),
               dlog_alpha=torch.empty(tuple(log_alpha.shape), dtype=f32, device=dev),
               db=torch.empty(tuple(b.shape), dtype=f32, device=dev),
               dw=torch.empty(tuple(w.shape), dtype=f32, device=dev),
               dS0=torch.empty((B, H, dk, dv), dtype=f32, device=dev))
    nbytes = gdr_chunk_bwd_workspace_bytes(B, H, T, dk, dv, chunk, flags)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    gdr_chunk_bwd(q, k, v, log_alpha, b, w, S0, dO, dS_final, out["dq"], out["dk"], out["dv"],
                  out["dlog_alpha"], out["db"], out["dw"], out["dS0"], B, H, T, dk, dv, chunk,
                  flags, ws, nbytes, stream)
    return out


@_on_its_stream
def chunk_bwd_varlen(q, k, v, log_alpha, b, w, cu_seqlens, S0, dO, dS_final=None, stream=None,
                     gate_logits: bool = False):
    """Packed sequences ([H,T,...] streams, cu_seqlens int32 on the GPU): the
    gradients of L = <dO, o> + <dS_final, S_final> as a dict of fp32 tensors
    dq, dk, dv, dlog_alpha, db, dw (in the inputs' shapes) and dS0 [nseq,H,dk,dv]."""
    H, T, dk = q.shape
    dv = v.shape[-1]
    if cu_seqlens.dtype != torch.int32:
        raise ValueError("cu_seqlens must be int32")
    nseq = cu_seqlens.numel() - 1
    flags = gate_flags(q, log_alpha, b, w, gate_logits)
    dev = q.device
    f32 = torch.float32
    out = dict(dq=torch.empty((H, T, dk), dtype=f32, device=dev),
               dk=torch.empty((H, T, dk), dtype=f32, device=dev),
               dv=torch.empty((H, T, dv), dtype=f32, device=dev),
               dlog_alpha=torch.empty(tuple(log_alpha.shape), dtype=f32, device=dev),
               db=torch.empty(tuple(b.shape), dtype=f32, device=dev),
               dw=torch.empty(tuple(w.shape), dtype=f32, device=dev),
               dS0=torch.empty((nseq, H, dk, dv), dtype=f32, device=dev))
    nbytes = gdr_chunk_bwd_varlen_workspace_bytes(nseq, H, T, dk, dv, flags)
    if nbytes == 0:
        raise GdrError("gdr_chunk_bwd_varlen_workspace_bytes", 2)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    gdr_chunk_bwd_varlen(q, k, v, log_alpha, b, w, S0, dO, dS_final, out["dq"], out["dk"],
                         out["dv"], out["dlog_alpha"], out["db"], out["dw"], out["dS0"],
                         cu_seqlens, nseq, H, T, dk, dv, flags, ws, nbytes, stream)
    return out


@_on_its_stream
def mixer_prologue(q_pre, k_pre, v_pre, conv_q, conv_k, conv_v, a_pre, b_pre, w_pre, stream=None,
                   gate_logits: bool = False):
    """[B,H,T,d] bf16 projection outputs (a_pre fp32; gate logits [B,H,T,d]
    or [B,H,T]) and fp32 [H,d,4] convolution taps -> dict q, k, v, log_alpha,
    b, w: the inputs of chunk_fwd.  gate_logits: only q, k, v are produced;
    log_alpha, b and w are the logits themselves, for the recurrence calls
    made with gate_logits=True."""
    B, H, T, dk = q_pre.shape
    dv = v_pre.shape[-1]
    flags = GDR_GATE_LOGITS if gate_logits else 0
    if a_pre.dim() == 3:
        flags |= GDR_ALPHA_SCALAR
    if b_pre.dim() == 3:
        flags |= GDR_B_SCALAR
    if w_pre.dim() == 3:
        flags |= GDR_W_SCALAR
    out = dict(q=torch.empty_like(q_pre), k=torch.empty_like(k_pre), v=torch.empty_like(v_pre))
    if gate_logits:
        gdr_mixer_prologue(q_pre, k_pre, v_pre, conv_q, conv_k, conv_v, None, None, None, out["q"],
                           out["k"], out["v"], None, None, None, B, H, T, dk, dv, flags, stream)
        out.update(log_alpha=a_pre, b=b_pre, w=w_pre)
        return out
    out.update(log_alpha=torch.empty_like(a_pre), b=torch.empty_like(b_pre), w=torch.empty_like(w_pre))
    gdr_mixer_prologue(q_pre, k_pre, v_pre, conv_q, conv_k, conv_v, a_pre, b_pre, w_pre, out["q"],
                       out["k"], out["v"], out["log_alpha"], out["b"], out["w"], B, H, T, dk, dv,
                       flags, stream)
    return out


@_on_its_stream
def mixer_epilogue(o, g, norm_weight, stream=None):
    """o fp32 [B,H,T,dv], g bf16 [B,H,T,dv], norm_weight fp32 [dv] -> y bf16."""
    B, H, T, dv = o.shape
    y = torch.empty(o.shape, dtype=torch.bfloat16, device=o.device)
    gdr_mixer_epilogue(o, g, norm_weight, y, B, H, T, dv, 0, stream)
    return y


@_on_its_stream
def mixer_prologue_bwd(q_pre, k_pre, v_pre, conv_q, conv_k, conv_v, dq, dk, dv, stream=None):
    """Gradients of the prologue's q, k, v paths: dict dq_pre, dk_pre, dv_pre
    (fp32 [B,H,T,d]) and dconv_q, dconv_k, dconv_v (fp32 [H,d,4])."""
    B, H, T, dk_ = q_pre.shape
    dv_ = v_pre.shape[-1]
    f32 = torch.float32
    out = dict(dq_pre=torch.empty(q_pre.shape, dtype=f32, device=q_pre.device),
               dk_pre=torch.empty(k_pre.shape, dtype=f32, device=q_pre.device),
               dv_pre=torch.empty(v_pre.shape, dtype=f32, device=q_pre.device),
               dconv_q=torch.empty_like(conv_q), dconv_k=torch.empty_like(conv_k),
               dconv_v=torch.empty_like(conv_v))
    nb = gdr_mixer_bwd_workspace_bytes(B, H, T, dk_, dv_)
    if nb == 0:
        raise GdrError("gdr_mixer_bwd_workspace_bytes", 2)
    ws = torch.empty(nb, dtype=torch.uint8, device=q_pre.device)
    gdr_mixer_prologue_bwd(q_pre, k_pre, v_pre, conv_q, conv_k, conv_v, dq, dk, dv, out["dq_pre"],
                           out["dk_pre"], out["dv_pre"], out["dconv_q"], out["dconv_k"],
                           out["dconv_v"], B, H, T, dk_, dv_, 0, ws, nb, stream)
    return out


@_on_its_stream
def mixer_epilogue_bwd(o, g, norm_weight, dy, stream=None):
    """Gradients of the epilogue: dict d_o, dg (fp32 [B,H,T,dv]), dnorm_weight (fp32 [dv])."""
    B, H, T, dv_ = o.shape
    f32 = torch.float32
    out = dict(d_o=torch.empty(o.shape, dtype=f32, device=o.device),
               dg=torch.empty(o.shape, dtype=f32, device=o.device),
               dnorm_weight=torch.empty((dv_,), dtype=f32, device=o.device))
    nb = gdr_mixer_bwd_workspace_bytes(B, H, T, dv_, dv_)
    if nb == 0:
        raise GdrError("gdr_mixer_bwd_workspace_bytes", 2)
    ws = torch.empty(nb, dtype=torch.uint8, device=o.device)
    gdr_mixer_epilogue_bwd(o, g, norm_weight, dy, out["d_o"], out["dg"], out["dnorm_weight"], B, H, T,
                           dv_, 0, ws, nb, stream)
    return out


# ---------------------------------------------------------------------------
# the attention layer of a hybrid stack
# ---------------------------------------------------------------------------


def _expect(name, t, shape, dtype, gpu):
    """The tensor a call takes: its shape, type, GPU and contiguity."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != gpu or not t.is_contiguous():
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.dtype is not dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.get_device() != gpu:
            raise ValueError(f"{name} must be on GPU {gpu}, got {t.device}")
        raise ValueError(f"{name} must be contiguous")


def _gpu_of(name, t):
    """The index of the GPU that a call's first tensor is on."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    return t.get_device()


def _launch(fn, gpu, stream, *args):
    """The library call `fn` with the given GPU current, on `stream` or that GPU's
    current one.  (The wrappers below take pointers and the stream's handle
    directly: a small call's time is that of the host.)"""
    if gpu != torch.cuda.current_device():
        with torch.cuda.device(gpu):
            return _launch(fn, gpu, stream, *args)
    call = getattr(_lib or _load(), fn)
    st = call(*args, torch._C._cuda_getCurrentRawStream(gpu) if stream is None else stream.cuda_stream)
    if st != 0:
        names = inspect.signature(globals()[fn]).parameters
        off = [n for n, a, t in zip(names, args, call.argtypes) if t is ctypes.c_void_p and a and a % 16]
        raise GdrError(fn, st, f"{', '.join(off)} must start at a multiple of 16 bytes (a slice may not)" if off else "")


def rope_frequencies(rot_dim, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                     trained: int = 0, low: float = 1.0, high: float = 32.0, device="cuda"):
    """(inv_freq fp32 [rot_dim / 2], scale) for :func:`rope`: base^(-2i / rot_dim),
    scaled to contexts `factor` times the trained ones by

    * "linear": every frequency divided by factor;
    * "base": the base raised to base * factor^(rot_dim / (rot_dim - 2)), which
      leaves the first frequency and divides the last by factor;
    * "parts": by how often a frequency turns over `trained` tokens: at least
      `high` times unchanged, at most `low` times divided by factor, between them
      a linear blend; with scale 0.1 ln(factor) + 1 on the turned channels."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    scale = 1.0
    if scaling == "base":
        if rot_dim < 4:
            raise ValueError("scaling 'base' needs rot_dim of at least 4")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = torch.pow(torch.tensor(base, dtype=torch.float64), -2.0 * i / rot_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if trained < 1 or not low < high:
            raise ValueError("scaling 'parts' needs the trained length and low < high")
        keep = ((trained * f / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1 - keep)
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.float().to(device), scale


@_on_its_stream
def rope(q, k, inv_freq, positions=None, position0: int = 0, interleaved: bool = False, inverse: bool = False,
         scale: float = 1.0, token_major: bool = False, q_out=None, k_out=None, stream=None):
    """Rotary positions.  q: [B,Hq,T,d], k: [B,Hk,T,d] or None, bf16 or fp32
    (token_major: [B,T,H,d]); packed streams [H,T,d] ([T,H,d]) count as B = 1;
    inv_freq: fp32 [rot_dim/2]; positions: int32 [B,T] (packed: [T]) or None for
    position0 + t.  inverse turns back: the gradients of q and k from those of the
    results.  Returns (q_out, k_out); they may be given, also as q and k themselves."""
    shape = q.shape
    n = len(shape)
    if n not in (3, 4) or (k is not None and k.dim() != n):
        raise ValueError("q and k must both be [B,H,T,d] or both packed [H,T,d]")
    gpu, dtype = _gpu_of("q", q), q.dtype
    lead, d = shape[:-3], shape[-1]
    B = lead[0] if n == 4 else 1
    T, Hq = (shape[-3], shape[-2]) if token_major else (shape[-2], shape[-3])
    flags = _act_flag(q) | (GDR_TOKEN_MAJOR if token_major else 0) | (GDR_ROPE_INTERLEAVED if interleaved else 0) \
        | (GDR_ROPE_INVERSE if inverse else 0)
    k_ptr = ko_ptr = None
    Hk = 0
    _expect("q", q, shape, dtype, gpu)
    if k is not None:
        Hk = k.shape[-2 if token_major else -3]
        _expect("k", k, lead + ((T, Hk, d) if token_major else (Hk, T, d)), dtype, gpu)
        if k_out is None:
            k_out = torch.empty_like(k)
        else:
            _expect("k_out", k_out, k.shape, dtype, gpu)
        k_ptr, ko_ptr = k.data_ptr(), k_out.data_ptr()
    if q_out is None:
        q_out = torch.empty_like(q)
    else:
        _expect("q_out", q_out, shape, dtype, gpu)
    half = inv_freq.numel()
    _expect("inv_freq", inv_freq, (half,), torch.float32, gpu)
    if positions is not None:
        _expect("positions", positions, lead + (T,), torch.int32, gpu)
        positions = positions.data_ptr()
    _launch("gdr_rope", gpu, stream, q.data_ptr(), k_ptr, q_out.data_ptr(), ko_ptr, inv_freq.data_ptr(), positions,
            _position(position0), B, Hq, Hk, T, d, 2 * half, scale, flags)
    return q_out, k_out if k is not None else None


def _attn_shapes(q, k, v, packed, token_major):
    """(B, Hq, Hkv, Tq, Tk, d, GPU) of attention's inputs, checked."""
    qs, ks = q.shape, k.shape
    if len(qs) != (3 if packed else 4) or len(ks) != len(qs):
        raise ValueError("q, k and v must be " + ("[H,T,d]" if packed else "[B,H,T,d]"))
    gpu = _gpu_of("q", q)
    h, t = (-2, -3) if token_major else (-3, -2)
    B, Hq, Hkv, Tq, Tk, d = (1 if packed else qs[0]), qs[h], ks[h], qs[t], ks[t], qs[-1]
    _expect("q", q, qs, torch.bfloat16, gpu)
    want = qs[:-3] + ((Tk, Hkv, d) if token_major else (Hkv, Tk, d))
    _expect("k", k, want, torch.bfloat16, gpu)
    _expect("v", v, want, torch.bfloat16, gpu)
    return B, Hq, Hkv, Tq, Tk, d, gpu


@_on_its_stream
def attn_fwd(q, k, v, window: int = 0, scale: Optional[float] = None, token_major: bool = False,
             return_lse: bool = True, stream=None):
    """Causal attention.  q: [B,Hq,Tq,d], k, v: [B,Hkv,Tk,d] bf16 (token_major:
    [B,T,H,d]); query i sees the keys up to i + Tk - Tq, the last `window` of them
    (0: all); scale: 1/sqrt(d) if None.  Returns (o as q, lse fp32 [B,Hq,Tq] or None)."""
    B, Hq, Hkv, Tq, Tk, d, gpu = _attn_shapes(q, k, v, False, token_major)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, Tq), dtype=torch.float32, device=q.device) if return_lse else None
    _launch("gdr_attn_fwd", gpu, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
            lse.data_ptr() if return_lse else None, B, Hq, Hkv, Tq, Tk, d, _window(window),
            d ** -0.5 if scale is None else scale, GDR_TOKEN_MAJOR if token_major else 0)
    return o, lse


@_on_its_stream
def attn_fwd_varlen(q, k, v, cu_seqlens, window: int = 0, scale: Optional[float] = None,
                    token_major: bool = False, return_lse: bool = True, stream=None):
    """Packed sequences: q: [Hq,T,d], k, v: [Hkv,T,d] bf16 (token_major: [T,H,d]);
    cu_seqlens: int32 [nseq+1] on the GPU.  Returns (o as q, lse fp32 [Hq,T] or None);
    rows from cu_seqlens[nseq] on are not written."""
    B, Hq, Hkv, T, Tk, d, gpu = _attn_shapes(q, k, v, True, token_major)
    if T != Tk:
        raise ValueError("packed q, k and v must have the same tokens")
    nseq = cu_seqlens.numel() - 1
    _expect("cu_seqlens", cu_seqlens, (nseq + 1,), torch.int32, gpu)
    o = torch.empty_like(q)
    lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device) if return_lse else None
    _launch("gdr_attn_fwd_varlen", gpu, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
            lse.data_ptr() if return_lse else None, cu_seqlens.data_ptr(), nseq, Hq, Hkv, T, d, _window(window),
            d ** -0.5 if scale is None else scale, GDR_TOKEN_MAJOR if token_major else 0)
    return o, lse


def _attn_bwd(q, k, v, o, lse, dO, cu_seqlens, window, scale, token_major, stream):
    packed = cu_seqlens is not None
    B, Hq, Hkv, Tq, Tk, d, gpu = _attn_shapes(q, k, v, packed, token_major)
    if packed and Tq != Tk:
        raise ValueError("packed q, k and v must have the same tokens")
    _expect("o", o, q.shape, torch.bfloat16, gpu)
    _expect("dO", dO, q.shape, torch.bfloat16, gpu)
    _expect("lse", lse, (Hq, Tq) if packed else (B, Hq, Tq), torch.float32, gpu)
    scale = d ** -0.5 if scale is None else scale
    flags = GDR_TOKEN_MAJOR if token_major else 0
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    nbytes = gdr_attn_bwd_workspace_bytes(B, Hq, Hkv, Tq, Tk, d)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device) if nbytes > 0 else None
    ptrs = [t.data_ptr() for t in (q, k, v, o, lse, dO, dq, dk, dv)]
    tail = (d, _window(window), scale, flags, ws.data_ptr() if nbytes > 0 else None, nbytes)
    if packed:
        nseq = cu_seqlens.numel() - 1
        _expect("cu_seqlens", cu_seqlens, (nseq + 1,), torch.int32, gpu)
        _launch("gdr_attn_bwd_varlen", gpu, stream, *ptrs, cu_seqlens.data_ptr(), nseq, Hq, Hkv, Tq, *tail)
    else:
        _launch("gdr_attn_bwd", gpu, stream, *ptrs, B, Hq, Hkv, Tq, Tk, *tail)
    return dict(dq=dq, dk=dk, dv=dv)


@_on_its_stream
def attn_bwd(q, k, v, o, lse, dO, window: int = 0, scale: Optional[float] = None, token_major: bool = False,
             stream=None):
    """Gradients of <dO, o>: dict dq, dk, dv (bf16, as q, k, v), from what
    :func:`attn_fwd` took and returned with the same window, scale and layout."""
    return _attn_bwd(q, k, v, o, lse, dO, None, window, scale, token_major, stream)


@_on_its_stream
def attn_bwd_varlen(q, k, v, o, lse, dO, cu_seqlens, window: int = 0, scale: Optional[float] = None,
                    token_major: bool = False, stream=None):
    """The same for :func:`attn_fwd_varlen`."""
    return _attn_bwd(q, k, v, o, lse, dO, cu_seqlens, window, scale, token_major, stream)


class KVCache(NamedTuple):
    """A paged 8-bit cache: e4m3 bytes and one power-of-two scale per (page, head).
    k: uint8 [n_pages,Hkv,64,d], v: uint8 [n_pages,Hkv,4,d,16] (value of token
    16 g + i and channel c at [g,c,i]), k_scale, v_scale: fp32 [n_pages,Hkv]."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def kv_cache(n_pages, Hkv, d, device="cuda") -> KVCache:
    """An empty cache (its contents count only where kv_append has written)."""
    P = GDR_KV_PAGE
    return KVCache(torch.empty((n_pages, Hkv, P, d), dtype=torch.uint8, device=device),
                   torch.empty((n_pages, Hkv, P // 16, d, 16), dtype=torch.uint8, device=device),
                   torch.empty((n_pages, Hkv), dtype=torch.float32, device=device),
                   torch.empty((n_pages, Hkv), dtype=torch.float32, device=device))


def _cache_shapes(cache, block_table, cache_len, gpu):
    """(n_pages, Hkv, d, nseq, max_pages) of a cache and its tables, checked."""
    ck, cv, ks, vs = cache
    n_pages, Hkv, P, d = ck.shape
    if P != GDR_KV_PAGE:
        raise ValueError(f"a page holds {GDR_KV_PAGE} tokens, got {P}")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [nseq, max_pages]")
    nseq, max_pages = block_table.shape
    _expect("cache.k", ck, ck.shape, torch.uint8, gpu)
    _expect("cache.v", cv, (n_pages, Hkv, P // 16, d, 16), torch.uint8, gpu)
    _expect("cache.k_scale", ks, (n_pages, Hkv), torch.float32, gpu)
    _expect("cache.v_scale", vs, (n_pages, Hkv), torch.float32, gpu)
    _expect("block_table", block_table, block_table.shape, torch.int32, gpu)
    _expect("cache_len", cache_len, (nseq,), torch.int32, gpu)
    return n_pages, Hkv, d, nseq, max_pages


def kv_append(k, v, cache: KVCache, block_table, cache_len, cu_seqlens=None, token_major: bool = False, stream=None):
    """Write new tokens behind the cache_len int32 [nseq] tokens of each sequence.
    k, v: bf16 [nseq,Hkv,d], one token each; or with cu_seqlens int32 [nseq+1]
    packed [Hkv,T,d] (token_major: [T,Hkv,d]).  block_table: int32 [nseq,max_pages].
    cache_len stays as it is: raise it by the new lengths afterwards."""
    gpu = _gpu_of("k", k)
    n_pages, Hkv, d, nseq, max_pages = _cache_shapes(cache, block_table, cache_len, gpu)
    cu = None
    if cu_seqlens is None:
        T, want = nseq, (nseq, Hkv, d)
    else:
        if k.dim() != 3:
            raise ValueError("packed k and v must be [Hkv,T,d] or token-major [T,Hkv,d]")
        T = k.shape[0 if token_major else 1]
        want = (T, Hkv, d) if token_major else (Hkv, T, d)
        _expect("cu_seqlens", cu_seqlens, (nseq + 1,), torch.int32, gpu)
        cu = cu_seqlens.data_ptr()
    _expect("k", k, want, torch.bfloat16, gpu)
    _expect("v", v, want, torch.bfloat16, gpu)
    _launch("gdr_kv_append", gpu, stream, k.data_ptr(), v.data_ptr(), *[t.data_ptr() for t in cache],
            block_table.data_ptr(), cache_len.data_ptr(), cu, nseq, Hkv, T, d, n_pages, max_pages,
            GDR_TOKEN_MAJOR if token_major else 0)


@_on_its_stream
def attn_decode(q, cache: KVCache, block_table, cache_len, window: int = 0, scale: Optional[float] = None,
                out_dtype=torch.float32, o=None, stream=None):
    """Attention of one token per sequence over the cache: q bf16 [N,Hq,d], the
    last of each sequence's cache_len tokens; sees all of them or the last
    `window`.  Calls of few sequences are slow behind a block_table much wider than
    they need.  Returns o [N,Hq,d] of out_dtype (fp32 or bf16)."""
    gpu = _gpu_of("q", q)
    n_pages, Hkv, d, N, max_pages = _cache_shapes(cache, block_table, cache_len, gpu)
    if q.dim() != 3:
        raise ValueError("q must be [N,Hq,d]")
    shape = (N, q.shape[1], d)
    Hq = shape[1]
    _expect("q", q, shape, torch.bfloat16, gpu)
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"out_dtype must be float32 or bfloat16, got {out_dtype}")
    ws = None
    if o is None:
        o = torch.empty(shape, dtype=out_dtype, device=q.device)
    else:
        _expect("o", o, shape, out_dtype, gpu)
    nbytes = gdr_attn_decode_workspace_bytes(N, Hq, Hkv, d, max_pages, window)
    if nbytes > 0:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    _launch("gdr_attn_decode", gpu, stream, q.data_ptr(), *[t.data_ptr() for t in cache], block_table.data_ptr(),
            cache_len.data_ptr(), o.data_ptr(), N, Hq, Hkv, d, n_pages, max_pages, _window(window),
            d ** -0.5 if scale is None else scale, GDR_OUT_BF16 if out_dtype is torch.bfloat16 else 0,
            None if ws is None else ws.data_ptr(), nbytes)
    return o
