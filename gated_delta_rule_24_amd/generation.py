"""Several continuations of one prompt: samples, beams, or a batch behind a common system
prompt, over the recurrent states and the paged cache of a hybrid stack.

* :func:`attn_decode_shared` — attention of one token per sequence where groups of
  sequences share their first pages, which are read once a group
* :func:`kv_fork` — the block table's rows continued, forked, grown and dropped
* :func:`kv_compact` — pages in use moved to the lowest places of the cache
* :func:`beam_select` — the best continuations of each prompt's beams
* :func:`state_reorder` — states moved to the rows that continue them

A step of a beam search, after a layer's keys and values were appended and attended to::

    tokens, rows, scores, ended = beam_select(logits, scores, ended=ended, end_token=2, keep_slots=True)
    state_reorder(S, rows, beams)                         # the recurrent layers' states
    table, length, missing = kv_fork(cache, table, length, rows.flatten(), room=1)

The calls are those of ``include/gdr.h`` with outputs and workspaces allocated for the
caller; like the package's other calls they run on the current stream or `stream`.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import (GDR_ACT_F32, GDR_KEEP_SLOTS, GDR_OUT_BF16, KVCache, _act_flag, _cache_shapes, _expect, _gpu_of, _launch,
               _on_its_stream, _window, gdr_attn_decode_shared_workspace_bytes, gdr_beam_select_workspace_bytes,
               gdr_kv_compact_workspace_bytes, gdr_kv_fork_workspace_bytes)


def _workspace(nbytes, like):
    # (0: sizes that the call itself refuses, with its own error.  new_empty here and below: it
    # takes half of torch.empty's time with a type and a device, and a small call's time is the host's)
    return like.new_empty(max(nbytes, 16), dtype=torch.uint8)


def _int32(name, x):
    # (ctypes would keep the low 32 bits without a word)
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError(f"{name} must fit 32 bits, got {x}")
    return x


def _held(held, n_pages, gpu):
    if held is None:
        return None
    if held.dtype is torch.bool:
        held = held.view(torch.uint8)
    _expect("held", held, (n_pages,), torch.uint8, gpu)
    return held.data_ptr()


@_on_its_stream
def attn_decode_shared(q, cache: KVCache, block_table, cache_len, group_start, shared_pages, window: int = 0,
                       scale: Optional[float] = None, out_dtype=torch.float32, o=None, stream=None):
    """:func:`attn_decode` for groups of sequences that share their first pages.
    q: bf16 [N,Hq,d]; group_start: int32 [groups+1], group g being sequences
    group_start[g] .. group_start[g+1]-1; shared_pages: int32 [groups], how many of
    their first pages are those in the row of the group's first sequence (which must hold them: a
    group whose first row was emptied begins behind it).
    Returns o [N,Hq,d] of out_dtype (fp32 or bf16)."""
    gpu = _gpu_of("q", q)
    n_pages, Hkv, d, N, max_pages = _cache_shapes(cache, block_table, cache_len, gpu)
    if q.dim() != 3:
        raise ValueError("q must be [N,Hq,d]")
    shape = (N, q.shape[1], d)
    Hq = shape[1]
    _expect("q", q, shape, torch.bfloat16, gpu)
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"out_dtype must be float32 or bfloat16, got {out_dtype}")
    groups = shared_pages.numel()
    _expect("shared_pages", shared_pages, (groups,), torch.int32, gpu)
    _expect("group_start", group_start, (groups + 1,), torch.int32, gpu)
    if o is None:
        o = q.new_empty(shape, dtype=out_dtype)
    else:
        _expect("o", o, shape, out_dtype, gpu)
    nbytes = gdr_attn_decode_shared_workspace_bytes(N, groups, Hq, Hkv, d, max_pages, window)
    ws = _workspace(nbytes, q)
    _launch("gdr_attn_decode_shared", gpu, stream, q.data_ptr(), *[t.data_ptr() for t in cache], block_table.data_ptr(),
            cache_len.data_ptr(), group_start.data_ptr(), shared_pages.data_ptr(), o.data_ptr(), N, groups, Hq, Hkv, d,
            n_pages, max_pages, _window(window), d ** -0.5 if scale is None else scale,
            GDR_OUT_BF16 if out_dtype is torch.bfloat16 else 0, ws.data_ptr(), nbytes)
    return o


@_on_its_stream
def kv_fork(cache: KVCache, block_table, cache_len, parent=None, room=1, held=None, table_out=None, len_out=None, stream=None):
    """The next block table: row n continues row parent[n] (int32 [N]; None: itself;
    outside the table: row n becomes empty) for the room tokens it is about to append (a
    number, or int32 [N]).  Whole pages are shared; a page that several rows are about to
    write on is copied for all but the lowest of them; fresh pages follow; pages that no row
    names any more are free, and dealt out from the lowest.  held: uint8 or bool [n_pages],
    pages that other tables hold.  Returns (table_out [N,max_pages], -1 behind a row's pages;
    len_out [N]; missing [N], the pages each row wanted and did not get: it must not be
    appended to then).  table_out and len_out may be given; without parent also as
    block_table and cache_len themselves.  The pages are one layer's: layers under one table take
    a call each, all from the old table (only the last may write over it), and get the same new one."""
    gpu = _gpu_of("cache.k", cache.k)
    n_pages, Hkv, d, N_in, max_pages = _cache_shapes(cache, block_table, cache_len, gpu)
    N = N_in
    if parent is not None:
        N = parent.numel()
        _expect("parent", parent, (N,), torch.int32, gpu)
        parent = parent.data_ptr()
    room_ptr, room_all = None, 0
    if isinstance(room, torch.Tensor):
        _expect("room", room, (N,), torch.int32, gpu)
        room_ptr = room.data_ptr()
    else:
        room_all = room
        if not 0 <= room < 1 << 31:
            raise ValueError(f"room must be 0 or more and fit 32 bits, got {room}")
    if table_out is None:
        table_out = block_table.new_empty((N, max_pages))
    else:
        _expect("table_out", table_out, (N, max_pages), torch.int32, gpu)
    if len_out is None:
        len_out = cache_len.new_empty(N)
    else:
        _expect("len_out", len_out, (N,), torch.int32, gpu)
    missing = cache_len.new_empty(N)
    nbytes = gdr_kv_fork_workspace_bytes(N, n_pages)
    ws = _workspace(nbytes, block_table)
    _launch("gdr_kv_fork", gpu, stream, *[t.data_ptr() for t in cache], block_table.data_ptr(), cache_len.data_ptr(), parent,
            room_ptr, _held(held, n_pages, gpu), table_out.data_ptr(), len_out.data_ptr(), missing.data_ptr(), N_in, N,
            room_all, Hkv, d, n_pages, max_pages, 0, ws.data_ptr(), nbytes)
    return table_out, len_out, missing


@_on_its_stream
def kv_compact(cache: KVCache, block_table, cache_len, held=None, table_out=None, stream=None):
    """Pages in use moved to the lowest free places (those that `held` marks stay), and the
    table that names them there.  Returns (table_out [N,max_pages], used int32 [1]: one past
    the last page in use afterwards).  table_out may be block_table; layers under one table take a
    call each, all from the old table, as for :func:`kv_fork`."""
    gpu = _gpu_of("cache.k", cache.k)
    n_pages, Hkv, d, N, max_pages = _cache_shapes(cache, block_table, cache_len, gpu)
    if table_out is None:
        table_out = block_table.new_empty((N, max_pages))
    else:
        _expect("table_out", table_out, (N, max_pages), torch.int32, gpu)
    used = cache_len.new_empty(1)
    nbytes = gdr_kv_compact_workspace_bytes(n_pages)
    ws = _workspace(nbytes, block_table)
    _launch("gdr_kv_compact", gpu, stream, *[t.data_ptr() for t in cache], block_table.data_ptr(), cache_len.data_ptr(),
            _held(held, n_pages, gpu), table_out.data_ptr(), used.data_ptr(), N, Hkv, d, n_pages, max_pages, 0,
            ws.data_ptr(), nbytes)
    return table_out, used


@_on_its_stream
def beam_select(logits, scores, n_select: Optional[int] = None, ended=None, end_token: int = -1, keep_slots: bool = False,
                stream=None):
    """The best n_select (None: K) continuations of each group of K beams.
    logits: bf16 or fp32 [G*K,V] (rows may be those of a wider tensor; at most 65,535), row g*K+k
    being beam k of group g; scores: fp32 [G,K], the beams' log probabilities; ended: bool
    [G,K], beams that end_token has ended (they go on as they are).
    Returns (tokens int32, rows int32: the row g*K+k that each continues, scores fp32,
    ended bool), all [G,n_select], from the best; with keep_slots (n_select = K) the first
    continuation of a beam in the beam's own place, the others in the places left."""
    gpu = _gpu_of("logits", logits)
    if logits.dim() != 2 or scores.dim() != 2:
        raise ValueError("logits must be [G*K,V] and scores [G,K]")
    G, K = scores.shape
    V = logits.shape[1]
    if logits.shape[0] != G * K:
        raise ValueError(f"logits must have the {G * K} rows of scores' beams, got {logits.shape[0]}")
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("logits' rows must be contiguous")
    _expect("scores", scores, (G, K), torch.float32, gpu)
    M = K if n_select is None else _int32("n_select", n_select)
    _int32("end_token", end_token)
    if ended is not None:
        _expect("ended", ended, (G, K), torch.bool, gpu)
        ended = ended.data_ptr()
    tokens = scores.new_empty((G, M), dtype=torch.int32)
    rows = scores.new_empty((G, M), dtype=torch.int32)
    out = scores.new_empty((G, M))
    done = scores.new_empty((G, M), dtype=torch.bool)
    nbytes = gdr_beam_select_workspace_bytes(G, K, M, V)
    ws = _workspace(nbytes, logits)
    _launch("gdr_beam_select", gpu, stream, logits.data_ptr(), scores.data_ptr(), ended, tokens.data_ptr(), rows.data_ptr(),
            out.data_ptr(), done.data_ptr(), G, K, M, V, logits.stride(0) if G * K > 1 else V, end_token,
            (GDR_ACT_F32 if _act_flag(logits) == GDR_ACT_F32 else 0) | (GDR_KEEP_SLOTS if keep_slots else 0),
            ws.data_ptr(), nbytes)
    return tokens, rows, out, done


def state_reorder(state, rows, beams: int, dim: int = 0, stream=None):
    """states moved to the rows that continue them, in place: row n becomes what row
    rows[n] was, for rows of the same group of `beams` rows.  state: [N,...], or with
    dim=1 [layers,N,...], of any type, a row's bytes a multiple of 16; rows: int32 of N
    values (:func:`beam_select`'s).  A row whose value is its own or not of its
    group stays as it is.  Returns state."""
    gpu = _gpu_of("state", state)
    _int32("beams", beams)
    if dim not in (0, 1) or state.dim() <= dim:
        raise ValueError("state must be [N,...], or with dim=1 [layers,N,...]")
    _expect("state", state, state.shape, state.dtype, gpu)
    N, layers = state.shape[dim], state.shape[0] if dim else 1
    _expect("rows", rows, rows.shape, torch.int32, gpu)
    if rows.numel() != N:
        raise ValueError(f"rows must have {N} values, got {rows.numel()}")
    row_bytes = state.numel() // max(N * layers, 1) * state.element_size()
    if row_bytes % 16 or row_bytes == 0:
        raise ValueError(f"a row of state must be a multiple of 16 bytes, got {row_bytes}")
    _launch("gdr_state_reorder", gpu, stream, state.data_ptr(), rows.data_ptr(), layers, N, beams, row_bytes, 0)
    return state
