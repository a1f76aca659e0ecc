"""Argument checks of the calls for several continuations of one prompt: every refusal
happens before a device is touched (fake aligned pointers, never dereferenced), so these
run without a GPU."""
import ctypes
import math

import pytest
import torch

import gated_delta_rule_24_amd as gdr
from tests.test_attn_abi import A, BIG, INVALID, MIS, UNSUPPORTED, WORKSPACE, _call, _lib

gen = gdr.generation

SHARED = "q kc vc ks vs table len starts shared o N groups Hq Hkv d pages width window scale flags ws nbytes".split()
SHARED_OK = dict(q=A, kc=A, vc=A, ks=A, vs=A, table=A, len=A, starts=A, shared=A, o=A, N=4, groups=2, Hq=8, Hkv=2, d=128,
                 pages=8, width=4, window=0, scale=0.1, flags=0, ws=A, nbytes=1 << 40)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(starts=None), INVALID), (dict(shared=None), INVALID), (dict(shared=MIS), INVALID),
    (dict(o=MIS), INVALID), (dict(table=None), INVALID), (dict(N=0), INVALID), (dict(groups=0), INVALID),
    (dict(groups=-1), INVALID), (dict(groups=4097), UNSUPPORTED), (dict(Hq=7), INVALID), (dict(pages=0), INVALID),
    (dict(width=0), INVALID), (dict(width=1 << 25), INVALID), (dict(window=-1), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=math.nan), INVALID), (dict(flags=0x1), INVALID), (dict(flags=0x8000), INVALID), (dict(d=32), UNSUPPORTED),
    (dict(N=1 << 20, Hq=1 << 20), INVALID), (dict(N=1 << 25, Hq=8), INVALID),
    (dict(ws=None), WORKSPACE), (dict(nbytes=63), WORKSPACE), (dict(ws=MIS), INVALID),
])
def test_attn_decode_shared_refusals(kw, status):
    assert _call("gdr_attn_decode_shared", SHARED, SHARED_OK, kw) == status


def test_attn_decode_shared_workspace_query():
    f = _lib().gdr_attn_decode_shared_workspace_bytes
    one = f(8, 1, 32, 8, 128, 800, 0)
    # a partial result of 32 rows, their maxima and sums, for each of 256 workgroups, and more
    assert one > 256 * 32 * (128 + 2) * 4
    assert f(8, 4097, 32, 8, 128, 800, 0) == 0
    assert f(8, 1, 32, 8, 128, 800, 64) < one                # a window bounds a sequence's own pages
    assert f(256, 1, 32, 8, 128, 800, 0) > 256 * 64 * (128 + 2) * 4
    for bad in ((0, 1, 32, 8, 128, 8, 0), (8, 0, 32, 8, 128, 8, 0), (8, 1, 31, 8, 128, 8, 0), (8, 1, 32, 8, 96, 8, 0),
                (8, 1, 32, 8, 128, 8, -1)):
        assert f(*bad) == 0


FORK = "kc vc ks vs table len parent room held out lout missing Nin N all Hkv d pages width flags ws nbytes".split()
B, C = ctypes.c_void_p(0x20000), ctypes.c_void_p(0x30000)
FORK_OK = dict(kc=A, vc=A, ks=A, vs=A, table=A, len=A, parent=A, room=A, held=A, out=B, lout=C, missing=A, Nin=3, N=5, all=1,
               Hkv=2, d=64, pages=9, width=4, flags=0, ws=A, nbytes=1 << 40)


@pytest.mark.parametrize("kw,status", [
    (dict(kc=None), INVALID), (dict(vs=None), INVALID), (dict(table=None), INVALID), (dict(len=None), INVALID),
    (dict(out=None), INVALID), (dict(lout=None), INVALID), (dict(missing=None), INVALID), (dict(parent=MIS), INVALID),
    (dict(room=MIS), INVALID), (dict(held=MIS), INVALID), (dict(out=A), INVALID), (dict(lout=A), INVALID),
    (dict(parent=None), INVALID), (dict(all=-1), INVALID), (dict(N=0), INVALID), (dict(Nin=0), INVALID),
    (dict(N=(1 << 20) + 1), INVALID), (dict(Hkv=0), INVALID), (dict(pages=0), INVALID), (dict(width=0), INVALID),
    (dict(width=1 << 25), INVALID), (dict(N=1 << 20, width=1 << 12), INVALID), (dict(flags=1), INVALID),
    (dict(Hkv=4096, N=1 << 20), INVALID), (dict(d=32), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(nbytes=100), WORKSPACE),
    (dict(ws=MIS), INVALID),
])
def test_kv_fork_refusals(kw, status):
    assert _call("gdr_kv_fork", FORK, FORK_OK, kw) == status


COMPACT = "kc vc ks vs table len held out used N Hkv d pages width flags ws nbytes".split()
COMPACT_OK = dict(kc=A, vc=A, ks=A, vs=A, table=A, len=A, held=A, out=A, used=A, N=3, Hkv=2, d=64, pages=9, width=4, flags=0,
                  ws=A, nbytes=1 << 40)


@pytest.mark.parametrize("kw,status", [
    (dict(kc=None), INVALID), (dict(ks=MIS), INVALID), (dict(table=None), INVALID), (dict(out=None), INVALID),
    (dict(used=None), INVALID), (dict(held=MIS), INVALID), (dict(N=0), INVALID), (dict(N=(1 << 20) + 1), INVALID),
    (dict(pages=-1), INVALID), (dict(pages=BIG), INVALID), (dict(width=0), INVALID), (dict(flags=2), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(nbytes=100), WORKSPACE), (dict(ws=MIS), INVALID),
])
def test_kv_compact_refusals(kw, status):
    assert _call("gdr_kv_compact", COMPACT, COMPACT_OK, kw) == status


def test_page_workspace_queries():
    lib = _lib()
    up = lambda n: (n + 15) // 16 * 16  # noqa: E731
    # per page a counter pair and the lowest writer, per 4,096 their free ones; three numbers a row
    assert lib.gdr_kv_fork_workspace_bytes(5, 5000) == 12 * 5000 + up(4 * 2) + 3 * up(4 * 5)
    assert lib.gdr_kv_fork_workspace_bytes(0, 10) == 0 and lib.gdr_kv_fork_workspace_bytes(5, 0) == 0
    assert lib.gdr_kv_compact_workspace_bytes(100) > 16 * 100 and lib.gdr_kv_compact_workspace_bytes(0) == 0


SELECT = "logits scores ended tokens rows sout eout G K M V stride end flags ws nbytes".split()
SELECT_OK = dict(logits=A, scores=A, ended=A, tokens=A, rows=A, sout=A, eout=A, G=2, K=3, M=3, V=100, stride=100, end=2, flags=0,
                 ws=A, nbytes=1 << 40)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), INVALID), (dict(logits=MIS), INVALID), (dict(scores=None), INVALID), (dict(ended=MIS), INVALID),
    (dict(tokens=None), INVALID), (dict(rows=None), INVALID), (dict(sout=None), INVALID), (dict(eout=None), INVALID),
    (dict(G=0), INVALID), (dict(K=0), INVALID), (dict(M=0), INVALID), (dict(V=0), INVALID), (dict(V=BIG), INVALID), (dict(V=(1 << 26) + 1, stride=1 << 27), UNSUPPORTED),
    (dict(stride=99), INVALID), (dict(end=100), INVALID), (dict(end=-2), INVALID), (dict(end=-1), INVALID),
    (dict(flags=0x2), INVALID), (dict(M=4, flags=0x8000), INVALID), (dict(M=301, K=3), UNSUPPORTED),
    (dict(K=1, M=5, V=4, stride=4), INVALID), (dict(K=65, M=1), UNSUPPORTED), (dict(M=65), UNSUPPORTED),
    (dict(G=40000), INVALID), (dict(ws=None), WORKSPACE), (dict(nbytes=10), WORKSPACE), (dict(ws=MIS), INVALID),
])
def test_beam_select_refusals(kw, status):
    if kw.get("M") == 301:                            # more than every candidate
        status = INVALID
    assert _call("gdr_beam_select", SELECT, SELECT_OK, kw) == status


REORDER = "state parent layers N K row flags".split()
REORDER_OK = dict(state=A, parent=A, layers=2, N=12, K=4, row=64, flags=0)


@pytest.mark.parametrize("kw,status", [
    (dict(state=None), INVALID), (dict(state=MIS), INVALID), (dict(parent=None), INVALID), (dict(parent=MIS), INVALID),
    (dict(layers=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(K=5), INVALID), (dict(row=0), INVALID),
    (dict(row=24), INVALID), (dict(row=1 << 41), INVALID), (dict(flags=1), INVALID), (dict(K=65, N=65), UNSUPPORTED),
    (dict(layers=1 << 20, N=1 << 20, K=1), INVALID), (dict(row=1 << 40), INVALID), (dict(N=1 << 24, K=1, row=1 << 20), INVALID),
])
def test_state_reorder_refusals(kw, status):
    assert _call("gdr_state_reorder", REORDER, REORDER_OK, kw) == status


def test_the_older_calls_do_not_know_the_new_flag():
    lib = _lib()
    assert lib.gdr_chunk_fwd(A, A, A, A, A, A, None, A, None, 1, 1, 64, 128, 128, 64, 0x8000, None, 0, None) == INVALID
    assert lib.gdr_attn_fwd(A, A, A, A, A, 1, 4, 2, 8, 8, 128, 0, 0.1, 0x8000, None) == INVALID


# ---------------------------------------------------------------------------
# the Python calls: tensors on the CPU, the GPU's part replaced
# ---------------------------------------------------------------------------


@pytest.fixture
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(gen, "_launch", lambda fn, gpu, stream, *a: made.append((fn, stream) + a))
    monkeypatch.setattr(gen, "_gpu_of", lambda name, t: t.get_device())
    return made


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _cache():
    return gdr.kv_cache(5, 2, 64, device="cpu")


def _q(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("call", [
    lambda: gen.attn_decode_shared(_q(3, 4, 64), _cache(), _i(3, 2), _i(3), _i(3), _i(1)),
    lambda: gen.attn_decode_shared(_q(3, 4, 64), _cache(), _i(3, 2), _i(3), _i(2).long(), _i(1)),
    lambda: gen.attn_decode_shared(_q(3, 4, 64), _cache(), _i(3, 2), _i(3), _i(3), _i(4)[::2]),
    lambda: gen.attn_decode_shared(_q(3, 4, 64), _cache(), _i(3, 2), _i(3), _i(2), _i(1), out_dtype=torch.float16),
    lambda: gen.attn_decode_shared(_q(3, 4, 64).float(), _cache(), _i(3, 2), _i(3), _i(2), _i(1)),
    lambda: gen.attn_decode_shared(_q(2, 4, 64), _cache(), _i(3, 2), _i(3), _i(2), _i(1)),
    lambda: gen.attn_decode_shared(_q(3, 4, 64), _cache(), _i(3, 2), _i(3), _i(2), _i(1), o=_q(3, 4, 64)),
    lambda: gen.kv_fork(_cache(), _i(3, 2), _i(2)),
    lambda: gen.kv_fork(_cache(), _i(3, 2), _i(3), parent=_i(4).long()),
    lambda: gen.kv_fork(_cache(), _i(3, 2), _i(3), parent=_i(4), room=_i(3)),
    lambda: gen.kv_fork(_cache(), _i(3, 2), _i(3), room=-1),
    lambda: gen.kv_fork(_cache(), _i(3, 2), _i(3), room=1 << 31),
    lambda: gen.kv_fork(_cache(), _i(3, 2), _i(3), held=_i(5)),
    lambda: gen.kv_fork(_cache(), _i(3, 2), _i(3), held=torch.zeros(4, dtype=torch.bool)),
    lambda: gen.kv_fork(_cache(), _i(3, 2), _i(3), parent=_i(4), table_out=_i(3, 2)),
    lambda: gen.kv_fork(_cache(), _i(3, 2), _i(3), len_out=_i(4)),
    lambda: gen.kv_compact(_cache(), _i(3, 2), _i(3), held=torch.zeros(6, dtype=torch.uint8)),
    lambda: gen.kv_compact(_cache(), _i(3, 2), _i(3), table_out=_i(3, 3)),
    lambda: gen.beam_select(torch.zeros(6, 9), torch.zeros(2, 2)),
    lambda: gen.beam_select(torch.zeros(6), torch.zeros(2, 3)),
    lambda: gen.beam_select(torch.zeros(9, 6).t(), torch.zeros(2, 3)),
    lambda: gen.beam_select(torch.zeros(6, 9).half(), torch.zeros(2, 3)),
    lambda: gen.beam_select(torch.zeros(6, 9), torch.zeros(2, 3).double()),
    lambda: gen.beam_select(torch.zeros(6, 9), torch.zeros(2, 3), ended=_i(2, 3)),
    lambda: gen.state_reorder(torch.zeros(6, 3), _i(6), 3),
    lambda: gen.state_reorder(torch.zeros(6, 4), _i(5), 3),
    lambda: gen.state_reorder(torch.zeros(6, 4), _i(6).long(), 3),
    lambda: gen.state_reorder(torch.zeros(4, 6).t(), _i(6), 3),
    lambda: gen.state_reorder(torch.zeros(6, 4), _i(6), 3, dim=2),
])
def test_python_refusals(call, calls):
    with pytest.raises(ValueError):
        call()
    assert not calls


def test_python_calls_name_their_tensors_in_the_librarys_order(calls):
    """Every call's arguments in number and kind as the library declares them."""
    lib = _lib()
    gen.attn_decode_shared(_q(3, 4, 64), _cache(), _i(3, 2), _i(3), _i(2), _i(1))
    gen.kv_fork(_cache(), _i(3, 2), _i(3), parent=_i(4), room=_i(4), held=torch.zeros(5, dtype=torch.bool))
    gen.kv_fork(_cache(), _i(3, 2), _i(3))
    gen.kv_compact(_cache(), _i(3, 2), _i(3))
    gen.beam_select(torch.zeros(6, 20)[:, :9], torch.zeros(2, 3), keep_slots=True)
    gen.state_reorder(torch.zeros(2, 6, 4, 5), _i(2, 3), 3, dim=1)
    assert len(calls) == 6
    for fn, _, *args in calls:
        types = getattr(lib, fn).argtypes
        assert len(args) + 1 == len(types), fn
        for t, a in zip(types, args):
            t(a)                                      # converts, or raises
        # the C-named call takes the same arguments in the same order
        import inspect
        assert len(inspect.signature(getattr(gdr, fn)).parameters) == len(types), fn
    assert calls[4][13] == 20 and calls[4][15] == gdr.GDR_ACT_F32 | gdr.GDR_KEEP_SLOTS
    assert calls[5][4:8] == (2, 6, 3, 80)
