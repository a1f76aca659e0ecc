"""Argument checks of the attention layer's calls: every refusal happens before
a device is touched (fake aligned pointers, never dereferenced), so these run
without a GPU."""
import ctypes
import math

import pytest

A = ctypes.c_void_p(0x10000)
MIS = ctypes.c_void_p(0x10004)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
BIG = (1 << 31) - 1


def _lib():
    from tests.test_abi import _lib as load
    return load()


def _call(name, order, base, kw):
    a = dict(base)
    a.update(kw)
    return getattr(_lib(), name)(*[a[x] for x in order], None)


ROPE = ("q k qo ko f pos p0 B Hq Hk T d rot scale flags").split()
ROPE_OK = dict(q=A, k=A, qo=A, ko=A, f=A, pos=A, p0=0, B=2, Hq=4, Hk=2, T=8, d=128, rot=64, scale=1.0, flags=0)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(ko=None), INVALID), (dict(f=None), INVALID), (dict(q=MIS), INVALID),
    (dict(pos=MIS), INVALID), (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(Hq=0, Hk=0), INVALID),
    (dict(Hq=-1), INVALID), (dict(flags=0x2), INVALID), (dict(flags=0x8000), INVALID), (dict(rot=0), INVALID),
    (dict(rot=144), INVALID), (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID),
    (dict(rot=24), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(d=256, rot=256), UNSUPPORTED),
    (dict(B=BIG, Hq=BIG), INVALID), (dict(B=1 << 15, T=1 << 20), INVALID),
])
def test_rope_refusals(kw, status):
    assert _call("gdr_rope", ROPE, ROPE_OK, kw) == status


FWD = "q k v o lse B Hq Hkv Tq Tk d window scale flags".split()
FWD_OK = dict(q=A, k=A, v=A, o=A, lse=A, B=1, Hq=4, Hkv=2, Tq=8, Tk=8, d=128, window=0, scale=0.1, flags=0)
SIZES = [
    (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=3), INVALID), (dict(window=-1), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID),
    (dict(scale=math.inf), INVALID), (dict(flags=0x2), INVALID), (dict(flags=0x2000), INVALID),
    (dict(flags=0x1), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(d=32), UNSUPPORTED), (dict(d=256), UNSUPPORTED),
    (dict(B=1 << 20, Hq=1 << 20, Hkv=1 << 20), INVALID),
]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(q=None), INVALID), (dict(v=None), INVALID), (dict(o=None), INVALID), (dict(lse=MIS), INVALID),
    (dict(k=MIS), INVALID), (dict(Tq=-1), INVALID), (dict(Tk=-1), INVALID), (dict(Tk=BIG), INVALID),
    (dict(Tq=BIG), INVALID),
])
def test_attn_fwd_refusals(kw, status):
    assert _call("gdr_attn_fwd", FWD, FWD_OK, kw) == status


FWDV = "q k v o lse cu nseq Hq Hkv T d window scale flags".split()
FWDV_OK = dict(q=A, k=A, v=A, o=A, lse=A, cu=A, nseq=2, Hq=4, Hkv=2, T=8, d=64, window=0, scale=0.1, flags=0)


@pytest.mark.parametrize("kw,status", [
    (dict(cu=None), INVALID), (dict(cu=MIS), INVALID), (dict(nseq=0), INVALID), (dict(nseq=(1 << 30) + 1), INVALID), (dict(q=None), INVALID),
    (dict(T=-1), INVALID), (dict(d=16), UNSUPPORTED), (dict(flags=0x1), UNSUPPORTED), (dict(Hq=5), INVALID),
])
def test_attn_fwd_varlen_refusals(kw, status):
    assert _call("gdr_attn_fwd_varlen", FWDV, FWDV_OK, kw) == status


BWD = "q k v o lse dO dq dk dv B Hq Hkv Tq Tk d window scale flags ws nbytes".split()
BWD_OK = dict(q=A, k=A, v=A, o=A, lse=A, dO=A, dq=A, dk=A, dv=A, B=1, Hq=4, Hkv=2, Tq=8, Tk=8, d=128, window=0,
              scale=0.1, flags=0, ws=A, nbytes=1 << 40)


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(lse=None), INVALID), (dict(dO=None), INVALID), (dict(dq=None), INVALID), (dict(dk=None), INVALID),
    (dict(dv=MIS), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=MIS), INVALID), (dict(nbytes=15), WORKSPACE),
])
def test_attn_bwd_refusals(kw, status):
    assert _call("gdr_attn_bwd", BWD, BWD_OK, kw) == status


BWDV = "q k v o lse dO dq dk dv cu nseq Hq Hkv T d window scale flags ws nbytes".split()


@pytest.mark.parametrize("kw,status", [
    (dict(cu=None), INVALID), (dict(cu=MIS), INVALID), (dict(nseq=0), INVALID), (dict(nseq=(1 << 30) + 1), INVALID), (dict(dk=None), INVALID),
    (dict(nbytes=0), WORKSPACE), (dict(d=48), UNSUPPORTED),
])
def test_attn_bwd_varlen_refusals(kw, status):
    base = {**BWD_OK, "cu": A, "nseq": 2, "T": 8}
    assert _call("gdr_attn_bwd_varlen", BWDV, base, kw) == status


def test_attn_bwd_workspace_query():
    f = _lib().gdr_attn_bwd_workspace_bytes
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    # D and the log-sum-exps of every query row, fp32
    assert f(1, 2, 2, 100, 100, 128) == up(2 * 2 * 100 * 4)
    # few key tiles and shared heads: the heads' partial dk and dv in fp32 (a split each)
    assert f(1, 4, 1, 100, 100, 64) == up(2 * 4 * 100 * 4) + 2 * 4 * 100 * 64 * 4
    # enough key tiles: no partials
    assert f(8, 16, 8, 8192, 8192, 128) == 2 * 8 * 16 * 8192 * 4
    for bad in ((0, 2, 2, 8, 8, 64), (1, 3, 2, 8, 8, 64), (1, 2, 2, -1, 8, 64), (1, 2, 2, 8, 8, 96)):
        assert f(*bad) == 0


APP = "k v kc vc ks vs table len cu nseq Hkv T d pages width flags".split()
APP_OK = dict(k=A, v=A, kc=A, vc=A, ks=A, vs=A, table=A, len=A, cu=A, nseq=3, Hkv=2, T=10, d=128, pages=8, width=4,
              flags=0)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(vc=None), INVALID), (dict(ks=None), INVALID), (dict(table=None), INVALID),
    (dict(len=None), INVALID), (dict(len=MIS), INVALID), (dict(cu=None), INVALID), (dict(nseq=0), INVALID),
    (dict(T=-1), INVALID), (dict(pages=0), INVALID), (dict(width=0), INVALID), (dict(flags=0x1), INVALID),
    (dict(flags=0x2), INVALID), (dict(d=32), UNSUPPORTED), (dict(Hkv=65536), INVALID),
    (dict(nseq=1 << 16, T=1 << 30), INVALID),
])
def test_kv_append_refusals(kw, status):
    assert _call("gdr_kv_append", APP, APP_OK, kw) == status


DEC = "q kc vc ks vs table len o N Hq Hkv d pages width window scale flags ws nbytes".split()
DEC_OK = dict(q=A, kc=A, vc=A, ks=A, vs=A, table=A, len=A, o=A, N=2, Hq=8, Hkv=2, d=128, pages=8, width=4, window=0,
              scale=0.1, flags=0, ws=A, nbytes=1 << 40)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(vs=None), INVALID), (dict(table=MIS), INVALID),
    (dict(N=0), INVALID), (dict(Hq=7), INVALID), (dict(pages=0), INVALID), (dict(width=0), INVALID),
    (dict(width=1 << 25), INVALID), (dict(window=-1), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=math.nan), INVALID), (dict(flags=0x1), INVALID), (dict(flags=0x1000), INVALID),
    (dict(d=256), UNSUPPORTED), (dict(N=1, width=4096, ws=None), WORKSPACE), (dict(N=1, width=4096, nbytes=0), WORKSPACE),
    (dict(N=1, width=4096, ws=MIS), INVALID),
])
def test_attn_decode_refusals(kw, status):
    assert _call("gdr_attn_decode", DEC, DEC_OK, kw) == status


def test_attn_decode_workspace_query():
    f = _lib().gdr_attn_decode_workspace_bytes
    assert f(64, 32, 8, 128, 1, 0) == 0                     # one page: one split
    one = f(1, 32, 8, 128, 1024, 0)
    assert one > 0 and one % ((128 + 2) * 32 * 4) == 0      # per split: an output row, its maximum and sum
    assert f(1, 32, 8, 128, 1024, 64) < one                 # a window bounds the pages read
    assert f(0, 32, 8, 128, 1024, 0) == 0 and f(1, 31, 8, 128, 1024, 0) == 0


def test_flags_of_the_attention_layer_are_not_the_recurrences():
    """The older calls keep refusing flags they do not know."""
    lib = _lib()
    for fl in (0x1000, 0x2000, 0x4000):
        assert lib.gdr_chunk_fwd(A, A, A, A, A, A, None, A, None, 1, 1, 64, 128, 128, 64, fl, None, 0, None) == INVALID
        assert lib.gdr_decode_step(A, A, A, A, A, A, A, A, 4, 2, 128, 128, fl, None) == INVALID
