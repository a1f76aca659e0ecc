"""Calls of more workgroups than one launch takes (2^24 - 1 of 256 threads) are refused by
their sizes before anything is launched, and those of as many are not.  (Fake aligned
pointers, never dereferenced; without a GPU an accepted call ends at the device check.)"""
import pytest
import torch

from tests.test_attn_abi import (APP, APP_OK, BWD, BWD_OK, BWDV, DEC, DEC_OK, FWD, FWD_OK, FWDV, FWDV_OK, ROPE, ROPE_OK, A, INVALID,
                                 _call)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="an accepted call would run")
DEVICE = 5


@pytest.mark.parametrize("name,order,base,over,most", [
    ("gdr_attn_fwd", FWD, FWD_OK, dict(B=1 << 20, Hq=16, Hkv=16, Tq=1, Tk=1), dict(B=(1 << 20) - 1, Hq=16, Hkv=16, Tq=1, Tk=1)),
    ("gdr_attn_fwd", FWD, FWD_OK, dict(B=1 << 16, Hq=16, Hkv=1, Tq=1921, Tk=1), dict(B=1 << 16, Hq=16, Hkv=1, Tq=1920, Tk=1)),
    ("gdr_attn_fwd_varlen", FWDV, FWDV_OK, dict(Hq=1 << 16, Hkv=1, T=32768 - 127), dict(Hq=1 << 16, Hkv=1, T=32768 - 128)),
    ("gdr_attn_bwd", BWD, BWD_OK, dict(B=1 << 19, Hq=16, Hkv=16, Tq=1, Tk=1), dict(B=(1 << 19) - 1, Hq=16, Hkv=16, Tq=1, Tk=1)),
    ("gdr_attn_bwd", BWD, BWD_OK, dict(B=1, Hq=4, Hkv=4, Tq=1 << 30, Tk=1), dict(B=1, Hq=4, Hkv=4, Tq=1 << 25, Tk=1)),
    ("gdr_attn_bwd_varlen", BWDV, {**BWD_OK, "cu": A, "nseq": 2}, dict(Hq=1 << 14, Hkv=1, T=1 << 15), dict(Hq=1 << 14, Hkv=1, T=1 << 13)),
    ("gdr_rope", ROPE, ROPE_OK, dict(B=1, Hq=1, Hk=0, T=1 << 30), dict(B=1, Hq=1, Hk=0, T=(1 << 29) - 32)),
    ("gdr_kv_append", APP, APP_OK, dict(nseq=1 << 23, Hkv=16, T=1 << 23, cu=None), dict(nseq=(1 << 23) - 1, Hkv=16, T=(1 << 23) - 1, cu=None)),
    ("gdr_kv_append", APP, APP_OK, dict(nseq=1 << 23, T=64), dict(nseq=(1 << 23) - 2, T=64)),
    ("gdr_attn_decode", DEC, DEC_OK, dict(N=1 << 20, Hq=16, Hkv=16, width=1), dict(N=(1 << 20) - 1, Hq=16, Hkv=16, width=1)),
    ("gdr_attn_decode", DEC, DEC_OK, dict(N=1 << 18, Hq=1 << 10, Hkv=1, width=1 << 16), dict(N=1 << 17, Hq=1 << 10, Hkv=1, width=1 << 16)),
])
def test_grids(name, order, base, over, most):
    assert _call(name, order, base, {**over, "nbytes": 1 << 62} if "ws" in order else over) == INVALID
    assert _call(name, order, base, {**most, "nbytes": 1 << 62} if "ws" in order else most) == DEVICE


def test_refused_calls_need_no_workspace():
    from tests.test_abi import _lib
    assert _lib().gdr_attn_bwd_workspace_bytes(1 << 19, 16, 16, 1, 1, 128) == 0
    assert _lib().gdr_attn_bwd_workspace_bytes((1 << 19) - 1, 16, 16, 1, 1, 128) > 0
