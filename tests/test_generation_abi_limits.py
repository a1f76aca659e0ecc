"""The sizes that the calls for several continuations support: the last of each is accepted, the
first past it refused.  (Fake aligned pointers, never dereferenced; without a GPU an accepted
call ends at the device check.)"""
import pytest
import torch

from tests.test_attn_abi import INVALID, UNSUPPORTED, _call, _lib
from tests.test_generation_abi import (COMPACT, COMPACT_OK, FORK, FORK_OK, REORDER, REORDER_OK, SELECT, SELECT_OK, SHARED,
                                       SHARED_OK)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="an accepted call would run")
DEVICE = 5
FORK_OK = {**FORK_OK, "Hkv": 1}
CALLS = dict(shared=("gdr_attn_decode_shared", SHARED, SHARED_OK), fork=("gdr_kv_fork", FORK, FORK_OK),
             compact=("gdr_kv_compact", COMPACT, {**COMPACT_OK, "Hkv": 1}), select=("gdr_beam_select", SELECT, SELECT_OK),
             reorder=("gdr_state_reorder", REORDER, REORDER_OK))


@pytest.mark.parametrize("call,most,over,status", [
    ("shared", dict(N=1, width=1 << 24), dict(N=1, width=(1 << 24) + 1), INVALID),
    # (waves, units and heads are numbered up to 2^24 - 1, some of them spare)
    ("shared", dict(N=(1 << 24) - (1 << 15), Hq=1, Hkv=1, width=1), dict(N=(1 << 24) - 1, Hq=1, Hkv=1, width=1), INVALID),
    ("shared", dict(N=(1 << 21) - (1 << 12), Hq=8, Hkv=8, width=1, groups=4096), dict(N=1 << 21, Hq=8, Hkv=8, width=1), INVALID),
    ("shared", dict(N=2, Hq=(1 << 23) - (1 << 14), Hkv=1), dict(N=2, Hq=1 << 23, Hkv=1), INVALID),
    ("shared", dict(N=2, Hq=(1 << 23) - (1 << 14), Hkv=(1 << 23) - (1 << 14)), dict(N=2, Hq=1 << 23, Hkv=1 << 23), INVALID),
    ("shared", dict(groups=4096), dict(groups=4097), UNSUPPORTED),
    ("fork", dict(N=1 << 20), dict(N=(1 << 20) + 1), INVALID),
    ("fork", dict(Nin=1 << 20), dict(Nin=(1 << 20) + 1), INVALID),
    ("fork", dict(Hkv=65535), dict(Hkv=65536), INVALID),
    ("fork", dict(pages=1 << 30), dict(pages=(1 << 30) + 1), INVALID),
    ("fork", dict(N=127, width=1 << 24), dict(N=127, width=(1 << 24) + 1), INVALID),
    ("fork", dict(N=1 << 20, width=2047), dict(N=1 << 20, width=2048), INVALID),
    ("fork", dict(Nin=1 << 20, width=2047), dict(Nin=1 << 20, width=2048), INVALID),
    ("compact", dict(N=1 << 20), dict(N=(1 << 20) + 1), INVALID),
    ("compact", dict(Hkv=65535), dict(Hkv=65536), INVALID),
    ("compact", dict(pages=1 << 30), dict(pages=(1 << 30) + 1), INVALID),
    ("compact", dict(N=127, width=1 << 24), dict(N=127, width=(1 << 24) + 1), INVALID),
    ("compact", dict(N=1 << 20, width=2047), dict(N=1 << 20, width=2048), INVALID),
    ("select", dict(G=65535, K=1, M=1), dict(G=65536, K=1, M=1), INVALID),
    ("select", dict(G=1023, K=64, M=64), dict(G=1024, K=64, M=64), INVALID),
    ("select", dict(V=1 << 26, stride=1 << 40), dict(V=1 << 26, stride=(1 << 40) + 1), INVALID),
    ("select", dict(V=1 << 26, stride=1 << 27), dict(V=(1 << 26) + 1, stride=1 << 27), UNSUPPORTED),
    ("reorder", dict(layers=1 << 22, N=64, K=64, row=16), dict(layers=(1 << 22) + 1, N=64, K=64, row=16), INVALID),
    ("reorder", dict(layers=1, N=4, K=4, row=16 * 256 * ((1 << 24) - 1)), dict(layers=1, N=4, K=4, row=16 * 256 * ((1 << 24) - 1) + 16), INVALID),
])
def test_the_last_size_and_the_first_past_it(call, most, over, status):
    name, order, base = CALLS[call]
    assert _call(name, order, base, most) == DEVICE
    assert _call(name, order, base, over) == status


def test_the_workspace_query_of_the_same_sizes():
    f = _lib().gdr_beam_select_workspace_bytes
    assert f(65535, 1, 1, 100) > 0 and f(65536, 1, 1, 100) == 0
