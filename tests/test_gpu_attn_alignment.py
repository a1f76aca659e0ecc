"""A tensor that does not start at a multiple of 16 bytes is refused by its name."""
import pytest
import torch

import gated_delta_rule_24_amd as gdr

pytestmark = pytest.mark.gpu


def _int(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


def _x(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")


def _off(*shape):
    n = _x(*shape).numel()
    return _x(n + 1)[1:].view(shape)


def test_slices_are_refused_by_name():
    q, f = _x(1, 2, 4, 64), gdr.rope_frequencies(32)[0]
    cache, table = gdr.kv_cache(3, 2, 64), _int(4, 1)
    k = _x(4, 2, 64)
    calls = [("positions", lambda: gdr.rope(q, None, f, _int(1, 9)[:, 5:])),
             ("q", lambda: gdr.rope(_off(1, 2, 4, 64), None, f)),
             ("k", lambda: gdr.attn_fwd(q, _off(1, 2, 4, 64), q)),
             ("cu_seqlens", lambda: gdr.attn_fwd_varlen(q[0], q[0], q[0], _int(9)[5:7])),
             ("dO", lambda: gdr.attn_bwd(q, q, q, q, torch.zeros((1, 2, 4), device="cuda"), _off(1, 2, 4, 64))),
             ("cache_len", lambda: gdr.kv_append(k, k, cache, table, _int(9)[5:])),
             ("block_table, cache_len", lambda: gdr.attn_decode(k, cache, _int(9, 1)[5:], _int(9)[5:]))]
    for name, call in calls:
        with pytest.raises(gdr.GdrError, match=rf"\(.*: {name} must start at a multiple of 16 bytes") as e:
            call()
        assert e.value.status == 1
    with pytest.raises(gdr.GdrError, match=r"\([^:]*\)$"):
        gdr.attn_fwd(q, q, q, window=-1)
    with pytest.raises(gdr.GdrError, match=r"\([^:]*\)$"):
        gdr.attn_fwd(q, q, q, scale=0.0)
