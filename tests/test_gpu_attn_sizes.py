"""Sizes past 32 bits at the Python entry points: a window past every length is none, a
first position that the library cannot number is refused."""
import pytest
import torch

import gated_delta_rule_24_amd as gdr
from tests.test_gpu_attn import _inputs

pytestmark = pytest.mark.gpu

FAR = [2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1, 2 ** 70 + 3]


@pytest.mark.parametrize("window", FAR)
def test_attention_windows_past_32_bits_are_none(window):
    x = {n: t.cuda() for n, t in _inputs(1, 2, 1, 100, 100, 64, 1).items()}
    cu = torch.tensor([0, 40, 100], dtype=torch.int32, device="cuda")
    q, k, v, dO = (x[n] for n in ("q", "k", "v", "dO"))
    o, lse = gdr.attn_fwd(q, k, v)
    o2, lse2 = gdr.attn_fwd(q, k, v, window=window)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g, g2 = gdr.attn_bwd(q, k, v, o, lse, dO), gdr.attn_bwd(q, k, v, o, lse, dO, window=window)
    assert all(torch.equal(g[n], g2[n]) for n in g)
    q, k, v, dO = q[0], k[0], v[0], dO[0]
    o, lse = gdr.attn_fwd_varlen(q, k, v, cu)
    o2, lse2 = gdr.attn_fwd_varlen(q, k, v, cu, window=window)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g, g2 = gdr.attn_bwd_varlen(q, k, v, o, lse, dO, cu), gdr.attn_bwd_varlen(q, k, v, o, lse, dO, cu, window=window)
    assert all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("window", FAR)
def test_decode_windows_past_32_bits_are_none(window):
    c = gdr.kv_cache(4, 1, 64)
    g = torch.Generator().manual_seed(2)
    k, v, q = (torch.randn(s, generator=g).to(torch.bfloat16).cuda() for s in ((1, 200, 64), (1, 200, 64), (1, 4, 64)))
    table = torch.tensor([[3, 1, 0, 2]], dtype=torch.int32, device="cuda")
    have, cu = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    gdr.kv_append(k, v, c, table, have, cu)
    have += 200
    assert torch.equal(gdr.attn_decode(q, c, table, have), gdr.attn_decode(q, c, table, have, window=window))


def test_windows_below_zero_are_refused():
    x = torch.zeros((1, 2, 8, 64), dtype=torch.bfloat16, device="cuda")
    for w in (-1, -2 ** 31, -2 ** 32 + 5, -2 ** 64 + 3):
        with pytest.raises(gdr.GdrError):
            gdr.attn_fwd(x, x, x, window=w)


def test_positions_past_32_bits_are_refused():
    x = torch.zeros((1, 2, 8, 64), dtype=torch.bfloat16, device="cuda")
    f, _ = gdr.rope_frequencies(32)
    for p in (2 ** 31, 2 ** 32 + 7, -2 ** 31 - 1):
        with pytest.raises(ValueError):
            gdr.rope(x, None, f, position0=p)
    a, _ = gdr.rope(x + 1, None, f, position0=2 ** 31 - 1)
    b, _ = gdr.rope(x + 1, None, f, torch.full((1, 8), 2 ** 31 - 1, dtype=torch.int32, device="cuda"))
    assert torch.equal(a[:, :, 0], b[:, :, 0])
