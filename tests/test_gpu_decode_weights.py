"""Single-token attention over the cache: the page that stands in for a missing one, and
the weights' 22 bits."""
import math

import pytest
import torch

import gated_delta_rule_24_amd as gdr
from tests.test_gpu_kv import _cache, _decode_check, _rand

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.mark.parametrize("value", [math.nan, math.inf, 0.0])
def test_what_stands_in_for_a_missing_page_does_not_matter(value):
    """Page 0, which no table names, full of NaN and with any scale."""
    lens = [70, 190, 5]
    c = _cache(10, 1, 64, seed=20)
    table = 1 + torch.randperm(9, generator=torch.Generator().manual_seed(21)).view(3, 3).int()
    q = _rand((3, 4, 64), 22)
    for bad in (10, -1, 2 ** 31 - 1, -2 ** 31):
        table[1, 1] = bad                                # a page among the tokens counts as masked
        table[2, 0] = bad                                # so does a sequence's only one: nothing is seen
        want = _decode_check(c, q, table, lens)
        assert not bool(want[2].any())
        c2 = gdr.KVCache(*[t.clone() for t in c])
        c2.k[0].fill_(0x7f), c2.v[0].fill_(0xff), c2.k_scale[0].fill_(value), c2.v_scale[0].fill_(value)
        got = gdr.attn_decode(q.cuda(), c2, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
        assert torch.equal(got, want)


@pytest.mark.parametrize("far", [0, 1000])
def test_a_weight_keeps_22_bits(far):
    """Two keys with scores 0 and s, values 0 and 1: o = w / (1 + w), w = exp(s), which shows
    the rounding of one weight.  (far: as many keys before them whose scores leave their
    weights 0, so that the pages are split over workgroups.)

    The bound: s itself is exact (8 by 4 significant bits).  In base 2 it is off by three
    roundings (log2 e, its product with the scale, with the dot product): 3 * 2^-24 |s2|; the
    exponent s2 + 15 by half a step of values below 16, 2^-21, and where the splits are joined
    by as much again; both times ln 2.  The exponential is off by 2^-22 (two units), the weight
    as two f16 parts by 2^-22, the products, the sum 1 + w and the quotient by four roundings
    of 2^-24; w's error counts once more in the sum.  Two bf16 parts would be off by up to 2^-16.
    """
    N, Hq, d = 32, 16, 64
    g = torch.Generator().manual_seed(5)
    width = (far + 2 + 63) // 64
    c = gdr.kv_cache(N * width, 1, d)
    c.k.fill_(0), c.v.fill_(0), c.k_scale.fill_(1.0), c.v_scale.fill_(1.0)
    table = torch.arange(N * width).view(N, width).int()
    one, big = 0x38, 0x7e                                # 1 and 448
    for n in range(N):
        for t in range(far):
            c.k[n * width + t // 64, 0, t % 64, 1] = big # against q's -2^10 there: a score of -57,344
        at, pg = (far + 1) % 64, n * width + (far + 1) // 64
        c.k[pg, 0, at, 0] = one
        c.v[pg, 0, at // 16, :, at % 16] = one
    q = torch.zeros((N, Hq, d), dtype=torch.bfloat16)
    q[:, :, 0] = -(torch.rand((N, Hq), generator=g) * 24 + 0.1).to(torch.bfloat16)
    q[:, :, 1] = -2.0 ** 10
    o = gdr.attn_decode(q.cuda(), c, table.cuda(), torch.full((N,), far + 2, dtype=torch.int32, device="cuda"))
    s = q[:, :, 0].to(F64) / 8
    w = torch.exp(s)
    want = w / (1 + w)
    rel = math.log(2) * (3 * 2.0 ** -24 * s.abs() / math.log(2) + 2 * 2.0 ** -21) + 2.0 ** -22
    tol = want * (2 * rel + 2.0 ** -22 + 4 * 2.0 ** -24)
    off = (o.cpu().to(F64) - want[..., None]).abs() - tol[..., None]
    assert float(off.max()) <= 0, f"{float((off / want[..., None]).max()):.3g} of the value over the bound"
