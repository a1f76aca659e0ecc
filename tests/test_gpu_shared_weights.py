"""Attention over shared pages: a bf16 result is the fp32 one rounded once, and a weight's 22
bits in either."""
import math

import pytest
import torch

import gated_delta_rule_24_amd as gdr
from tests import test_gpu_shared as base

pytestmark = pytest.mark.gpu
gen = gdr.generation
F64 = torch.float64

# sizes of the groups, pages that each shares, query heads on key heads: own pages alone, 32 rows a
# wave without and (more than 64 groups) with a kernel for the plan, 64 rows a wave, several tiles of them
SIZES = [([3], [0], 8, 2), ([4, 1, 6], [3, 0, 1], 9, 3), ([1] * 70, [1] * 70, 2, 1), ([5, 4], [4, 2], 140, 1), ([150], [9], 4, 2)]


@pytest.mark.parametrize("sizes,shared,Hq,Hkv", SIZES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [0, 100])
def test_a_bf16_result_is_the_fp32_one_rounded(sizes, shared, Hq, Hkv, d, window):
    """The arithmetic does not depend on the result's type: bit for bit."""
    g = torch.Generator().manual_seed(len(sizes) + Hq)
    lens = []
    for n, p in zip(sizes, shared):
        lens += [p * 64 + int(x) for x in torch.randint(0, 400, (n,), generator=g)]
    total, table = base._tables(sizes, shared, lens, 3)
    c, q = base._cache(total, Hkv, d, 4), base._rand((len(lens), Hq, d), 5)
    full, one = [base._call(c, q, table, lens, base._starts(sizes), shared, window, out=t) for t in (torch.float32, torch.bfloat16)]
    assert torch.equal(one, full.to(torch.bfloat16))


@pytest.mark.parametrize("shared", [0, 1])
@pytest.mark.parametrize("Hq", [16, 70])
@pytest.mark.parametrize("far", [0, 1000])
def test_a_weight_keeps_22_bits(far, Hq, shared):
    """Two keys with scores 0 and s, values 0 and 1: o = w / (1 + w), w = exp(s), which shows
    the rounding of one weight; `far` keys before them have weights of 0.  They are among a group's
    shared pages or each sequence's own.

    The bound: s itself is exact (8 by 4 significant bits).  In base 2 it is off by three roundings
    (log2 e, its product with the scale, with the dot product): 3 * 2^-24 |s2|; the exponent s2 + b
    of the weight by half a step of values below 16, 2^-21, and the one that takes it back
    to the maximum, and where runs of pages are joined, by as much again: three times, times ln 2.
    The exponentials are off by 2^-22 each (the weight, and those two), the weight as two f16 parts by
    2^-22 (a step of 2^-24 below f16's normal range is 2^-36 of the largest), the products, the sum
    1 + w and the quotient by four roundings of 2^-24, the sum's own factors by two more; w's
    error counts once more in the sum.  One f16 part would be off by up to 2^-12."""
    N, d = 8, 64
    g = torch.Generator().manual_seed(5)
    width = (far + 2 + 63) // 64
    groups = 2 if shared else N
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
    starts = torch.arange(0, N + 1, N // groups)
    o = base._call(c, q, table, [far + 2] * N, starts, [width if shared else 0] * groups)
    s = q[:, :, 0].to(F64) / 8
    w = torch.exp(s)
    want = w / (1 + w)
    rel = math.log(2) * (3 * 2.0 ** -24 * s.abs() / math.log(2) + 3 * 2.0 ** -21) + 3 * 2.0 ** -22
    tol = want * (2 * rel + 2.0 ** -22 + 2.0 ** -35 / w + 6 * 2.0 ** -24)
    off = (o.cpu().to(F64) - want[..., None]).abs() - tol[..., None]
    assert float(off.max()) <= 0, f"{float((off / want[..., None]).max()):.3g} of the value over the bound"
