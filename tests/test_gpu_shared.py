"""Attention of one token per sequence over pages that groups of sequences share,
against each sequence's own softmax in 64 bits."""
import math

import pytest
import torch

import gated_delta_rule_24_amd as gdr
from tests import attn_reference as attn
from tests import generation_reference as ref

pytestmark = pytest.mark.gpu
gen = gdr.generation
F64 = torch.float64


def _rand(shape, seed, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _cache(n_pages, H, d, seed):
    g = torch.Generator().manual_seed(seed)
    c = gdr.kv_cache(n_pages, H, d, device="cpu")
    for x in (c.k, c.v):
        x.copy_((torch.randn(x.shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    for x in (c.k_scale, c.v_scale):
        x.copy_(torch.pow(2.0, torch.randint(-8, -4, x.shape, generator=g).float()))
    return c


def _tables(sizes, shared, lens, seed, spare=2):
    """Shuffled pages; only the group's first row names the shared ones, the others have
    entries there that are no pages."""
    N, width = sum(sizes), max([1] + [ref.pages_of(n) for n in lens] + [p for p in shared])
    total = N * width + spare
    order = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).int()
    table = order[:N * width].view(N, width).clone()
    at = 0
    for size, p in zip(sizes, shared):
        table[at + 1:at + size, :p] = -5
        at += size
    return total, table


def _call(c, q, table, lens, starts, shared, window=0, scale=None, out=torch.float32):
    dev = c if c.k.is_cuda else gdr.KVCache(*[x.cuda() for x in c])
    ints = [torch.as_tensor(x, dtype=torch.int32).cuda() for x in (table, lens, starts, shared)]
    return gen.attn_decode_shared(q.cuda(), dev, *ints, window=window, scale=scale, out_dtype=out)


def _check(c, q, table, lens, starts, shared, window=0, scale=None):
    host = attn.Cache(*c)
    for out in (torch.float32, torch.bfloat16):
        got = _call(c, q, table, lens, starts, shared, window, scale, out)
        want, tol = ref.shared_decode(q.to(F64), host, table, lens, starts, shared, window, scale, out is torch.bfloat16)
        off = (got.cpu().to(F64) - want).abs()
        assert bool((off <= tol).all()), f"{out}: {float((off / tol.clamp_min(1e-300)).max()):.3g} of the bound"
    return got


def _starts(sizes):
    s = [0]
    for n in sizes:
        s.append(s[-1] + n)
    return s


SIZES = [
    # sizes of the groups, pages that each shares, query heads on key heads
    ([1], [0], 1, 1), ([1], [3], 4, 4), ([4], [2], 8, 2), ([4, 1, 6], [3, 0, 1], 9, 3), ([2, 0, 3], [2, 4, 1], 16, 1),
    ([5, 5], [4, 2], 20, 1), ([33], [3], 4, 2), ([3] * 30, [i % 3 for i in range(30)], 4, 4), ([70], [2], 3, 1),
    ([1] * 70, [1] * 70, 2, 1), ([12], [9], 40, 2),
]


@pytest.mark.parametrize("sizes,shared,Hq,Hkv", SIZES)
@pytest.mark.parametrize("d", [64, 128])
def test_against_each_sequence_alone(sizes, shared, Hq, Hkv, d):
    g = torch.Generator().manual_seed(len(sizes) + Hq)
    lens = []
    for n, p in zip(sizes, shared):
        lens += [p * 64 + int(x) for x in torch.randint(1, 150, (n,), generator=g)]
    total, table = _tables(sizes, shared, lens, 3)
    q = _rand((len(lens), Hq, d), 5)
    _check(_cache(total, Hkv, d, 4), q, table, lens, _starts(sizes), shared)


@pytest.mark.parametrize("window", [1, 63, 64, 100, 200, 1 << 40])
def test_windows_and_lengths_of_any_kind(window):
    """Sequences that end inside the shared pages or have none of them, windows that reach
    into them or not."""
    sizes, shared = [7, 4, 9], [4, 0, 2]
    lens = [0, 1, 63, 64, 65, 256, 300, 0, 5, 128, 129, 400, 130, 1, 0, 200, 127, 128, 3, 64]
    for Hq, Hkv, d in ((8, 2, 64), (6, 1, 128), (20, 1, 64)):
        total, table = _tables(sizes, shared, lens, 8)
        out = _check(_cache(total, Hkv, d, 9), _rand((20, Hq, d), 10), table, lens, _starts(sizes), shared, min(window, 1 << 30))
        assert not bool(out[torch.tensor([n == 0 for n in lens])].any())
    if window > 1 << 31:
        c, q = _cache(total, 1, 64, 9), _rand((20, 20, 64), 10)
        assert torch.equal(_call(c, q, table, lens, _starts(sizes), shared, window), _call(c, q, table, lens, _starts(sizes), shared))


def test_long_prefix_split_over_workgroups():
    sizes, shared, lens = [6, 2], [130, 77], [130 * 64 + n for n in (1, 70, 64, 3, 200, 9)] + [77 * 64 + 5, 77 * 64 + 600]
    for Hq, Hkv, d in ((4, 1, 128), (16, 1, 64)):
        total, table = _tables(sizes, shared, lens, 11)
        _check(_cache(total, Hkv, d, 12), _rand((8, Hq, d), 13), table, lens, _starts(sizes), shared)


def test_sequences_in_no_group_share_nothing():
    lens = [200, 130, 90, 200, 64]
    total, table = _tables([2, 2, 1], [0, 2, 0], lens, 14)
    c, q = _cache(total, 2, 64, 15), _rand((5, 8, 64), 16)
    got = _call(c, q, table, lens, [2, 4], [2])
    full = _call(c, q, table, lens, [0, 2, 4, 5], [0, 2, 0])
    assert torch.equal(got, full)
    _check(c, q, table, lens, [2, 4], [2])


@pytest.mark.parametrize("starts,shared", [([0, 9, 3], [2, 2]), ([-4, 2, 100], [1, 2]), ([5, 5, 5], [3, 3]), ([3, 1, 2], [1 << 30, -3]),
                                           ([-2 ** 31, 2 ** 31 - 1, 4], [-2 ** 31, 2 ** 31 - 1])])
def test_any_content_of_groups_stays_inside(starts, shared):
    """Bounds that are none: nothing but the result is wrong (sequences in one group alone are right)."""
    lens = [200, 130, 90, 200, 64]
    total, table = _tables([5], [0], lens, 14)
    guard = torch.full((5 + 2, 8, 64), 7.0, device="cuda")
    c = gdr.KVCache(*[x.cuda() for x in _cache(total, 2, 64, 15)])
    ints = [torch.as_tensor(x, dtype=torch.int32).cuda() for x in (table, lens, starts, shared)]
    gen.attn_decode_shared(_rand((5, 8, 64), 16).cuda(), c, *ints, o=guard[1:6])
    assert bool((guard[0] == 7).all()) and bool((guard[6] == 7).all())


@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (12, 2)])
def test_what_a_sequence_does_not_see_does_not_matter(window, Hq, Hkv):
    """NaN and other bytes in slots that one sequence of the group sees and another does
    not: the one that does not has the same bits, the one that does has NaN."""
    sizes, shared, d = [6, 2], [3, 1], 64
    lens = [70, 192, 200, 130, 1, 64, 64, 100]
    total, table = _tables(sizes, shared, lens, 20)
    c, q, st = _cache(total, Hkv, d, 21), _rand((8, Hq, d), 22), _starts(sizes)
    plain = _check(c, q, table, lens, st, shared, window)
    full = ref.shared_table(table, st, shared)
    for tok in (60, 69, 70, 150, 191):                # tokens of the first group's prefix
        pg, slot = int(full[0, tok // 64]), tok % 64
        for side in "kv":
            for byte in (0x7f, 0xff, 0x7e):
                c2 = gdr.KVCache(*[x.clone() for x in c])
                if side == "k":
                    c2.k[pg, :, slot] = byte
                else:
                    c2.v[pg, :, slot // 16, 5:9, slot % 16] = byte
                got = _call(c2, q, table, lens, st, shared, window, out=torch.bfloat16)
                for n in range(8):
                    sees = n < 6 and tok < lens[n] and (not window or tok >= lens[n] - window)
                    if not sees:
                        assert torch.equal(got[n], plain[n]), (tok, side, byte, n)
                    elif byte != 0x7e:
                        hit = got[n].isnan().cpu()
                        if side == "k":
                            assert bool(hit.all())
                        else:
                            assert bool(hit[:, 5:9].all()) and int(hit.sum()) == 4 * Hq


@pytest.mark.parametrize("value", [math.nan, math.inf, 0.0])
def test_absent_pages_and_scales_of_unseen_ones(value):
    """A page outside the cache counts as masked; so does the scale of a page that a
    sequence does not see."""
    sizes, shared, lens, d = [5], [3], [70, 192, 230, 10, 130], 64
    total, table = _tables(sizes, shared, lens, 30)
    table = table.clamp_max(total - 2)                # the last page is nobody's
    c, q, st = _cache(total, 1, d, 31), _rand((5, 8, d), 32), _starts(sizes)
    for bad in (total, -1, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[0, 1] = bad                                 # a shared page
        t[2, 3] = bad                                 # one of a sequence's own
        got = _check(c, q, t, lens, st, shared)
        c2 = gdr.KVCache(*[x.clone() for x in c])
        c2.k[0].fill_(0x7f), c2.v[0].fill_(0xff), c2.k_scale[0].fill_(value), c2.v_scale[0].fill_(value)
        if not bool((ref.shared_table(t, st, shared) == 0).any()):
            assert torch.equal(_call(c2, q, t, lens, st, shared, out=torch.bfloat16), got)
    plain = _call(c, q, table, lens, st, shared)
    c.k_scale[int(table[0, 2])] = value               # the third shared page: sequences 1, 2 and 4 see it
    c.v_scale[int(table[0, 2])] = value
    got = _call(c, q, table, lens, st, shared)
    assert torch.equal(got[[0, 3]], plain[[0, 3]])


def test_pages_with_scales_far_apart():
    """A page of zeros has the smallest scale; another's values are large: neither the
    weights nor their sum lose by it."""
    sizes, shared, lens, d = [4], [4], [300, 256, 257, 290], 64
    total, table = _tables(sizes, shared, lens, 40)
    for exps in ((-96, 10, -5, 0), (20, -96, -96, -3), (-5, -5, -96, 60)):
        c = _cache(total, 1, d, 41)
        for i, e in enumerate(exps):
            pg = int(table[0, i])
            c.v_scale[pg] = 2.0 ** e
            if e == -96:
                c.v[pg] = 0
        _check(c, _rand((4, 4, d), 42), table, lens, [0, 4], shared)


def test_the_same_as_single_decode_where_nothing_is_shared():
    lens = [200, 130, 90, 500, 64, 0]
    total, table = _tables([6], [0], lens, 50)
    c, q = _cache(total, 2, 128, 51), _rand((6, 8, 128), 52)
    got = _call(c, q, table, lens, [0, 6], [0])
    one = gdr.attn_decode(q.cuda(), gdr.KVCache(*[x.cuda() for x in c]), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    want, tol = ref.shared_decode(q.to(F64), attn.Cache(*c), table, lens, [0, 6], [0])
    assert bool(((got - one).abs().cpu().to(F64) <= 2 * tol).all())


def test_scales_of_the_scores():
    sizes, shared, lens, d = [3, 2], [1, 2], [100, 80, 64, 128, 150], 64
    total, table = _tables(sizes, shared, lens, 60)
    for scale in (0.02, 0.5, 2.0):
        _check(_cache(total, 2, d, 61), _rand((5, 4, d), 62), table, lens, _starts(sizes), shared, 0, scale)
