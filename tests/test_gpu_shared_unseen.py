"""Attention over shared pages: the page that is read in place of an absent one, and bytes in slots
that a sequence does not see, for either type of result, in sequences' own pages and shared ones,
with 32 and with 64 rows a wave."""
import math

import pytest
import torch

import gated_delta_rule_24_amd as gdr
from tests import generation_reference as ref
from tests import test_gpu_shared as base

pytestmark = pytest.mark.gpu
HEADS = [(2, 2), (12, 2), (70, 1), (400, 2)]          # the last two: 64 rows a wave


def _tables(sizes, shared, lens, seed):
    """As test_gpu_shared's, but nobody has page 0."""
    total, table = base._tables(sizes, shared, lens, seed)
    return total + 1, torch.where(table >= 0, table + 1, table)


@pytest.mark.parametrize("value", [math.nan, math.inf, 0.0])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_what_stands_in_for_an_absent_page_does_not_matter(Hq, Hkv, value):
    sizes, shared, lens, d = [5, 2], [3, 1], [70, 192, 230, 10, 130, 64, 200], 64
    total, table = _tables(sizes, shared, lens, 30)
    c, q, st = base._cache(total, Hkv, d, 31), base._rand((7, Hq, d), 32), base._starts(sizes)
    c2 = gdr.KVCache(*[x.clone() for x in c])
    c2.k[0].fill_(0x7f), c2.v[0].fill_(0xff), c2.k_scale[0].fill_(value), c2.v_scale[0].fill_(value)
    for bad in (total, -1, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[0, 0] = t[0, 2] = bad                       # shared pages, the first and the last
        t[2, 3] = bad                                 # one of a sequence's own
        t[5, 0] = bad                                 # the second group's only one: sequence 5 sees nothing
        assert not bool((ref.shared_table(t, st, shared) == 0).any())
        base._check(c, q, t, lens, st, shared)
        for out in (torch.float32, torch.bfloat16):
            want = base._call(c, q, t, lens, st, shared, out=out)
            assert not bool(want[5].any()) and not bool(want.isnan().any())
            assert torch.equal(base._call(c2, q, t, lens, st, shared, out=out), want)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_bytes_that_one_sequence_sees_and_another_does_not(Hq, Hkv, window, out):
    sizes, shared, d = [6, 2], [3, 1], 64
    lens = [70, 192, 200, 130, 1, 64, 64, 100]
    total, table = _tables(sizes, shared, lens, 20)
    c, q, st = base._cache(total, Hkv, d, 21), base._rand((8, Hq, d), 22), base._starts(sizes)
    plain = base._call(c, q, table, lens, st, shared, window, out=out)
    full = ref.shared_table(table, st, shared)
    # tokens of the first group's prefix, and one of sequence 2's own
    for tok, owner in ((60, None), (69, None), (70, None), (191, None), (195, 2)):
        pg, slot = int(full[2, tok // 64]), tok % 64
        for side in "kv":
            for byte in (0x7f, 0xff, 0x7e):
                c2 = gdr.KVCache(*[x.clone() for x in c])
                if side == "k":
                    c2.k[pg, :, slot] = byte
                else:
                    c2.v[pg, :, slot // 16, 5:9, slot % 16] = byte
                got = base._call(c2, q, table, lens, st, shared, window, out=out)
                for n in range(8):
                    sees = (n < 6 if owner is None else n == owner) and tok < lens[n] and (not window or tok >= lens[n] - window)
                    if not sees:
                        assert torch.equal(got[n], plain[n]), (tok, side, byte, n)
                    elif byte != 0x7e:
                        hit = got[n].isnan().cpu()
                        assert bool(hit.all()) if side == "k" else bool(hit[:, 5:9].all()) and int(hit.sum()) == 4 * Hq
                    else:
                        assert not bool(got[n].isnan().any())


@pytest.mark.parametrize("Hq", [8, 150])
def test_a_group_whose_first_sequence_was_dropped(Hq):
    """Its emptied row has no shared pages; the group that begins behind it has them all."""
    sizes, shared, d = [4], [2], 64
    total, table = _tables(sizes, [0], [200, 150, 140, 190], 40)
    table[:, :2] = table[0, :2]
    c, q = base._cache(total, 1, d, 41), base._rand((4, Hq, d), 42)
    lens = torch.tensor([200, 150, 140, 190], dtype=torch.int32)
    parent = torch.tensor([-1, 1, 2, 3], dtype=torch.int32).cuda()
    dev = gdr.KVCache(*[x.cuda() for x in c])
    table, lens, missing = gdr.generation.kv_fork(dev, table.cuda(), lens.cuda(), parent, room=0)
    table, lens = table.cpu(), lens.tolist()
    assert lens == [0, 150, 140, 190] and bool((table[0] == -1).all()) and not bool(missing.any())
    whole = base._check(c, q, table, lens, [1, 4], shared)
    base._check(c, q, table, lens, [0, 4], shared)    # (the shared pages count as masked)
    assert not bool(whole[0].any())
