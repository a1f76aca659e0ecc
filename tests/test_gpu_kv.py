"""gdr_kv_append and gdr_attn_decode on the GPU against the cache and the
attention in 64 bits: the cache bit for bit, outputs within derived bounds."""
import math

import pytest
import torch

import gated_delta_rule_24_amd as gdr
from tests import attn_reference as ref

pytestmark = pytest.mark.gpu
F64 = torch.float64


def _cache(n_pages, H, d, seed=None):
    """Every slot's byte set: a recognisable pattern, or random e4m3 values."""
    c = gdr.kv_cache(n_pages, H, d)
    if seed is None:
        c.k.fill_(0x33), c.v.fill_(0x33), c.k_scale.fill_(0.25), c.v_scale.fill_(0.25)
        return c
    g = torch.Generator().manual_seed(seed)
    for t in (c.k, c.v):
        t.copy_((torch.randn(t.shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    for t in (c.k_scale, c.v_scale):
        t.copy_(torch.pow(torch.tensor(2.0), torch.randint(-8, -4, t.shape, generator=g).float()))
    return c


def _table(nseq, width, n_pages, seed):
    return torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed))[:nseq * width].view(nseq, width).int()


def _same(c, want):
    for got, val in ((c.k.cpu().view(torch.float8_e4m3fn).to(F64), want.k),
                     (c.v.cpu().view(torch.float8_e4m3fn).to(F64).transpose(3, 4).flatten(2, 3), want.v)):
        assert torch.equal(torch.isnan(got), torch.isnan(val))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(val))
    assert torch.equal(c.k_scale.cpu().to(F64), want.ks) and torch.equal(c.v_scale.cpu().to(F64), want.vs)


def _rand(shape, seed, by=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * by).to(torch.bfloat16)


@pytest.mark.parametrize("H,d", [(1, 64), (3, 128)])
@pytest.mark.parametrize("by", [1e-3, 1.0, 50.0])
def test_one_token_each(H, d, by):
    """Appended one by one across a page's end: scales grow, older tokens are rounded again."""
    have = [0, 1, 14, 15, 16, 62, 63, 64, 127, 65]
    n = len(have)
    c, table = _cache(n * 3, H, d, seed=1), _table(n, 3, n * 3, 2)
    want = ref.Cache(*c)
    td = table.cuda()
    for step in range(4):
        k, v = _rand((n, H, d), 10 + step, by * 2.0 ** step), _rand((n, H, d), 20 + step, by)
        lens = torch.tensor([x + step for x in have], dtype=torch.int32, device="cuda")
        gdr.kv_append(k.cuda(), v.cuda(), c, td, lens)
        want.append(list(k.to(F64)[:, :, None]), list(v.to(F64)[:, :, None]), table, lens.tolist())
        _same(c, want)


@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("new,have", [([1, 0, 64, 65, 200], [0, 5, 64, 63, 10]), ([300], [0]), ([0, 0, 7], [3, 0, 60]),
                                      ([3] * 300, [i % 70 for i in range(300)])])
def test_prompts(new, have, token_major):
    H, d, n = 2, 64, len(new)
    width = max((a + b + 63) // 64 for a, b in zip(new, have))
    c, table = _cache(n * width + 2, H, d, seed=3), _table(n, width, n * width + 2, 4)
    want = ref.Cache(*c)
    T = sum(new)
    k, v = _rand((H, T, d), 5), _rand((H, T, d), 6, 3.0)
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    give = (lambda x: x.transpose(0, 1).contiguous().cuda()) if token_major else (lambda x: x.cuda())
    gdr.kv_append(give(k), give(v), c, table.cuda(), torch.tensor(have, dtype=torch.int32, device="cuda"),
                  torch.tensor(cu, dtype=torch.int32, device="cuda"), token_major=token_major)
    want.append([k[:, a:b].to(F64) for a, b in zip(cu, cu[1:])], [v[:, a:b].to(F64) for a, b in zip(cu, cu[1:])], table, have)
    _same(c, want)


def test_extreme_values():
    """Zeros, the largest and smallest values, infinities and NaN."""
    H, d = 1, 64
    c, table = _cache(2, H, d, seed=7), torch.tensor([[1]], dtype=torch.int32)
    want = ref.Cache(*c)
    k = torch.zeros((H, 4, d), dtype=torch.bfloat16)
    k[0, 1] = 3.3895e38
    k[0, 2, :8] = torch.tensor([math.inf, -math.inf, math.nan, 1e-40, 1.0, -3e38, 2.0 ** -133, -0.0])
    v = torch.zeros((H, 4, d), dtype=torch.bfloat16)
    v[0, :, 3] = 2.0 ** -120
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    gdr.kv_append(k.cuda(), v.cuda(), c, table.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"), cu)
    want.append([k.to(F64)], [v.to(F64)], table, [0])
    _same(c, want)


def test_slots_behind_the_tokens_and_bad_pages_are_left_alone():
    H, d = 2, 64
    c = _cache(4, H, d)
    before = [t.clone() for t in c]
    table = torch.tensor([[0, -1], [7, 2], [3, 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([60, 0, 128], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 10, 20, 30], dtype=torch.int32, device="cuda")
    gdr.kv_append(_rand((H, 30, d), 8).cuda(), _rand((H, 30, d), 9).cuda(), c, table, lens, cu)
    torch.cuda.synchronize()
    # only sequence 0's first four tokens have a page: slots 60 .. 63 of page 0
    for i in (1, 2, 3):
        assert torch.equal(c.k[i], before[0][i]) and torch.equal(c.v[i], before[1][i])
        assert torch.equal(c.k_scale[i], before[2][i]) and torch.equal(c.v_scale[i], before[3][i])
    assert not torch.equal(c.k[0, :, 60:], before[0][0, :, 60:])
    assert torch.equal(c.v[0, :, :3], before[1][0, :, :3])         # scale 0.25 is large enough: nothing re-rounded
    # new tokens at a page's start leave the slots behind them
    c2 = _cache(1, H, d)
    gdr.kv_append(_rand((1, H, d), 1).cuda(), _rand((1, H, d), 2).cuda(), c2,
                  torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert bool((c2.k[:, :, 1:] == 0x33).all()) and bool((c2.v[:, :, 0, :, 1:] == 0x33).all()) and bool((c2.v[:, :, 1:] == 0x33).all())


def test_bad_lengths_and_offsets_stay_inside():
    H, d = 1, 64
    c = _cache(3, H, d)
    table = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    for lens, cu in (([-7, 2 ** 31 - 1], [0, 5, 10]), ([0, 0], [-3, 4, 99]), ([0, 0], [8, 2, 10])):
        gdr.kv_append(_rand((H, 10, d), 1).cuda(), _rand((H, 10, d), 2).cuda(), c, table,
                      torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.tensor(cu, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert bool((c.k[2] == 0x33).all()) and bool((c.v[2] == 0x33).all())


def _decode_check(c, q, table, lens, window=0, scale=None, poison=False):
    want, tol = ref.decode(q.to(F64), ref.Cache(*c), table, lens, window, scale)
    args = (q.cuda(), c, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    o = gdr.attn_decode(*args, window=window, scale=scale)
    assert o.dtype == torch.float32
    off = (o.cpu().to(F64) - want).abs() - tol
    assert float(off.max()) <= 0, f"{float(off.max()):.3g} over its bound"
    b = gdr.attn_decode(*args, window=window, scale=scale, out_dtype=torch.bfloat16)
    assert torch.equal(b, o.to(torch.bfloat16))
    return o


@pytest.mark.parametrize("Hq,H,d", [(1, 1, 64), (4, 1, 128), (8, 2, 64), (16, 1, 128), (17, 1, 64), (40, 2, 128), (6, 6, 64)])
@pytest.mark.parametrize("window", [0, 50])
def test_decode(Hq, H, d, window):
    lens = [1, 2, 63, 64, 65, 200, 0, 448]
    n = len(lens)
    c, table = _cache(n * 7, H, d, seed=11), _table(n, 7, n * 7, 12)
    _decode_check(c, _rand((n, Hq, d), 13), table, lens, window)


@pytest.mark.parametrize("window", [1, 64, 65, 128, 1000, 3000, 100000])
def test_decode_long_and_windows(window):
    """Many pages for one sequence: split over workgroups and joined."""
    c, table = _cache(100, 1, 64, seed=14), _table(1, 90, 100, 15)
    _decode_check(c, _rand((1, 4, 64), 16), table, [5700], window)


@pytest.mark.parametrize("scale", [1e-3, 1.0, 30.0])
def test_decode_scales(scale):
    c, table = _cache(8, 2, 128, seed=17), _table(2, 4, 8, 18)
    _decode_check(c, _rand((2, 4, 128), 19), table, [130, 256], 0, scale)


def test_decode_page_scales_far_apart():
    """One page's values 2^40 times another's, and the other way round for the keys'
    weights: every page counts to fp32."""
    c, table = _cache(8, 1, 64, seed=40), _table(2, 4, 8, 41)
    c.v_scale[table[0, 0]], c.v_scale[table[0, 1]] = 2.0 ** 20, 2.0 ** -20
    c.v_scale[table[1, 2]], c.k_scale[table[1, 2]] = 2.0 ** 30, 2.0 ** -20
    c.k_scale[table[0, 0]] = 2.0 ** -3
    q = _rand((2, 4, 64), 42)
    _decode_check(c, q, table, [200, 256])
    c.v_scale[table[0, 1]] = 2.0 ** -96
    c.v_scale[table[1, 0]] = 2.0 ** 110
    _decode_check(c, q, table, [200, 256])


def test_decode_ignores_what_is_masked():
    """Bytes behind the last token or before the window, pages that are not there:
    NaN everywhere in them changes nothing."""
    d, lens = 64, [70, 130, 5]
    c, table = _cache(10, 1, d, seed=20), _table(3, 3, 9, 21)
    q = _rand((3, 4, d), 22)
    want = _decode_check(c, q, table, lens, 60)
    kf, vf = c.k.clone(), c.v.clone()
    for i, n in enumerate(lens):
        for t in range(3 * 64):
            if t >= n or t < n - 60:
                pg = int(table[i, t // 64])
                kf[pg, :, t % 64] = 0x7f
                vf[pg, :, (t % 64) // 16, :, t % 16] = 0xff
    c2 = gdr.KVCache(kf, vf, c.k_scale, c.v_scale)
    # pages past the last token, named in the table or not, are never read
    table2 = table.clone()
    table2[2, 1:] = torch.tensor([-1, 2 ** 31 - 1])
    got = gdr.attn_decode(q.cuda(), c2, table2.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), window=60)
    assert torch.equal(got, want)
    # a missing page among the tokens counts as masked; its scale and bytes do not matter
    table3 = table.clone()
    table3[1, 1] = 10
    o = _decode_check(c, q, table3, lens)
    c.k[0].fill_(0x7f), c.v[0].fill_(0x7f), c.v_scale[0].fill_(math.nan)
    if 0 not in table3[:, :].tolist()[0] + table3.tolist()[1] + table3.tolist()[2]:
        assert torch.equal(gdr.attn_decode(q.cuda(), c, table3.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")), o)


def test_decode_nan_reaches_its_reader_only():
    d = 64
    c, table = _cache(6, 1, d, seed=23), _table(2, 3, 6, 24)
    q = _rand((2, 2, d), 25)
    lens = torch.tensor([100, 100], dtype=torch.int32, device="cuda")
    want = gdr.attn_decode(q.cuda(), c, table.cuda(), lens)
    c.v[int(table[0, 0]), 0, 2, 7, 3] = 0x7f                       # token 35, channel 7
    got = gdr.attn_decode(q.cuda(), c, table.cuda(), lens)
    assert torch.equal(got[1], want[1]) and bool(torch.isnan(got[0, :, 7]).all())
    rest = [i for i in range(d) if i != 7]
    assert torch.equal(got[0][:, rest], want[0][:, rest])
    q[0, 1, 0] = math.nan
    got = gdr.attn_decode(q.cuda(), c, table.cuda(), lens)
    assert bool(torch.isnan(got[0, 1]).all()) and torch.equal(got[1], want[1]) and torch.equal(got[0, 0, rest], want[0, 0, rest])


def test_lengths_outside_the_table_stay_inside():
    c, table = _cache(4, 1, 64, seed=26), _table(2, 2, 4, 27)
    q = _rand((2, 2, 64), 28)
    for lens in ([-5, 2 ** 31 - 1], [129, 1000]):
        _decode_check(c, q, table, lens)
        _decode_check(c, q, table, lens, 100)


def test_far_pages_of_a_large_cache():
    """Byte offsets past 2^32: the last pages of a cache of more than 4 GiB a side."""
    H, d = 8, 128
    pages = (1 << 32) // (H * 64 * d) + 40
    c = gdr.kv_cache(pages, H, d)
    table = torch.tensor([[pages - 1, pages - 2, 3]], dtype=torch.int32)
    T = 150
    k, v = _rand((H, T, d), 29), _rand((H, T, d), 30)
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    gdr.kv_append(k.cuda(), v.cuda(), c, table.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"), cu)
    q = _rand((1, 16, d), 31)
    o = gdr.attn_decode(q.cuda(), c, table.cuda(), torch.tensor([T], dtype=torch.int32, device="cuda"))
    sub = gdr.KVCache(*[torch.stack([t[pages - 1], t[pages - 2], t[3]]) for t in c])
    want, tol = ref.decode(q.to(F64), ref.Cache(*sub), torch.tensor([[0, 1, 2]]), [T])
    assert bool(((o.cpu().to(F64) - want).abs() <= tol).all())
    small = _cache(3, H, d)
    gdr.kv_append(k.cuda(), v.cuda(), small, torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda"),
                  torch.zeros(1, dtype=torch.int32, device="cuda"), cu)
    assert torch.equal(small.k[:2], sub.k[:2]) and torch.equal(small.k_scale, sub.k_scale)
    assert torch.equal(small.k[2, :, :T - 128], sub.k[2, :, :T - 128])


def test_refusals():
    c = _cache(4, 2, 64, seed=1)
    table, lens = torch.zeros((2, 2), dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    q, k = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: gdr.attn_decode(q.float(), c, table, lens), lambda: gdr.attn_decode(q, c, table.long(), lens),
                lambda: gdr.attn_decode(q, c, table, lens[:1]), lambda: gdr.attn_decode(q, c, table, lens, out_dtype=torch.float16),
                lambda: gdr.kv_append(k, k[:1], c, table, lens), lambda: gdr.kv_append(k, k, c, table, lens.cpu()),
                lambda: gdr.kv_append(k, k, c._replace(k_scale=c.k_scale.double()), table, lens),
                lambda: gdr.kv_append(k, k, c, table, lens, torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gdr.GdrError):
        gdr.attn_decode(q[:, :3].contiguous(), c, table, lens)     # 3 query heads, 2 key heads


def test_graph_of_generation_steps():
    """Append and attend captured once, replayed step after step, against eager steps;
    two graphs of different sequences, each with its own workspace, in turn."""
    d, H, n = 64, 2, 3

    def setup(seed):
        c, table = _cache(n * 20, H, d, seed=seed), _table(n, 20, n * 20, seed).cuda()
        return c, table, torch.tensor([60, 5, 1000], dtype=torch.int32, device="cuda")

    runs = []
    for seed in (33, 34):
        c, table, lens = setup(seed)
        k, v, q = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((n, H, d), (n, H, d), (n, 8, d)))
        gdr.kv_append(k, v, c, table, lens)
        gdr.attn_decode(q, c, table, lens + 1)
        c, table, lens = setup(seed)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gdr.kv_append(k, v, c, table, lens)
            lens.add_(1)
            o = gdr.attn_decode(q, c, table, lens)
        lens.copy_(setup(seed)[2])
        runs.append((graph, k, v, q, lens, o, c, setup(seed), table))      # the captured table stays alive
    for step in range(5):
        for r, (graph, k, v, q, lens, o, c, (c2, table2, lens2), _) in enumerate(runs):
            for t, s in ((k, 1), (v, 2), (q, 3)):
                t.copy_(_rand(t.shape, 100 * step + 10 * r + s))
            graph.replay()
            gdr.kv_append(k, v, c2, table2, lens2)
            lens2 += 1
            want = gdr.attn_decode(q, c2, table2, lens2)
            torch.cuda.synchronize()
            assert torch.equal(o, want) and torch.equal(lens, lens2) and all(torch.equal(a, b) for a, b in zip(c, c2))
