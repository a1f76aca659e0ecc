"""Several layers' caches under one block table: a call for each, all from the old table."""
import pytest
import torch

import gated_delta_rule_24_amd as gdr
from tests import attn_reference as attn
from tests import generation_reference as ref
from tests import test_gpu_pages as pages
from tests import test_gpu_shared as shared

pytestmark = pytest.mark.gpu
gen = gdr.generation
LAYERS = 3


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("small", [True, False])
def test_tables_are_alike_and_every_layers_pages_follow(small, in_place):
    """in_place: the last layer's call writes over the old table."""
    # (more pages than one workgroup counts; the cache's pages are small)
    n_pages = 40 if small else 12300
    g = torch.Generator().manual_seed(7)
    lens = torch.tensor([130, 64, 200, 90, 1], dtype=torch.int32)
    order = torch.randperm(n_pages, generator=g).int()[:20].view(5, 4)
    table = torch.full((5, 4), -1, dtype=torch.int32)
    for n, p in enumerate(lens.tolist()):
        table[n, :ref.pages_of(p)] = order[n, :ref.pages_of(p)]
    table[4, 0] = table[3, 0]                         # two rows on one page
    lens[4] = 64
    held = [0] * n_pages
    held[int(table[2, 1])] = held[3] = 1
    layers = [pages._cache(n_pages, 1, 64, k) for k in range(LAYERS)]
    dev = [pages._on(c) for c in layers]
    parent = None if in_place else [0, 0, 2, 2, 3, 7, 1]
    room = [3, 1, 0, 70, 1] if in_place else [1, 2, 1, 100, 1, 1, 1]
    want, n, missing, copies = ref.fork(table, lens, n_pages, parent, room, held)
    old, old_len = table.cuda(), lens.cuda()
    args = dict(parent=None if parent is None else pages._int(parent).cuda(), room=pages._int(room).cuda(),
                held=torch.tensor(held, dtype=torch.uint8).cuda())
    for k, c in enumerate(dev):
        last = dict(table_out=old, len_out=old_len) if in_place and k == LAYERS - 1 else {}
        got = gen.kv_fork(c, old, old_len, **args, **last)
        assert torch.equal(got[0].cpu(), want) and torch.equal(got[1].cpu(), n) and torch.equal(got[2].cpu(), missing)
    layers = [pages._moved(c, copies) for c in layers]
    assert copies or in_place
    assert all(pages._same(c, h) for c, h in zip(dev, layers))
    old, old_len = got[0], got[1]
    want, used, moves = ref.compact(want, n, n_pages, held)
    for k, c in enumerate(dev):
        got = gen.kv_compact(c, old, old_len, held=args["held"], table_out=old if in_place and k == LAYERS - 1 else None)
        assert torch.equal(got[0].cpu(), want) and int(got[1]) == used
    assert moves and all(pages._same(c, pages._moved(h, moves)) for c, h in zip(dev, layers))


def test_a_fork_of_a_stack_of_attention_layers():
    """Beams of two prompts over two attention layers: forked, appended to and attended to a token at a
    time, each layer against every beam's own history."""
    H, Hq, d, K, V = 2, 4, 64, 3, 30
    g = torch.Generator().manual_seed(11)
    words = [[torch.randn((V, h, d), generator=g).to(torch.bfloat16).cuda() for h in (Hq, H, H)] for _ in range(2)]
    prompts = [torch.randint(0, V, (n,), generator=g).tolist() for n in (63, 130)]
    caches = [gdr.kv_cache(30, H, d) for _ in words]
    lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32)
    table = torch.full((2, 4), -1, dtype=torch.int32)
    at = iter(torch.randperm(30, generator=g).tolist())
    for n, p in enumerate(prompts):
        for i in range(ref.pages_of(len(p))):
            table[n, i] = next(at)
    table, zero = table.cuda(), torch.zeros(2, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 63, 193], dtype=torch.int32).cuda()
    tokens = torch.tensor(prompts[0] + prompts[1], device="cuda")
    for (q, k, v), c in zip(words, caches):
        gdr.kv_append(k[tokens], v[tokens], c, table, zero, cu, token_major=True)
    length, history = lens.cuda(), [list(p) for p in prompts]
    starts, common = torch.tensor([0, K, 2 * K], dtype=torch.int32).cuda(), (lens // 64).int().cuda()
    parent = [0] * K + [1] * K
    for step in range(5):
        rows = torch.tensor(parent, dtype=torch.int32).cuda()
        out = [gen.kv_fork(c, table, length, rows, room=1) for c in caches]
        assert all(torch.equal(a, b) for a, b in zip(out[0], out[1])) and not bool(out[0][2].any())
        table, length = out[0][:2]
        history = [list(history[p]) for p in parent]
        new = torch.randint(0, V, (2 * K,), generator=g)
        for h, t in zip(history, new.tolist()):
            h.append(t)
        for (q, k, v), c in zip(words, caches):
            gdr.kv_append(k[new.cuda()], v[new.cuda()], c, table, length)
        length = length + 1
        for (q, k, v), c in zip(words, caches):
            got = gen.attn_decode_shared(q[new.cuda()], c, table, length, starts, common)
            zeros = gdr.kv_cache(2 * K * 4, H, d, device="cpu")
            for x in zeros:
                x.zero_()
            host = attn.Cache(*zeros)
            own = torch.arange(2 * K * 4, dtype=torch.int32).view(2 * K, 4)
            for n, h in enumerate(history):           # prompt, then token by token: as the scales grew
                kk, vv = [x[h].cpu().to(torch.float64).transpose(0, 1) for x in (k, v)]
                p = len(prompts[n // K])
                host.append([kk[:, :p]], [vv[:, :p]], own[n:n + 1], [0])
                for t in range(p, len(h)):
                    host.append([kk[:, t:t + 1]], [vv[:, t:t + 1]], own[n:n + 1], [t])
            want, tol = ref.shared_decode(q[new.cuda()].cpu().to(torch.float64), host, own, [len(h) for h in history],
                                          list(range(2 * K + 1)), [0] * (2 * K))
            assert bool(((got.cpu().to(torch.float64) - want).abs() <= tol).all()), step
        parent = [0, 0, 2, 3, 5, 5] if step % 2 else [1, 1, 2, 4, 3, 3]


def test_a_row_whose_table_is_full_is_given_nothing():
    """It wants no page that the table has no place for, and misses none; tokens past it are dropped."""
    c = pages._cache(9, 1, 64, 3)
    dev = pages._on(c)
    table = torch.tensor([[5, 2], [5, 7], [1, -1]], dtype=torch.int32)
    lens = torch.tensor([128, 127, 64], dtype=torch.int32)
    got = gen.kv_fork(dev, table.cuda(), lens.cuda(), room=200)
    # (the third row has one place left)
    assert got[0].tolist() == [[5, 2], [5, 7], [1, 0]] and got[2].tolist() == [0, 0, 0]
    assert pages._same(dev, c)
    k = shared._rand((3, 1, 64), 4).cuda()
    gdr.kv_append(k, k, dev, got[0], torch.tensor([128, 128, 128], dtype=torch.int32).cuda())
    assert pages._same(dev, c)
