"""Block tables forked, grown and dropped, and the cache compacted, against the host's
dealing out of pages one after the other: tables, lengths, and every byte of the cache."""
import pytest
import torch

import gated_delta_rule_24_amd as gdr
from tests import generation_reference as ref

pytestmark = pytest.mark.gpu
gen = gdr.generation


def _cache(n_pages, H, d, seed):
    g = torch.Generator().manual_seed(seed)
    c = gdr.kv_cache(n_pages, H, d, device="cpu")
    for x in (c.k, c.v):
        x.copy_(torch.randint(0, 256, x.shape, generator=g).to(torch.uint8))
    for x in (c.k_scale, c.v_scale):
        x.copy_(torch.randn(x.shape, generator=g))
    return c


def _moved(c, moves):
    out = gdr.KVCache(*[x.clone() for x in c])
    for a, b in moves:
        for x, y in zip(out, c):
            x[b] = y[a]
    return out


def _same(dev, host):
    return all(torch.equal(x.cpu().view(torch.uint8), y.view(torch.uint8)) for x, y in zip(dev, host))


def _on(c):
    return gdr.KVCache(*[x.cuda() for x in c])


def _int(x):
    return torch.as_tensor(x, dtype=torch.int32)


def _fork_check(c, table, lens, parent=None, room=1, held=None):
    """Twice: the call keeps nothing, so that it gives the same again."""
    n_pages = c.k.shape[0]
    want, n, missing, copies = ref.fork(table, lens, n_pages, parent, room, held)
    dev = _on(c)
    args = dict(parent=None if parent is None else _int(parent).cuda(), room=room if isinstance(room, int) else _int(room).cuda(),
                held=None if held is None else torch.tensor(held, dtype=torch.uint8).cuda())
    after = _moved(c, copies)
    for _ in range(2):
        got = gen.kv_fork(dev, table.cuda(), lens.cuda(), **args)
        assert torch.equal(got[0].cpu(), want) and torch.equal(got[1].cpu(), n) and torch.equal(got[2].cpu(), missing)
        assert _same(dev, after)
    return want, n, missing


def _tables(g, rows, width, n_pages, lens):
    """Rows with pages of their own, some of them shared with the row before."""
    order = torch.randperm(n_pages, generator=g).tolist()
    t = torch.full((rows, width), -1, dtype=torch.int32)
    for i in range(rows):
        need = min(width, ref.pages_of(int(lens[i])))
        for j in range(need):
            if i and int(torch.randint(0, 3, (), generator=g)) == 0 and t[i - 1, j] >= 0:
                t[i, j] = t[i - 1, j]
            elif order:
                t[i, j] = order.pop()
    return t


@pytest.mark.parametrize("H,d", [(1, 64), (3, 128), (8, 128)])
def test_beams_of_one_prompt(H, d):
    """A prompt forked into four beams, which each go on in a page of their own."""
    c = _cache(12, H, d, 1)
    table = _int([[7, 2, 9, -1, -1]])
    lens = _int([140])
    t, n, missing = _fork_check(c, table, lens, parent=[0, 0, 0, 0])
    # the lowest beam keeps the last page, the others copy it into the lowest free ones
    assert t.tolist() == [[7, 2, 9, -1, -1], [7, 2, 0, -1, -1], [7, 2, 1, -1, -1], [7, 2, 3, -1, -1]]
    assert n.tolist() == [140] * 4 and not bool(missing.any())
    # a full page is shared, and a fresh one follows
    t, _, _ = _fork_check(c, table, _int([128]), parent=[0, 0, 0])
    assert t.tolist() == [[7, 2, 0, -1, -1], [7, 2, 1, -1, -1], [7, 2, 3, -1, -1]]
    # dropped rows give their pages back
    t, n, _ = _fork_check(c, _int([[0, 1], [2, 3]]), _int([100, 128]), parent=[-1, 1, 2, -2 ** 31], room=64)
    assert t.tolist() == [[-1, -1], [2, 3], [-1, -1], [-1, -1]] and n.tolist() == [0, 128, 0, 0]
    t, n, _ = _fork_check(c, _int([[0, 1, -1], [2, 3, -1]]), _int([100, 128]), parent=[-1, 1], room=64)
    assert t.tolist() == [[-1] * 3, [2, 3, 0]]


def test_rows_that_write_and_rows_that_do_not():
    c = _cache(8, 2, 64, 2)
    table, lens = _int([[5, 6]]), _int([70])
    # the other row does not write: the page stays its own
    t, _, _ = _fork_check(c, table, lens, parent=[0, 0], room=[1, 0])
    assert t.tolist() == [[5, 0], [5, 6]]
    t, _, _ = _fork_check(c, table, lens, parent=[0, 0], room=[0, 0])
    assert t.tolist() == [[5, 6], [5, 6]]
    # a page that others hold is copied, and not dealt out
    t, _, _ = _fork_check(c, table, lens, held=[1, 0, 0, 0, 0, 0, 1, 0])
    assert t.tolist() == [[5, 1]]
    # taken back below what the other row still has on the page
    t, _, _ = _fork_check(c, _int([[5, 6], [5, 6]]), _int([70, 100]))
    assert t.tolist() == [[5, 6], [5, 0]]
    t, _, _ = _fork_check(c, _int([[5, 6], [5, 6]]), _int([70, 128]))
    assert t.tolist() == [[5, 0], [5, 6]]


@pytest.mark.parametrize("seed", range(24))
def test_fork_of_random_tables(seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (), generator=g))  # noqa: E731
    N_in, N, width = r(1, 40), r(1, 60), r(1, 9)
    n_pages = r(1, 300) if seed % 3 else r(1, 40)
    lens = torch.randint(-5, width * 64 + 30, (N_in,), generator=g).int()
    table = _tables(g, N_in, width, n_pages, lens)
    if seed % 4 == 0:                                 # entries that are no pages, the same page twice
        table[r(0, N_in - 1), r(0, width - 1)] = (n_pages, -7, 2 ** 31 - 1)[seed % 3]
        table[r(0, N_in - 1)] = r(0, n_pages - 1)
    parent = None if N == N_in or seed % 5 == 0 else torch.randint(-2, N_in + 1, (N,), generator=g).tolist()
    rows = N_in if parent is None else N
    room = r(0, 200) if seed % 2 else torch.randint(-3, 130, (rows,), generator=g).tolist()
    held = (torch.rand((n_pages,), generator=g) < 0.2).int().tolist() if seed % 3 == 1 else None
    _fork_check(_cache(n_pages, r(1, 3), (64, 128)[seed % 2], seed), table, lens, parent, room, held)


@pytest.mark.parametrize("n_pages,N,width", [(4095, 300, 13), (4096, 257, 3), (9000, 5000, 2), (20000, 70, 300), (8193, 2, 2500)])
def test_fork_of_many_rows_and_pages(n_pages, N, width):
    g = torch.Generator().manual_seed(N)
    lens = torch.randint(0, min(width * 64, n_pages * 64 // N * 2) + 1, (N,), generator=g).int()
    table = _tables(g, N, width, n_pages, lens)
    parent = torch.randint(-1, N, (N,), generator=g).tolist()
    _fork_check(_cache(n_pages, 1, 64, 3), table, lens, parent, 70)


def test_fork_in_place_without_parents():
    c = _cache(20, 2, 64, 4)
    table, lens = _int([[3, -1, -1], [3, 4, -1], [-1, -1, -1]]), _int([64, 65, 0])
    want, n, _, copies = ref.fork(table, lens, 20, None, 64)
    dev, t, L = _on(c), table.cuda(), lens.cuda()
    out = gen.kv_fork(dev, t, L, room=64, table_out=t, len_out=L)
    assert out[0].data_ptr() == t.data_ptr() and torch.equal(t.cpu(), want) and torch.equal(L.cpu(), n)
    assert _same(dev, _moved(c, copies))


def test_fork_when_pages_run_out():
    c = _cache(5, 1, 64, 5)
    table, lens = _int([[0, 1, -1, -1, -1]]), _int([100])
    t, _, missing = _fork_check(c, table, lens, parent=[0, 0, 0, 0, 0], room=100)
    # each wants two pages for its tokens, all but the first a copy before them: three are free
    assert missing.tolist() == [0, 2, 3, 3, 3]
    assert t.tolist() == [[0, 1, 2, 3, -1], [0, 4, -1, -1, -1]] + [[0, 1, -1, -1, -1]] * 3


# ---------------------------------------------------------------------------


def _compact_check(c, table, lens, held=None, in_place=False):
    want, used, moves = ref.compact(table, lens, c.k.shape[0], held)
    dev, t = _on(c), table.cuda()
    h = None if held is None else torch.tensor(held, dtype=torch.bool).cuda()
    after = _moved(c, moves)
    for _ in range(1 if in_place else 2):
        got = gen.kv_compact(dev, t, lens.cuda(), held=h, table_out=t if in_place else None)
        assert torch.equal(got[0].cpu(), want) and int(got[1]) == used
        assert _same(dev, after)
    return want, used


def test_compact_small():
    c = _cache(10, 2, 64, 6)
    t, used = _compact_check(c, _int([[8, 3], [8, 9]]), _int([100, 128]))
    # 9, 8 and 3 are in use, 0, 1 and 2 the lowest free: 9 -> 0, 8 -> 1, 3 -> 2
    assert t.tolist() == [[1, 2], [1, 0]] and used == 3
    t, used = _compact_check(c, _int([[8, 3], [8, 9]]), _int([100, 128]), held=[1] + [0] * 6 + [1, 0, 0])
    # 0 and 7 stay: 9 -> 1, 8 -> 2, and 3 is below the next free one
    assert t.tolist() == [[2, 3], [2, 1]] and used == 8
    t, used = _compact_check(c, _int([[0, 1]]), _int([128]))         # nothing to move
    assert t.tolist() == [[0, 1]] and used == 2
    t, used = _compact_check(c, _int([[5, 1]]), _int([0]))           # nothing in use
    assert t.tolist() == [[-1, -1]] and used == 0
    t, used = _compact_check(c, _int([list(range(9, -1, -1))]), _int([640]))   # all in use
    assert used == 10


@pytest.mark.parametrize("seed", range(16))
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_of_random_tables(seed, in_place):
    g = torch.Generator().manual_seed(100 + seed)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (), generator=g))  # noqa: E731
    N, width, n_pages = r(1, 40), r(1, 9), (r(1, 300), r(300, 12000))[seed % 2]
    lens = torch.randint(-5, width * 64 + 30, (N,), generator=g).int()
    table = _tables(g, N, width, n_pages, lens)
    if seed % 4 == 0:
        table[r(0, N - 1), r(0, width - 1)] = (n_pages, -7, 2 ** 31 - 1)[seed % 3]
    held = (torch.rand((n_pages,), generator=g) < 0.1).int().tolist() if seed % 3 == 1 else None
    _compact_check(_cache(n_pages, r(1, 2), 64, seed), table, lens, held, in_place)


def test_compact_of_a_large_cache():
    g = torch.Generator().manual_seed(7)
    lens = torch.randint(0, 40 * 64, (200,), generator=g).int()
    _compact_check(_cache(12289, 2, 64, 8), _tables(g, 200, 40, 12289, lens), lens)
