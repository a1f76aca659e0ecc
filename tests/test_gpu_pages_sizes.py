"""Block tables forked and the cache compacted at the sizes where one workgroup or several
read the tables: the last that one takes, and the first past each of its limits."""
import pytest
import torch

from tests import generation_reference as ref
from tests.test_gpu_pages import _cache, _compact_check, _fork_check, _tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("n_pages,N,width", [
    (12288, 2048, 20), (12288, 2048, 3), (12289, 10, 7), (500, 2049, 3), (3000, 41, 1000), (1, 1, 1), (1, 3, 2), (1024, 1, 40960)])
def test_fork(n_pages, N, width, held):
    g = torch.Generator().manual_seed(N + width)
    lens = torch.randint(0, min(width * 64, max(n_pages * 64 // N * 2, 64)) + 1, (N,), generator=g).int()
    table = _tables(g, N, width, n_pages, lens)
    parent = torch.randint(-1, N, (N,), generator=g).tolist()
    room = torch.randint(0, 150, (N,), generator=g).tolist()
    marks = (torch.rand((n_pages,), generator=g) < 0.1).int().tolist() if held else None
    _fork_check(_cache(n_pages, 1, 64, 3), table, lens, parent, room, marks)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n_pages,N,width", [(12288, 20, 1024), (12288, 20, 1025), (12289, 20, 30), (300, 2048, 10), (300, 2049, 3),
                                             (1, 1, 1), (1025, 3, 400)])
def test_compact(n_pages, N, width, in_place):
    g = torch.Generator().manual_seed(N + width)
    lens = torch.randint(0, min(width * 64, max(n_pages * 64 // N * 2, 64)) + 1, (N,), generator=g).int()
    held = (torch.rand((n_pages,), generator=g) < 0.1).int().tolist() if in_place else None
    _compact_check(_cache(n_pages, 1, 64, 8), _tables(g, N, width, n_pages, lens), lens, held, in_place)


def test_every_row_writes_on_one_page():
    """2,048 rows behind one that is partly full: as many copies as there are free pages."""
    table, lens = torch.tensor([[7, 3]], dtype=torch.int32), torch.tensor([100], dtype=torch.int32)
    _, _, missing = _fork_check(_cache(1500, 1, 64, 5), table, lens, [0] * 2048, 1)
    assert int((missing == 0).sum()) == 1 + 1498


def test_one_page_named_everywhere():
    """Counters' largest values: 40,960 entries name the same page."""
    table = torch.full((2048, 20), 4, dtype=torch.int32)
    lens = torch.full((2048,), 20 * 64, dtype=torch.int32)
    lens[5:900] -= 3                                  # (895 write into it, and so do entries that are whole)
    _fork_check(_cache(1000, 1, 64, 6), table, lens, None, 2)
    want = ref.compact(table, lens, 1000)
    assert want[1] == 1 and want[2] == [(4, 0)]
    _compact_check(_cache(1000, 1, 64, 6), table, lens)
