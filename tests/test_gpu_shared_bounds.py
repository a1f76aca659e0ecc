"""Attention over shared pages with any numbers as groups' bounds: bounds are held within 0 .. N and
not below the one before, shared pages within 0 .. max_pages, and every sequence's result is that
of the groups which this leaves."""
import pytest
import torch

from tests import attn_reference as attn
from tests import generation_reference as ref
from tests import test_gpu_shared as base

pytestmark = pytest.mark.gpu


def _held(starts, shared, N, width):
    """The groups that the bounds stand for."""
    out, top = [], 0
    for s in starts:
        top = max(top, min(max(int(s), 0), N))
        out.append(top)
    return out, [min(max(int(p), 0), width) for p in shared]


def _bounds_check(c, q, table, lens, starts, shared, window=0):
    first, pages = _held(starts, shared, *table.shape)
    got = base._call(c, q, table, lens, starts, shared, window).cpu().to(torch.float64)
    want, tol = ref.shared_decode(q.to(torch.float64), attn.Cache(*c), table, lens, first, pages, window)
    off = (got - want).abs()
    assert bool((off <= tol).all()), float((off / tol.clamp_min(1e-300)).max())


@pytest.mark.parametrize("Hq", [8, 200])                            # 32 and 64 rows a wave
@pytest.mark.parametrize("starts,shared", [
    ([0, 9, 3], [2, 2]), ([-4, 2, 100], [1, 2]), ([5, 5, 5], [3, 3]), ([3, 1, 2], [1 << 30, -3]), ([2, 0, 4], [1, 1]), ([0, 4, 2, 5], [1, 2, 1]),
    ([-2 ** 31, 2 ** 31 - 1, 4], [-2 ** 31, 2 ** 31 - 1]), ([-2 ** 31, 2 ** 31 - 1, 4], [2 ** 31 - 1, -2 ** 31]), ([1, 4], [3])])
def test_every_sequence_has_the_result_of_the_groups_that_are_left(Hq, starts, shared):
    lens = [200, 130, 90, 200, 64]
    total, table = base._tables([5], [0], lens, 14)
    c, q = base._cache(total, 2, 64, 15), base._rand((5, Hq, 64), 16)
    for window in (0, 77):
        _bounds_check(c, q, table, lens, starts, shared, window)


@pytest.mark.parametrize("groups", [3, 64, 65, 300])
def test_bounds_in_no_order(groups):
    """As many as a workgroup plans for by itself, and more."""
    N, width, g = 40, 6, torch.Generator().manual_seed(groups)
    c = base._cache(5, 2, 64, groups)
    table = torch.randint(0, 5, (N, width), generator=g, dtype=torch.int32)
    lens = torch.randint(0, width * 64, (N,), generator=g).tolist()
    q = base._rand((N, 4, 64), groups)
    for high in (N, 10 ** 9):
        starts = torch.randint(-high, high, (groups + 1,), generator=g).tolist()
        _bounds_check(c, q, table, lens, starts, torch.randint(-3, 9, (groups,), generator=g).tolist())
    # mostly rising, with some that fall back
    starts = (torch.arange(groups + 1) * N // groups + torch.randint(-3, 4, (groups + 1,), generator=g)).tolist()
    _bounds_check(c, q, table, lens, starts, torch.randint(0, 5, (groups,), generator=g).tolist())
