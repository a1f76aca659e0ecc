"""Attention over shared pages where a group has hundreds of rows on a key head (64 of them a
wave): the same checks as for small groups."""
import pytest
import torch

from tests import test_gpu_shared as base

pytestmark = pytest.mark.gpu

SIZES = [([3], [2], 130, 1), ([5, 4], [4, 2], 140, 1), ([150], [3], 4, 2), ([1, 0, 2, 3], [2, 9, 0, 5], 300, 1), ([65, 3, 66], [7, 0, 2], 8, 1)]


@pytest.mark.parametrize("sizes,shared,Hq,Hkv", SIZES)
@pytest.mark.parametrize("d", [64, 128])
def test_against_each_sequence_alone(sizes, shared, Hq, Hkv, d):
    base.test_against_each_sequence_alone(sizes, shared, Hq, Hkv, d)


@pytest.mark.parametrize("window", [0, 70])
def test_what_a_sequence_does_not_see_does_not_matter(window):
    base.test_what_a_sequence_does_not_see_does_not_matter(window, 70, 1)


@pytest.mark.parametrize("window", [0, 1, 64, 100, 300])
@pytest.mark.parametrize("d", [64, 128])
def test_windows_and_lengths(window, d):
    sizes, shared = [6, 3], [5, 2]
    lens = [320, 0, 1, 250, 700, 64, 128, 5, 129]
    total, table = base._tables(sizes, shared, lens, 12)
    q = base._rand((9, 120, d), 13)
    base._check(base._cache(total, 2, d, 14), q, table, lens, base._starts(sizes), shared, window)


def test_a_table_of_many_pages():
    """Rows of a wave follow the table's width as well: 100 rows behind 1,030 entries."""
    sizes, shared = [10], [6]
    lens = [400 + 7 * i for i in range(10)]
    total, table = base._tables(sizes, shared, lens, 15)
    wide = torch.full((10, 1030), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    q = base._rand((10, 10, 128), 16)
    base._check(base._cache(total, 1, 128, 17), q, wide, lens, base._starts(sizes), shared)


def test_absent_page_and_scales_far_apart():
    sizes, shared, lens = [5], [4], [250, 256, 300, 70, 320]
    total, table = base._tables(sizes, shared, lens, 18)
    c = base._cache(total, 1, 64, 19)
    table[0, 1] = total                               # a shared page that is none
    c.v_scale[int(table[0, 2])] = 2.0 ** -90
    q = base._rand((5, 100, 64), 20)
    base._check(c, q, table, lens, base._starts(sizes), shared)
