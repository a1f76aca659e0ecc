"""A key or value that a query does not see has no effect on it: not on one bit of its
results, whatever its (finite) size."""
import pytest
import torch

from tests.test_gpu_attn import _back, _forward, _inputs

pytestmark = pytest.mark.gpu


def _rows(t, packed, rows):
    return _back(t, packed, False)[:, :, rows]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,cu,T", [(0, None, 128), (40, None, 128), (100, None, 128), (0, [0, 100, 128], 128),
                                         (0, None, 300), (0, [0, 230, 300], 300)])
def test_forward_rows_do_not_depend_on_keys_they_do_not_see(window, cu, T, d):
    """The last key, which the last query alone sees, or the second sequence's keys: made
    to match the queries that see them, so that those rows' maximum jumps."""
    x = _inputs(1, 2, 1, T, T, d, 30)
    keep = torch.arange(T) < (cu[1] if cu else T - 1)
    o, lse = _forward(x, window, cu)
    for n, by in (("k", 8.0), ("k", 200.0), ("v", 1e4), ("v", 3e38)):
        y = {m: t.clone() for m, t in x.items()}
        if n == "k":
            y["k"][0, 0, ~keep] = x["q"][0, 0, ~keep] * by
        else:
            y["v"][0, 0, ~keep] = by
        o2, lse2 = _forward(y, window, cu)
        packed = cu is not None
        assert torch.equal(_rows(o, packed, keep), _rows(o2, packed, keep)), (n, by)
        assert torch.equal(lse.cpu()[..., keep], lse2.cpu()[..., keep]), (n, by)
        if n == "k" and by > 8:
            assert not torch.equal(_rows(o, packed, ~keep), _rows(o2, packed, ~keep))
