"""A key or value that a query does not see, and a query that does not see a key,
have no effect on it: not on one bit of its results, whatever their (finite) size."""
import pytest
import torch

from tests.test_gpu_attn import _back, _backward, _forward, _inputs

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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,cu,T", [(0, None, 128), (40, None, 128), (0, [0, 100, 128], 128), (30, None, 300),
                                         (0, [0, 230, 300], 300)])
def test_gradients_of_queries_do_not_depend_on_keys_they_do_not_see(window, cu, T, d):
    """Values near the type's largest: dO.v of a pair that is not seen overflows, and must
    not reach dq through 0 * infinity."""
    x = _inputs(1, 2, 1, T, T, d, 31)
    keep = torch.arange(T) < (cu[1] if cu else T - 1)
    packed = cu is not None
    o, lse = _forward(x, window, cu)
    want = _backward(x, o, lse, window, cu)
    assert bool(torch.isfinite(want["dq"]).all())
    for n, value in (("v", 3e38), ("v", -3e38), ("k", 3e38), ("v", torch.finfo(torch.bfloat16).min)):
        y = {m: t.clone() for m, t in x.items()}
        y[n][0, 0, ~keep] = value
        got = _backward(y, o, lse, window, cu)
        assert torch.equal(_rows(got["dq"], packed, keep), _rows(want["dq"], packed, keep)), (n, value)
        if packed:                                   # the first sequence's keys are seen by its own queries only
            for m in ("dk", "dv"):
                assert torch.equal(_rows(got[m], packed, keep), _rows(want[m], packed, keep)), (n, value, m)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,cu,T,row", [(0, None, 128, 0), (0, None, 300, 0), (20, None, 300, 140),
                                             (0, [0, 100, 128], 128, 99), (0, [0, 90, 128], 128, 0)])
def test_gradients_of_keys_do_not_depend_on_queries_that_do_not_see_them(window, cu, T, row, d):
    """One query's dO is near the type's largest in a channel where the values it sees are
    0 and the others 2: its D is 0 and dO.v of the pairs that are not seen infinite."""
    x = _inputs(1, 2, 1, T, T, d, 32)
    packed = cu is not None
    end = [e for e in cu if e <= row][-1] if cu else 0
    seen = torch.zeros(T, dtype=torch.bool)
    seen[max(end, row - window + 1 if window else 0):row + 1] = True
    x["v"][0, 0, :, 7] = torch.where(seen, 0.0, 2.0).to(torch.bfloat16)
    o, lse = _forward(x, window, cu)
    want = _backward(x, o, lse, window, cu)
    x["dO"][0, :, row, 7] = 3e38
    got = _backward(x, o, lse, window, cu)
    for m in ("dk", "dv"):
        assert torch.equal(_rows(got[m], packed, ~seen), _rows(want[m], packed, ~seen)), m
    others = torch.arange(T) != row
    assert torch.equal(_rows(got["dq"], packed, others), _rows(want["dq"], packed, others))
    assert bool(torch.isfinite(got["dq"]).all()) and bool(torch.isfinite(got["dk"]).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,cu,T,row", [(0, None, 128, 0), (0, None, 300, 0), (20, None, 300, 140),
                                             (0, [0, 100, 128], 128, 99), (0, [0, 90, 128], 128, 0)])
def test_a_query_whose_own_sum_overflows_reaches_only_the_keys_that_it_sees(window, cu, T, row, d):
    """dO near the type's largest in every channel of one query: its D overflows."""
    x = _inputs(1, 2, 1, T, T, d, 33)
    packed = cu is not None
    start = [e for e in cu if e <= row][-1] if cu else 0
    seen = torch.zeros(T, dtype=torch.bool)
    seen[max(start, row - window + 1 if window else 0):row + 1] = True
    o, lse = _forward(x, window, cu)
    want = _backward(x, o, lse, window, cu)
    x["dO"][0, :, row] = 3e38
    got = _backward(x, o, lse, window, cu)
    for m in ("dk", "dv"):
        assert torch.equal(_rows(got[m], packed, ~seen), _rows(want[m], packed, ~seen)), m
    others = torch.arange(T) != row
    assert torch.equal(_rows(got["dq"], packed, others), _rows(want["dq"], packed, others))
