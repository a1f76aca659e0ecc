"""Beam search's selection and the reordering of states against their definitions."""
import math

import pytest
import torch

import gated_delta_rule_24_amd as gdr
from tests import generation_reference as ref

pytestmark = pytest.mark.gpu
gen = gdr.generation
F64, INF = torch.float64, math.inf


def _logits(R, V, dtype, seed, by=2.5):
    return (torch.randn((R, V), generator=torch.Generator().manual_seed(seed)) * by).to(dtype)


def _check(x, scores, M, ended=None, end=-1, keep=False, view=None):
    """Whole numbers equal; scores within the bound.  (The order is settled where no two
    beams' scores are closer than the bound: that is checked on the definition.)

    The log-sum: each term's exponent d = x - max is off by one rounding and its product with
    log2 e by one, the exponential by 2^-22: weighted by the terms, 2^-22 + 2^-23 max|d| of
    the sum; a thread adds at most V / 256 + 8 terms and a run's threads and the rescalings
    ten more, 2^-24 each.  The result is rounded once."""
    V = x.shape[1]
    want = ref.select(x.to(F64), scores, M, ended, end, keep)
    fin = x.to(F64)[torch.isfinite(x)]
    spread = float(fin.max() - fin.min()) if fin.numel() else 0.0
    tol = 2.0 ** -22 + 2.0 ** -23 * min(spread, 100.0) + (V / 256 + 18) * 2.0 ** -24
    assert want[4] > 2 * tol, "the inputs leave the order open"
    dev = x.cuda() if view is None else view
    got = gen.beam_select(dev, scores.cuda(), M, None if ended is None else ended.cuda(), end, keep)
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])
    assert torch.equal(got[3].cpu(), want[3])
    s, w = got[2].cpu().to(F64), want[2]
    assert torch.equal(s == -INF, w == -INF)
    fine = w > -INF
    assert bool(((s - w).abs()[fine] <= tol * 1.01 + 2.0 ** -24 * w.abs()[fine]).all())
    return got


def _scores(G, K, seed):
    return (-20 * torch.rand((G, K), generator=torch.Generator().manual_seed(seed))).float()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,K,M,V", [
    (1, 1, 1, 1), (2, 1, 3, 3), (1, 2, 4, 2), (3, 4, 4, 7), (2, 3, 6, 255), (1, 4, 8, 256), (5, 2, 2, 257), (1, 64, 64, 300),
    (2, 5, 10, 2047), (1, 1, 64, 2049), (3, 7, 7, 8191), (1, 4, 4, 32001), (1, 2, 64, 40000), (40, 1, 5, 1000),
    (2, 64, 64, 4099)])
def test_select_against_all_candidates_sorted(G, K, M, V, dtype):
    _check(_logits(G * K, V, dtype, V + M), _scores(G, K, V), M, end=min(2, V - 1))


@pytest.mark.parametrize("V", [5, 1000, 9001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_select_ties_go_to_the_lowest_token(V, dtype):
    x = torch.zeros((3, V), dtype=dtype)
    x[1, ::2] = -0.0                                  # equal to +0
    x[2] = _logits(1, V, dtype, 4, by=0.02)[0].round()
    for M in (1, 5):
        _check(x, torch.tensor([[-1.0, -1.125, -1.3]]), M)
    _check(torch.cat([x[2:], x[2:]]), torch.tensor([[-1.5, -1.5]]), 4)      # two beams alike: the lower beam first
    got = gen.beam_select(torch.cat([x[2:], x[2:]]).cuda(), torch.tensor([[-1.5, -1.5]]).cuda(), 2)
    assert got[1].cpu().tolist() == [[0, 1]] or got[1].cpu().tolist() == [[0, 0]]


@pytest.mark.parametrize("M", [1, 8, 64])
@pytest.mark.parametrize("down", [False, True])
def test_select_of_logits_in_order(M, down):
    """Rising logits: every value passes the bound that the ones before it left."""
    x = torch.linspace(-30, 5, 50000, dtype=torch.float32)[None].repeat(2, 1)
    x[1] += 0.01 * torch.arange(50000) % 3
    if down:
        x = x.flip(1).contiguous()
    _check(x, torch.tensor([[-1.0, -2.01]]), M)


@pytest.mark.parametrize("pad", [1, 3, 7, 8, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_select_rows_of_a_wider_tensor(pad, dtype):
    """Rows that start anywhere; what lies between them is not read as theirs."""
    V = 3001
    wide = torch.full((12, V + pad), math.nan, dtype=dtype)
    wide[:, :V] = _logits(12, V, dtype, pad)
    dev = wide.cuda()
    _check(wide[:, :V], _scores(3, 4, pad), 4, view=dev[:, :V])
    exact = torch.full((12, V), INF, dtype=dtype)     # the last row ends where the memory does
    exact.copy_(wide[:, :V])
    _check(exact, _scores(3, 4, pad), 4)


def test_select_masked_rows_and_values():
    x = _logits(8, 600, torch.float32, 9)
    x[0, 3:] = -INF                                   # three candidates left
    x[1] = -INF                                       # none
    x[2, 77] = math.nan
    x[3, 5] = INF
    x[5, :] = -3.4e38                                 # the type's lowest value everywhere
    x[6, 1:] = -3.4e38
    for M in (1, 2, 4, 9, 64):
        _check(x, torch.tensor([[-1.0, 0.0, 0.0, 0.0], [-2.0, -1.0, -7.0, -INF]]), M)
    _check(x, torch.tensor([[-INF, -INF, 0.0, math.nan], [-INF, INF, -INF, -INF]]), 7)
    _check(torch.full((4, 50), -INF), torch.zeros((1, 4)), 10)


@pytest.mark.parametrize("keep", [False, True])
def test_select_ended_beams(keep):
    """An ended beam goes on with its own score; its logits are not read."""
    x = _logits(12, 500, torch.bfloat16, 5)
    ended = torch.zeros((3, 4), dtype=torch.bool)
    ended[0, 1] = ended[1] = True
    x[1] = math.nan
    scores = torch.tensor([[-3.0, -3.1, -9.0, -1.0], [-4.0, -2.0, -3.0, -1.0], [-5.0, -5.2, -5.1, -1.0]])
    got = _check(x, scores, 4, ended, 7, keep)
    assert got[0][1].tolist() == [7] * 4 and bool(got[3][1].all())
    if not keep:
        for M in (1, 6, 30):
            _check(x, scores, M, ended, 0)
            _check(x, scores, M, ended, 499)


def test_select_keeps_beams_in_their_places():
    for seed in range(6):
        K = (2, 3, 8, 16, 33, 64)[seed]
        x, s = _logits(2 * K, 700, torch.float32, seed), _scores(2, K, seed)
        tokens, rows, _, _ = _check(x, s, K, keep=True)
        own = torch.arange(2 * K).view(2, K).int()
        for g in range(2):
            alive = set(rows[g].tolist())
            for k in range(K):                        # a beam that goes on is in its own place
                assert (int(own[g, k]) in alive) == (int(rows[g, k]) == int(own[g, k]))


def test_select_many_rows():
    """More groups than compute units; each against its own call."""
    x, s = _logits(700 * 3, 1500, torch.bfloat16, 1), _scores(700, 3, 2)
    got = gen.beam_select(x.cuda(), s.cuda(), 3)
    for g in (0, 1, 350, 699):
        one = ref.select(x[3 * g:3 * g + 3].to(F64), s[g:g + 1], 3)
        assert torch.equal(got[0][g:g + 1].cpu(), one[0]) and torch.equal(got[1][g:g + 1].cpu(), one[1] + 3 * g)


# ---------------------------------------------------------------------------


@pytest.mark.parametrize("K", [1, 2, 4, 5, 8, 13, 16, 30, 32, 33, 64])
@pytest.mark.parametrize("shape,dtype", [((4,), torch.float32), ((3, 8), torch.bfloat16), ((5, 7, 16), torch.float32),
                                         ((2, 64, 64), torch.float32), ((16,), torch.uint8)])
def test_reorder_any_map_of_a_group(K, shape, dtype):
    g = torch.Generator().manual_seed(K)
    for layers, groups in ((1, 1), (3, 2), (1, 5)):
        N = groups * K
        state = torch.randint(0, 200, (layers, N) + shape, generator=g).to(dtype)
        rows = torch.randint(0, K, (N,), generator=g) + K * (torch.arange(N) // K)
        want = state[:, rows]
        dev = state.cuda()
        out = gen.state_reorder(dev, rows.int().cuda(), K, dim=1)
        assert out.data_ptr() == dev.data_ptr() and torch.equal(dev.cpu(), want)
        one = state[0].cuda()
        gen.state_reorder(one, rows.int().cuda().view(groups, K), K)
        assert torch.equal(one.cpu(), want[0])


def test_reorder_leaves_rows_whose_source_is_not_of_their_group():
    state = torch.arange(8 * 4, dtype=torch.float32).view(8, 4)
    rows = torch.tensor([4, -1, 2 ** 31 - 1, 0, -2 ** 31, 4, 3, 8], dtype=torch.int32)
    dev = state.cuda()
    gen.state_reorder(dev, rows.cuda(), 4)
    assert torch.equal(dev.cpu(), state[[0, 1, 2, 0, 4, 4, 6, 7]])
