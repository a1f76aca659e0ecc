"""Beam search's selection where a run of a row's logits is walked in several pieces, and where
the join has as many runs as a group may have."""
import math

import pytest
import torch

import gated_delta_rule_24_amd as gdr

pytestmark = pytest.mark.gpu
gen = gdr.generation
F64, BF16, F32 = torch.float64, torch.bfloat16, torch.float32


def _runs(G, K, V, dtype):
    """(runs of a row, values of each, values that a workgroup takes at once)."""
    segs = gdr.gdr_beam_select_workspace_bytes(G, K, 1, V) // (16 * G * K)
    wide = 8 if dtype is BF16 else 4
    return segs, wide * -(-(-(-V // wide) + 1) // segs), 1024 * wide


def _best(x, scores, M):
    """x [K, V], scores [K] of one group: the best M of all candidates in 64 bits, and the least
    gap between neighbours of different beams among those and the first one left."""
    x = x.to(F64)
    lse = torch.logsumexp(x, 1)
    value, token = x.sort(dim=1, descending=True, stable=True)       # equal ones: the lower token first
    cand = []
    for k in range(len(x)):
        cand += [(float(scores[k]) + float(v) - float(lse[k]), k, float(v), int(t)) for v, t in zip(value[k, :M + 1], token[k, :M + 1])]
    cand.sort(key=lambda c: (-c[0], c[1], -c[2], c[3]))
    gap = min([a[0] - b[0] for a, b in zip(cand[:M], cand[1:M + 1]) if a[1] != b[1] and a[0] != b[0]], default=math.inf)
    return cand[:M], gap


def _check(x, scores, M, groups, dev=None):
    """As in test_gpu_beam: whole numbers equal, scores within the log-sum's bound."""
    G, K = scores.shape
    V = x.shape[1]
    got = [t.cpu() for t in gen.beam_select(x.cuda() if dev is None else dev, scores.cuda(), M)]
    for g in groups:
        rows = x[g * K:(g + 1) * K]
        fin = rows[torch.isfinite(rows)].to(F64)
        tol = 2.0 ** -22 + 2.0 ** -23 * min(float(fin.max() - fin.min()), 100.0) + (V / 256 + 18) * 2.0 ** -24
        want, gap = _best(rows, scores[g], M)
        assert gap > 2 * tol, "the inputs leave the order open"
        assert got[0][g].tolist() == [c[3] for c in want] and got[1][g].tolist() == [g * K + c[1] for c in want]
        w = torch.tensor([c[0] for c in want], dtype=F64)
        assert bool(((got[2][g].to(F64) - w).abs() <= 1.01 * tol + 2.0 ** -24 * w.abs()).all())


def _scores(G, K, seed):
    return (-20 * torch.rand((G, K), generator=torch.Generator().manual_seed(seed))).float()


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_long_runs_of_many_rows(dtype, pad):
    """64 searches of 8 beams, rows that start anywhere."""
    G, K, V = 64, 8, 70001
    segs, run, chunk = _runs(G, K, V, dtype)
    assert run > 4 * chunk and segs > 1
    wide = torch.full((G * K, V + pad), math.nan, dtype=dtype)
    wide[:, :V] = (torch.randn((G * K, V), generator=torch.Generator().manual_seed(1)) * 2.5).to(dtype)
    for M in (1, 8, 20):
        _check(wide[:, :V], _scores(G, K, 3), M, (0, 1, 31, 63), wide.cuda()[:, :V])


def _pattern(kind, V, dtype, segs, run, chunk, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(V, generator=g)
    if kind == "rising":
        x = torch.linspace(-30, 6, V)
    elif kind == "falling":
        x = torch.linspace(6, -30, V)
    elif kind == "equal":
        x = torch.full((V,), 0.5)
    elif kind == "steps":                             # each chunk above the one before it
        x = (torch.arange(V) // chunk).float() * 0.25 + (x > 3).float() * 0.125
    elif kind == "few, then many":
        # every run: a first piece, one with ten that pass, one in which more rise above all before
        # than there is room for, one with none, one that rises again
        for s in range(segs):
            at = s * run
            part = [x[at + i * chunk:min(at + (i + 1) * chunk, at + run)] for i in range(run // chunk + 1)]
            part[1].fill_(-10.0)
            part[1][100:110] = 5.0
            part[2][:2000] = torch.linspace(5.5, 7.5, 2000)[:len(part[2][:2000])]
            part[3].fill_(-11.0)
            part[4][:] = torch.linspace(4, 8, len(part[4]))
    return x.to(dtype)


@pytest.mark.parametrize("M", [1, 8, 64])
@pytest.mark.parametrize("kind", ["random", "rising", "falling", "equal", "steps", "few, then many"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_long_runs_of_64_beams(kind, M, dtype):
    """What a piece leaves behind for the next: the bound, the best so far, those listed beside
    them, and pieces with more candidates than there is room for."""
    G, K, V = 1, 64, 90001
    segs, run, chunk = _runs(G, K, V, dtype)
    assert run > 4 * chunk + 1000 and segs == 2
    x = torch.stack([_pattern(kind, V, dtype, segs, run, chunk, k) for k in range(K)])
    order = torch.randperm(K, generator=torch.Generator().manual_seed(M)).float()[None]
    _check(x, -20 * order, M, (0,))                   # all of the first beam's, then all of the last one's
    _check(x, -20 * (K - 1 - order), M, (0,))
    # some of many beams, which have the same row of multiples of 1/64 (in bf16 of multiples of that):
    # m / (129 64) is between scores of beams m apart, or more
    same = ((x[:1].float() * 64).round() / 64).to(dtype).repeat(K, 1)
    _check(same, -(13 + 1 / 129) / 64 * order, M, (0,))


@pytest.mark.parametrize("M", [1, 7, 63, 64])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_as_many_runs_as_a_group_may_have(M, dtype):
    """128 runs of a group, more than it selects: those whose first is among the best are joined."""
    G, K, V = 2, 64, 9001
    segs, _, _ = _runs(G, K, V, dtype)
    assert segs * K == 128
    x = (torch.randn((G * K, V), generator=torch.Generator().manual_seed(2)) * 2.5).to(dtype)
    _check(x, _scores(G, K, 5), M, (0, 1))
    close = -0.01 * torch.arange(G * K).float().view(G, K)           # many runs pass
    x[:, 77] += 9.0
    _check(x, close, M, (0, 1))


def test_one_row_of_as_many_runs():
    V = 128 * 8192 - 9
    segs, _, _ = _runs(1, 1, V, F32)
    assert segs == 128
    x = torch.randn((1, V), generator=torch.Generator().manual_seed(4))
    for M in (1, 64):
        _check(x, torch.tensor([[-1.0]]), M, (0,))
