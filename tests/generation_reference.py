"""The operators for several continuations of one prompt from their definitions, on the
host: attention over shared pages in 64 bits with the bound of its roundings, the block
tables and pages as a program would deal them out one after the other, and beam
search's selection over all candidates."""
import math

import torch

from tests.attn_reference import FP32

F64 = torch.float64
PAGE = 64


def shared_table(table, group_start, shared):
    """The table that each sequence reads by: its group's first row in front."""
    t = table.clone()
    for a, b, p in zip(group_start, group_start[1:], shared):
        for n in range(a, b):
            t[n, :p] = table[a, :p]
    return t


def shared_decode(q, cache, table, lens, group_start, shared, window=0, scale=None, bf16=False):
    """q [N, Hq, d] in 64 bits, cache an attn_reference.Cache -> o and the bound of an fp32
    (bf16) result.

    Scores: a dot product of d exact products and the roundings of scale, log2 e and their
    product, (d + 4) 2^-24 of the terms' magnitudes.  A weight's factor is formed from sums
    of the maxima and the scale's logarithm, four roundings of values up to those; it, the
    weight and the joins of waves and of partial results are exponentials of 2^-22 each
    (six at most).  A weight as two f16 values keeps 22 bits, as one 11, relative to the
    largest down to 2^-26; below, half a step of 2^-24 is 2^-37 of it (it stands at 2^12 or
    above)."""
    N, Hq, d = q.shape
    H = cache.k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    t = shared_table(table, group_start, shared)
    o, tol = torch.zeros_like(q), torch.zeros_like(q)
    for i in range(N):
        n = min(int(lens[i]), t.shape[1] * PAGE)
        if n <= 0:
            continue
        lo = max(0, int(lens[i]) - window) if window else 0
        k, v, ok = cache.tokens(t[i], n)
        at = torch.arange(n)
        at = at[ok & (at >= lo)]
        if not len(at):
            continue
        k, v = k[:, at].repeat_interleave(Hq // H, 0), v[:, at].repeat_interleave(Hq // H, 0)
        s = (q[i][:, None] * k).sum(-1) * scale
        p = torch.softmax(s, -1)
        o[i] = (p[..., None] * v).sum(1)
        mag = ((q[i].abs()[:, None] * k.abs()).sum(-1) * scale).amax(-1)
        far = max(abs(math.log2(float(x))) for x in cache.vs.flatten() if math.isfinite(float(x)) and float(x) > 0)
        rel = (d + 12) * FP32 * mag + 6 * 2.0 ** -22 + 4 * FP32 * (far + 16)
        A = (p[..., None] * v.abs()).sum(1)
        top = (p[..., None] * cache.vs.amax() * 448).amax(1)
        tol[i] = (2.0 ** -11 if bf16 else 2.0 ** -22) * A + (2.1 * rel[:, None] + (len(at) + 16) * FP32) * A \
            + len(at) * 2.0 ** -37 * top + (2.0 ** -8 if bf16 else 4 * FP32) * o[i].abs() * 1.01
    return o, tol


def pages_of(n):
    return (n + PAGE - 1) // PAGE


def _rows(table, lens, n_pages):
    """Each row's pages: as many as its tokens need, entries that are no page as -1."""
    width = table.shape[1]
    out, held = [], []
    for row, n in zip(table.tolist(), lens.tolist()):
        n = max(0, min(n, width * PAGE))
        held.append(n)
        out.append([x if 0 <= x < n_pages else -1 for x in row[:pages_of(n)]])
    return out, held


def fork(table, lens, n_pages, parent=None, room=1, held=None):
    """-> new table, lengths, missing, copies [(source, place)]."""
    width = table.shape[1]
    old, n_old = _rows(table, lens, n_pages)
    parent = list(range(len(old))) if parent is None else list(parent)
    room = [room] * len(parent) if isinstance(room, int) else [max(0, int(r)) for r in room]
    held = [0] * n_pages if held is None else list(held)
    live = [0 <= p < len(old) for p in parent]
    rows = [list(old[p]) if ok else [] for p, ok in zip(parent, live)]
    n = [n_old[p] if ok else 0 for p, ok in zip(parent, live)]
    names, writers = [0] * n_pages, {}
    for i, row in enumerate(rows):
        for page in row:
            if page >= 0:
                names[page] += 1
        if n[i] % PAGE and room[i] and row[n[i] // PAGE] >= 0:
            writers.setdefault(row[n[i] // PAGE], []).append(i)
    free = iter([p for p in range(n_pages) if not names[p] and not held[p]])
    missing, copies = [0] * len(rows), []
    out = torch.full((len(rows), width), -1, dtype=torch.int32)
    for i, row in enumerate(rows):
        row = list(row)
        if live[i] and room[i]:
            if n[i] % PAGE and row[-1] >= 0:
                page = row[-1]
                if held[page] or len(writers[page]) != names[page] or writers[page][0] != i:
                    to = next(free, -1)
                    missing[i] += to < 0
                    if to >= 0:
                        copies.append((page, to))
                        row[-1] = to
            for _ in range(min(width, pages_of(n[i] + room[i])) - len(row)):
                to = next(free, -1)
                missing[i] += to < 0
                row.append(to)
        out[i, :len(row)] = torch.tensor(row, dtype=torch.int32)
    return out, torch.tensor(n, dtype=torch.int32), torch.tensor(missing, dtype=torch.int32), copies


def compact(table, lens, n_pages, held=None):
    """-> new table, used, moves [(source, place)]."""
    rows, _ = _rows(table, lens, n_pages)
    held = [0] * n_pages if held is None else list(held)
    named = {p for row in rows for p in row if p >= 0}
    free = [p for p in range(n_pages) if p not in named and not held[p]]
    high = sorted((p for p in named if not held[p]), reverse=True)
    moves = [(b, a) for a, b in zip(free, high) if a < b]
    to = dict(moves)
    out = torch.full(table.shape, -1, dtype=torch.int32)
    for i, row in enumerate(rows):
        out[i, :len(row)] = torch.tensor([to.get(p, p) for p in row], dtype=torch.int32)
    used = max([0] + [to.get(p, p) + 1 for p in named] + [p + 1 for p in range(n_pages) if held[p]])
    return out, used, moves


def select(x, scores, M, ended=None, end=-1, keep=False):
    """x [G K, V] in 64 bits, scores [G, K]: every candidate of a group sorted.
    -> tokens, rows, scores (64 bits), ended, and the smallest gap between two scores of
    different beams among the taken and the first one left."""
    G, K = scores.shape
    V = x.shape[1]
    out, gap = [], math.inf
    for g in range(G):
        cand = []
        for k in range(K):
            row, base = x[g * K + k], float(scores[g, k])
            top = float(row.max()) if not bool(row.isnan().any()) else math.nan
            lse = top + math.log(float((row - top).exp().sum())) if math.isfinite(top) else math.nan
            if not math.isfinite(base) or (not math.isfinite(lse) and not (ended is not None and bool(ended[g, k]))):
                cand += [(-math.inf, k, 0.0, t) for t in range(min(V, M))]
            elif ended is not None and bool(ended[g, k]):
                cand += [(base, k, 1.0, end)] + [(-math.inf, k, 0.0, t) for t in range(min(V, M + 1)) if t != end]
            else:
                best = sorted(range(V), key=lambda t: (-float(row[t]), t))[:M]
                cand += [(base + float(row[t]) - lse, k, float(row[t]), t) for t in best]
        cand.sort(key=lambda c: (-c[0], c[1], -c[2], c[3]))
        for a, b in zip(cand[:M], cand[1:M + 1]):
            if a[1] != b[1] and a[0] != b[0]:
                gap = min(gap, a[0] - b[0])
        took = cand[:M]
        if keep:
            place, rest = [None] * M, []
            for c in took:
                if place[c[1]] is None:
                    place[c[1]] = c
                else:
                    rest.append(c)
            took = [c if c is not None else rest.pop(0) for c in place]
        out.append(took)
    tokens = torch.tensor([[c[3] for c in t] for t in out], dtype=torch.int32)
    rows = torch.tensor([[g * K + c[1] for c in t] for g, t in enumerate(out)], dtype=torch.int32)
    value = torch.tensor([[c[0] for c in t] for t in out], dtype=F64)
    over = torch.tensor([[(ended is not None and bool(ended[g, c[1]])) or c[3] == end for c in t] for g, t in enumerate(out)])
    return tokens, rows, value, over, gap
