"""The operators for several continuations of one prompt together, as a search uses them:
a small hybrid model (a recurrent layer and an attention layer) that searches with beams,
in eager steps, in a captured graph and on two streams, and the attention at sizes that
its kernels walk in several pieces."""
import math

import pytest
import torch

import gated_delta_rule_24_amd as gdr
from tests import attn_reference as attn
from tests import generation_reference as ref

pytestmark = pytest.mark.gpu
gen = gdr.generation
F64, BF16 = torch.float64, torch.bfloat16
H, HQ, HKV, D = 2, 4, 2, 64
LAYERS = 3


def _rand(shape, seed, by=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * by


class Model:
    """Keys, values, queries and gates are a token's own; logits a product with both layers'
    outputs."""

    def __init__(self, V, seed):
        bf = lambda *s, by=1.0, k=0: _rand((V, *s), seed + k, by).to(BF16).cuda()  # noqa: E731
        self.q, self.k, self.v = bf(HQ, D, k=1), bf(HKV, D, k=2), bf(HKV, D, k=3)
        self.r = [bf(H, D, by=0.1, k=4), bf(H, D, by=0.1, k=5), bf(H, D, k=6),
                  torch.nn.functional.logsigmoid(_rand((V, H, D), seed + 7) + 2).cuda(), torch.sigmoid(_rand((V, H, D), seed + 8)).to(BF16).cuda(),
                  torch.sigmoid(_rand((V, H, D), seed + 9)).to(BF16).cuda()]
        self.out = (_rand((HQ * D + H * D, V), seed + 10, 0.2)).cuda()

    def recur(self, tokens, S):
        """One step of every layer of S [LAYERS, N, H, D, D]; the last one's output."""
        x = [t[tokens] for t in self.r]
        for layer in S:
            o = gdr.decode_step(*x, layer)
        return o

    def logits(self, o, r):
        # (sums by halves: no library call that a graph could not hold)
        x = torch.cat([o.flatten(1), r.flatten(1)], 1)[:, :, None] * self.out[None]
        x = x.view(len(o), 3, -1, x.shape[2])
        while x.shape[2] > 1:
            x = x[:, :, :x.shape[2] // 2] + x[:, :, x.shape[2] // 2:]
        return (x[:, 0, 0] + x[:, 1, 0]) + x[:, 2, 0]

    def replay(self, histories):
        """States [LAYERS, N, H, D, D] behind all but the last token of each of N histories, each
        row alone in a batch of N."""
        S = torch.zeros((LAYERS, len(histories), H, D, D), device="cuda")
        out = S.clone()
        for t in range(max(len(h) for h in histories)):
            for n, h in enumerate(histories):
                if len(h) - 1 == t:
                    out[:, n] = S[:, n]
            self.recur(torch.tensor([h[min(t, len(h) - 1)] for h in histories], device="cuda"), S)
        return out


class Search:
    """Tables, cache, states and scores of G prompts with K beams each."""

    def __init__(self, model, prompts, K, n_pages, width, order):
        self.m, self.K, G = model, K, len(prompts)
        N = G * K
        self.cache = gdr.kv_cache(n_pages, HKV, D)
        lens = torch.tensor([len(p) - 1 for p in prompts], dtype=torch.int32)
        table = torch.full((G, width), -1, dtype=torch.int32)
        at = iter(order)
        for g, n in enumerate(lens.tolist()):
            for i in range(ref.pages_of(n)):
                table[g, i] = next(at)
        table, self.len = table.cuda(), torch.zeros(G, dtype=torch.int32, device="cuda")
        # the prompts but for their last tokens, which the first step takes
        cu = torch.tensor([0] + lens.cumsum(0).tolist(), dtype=torch.int32).cuda()
        tokens = torch.tensor([t for p in prompts for t in p[:-1]], device="cuda")
        gdr.kv_append(model.k[tokens], model.v[tokens], self.cache, table, self.len, cu, token_major=True)
        self.S = model.replay([p for p in prompts for _ in range(K)])
        parent = torch.arange(G, dtype=torch.int32).repeat_interleave(K).cuda()
        self.table, self.len, missing = gen.kv_fork(self.cache, table, lens.cuda(), parent, room=1)
        assert not bool(missing.any())
        self.tokens = torch.tensor([p[-1] for p in prompts], dtype=torch.int32).repeat_interleave(K).cuda()
        self.scores = torch.full((G, K), -math.inf, device="cuda")
        self.scores[:, 0] = 0                         # one beam of each is there, the others are copies
        self.ended = torch.zeros((G, K), dtype=torch.bool, device="cuda")
        self.starts = torch.arange(0, N + 1, K, dtype=torch.int32).cuda()
        self.shared = (lens // 64).int().cuda()

    def step(self, end):
        t = self.tokens.long()
        gdr.kv_append(self.m.k[t], self.m.v[t], self.cache, self.table, self.len)
        self.len += 1
        o = gen.attn_decode_shared(self.m.q[t], self.cache, self.table, self.len, self.starts, self.shared)
        r = self.m.recur(t, self.S)
        x = self.m.logits(o, r)
        took = gen.beam_select(x, self.scores, ended=self.ended, end_token=end, keep_slots=True)
        gen.state_reorder(self.S, took[1].flatten(), self.K, dim=1)
        table, length, missing = gen.kv_fork(self.cache, self.table, self.len, took[1].flatten(), room=1)
        self.tokens.copy_(took[0].flatten()), self.scores.copy_(took[2]), self.ended.copy_(took[3])
        self.table.copy_(table), self.len.copy_(length)
        return o, r, x, took, missing


class Plain:
    """Every beam with a history, pages and states of its own."""

    def __init__(self, model, prompts, K):
        self.m, self.K = model, K
        self.history = [list(p) for p in prompts for _ in range(K)]
        self.width = 4
        N = len(self.history)
        self.table = torch.arange(N * self.width, dtype=torch.int32).view(N, self.width)
        zeros = gdr.kv_cache(N * self.width, HKV, D, device="cpu")
        for x in zeros:
            x.zero_()
        self.cache, self.len = attn.Cache(*zeros), [0] * N
        for i, p in enumerate(self.history):
            self._append(i, p[:-1])

    def _append(self, i, tokens):
        k, v = [x[tokens].cpu().to(F64).transpose(0, 1) for x in (self.m.k, self.m.v)]
        self.cache.append([k], [v], self.table[i:i + 1], [self.len[i]])
        self.len[i] += len(tokens)

    def step(self):
        """The last tokens appended: queries, tables and lengths of this step's attention."""
        for i, h in enumerate(self.history):
            self._append(i, h[-1:])
        q = self.m.q[torch.tensor([h[-1] for h in self.history])].cpu().to(F64)
        one = list(range(len(self.history) + 1))
        return ref.shared_decode(q, self.cache, self.table, self.len, one, [0] * len(self.history))

    def go_on(self, tokens, rows):
        old = [list(h) for h in self.history]
        self.history = [old[r] + [t] for t, r in zip(tokens, rows)]
        self.len = [self.len[r] for r in rows]
        for x in (self.cache.k, self.cache.v, self.cache.ks, self.cache.vs):
            x.copy_(x.view(len(rows), self.width, *x.shape[1:])[rows].flatten(0, 1).clone())


PROMPTS = (62, 3, 130)


def _prompts(V, lens=PROMPTS):
    g = torch.Generator().manual_seed(5)
    return [torch.randint(0, V, (n,), generator=g).tolist() for n in lens]


@pytest.mark.parametrize("K", [1, 4, 5])
def test_a_beam_search(K):
    """Each step's attention against the beams' own histories, its selection against all
    candidates, and at the end every state, bit for bit, against its history alone."""
    V, end = 50, 7
    model, prompts = Model(V, 3), _prompts(50)
    G, N = len(prompts), len(prompts) * K
    n_pages = 6 + 3 * N
    s = Search(model, prompts, K, n_pages, 4, torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).tolist())
    plain, moved = Plain(model, prompts, K), 0
    for step in range(9):
        # (equal scores, as of a prompt's first copies, are settled by the order of beams)
        before, ended = s.scores.cpu().clone(), s.ended.cpu().clone()
        o, r, x, took, missing = s.step(end)
        want, tol = plain.step()
        assert bool(((o.cpu().to(F64) - want).abs() <= tol).all()), step
        assert not bool(missing.any())
        tokens, rows, score, over, gap = ref.select(x.cpu().to(F64), before, K, ended, end, True)
        # (the bound of the selection's own test)
        spread = float(x.max() - x.min())
        assert gap > 2 * (2.0 ** -22 + 2.0 ** -23 * spread + (V / 256 + 18) * 2.0 ** -24)
        assert torch.equal(took[0].cpu(), tokens) and torch.equal(took[1].cpu(), rows) and torch.equal(took[3].cpu(), over)
        plain.go_on(tokens.flatten().tolist(), rows.flatten().tolist())
        moved += int((rows.flatten() != torch.arange(N)).sum())
        if step == 4:
            # the pages in use at the front: nothing else changes
            s.table, used = gen.kv_compact(s.cache, s.table, s.len, table_out=s.table)
            named = set(s.table[s.table >= 0].tolist())
            assert int(used) == len(named) == max(named) + 1
            s.table, s.len, missing = gen.kv_fork(s.cache, s.table, s.len, room=1)
            assert not bool(missing.any())
    assert K == 1 or moved > 0
    assert torch.equal(s.tokens.cpu().int(), torch.tensor([h[-1] for h in plain.history], dtype=torch.int32))
    assert torch.equal(model.replay(plain.history), s.S)


def test_a_captured_step_replayed():
    """A step of a search in a graph, replayed with eager work in between, against the same
    steps made eagerly: the same arithmetic, so the same bits.  Another search's graph with
    workspaces of its own is replayed by turns."""
    V, K, end = 40, 4, 3
    model = Model(V, 9)
    order = torch.randperm(60, generator=torch.Generator().manual_seed(2)).tolist()
    prompts = [_prompts(V), _prompts(V, (70, 65, 2))]
    graphs, searches, eager = [], [], [Search(model, p, K, 60, 4, order) for p in prompts]
    side = torch.cuda.Stream()
    for p in prompts:
        warm = Search(model, p, K, 60, 4, order)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            warm.step(end)
        torch.cuda.current_stream().wait_stream(side)
        s = Search(model, p, K, 60, 4, order)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            out = s.step(end)
        graphs.append((graph, out)), searches.append(s)
    for _ in range(5):
        for (graph, out), s, e in zip(graphs, searches, eager):
            graph.replay()
            want = e.step(end)
            torch.cuda.synchronize()
            for a, b in zip((*out[:3], *out[3], out[4]), (*want[:3], *want[3], want[4])):
                assert torch.equal(a, b)
            assert torch.equal(s.table, e.table) and torch.equal(s.len, e.len) and torch.equal(s.S, e.S)
            junk = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(4)]   # other work's memory
            del junk


def test_two_searches_at_once_on_two_streams():
    V, K, end = 40, 4, 3
    model = Model(V, 9)
    order = torch.randperm(60, generator=torch.Generator().manual_seed(2)).tolist()
    prompts = [_prompts(V), _prompts(V, (70, 65, 2))]
    alone = [Search(model, p, K, 60, 4, order) for p in prompts]
    both = [Search(model, p, K, 60, 4, order) for p in prompts]
    for s in alone:
        for _ in range(6):
            s.step(end)
    streams = [torch.cuda.Stream() for _ in both]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(6):
        for s, st in zip(both, streams):
            with torch.cuda.stream(st):
                s.step(end)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert torch.equal(a.tokens, b.tokens) and torch.equal(a.scores, b.scores)
        assert torch.equal(a.table, b.table) and torch.equal(a.S, b.S)


def test_the_stream_argument():
    """Inputs ready on another stream, the calls on it, and the results read behind it."""
    V, K = 300, 4
    x, scores = _rand((8, V), 1, 2.5).cuda(), -_rand((2, K), 2).abs().cuda()
    S, rows = _rand((8, 4, 64), 3).cuda(), torch.tensor([1, 0, 3, 3, 4, 4, 4, 7], dtype=torch.int32).cuda()
    cache = gdr.kv_cache(30, HKV, D)
    for t, by in zip(cache, (120, 119, 1, 2)):      # (bytes below that of NaN)
        t.copy_((torch.rand(t.shape, generator=torch.Generator().manual_seed(by)) * by).to(t.dtype))
    table = torch.randperm(30, generator=torch.Generator().manual_seed(4))[:24].view(8, 3).int().cuda()
    lens = torch.tensor([5, 64, 100, 192, 0, 1, 65, 130], dtype=torch.int32).cuda()
    q, starts, shared = _rand((8, HQ, D), 5).to(BF16).cuda(), torch.tensor([0, 4, 8], dtype=torch.int32).cuda(), torch.tensor([0, 0], dtype=torch.int32).cuda()
    copies = lambda ts: type(ts)(*[t.clone() for t in ts])  # noqa: E731
    calls = [lambda S, c, **k: gen.beam_select(x, scores, **k), lambda S, c, **k: gen.state_reorder(S, rows, K, **k),
             lambda S, c, **k: gen.attn_decode_shared(q, c, table, lens, starts, shared, **k),
             lambda S, c, **k: gen.kv_fork(c, table, lens, room=3, **k), lambda S, c, **k: gen.kv_compact(c, table, lens, **k)]
    for call in calls:
        outs = []
        for stream in (None, torch.cuda.Stream()):
            S1, c1 = S.clone(), copies(cache)
            torch.cuda.synchronize()
            out = call(S1, c1, stream=stream)
            torch.cuda.synchronize()
            outs.append([*([out] if isinstance(out, torch.Tensor) else out), S1, *c1])
        for a, b in zip(*outs):
            assert torch.equal(a, b)


def _repeated(q, host, table, lens, bf16):
    """One sequence after the other, pages that a row names several times counted as often:
    o = sum_pages c sum_j p_j v_j / sum_pages c sum_j p_j.  The bound as in
    generation_reference.shared_decode."""
    N, Hq, d = q.shape
    rep = Hq // host.k.shape[1]
    k = (host.k * host.ks[:, :, None, None]).repeat_interleave(rep, 1)
    v = (host.v * host.vs[:, :, None, None]).repeat_interleave(rep, 1)
    o, tol = torch.zeros_like(q), torch.zeros_like(q)
    far = max(abs(math.log2(float(x))) for x in host.vs.flatten())
    for n in range(N):
        L = int(lens[n])
        count = torch.zeros((host.k.shape[0], 64), dtype=F64)
        whole = table[n, :L // 64].long()
        count += torch.bincount(whole, minlength=host.k.shape[0]).to(F64)[:, None]
        if L % 64:
            count[int(table[n, L // 64]), :L % 64] += 1
        s = (q[n][None, :, None] * k).sum(-1) * d ** -0.5               # [pages, Hq, 64]
        seen = (count > 0)[:, None].expand_as(s)
        top = s.masked_fill(~seen, -math.inf).amax((0, 2))
        w = torch.where(seen, count[:, None] * (s - top[None, :, None]).exp(), 0.0)
        w = w / w.sum((0, 2), keepdim=True)
        o[n], A = (w[..., None] * v).sum((0, 2)), (w[..., None] * v.abs()).sum((0, 2))
        mag = ((q[n].abs()[None, :, None] * k.abs()).sum(-1) * d ** -0.5).amax((0, 2))
        rel = (d + 12) * attn.FP32 * mag + 6 * 2.0 ** -22 + 4 * attn.FP32 * (far + 16)
        tol[n] = (2.0 ** -11 if bf16 else 2.0 ** -22) * A + (2.1 * rel[:, None] + (L + 16) * attn.FP32) * A \
            + L * 2.0 ** -37 * 448 * host.vs.amax() + (2.0 ** -8 if bf16 else 4 * attn.FP32) * o[n].abs() * 1.01
    return o, tol


@pytest.mark.parametrize("sizes,shared,own,Hq,Hkv", [
    ([2], [20001], 70, 4, 4),          # a wave has more shared pages than it looks up at once
    ([1, 700, 400], [0, 1, 2], 5000, 1, 1),        # more own ones, of many sequences
    ([90, 3], [3000, 41], 65, 16, 2),   # 64 rows a wave, runs over the ends of units
    ([3] * 600, [9] * 600, 20, 2, 1)])             # more units than workgroups
@pytest.mark.parametrize("out", [torch.float32, BF16])
def test_attention_over_many_pages(sizes, shared, own, Hq, Hkv, out):
    """Long tables whose entries name a few pages over and over.  Three pages with scores 8 times
    as large, which outweigh all others, stand once each in a row: behind the entries that
    a wave has looked up at first, at the end of the shared pages, and at the row's end."""
    N, d, n_pages = sum(sizes), 64, 23
    g = torch.Generator().manual_seed(N)
    cache = gdr.kv_cache(n_pages, Hkv, d, device="cpu")
    for x in (cache.k, cache.v):
        x.copy_((torch.randn(x.shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    for x in (cache.k_scale, cache.v_scale):
        x.copy_(torch.pow(2.0, torch.randint(-8, -4, x.shape, generator=g).float()))
    starts = [0] + torch.tensor(sizes).cumsum(0).tolist()
    lens = [0] * N
    for a, b, p in zip(starts, starts[1:], shared):
        for n in range(a, b):
            lens[n] = p * 64 + int(torch.randint(0, own + 1, (1,), generator=g))
    cache.k_scale[20:] *= 8
    width = max(ref.pages_of(n) for n in lens)
    table = torch.randint(0, 20, (N, width), generator=g, dtype=torch.int32)
    for a, p in zip(starts, shared):
        if p:
            table[a, 300 if p > 300 else p // 2] = 20
            table[a, p - 1] = 21
    for n in range(N):
        if lens[n]:
            table[n, ref.pages_of(lens[n]) - 1] = 22
    read = ref.shared_table(table, starts, shared)
    q = torch.randn((N, Hq, d), generator=g).to(BF16)
    ints = [torch.as_tensor(x, dtype=torch.int32).cuda() for x in (table, lens, starts, shared)]
    got = gen.attn_decode_shared(q.cuda(), gdr.KVCache(*[x.cuda() for x in cache]), *ints, out_dtype=out).cpu().to(F64)
    some = sorted(set(list(range(0, N, max(1, N // 12))) + [N - 1, int(torch.tensor(lens).argmax())]))
    want, tol = _repeated(q[some].to(F64), attn.Cache(*cache), read[some], [lens[n] for n in some], out is BF16)
    off = (got[some] - want).abs()
    assert bool((off <= tol).all()), float((off / tol.clamp_min(1e-300)).max())


def test_pages_past_32_bits():
    """A cache of more than 2^32 bytes a side: the last pages read, copied and moved."""
    Hkv, d = 8, 128
    n_pages = (1 << 32) // (Hkv * 64 * d) + 40
    cache = gdr.kv_cache(n_pages, Hkv, d)
    cache.k_scale.zero_(), cache.v_scale.zero_()
    last = list(range(n_pages - 4, n_pages))
    g = torch.Generator().manual_seed(8)
    for x in (cache.k, cache.v):
        for p in last:
            x[p] = (torch.randn(x[p].shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    for x in (cache.k_scale, cache.v_scale):
        x[last] = torch.pow(2.0, torch.randint(-8, -4, (4, Hkv), generator=g).float()).cuda()
    few = gdr.KVCache(*[x[last].clone() for x in cache])
    table = torch.tensor([[last[3], last[0]], [last[3], last[1]], [last[2], -1]], dtype=torch.int32)
    lens, starts, shared = [128, 100, 30], [0, 2, 3], [1, 0]
    q = torch.randn((3, 8, d), generator=g).to(BF16)
    ints = [torch.as_tensor(x, dtype=torch.int32).cuda() for x in (table, lens, starts, shared)]
    got = gen.attn_decode_shared(q.cuda(), cache, *ints)
    want, tol = ref.shared_decode(q.to(F64), attn.Cache(*few), torch.where(table >= 0, table - last[0], table), lens, starts, shared)
    assert bool(((got.cpu().to(F64) - want).abs() <= tol).all())
    # the third row twice: its page is copied to the lowest free one; then everything to the front
    held = torch.ones(n_pages, dtype=torch.uint8)
    held[last] = 0
    held[5:8] = 0
    t, n, missing = gen.kv_fork(cache, ints[0], ints[1], torch.tensor([0, 1, 2, 2], dtype=torch.int32).cuda(), room=0, held=held.cuda())
    assert not bool(missing.any()) and t[2, 0] == t[3, 0] == last[2]
    t, n, missing = gen.kv_fork(cache, t, n, room=1, held=held.cuda())
    # (rows 2 and 3 are about to write on one page: the lower keeps it)
    assert not bool(missing.any()) and t.tolist() == [[last[3], last[0]], [last[3], last[1]], [last[2], -1], [5, -1]]
    t, used = gen.kv_compact(cache, t, n, held=held.cuda())
    # (free: 6 and 7; they take the two highest)
    assert t.tolist() == [[6, last[0]], [6, last[1]], [7, -1], [5, -1]] and int(used) == last[1] + 1
    got = gen.attn_decode_shared(q[[0, 1, 2, 2]].cuda(), cache, t, n, *[torch.as_tensor(x, dtype=torch.int32).cuda() for x in ([0, 2, 4], [1, 0])])
    four = [0, 1, 2, 2]
    assert bool(((got.cpu().to(F64) - want[four]).abs() <= tol[four]).all())


@pytest.mark.parametrize("out", [torch.float32, BF16])
@pytest.mark.parametrize("Hq,Hkv,d", [(2, 1, 64), (8, 2, 128), (64, 1, 64), (130, 1, 64), (200, 2, 128)])
def test_a_neighbours_page_changes_no_bit(Hq, Hkv, d, out):
    """A page that only the group's other sequences see, with a scale far from the rest: theirs
    take another way through the pages behind it, the first one's results stay bit for bit."""
    g = torch.Generator().manual_seed(3)
    cache = gdr.kv_cache(12, Hkv, d, device="cpu")
    for x in (cache.k, cache.v):
        x.copy_((torch.randn(x.shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    for x in (cache.k_scale, cache.v_scale):
        x.fill_(2.0 ** -6)
    # pages 1 .. 6 and 4 .. 9 of the shared ten: the second has page 1 for itself
    lens, window = [640, 448, 448], 384
    table = torch.arange(10, dtype=torch.int32).repeat(3, 1)
    q = torch.randn((3, Hq, d), generator=g).to(BF16)
    ints = [torch.as_tensor(x, dtype=torch.int32).cuda() for x in (table, lens, [0, 3], [10])]
    outs = []
    for scale in (2.0 ** -6, 2.0 ** 80, 2.0 ** -96, 0.0):
        c = gdr.KVCache(*[x.cuda() for x in cache])
        c.v_scale[1] = scale
        outs.append(gen.attn_decode_shared(q.cuda(), c, *ints, window=window, out_dtype=out))
    for o in outs[1:]:
        assert torch.equal(o[0], outs[0][0])
        assert not torch.equal(o[1], outs[0][1])


@pytest.mark.parametrize("groups", [1, 20, 64, 65, 150])
@pytest.mark.parametrize("window", [0, 3000])
def test_groups_of_uneven_length(groups, window):
    """Workgroups' runs that end and start inside units of different groups, some of which share
    nothing, have no sequence, or see nothing of what they share; as many groups as one wave plans
    for, and more."""
    d, n_pages, Hq, Hkv = 64, 9, 8, 4
    g = torch.Generator().manual_seed(groups)
    cache = gdr.kv_cache(n_pages, Hkv, d, device="cpu")
    for x in (cache.k, cache.v):
        x.copy_((torch.randn(x.shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    for x in (cache.k_scale, cache.v_scale):
        x.copy_(torch.pow(2.0, torch.randint(-8, -4, x.shape, generator=g).float()))
    sizes = torch.randint(0, 4, (groups,), generator=g).tolist()
    sizes[0] = 2
    shared = [int(torch.randint(0, 250, (1,), generator=g)) * (i % 5 != 3) for i in range(groups)]
    starts = [1] + (1 + torch.tensor(sizes).cumsum(0)).tolist()                  # the first and the last are in no group
    N = starts[-1] + 1
    lens = torch.randint(0, 260 * 64, (N,), generator=g).tolist()
    table = torch.randint(0, n_pages, (N, 260), generator=g, dtype=torch.int32)
    q = torch.randn((N, Hq, d), generator=g).to(BF16)
    ints = [torch.as_tensor(x, dtype=torch.int32).cuda() for x in (table, lens, starts, shared)]
    got = gen.attn_decode_shared(q.cuda(), gdr.KVCache(*[x.cuda() for x in cache]), *ints, window=window).cpu().to(F64)
    some = sorted(set(list(range(0, N, max(1, N // 10))) + [N - 1]))
    read = ref.shared_table(table, starts, shared)
    want, tol = ref.shared_decode(q[some].to(F64), attn.Cache(*cache), read[some], [lens[n] for n in some], list(range(len(some) + 1)),
                                  [0] * len(some), window)
    off = (got[some] - want).abs()
    assert bool((off <= tol).all()), float((off / tol.clamp_min(1e-300)).max())


@pytest.mark.parametrize("groups", [3, 64, 65, 300])
def test_bounds_in_no_order_stay_inside(groups):
    """Any numbers as bounds: every sequence has some result of its own rows, nothing else is
    touched, and a call with bounds in order behind it is right."""
    d, N = 64, 40
    g = torch.Generator().manual_seed(groups)
    cache = gdr.kv_cache(5, 2, d)
    for x in (cache.k, cache.v):
        x.copy_(torch.randint(0, 100, x.shape, generator=g).to(torch.uint8))
    for x in (cache.k_scale, cache.v_scale):
        x.fill_(0.01)
    table = torch.randint(0, 5, (N, 6), generator=g, dtype=torch.int32).cuda()
    lens = torch.randint(0, 6 * 64, (N,), generator=g).int().cuda()
    q = torch.randn((N, 4, d), generator=g).to(BF16).cuda()
    for high in (N, 10 ** 9):
        starts = torch.randint(-high, high, (groups + 1,), generator=g).int().cuda()
        shared = torch.randint(-3, 9, (groups,), generator=g).int().cuda()
        room = torch.full((N + 2, 4, d), 7.0, device="cuda")
        gen.attn_decode_shared(q, cache, table, lens, starts, shared, o=room[1:-1])
        assert bool((room[0] == 7).all()) and bool((room[-1] == 7).all())
    starts = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    alone = gen.attn_decode_shared(q, cache, table, lens, starts, shared)
    want, tol = ref.shared_decode(q.cpu().to(F64), attn.Cache(*cache), table.cpu(), lens.tolist(), list(range(N + 1)), [0] * N)
    assert bool(((alone.cpu().to(F64) - want).abs() <= tol).all())
