"""Several continuations of one prompt, operator by operator: the cases that are timed, the operators'
plain forms and their values in 64 bits.

A hybrid stack that samples several continuations of a prompt, searches with beams or serves a batch
behind a common system prompt needs, next to the recurrence's and the attention layer's single steps:

* ``shared``   attention of one query token per sequence where groups of sequences share their first
               cache pages, which are read once for the group;
* ``fork``     the block tables of the continuations: shared pages, copies of the pages that several
               are about to write, fresh pages, pages let go;
* ``compact``  used pages moved to the lowest places;
* ``select``   the best continuations of each prompt over its beams and the vocabulary;
* ``reorder``  recurrent states moved to the rows that continue them.

``run`` computes the plain forms with elementary torch operations, or, where ``own`` is true, calls
the framework.
"""
import math
import random

import torch

own = False

PAGE = 64           # tokens of a cache page: keys [64, d], values [4, d, 16] (16 tokens side by side)
FP8_MAX = 448.0     # largest e4m3 value


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # four beams of each of 16 prompts of ordinary length, some way into their answers
        dict(name="shared 16x4 beams", op="shared", groups=16, size=4, ragged=False, Hq=32, Hkv=8, d=128,
             prefix=4000, own=200, window=0, out="bf16"),
        # eight samples of one very long prompt: latency, and 32-bit results
        dict(name="shared 8 of 50000", op="shared", groups=1, size=8, ragged=False, Hq=32, Hkv=8, d=128,
             prefix=50000, own=100, window=0, out="fp32"),
        # a serving batch behind three system prompts of different use
        dict(name="shared 256 behind 3", op="shared", groups=3, size=85, ragged=True, Hq=32, Hkv=8, d=128,
             prefix=16384, own=1000, window=0, out="bf16"),
        # one step of a small beam search: latency
        dict(name="fork 4 beams", op="fork", groups=1, size=4, Hkv=4, d=64, prefix=1000, own=90, spare=24, held=0,
             dead=0, room=1),
        # a step of 64 searches of 4 beams: most rows copy a page
        dict(name="fork 64x4 beams", op="fork", groups=64, size=4, Hkv=8, d=128, prefix=2000, own=300, spare=700,
             held=50, dead=9, room=1),
        # a cache with holes all over after long use, half of it in use
        dict(name="compact 6000 pages", op="compact", groups=40, size=3, Hkv=8, d=128, prefix=3500, own=700,
             spare=2700, held=30),
        # a small cache that is nearly full: few pages move
        dict(name="compact small", op="compact", groups=3, size=1, Hkv=2, d=64, prefix=700, own=65, spare=5, held=0),
        # four beams of one prompt: latency, odd vocabulary
        dict(name="select 1x4", op="select", G=1, K=4, M=4, V=32001, pad=0, dtype="bf16", ended=0.0, keep=True),
        # 64 searches of 8 beams over a large vocabulary
        dict(name="select 64x8", op="select", G=64, K=8, M=8, V=131072, pad=0, dtype="bf16", ended=0.05, keep=True),
        # 32-bit logits, padded rows, twice as many candidates as beams, as searches with stop rules take
        dict(name="select 16x5 fp32", op="select", G=16, K=5, M=10, V=50001, pad=63, dtype="fp32", ended=0.0, keep=False),
        # the states of a small stack's three layers for one search of five beams, in one tensor
        dict(name="reorder 1x5", op="reorder", G=1, K=5, layers=3, H=6, dk=64, dv=128, moved=0.5),
        # a layer's states of 64 searches of 4 beams
        dict(name="reorder 64x4", op="reorder", G=64, K=4, layers=1, H=32, dk=128, dv=128, moved=0.4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "fork", "compact", "select", "select", "reorder"])
    if op == "shared":
        groups, size = _log(rng, 1, 32), _log(rng, 1, 64)
        Hkv = rng.choice([1, 2, 4, 8])
        case = dict(op=op, groups=groups, size=size, ragged=rng.random() < 0.5, Hq=Hkv * rng.choice([1, 3, 4, 8, 16]),
                    Hkv=Hkv, d=rng.choice([64, 128]), prefix=_log(rng, 1, 50000), own=_log(rng, 1, 1500),
                    window=rng.choice([0, 0, _log(rng, 1, 4096)]), out=rng.choice(["bf16", "fp32"]))
        while work(case)["flops"] > 5e10 or groups * case["prefix"] > 150000:
            case["prefix"], case["own"] = case["prefix"] * 2 // 3 + 1, case["own"] * 2 // 3 + 1
        return case
    if op in ("fork", "compact"):
        groups, size = _log(rng, 1, 64), rng.randint(1, 8)
        case = dict(op=op, groups=groups, size=size, Hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]),
                    prefix=_log(rng, 1, 4000), own=_log(rng, 1, 400), spare=_log(rng, groups * size * 3, 2600),
                    held=rng.choice([0, _log(rng, 1, 100)]))
        return dict(case, dead=rng.choice([0, rng.randint(0, groups * size // 4)]), room=_log(rng, 1, 130)) \
            if op == "fork" else case
    if op == "select":
        G, K = _log(rng, 1, 64), rng.randint(1, 16)
        V = min(_log(rng, 200, 131072), 60000000 // (G * K))
        keep = rng.random() < 0.6
        return dict(op=op, G=G, K=K, M=K if keep else rng.randint(1, min(64, 2 * K)), V=V, pad=rng.choice([0, 0, 17, 64]),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), ended=rng.choice([0.0, 0.2]), keep=keep)
    G, K = _log(rng, 1, 64), rng.randint(1, 12)
    layers, H, dk, dv = rng.choice([1, 1, 3]), rng.choice([2, 8, 16, 32]), rng.choice([64, 128]), rng.choice([64, 128])
    while G * K * layers * H * dk * dv > 130000000:
        G, H = max(1, G * 2 // 3), max(1, H * 2 // 3)
    return dict(op=op, G=G, K=K, layers=layers, H=H, dk=dk, dv=dv, moved=rng.choice([0.2, 0.5, 0.8]))


def _sizes(case):
    """Sequences of each group."""
    n, G = case["size"] * case["groups"], case["groups"]
    if not case.get("ragged"):
        return [case["size"]] * G
    r = random.Random(n * 31 + G)
    weights = [r.uniform(0.2, 3.0) for _ in range(G)]
    got = [max(1, int(n * w / sum(weights))) for w in weights]
    got[-1] += max(0, n - sum(got))
    return got


def _lengths(case):
    """(pages that each group shares, tokens of each sequence group by group)."""
    r = random.Random(case["groups"] * 7919 + case["prefix"])
    pages, lens = [], []
    for g, n in enumerate(_sizes(case)):
        tokens = case["prefix"] if g == 0 else r.randint(max(1, case["prefix"] // 2), case["prefix"])
        pages.append(tokens // PAGE)
        if case["op"] == "shared":
            lens.append([tokens + r.randint(1, case["own"]) for _ in range(n)])
        else:               # the beams of a search are equally long
            lens.append([tokens + r.randint(1, case["own"])] * n)
    return pages, lens


def _pages_of(n):
    return (n + PAGE - 1) // PAGE


def _parents(case):
    """The row that each row continues: a few of a group's beams live on, in their own rows as well."""
    size, G = (case["K"], case["G"]) if "K" in case else (case["size"], case["groups"])
    r = random.Random(size * 1009 + G)
    rows = []
    for g in range(G):
        stay = [r.random() >= case.get("moved", 0.5) for _ in range(size)]
        if not any(stay):
            stay[r.randrange(size)] = True
        alive = [k for k in range(size) if stay[k]]
        rows += [g * size + (k if stay[k] else r.choice(alive)) for k in range(size)]
    for n in r.sample(range(len(rows)), case.get("dead", 0)):
        rows[n] = -1
    return rows


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "shared":
        pages, lens = _lengths(case)
        d, W = case["d"], case["window"] or 1 << 60
        once, seen = 0, 0
        for p, group in zip(pages, lens):
            first = min(max(0, n - W) for n in group)
            once += max(0, p * PAGE - first)
            for n in group:
                seen += min(n, W)
                once += min(n - p * PAGE, W)
        rows = sum(map(len, lens)) * case["Hq"]
        return {"bytes": once * case["Hkv"] * d * 2 + rows * d * (2 + (2 if case["out"] == "bf16" else 4)),
                "flops": 4 * d * case["Hq"] * seen}
    if op in ("fork", "compact"):
        pages, lens = _lengths(case)
        flat = [n for group in lens for n in group]
        page = case["Hkv"] * (2 * PAGE * case["d"] + 8)
        table = len(flat) * 8 * (_pages_of(max(flat)) + 3)
        if op == "fork":
            par = _parents(case)
            live = [p for p in par if p >= 0]
            copies = sum(1 for i, p in enumerate(live) if flat[p] % PAGE and p in live[:i])
            return {"bytes": table + copies * page * 2, "flops": len(flat)}
        used = sum(p + sum(_pages_of(n) - p for n in group) for p, group in zip(pages, lens))
        total = used + case["spare"] + case["held"]
        moved = used * case["spare"] // total         # the free places below the number of pages in use
        return {"bytes": table + moved * page * 2, "flops": used}
    if op == "select":
        rows = case["G"] * case["K"]
        n = rows * case["V"] * (1 - case["ended"])
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + rows * 5 + case["G"] * case["M"] * 13, "flops": 4 * n}
    par = _parents(case)
    moved = [(n, p) for n, p in enumerate(par) if n != p]
    row = case["H"] * case["dk"] * case["dv"] * 4 * case["layers"]
    return {"bytes": (len(moved) + len({p for _, p in moved})) * row + 4 * len(par), "flops": len(par)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _tables(case, seed, wider):
    """(pages of the cache, block table, pages of others) with each group's first pages shared and every
    page at a random place; entries behind a row's last page are -1."""
    pages, lens = _lengths(case)
    flat = [n for group in lens for n in group]
    used = sum(p + sum(_pages_of(n) - p for n in group) for p, group in zip(pages, lens))
    total = used + case.get("spare", 3) + case.get("held", 0)
    order = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(flat), _pages_of(max(flat)) + wider), -1, dtype=torch.int32)
    at = row = 0
    for p, group in zip(pages, lens):
        shared = order[at:at + p]
        at += p
        for n in group:
            mine = _pages_of(n)
            table[row, :p] = shared
            table[row, p:mine] = order[at:at + mine - p]
            at, row = at + mine - p, row + 1
    held = torch.zeros(total, dtype=torch.uint8)
    held[order[at:at + case.get("held", 0)].long()] = 1
    return total, table.cuda(), held.cuda(), flat


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, op = "cuda", case["op"]
    s = {"case": case}
    if op == "select":
        R, V = case["G"] * case["K"], case["V"]
        # (rows of a wider projection where it is padded)
        x = torch.randn((R, V + case["pad"]), generator=g, device=dev) * 2.5
        s["logits"] = x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)[:, :V]
        s["scores"] = (-20 * torch.rand((case["G"], case["K"]), generator=g, device=dev)).sort(-1, descending=True)[0]
        s["ended"] = torch.rand((case["G"], case["K"]), generator=g, device=dev) < case["ended"]
        s["end"] = 2
        return s
    if op == "reorder":
        s["rows"] = torch.tensor(_parents(case), dtype=torch.int32, device=dev)
        s["state"] = torch.randn((case["layers"], case["G"] * case["K"], case["H"], case["dk"], case["dv"]), generator=g, device=dev)
        return s
    total, s["table"], s["held"], lens = _tables(case, seed, 3 if op == "fork" else 0)
    s["len"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    Hkv, d = case["Hkv"], case["d"]

    def cache(shape):
        x = torch.empty(shape, dtype=torch.uint8, device=dev)
        for i in range(0, shape[0], 512):
            part = torch.randn(x[i:i + 512].shape, generator=g, device=dev) * 80.0
            x[i:i + 512] = part.clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        return x

    def scales():
        e = torch.randint(-8, -5, (total, Hkv), generator=g, device=dev)
        return ((e.to(torch.int32) + 127) << 23).view(torch.float32)

    s["k"], s["v"] = cache((total, Hkv, PAGE, d)), cache((total, Hkv, PAGE // 16, d, 16))
    s["k_scale"], s["v_scale"] = scales(), scales()
    if op == "shared":
        ends = [0]
        for n in _sizes(case):
            ends.append(ends[-1] + n)
        s["groups"] = torch.tensor(ends, dtype=torch.int32, device=dev)
        s["pages"] = torch.tensor(_lengths(case)[0], dtype=torch.int32, device=dev)
        s["q"] = torch.randn((len(lens), case["Hq"], d), generator=g, device=dev).to(torch.bfloat16)
    if op == "fork":
        s["rows"] = torch.tensor(_parents(case), dtype=torch.int32, device=dev)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------


def _gathered(s, t):
    """Keys and values [H, tokens, d] in 32 bits of the pages t."""
    k = s["k"][t].view(torch.float8_e4m3fn).float() * s["k_scale"][t][..., None, None]
    v = s["v"][t].view(torch.float8_e4m3fn).float() * s["v_scale"][t][..., None, None, None]
    return k.transpose(0, 1).flatten(1, 2), v.permute(1, 0, 2, 4, 3).flatten(1, 3)


def _plain_shared(s):
    """Group by group, the shared pages' scores as one product, each sequence's own behind them."""
    c = s["case"]
    Hkv, d, G = c["Hkv"], c["d"], c["Hq"] // c["Hkv"]
    pages, lens = _lengths(c)
    by, rows, row = 1 / math.sqrt(d), [], 0
    for p, group in zip(pages, lens):
        n, t = len(group), s["table"][row:row + len(group)].long()
        q = s["q"][row:row + n].float().view(n, Hkv, G, d).permute(1, 0, 2, 3).contiguous()      # [H, n, G, d]
        L = s["len"][row:row + n].long()[None, :, None, None]
        k, v = _gathered(s, t[0, :p])
        a = torch.matmul(q.flatten(1, 2), k.transpose(1, 2).contiguous()).view(Hkv, n, G, p * PAGE)
        own = t[:, p:_pages_of(max(group))].clamp_min(0)
        w = own.shape[1]
        ko, vo = _gathered(s, own.flatten())
        ko, vo = (x.view(Hkv, n, w * PAGE, d) for x in (ko, vo))
        b = torch.matmul(q, ko.transpose(2, 3).contiguous())
        x = torch.cat((a, b), -1).mul_(by)
        j = torch.arange(x.shape[-1], device=x.device)
        hidden = j >= L
        if c["window"]:
            hidden = hidden | (j < L - c["window"])
        x.masked_fill_(hidden, -math.inf)
        x = x.sub_(x.amax(-1, keepdim=True)).exp_()
        total = x.sum(-1, keepdim=True)
        o = torch.matmul(x[..., :p * PAGE].flatten(1, 2), v).view(Hkv, n, G, d) + torch.matmul(x[..., p * PAGE:], vo)
        rows.append((o / total).permute(1, 0, 2, 3).reshape(n, c["Hq"], d))
        row += n
    return torch.cat(rows).to(torch.bfloat16 if c["out"] == "bf16" else torch.float32)


def _cache_outputs(s):
    """The cache's values beside their scales."""
    return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_fork(s):
    c, P = s["case"], s["k"].shape[0]
    N, width = s["rows"].numel(), s["table"].shape[1]
    dev = s["table"].device
    parent = s["rows"].long()
    ok = (parent >= 0) & (parent < s["table"].shape[0])
    at = parent.clamp(0, s["table"].shape[0] - 1)
    n = torch.where(ok, s["len"].long()[at], 0)
    col = torch.arange(width, device=dev)[None]
    table = torch.where(col < ((n + PAGE - 1) // PAGE)[:, None], s["table"][at].long(), -1)
    named = torch.where(table >= 0, table, P).flatten()
    uses = torch.zeros(P + 1, dtype=torch.long, device=dev).index_add_(0, named, torch.ones_like(named))
    free = (uses[:P] == 0) & (s["held"] == 0)
    rank = torch.where(free, free.cumsum(0) - 1, P)
    lowest = torch.full((P + 1,), -1, dtype=torch.long, device=dev).scatter_(0, rank, torch.arange(P, device=dev))
    # a page that a row goes on writing: its copy, unless the row is the lowest of those that name it
    part = ok & (n % PAGE != 0)
    row = torch.arange(N, device=dev)
    last = torch.where(part, table.gather(1, (n // PAGE).clamp_max(width - 1)[:, None])[:, 0], P)
    writers = torch.zeros(P + 1, dtype=torch.long, device=dev).index_add_(0, last, torch.ones_like(last))
    first = torch.full((P + 1,), N, dtype=torch.long, device=dev).scatter_reduce_(0, last, row, "amin")
    held = torch.cat((s["held"], s["held"].new_zeros(1)))
    keeps = (uses[last] == writers[last]) & (first[last] == row) & (held[last] == 0)
    copy = part & ~keeps
    begin = (n + PAGE - 1) // PAGE
    fresh = torch.where(ok, ((n + c["room"] + PAGE - 1) // PAGE).clamp_max(width) - begin, 0)
    want = copy.long() + fresh
    offset = want.cumsum(0) - want
    # entry by entry: the place in the list of wanted pages
    number = torch.where(col == (n // PAGE)[:, None], torch.where(copy[:, None], offset[:, None], P), P)
    new = (col >= begin[:, None]) & (col < (begin + fresh)[:, None])
    number = torch.where(new, offset[:, None] + copy[:, None] + col - begin[:, None], number)
    got = lowest[number.clamp_max(P)]
    got = torch.where(number < P, got, -1)
    done = (copy & (got.gather(1, (n // PAGE).clamp_max(width - 1)[:, None])[:, 0] >= 0)).nonzero()[:, 0]
    source, place = table[done, (n // PAGE)[done]], got[done, (n // PAGE)[done]]
    for x in ("k", "v", "k_scale", "v_scale"):
        s[x][place] = s[x][source]
    table = torch.where(got >= 0, got, table)
    missing = torch.minimum(want, (offset + want - free.sum()).clamp_min(0))
    return dict(_cache_outputs(s), table=table.to(torch.int32), len=n.to(torch.int32), missing=missing.to(torch.int32))


def _plain_compact(s):
    P, dev = s["k"].shape[0], s["table"].device
    n = s["len"].long()
    col = torch.arange(s["table"].shape[1], device=dev)[None]
    table = torch.where(col < ((n + PAGE - 1) // PAGE)[:, None], s["table"].long(), -1)
    used = torch.zeros(P + 1, dtype=torch.bool, device=dev)
    used[torch.where(table >= 0, table, P).flatten()] = True
    used = used[:P]
    free = (~used & (s["held"] == 0)).nonzero()[:, 0]
    high = (used & (s["held"] == 0)).nonzero()[:, 0].flip(0)
    m = min(free.numel(), high.numel())
    move = free[:m] < high[:m]
    to, source = free[:m][move], high[:m][move]
    for x in ("k", "v", "k_scale", "v_scale"):
        s[x][to] = s[x][source]
    to_of = torch.arange(P, device=dev)
    to_of[source] = to
    table = torch.where(table >= 0, to_of[table.clamp_min(0)], -1)
    in_use = torch.where(s["held"] != 0, torch.arange(1, P + 1, device=dev), 0).amax()
    return dict(_cache_outputs(s), table=table.to(torch.int32), used=torch.maximum(in_use, table.amax() + 1).to(torch.int32)[None])


def _plain_select(s):
    c = s["case"]
    G, K, M, V = c["G"], c["K"], c["M"], c["V"]
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    lse = ((x - top).exp_().sum(-1, keepdim=True).log_() + top)[:, 0]
    base, ended = s["scores"].double().view(-1), s["ended"].view(-1)
    none = ~torch.isfinite(base) | (~ended & ~torch.isfinite(lse))
    # the best M of each row: the logit's bits as a whole number that orders alike, then the lowest token
    t = torch.arange(V, device=x.device)
    bits = (s["logits"].float() + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, bits ^ 0x7fffffff, bits)
    key = torch.where(ended[:, None], (t == s["end"]).long(), key)
    key = torch.where(none[:, None], 0, key) * (1 << 32) + (V - t)
    m = min(M, V)
    tok = key.topk(m, -1)[1]
    score = base[:, None] + x.gather(1, tok) - lse[:, None]
    score = torch.where(ended[:, None], torch.where(tok == s["end"], base[:, None], -math.inf), score)
    score = torch.where(none[:, None], -math.inf, score).view(G, K * m)
    score, at = (y[:, :M] for y in score.sort(dim=-1, descending=True, stable=True))
    tok, beam = tok.view(G, K * m).gather(1, at), at // m
    if c["keep"]:
        # the first taken continuation of a beam in the beam's own row, the others in the rows left
        i = torch.arange(M, device=x.device)
        again = ((beam[:, :, None] == beam[:, None, :]) & (i[None, :] < i[:, None])[None]).any(-1)
        left = ~(beam[:, :, None] == i).any(1)
        slots = torch.where(left, i, K + i).sort(-1)[0]
        slot = torch.where(again, slots.gather(1, (again.long().cumsum(-1) - 1).clamp_min(0)), beam)
        tok, beam, score = (torch.empty_like(y).scatter_(1, slot, y) for y in (tok, beam, score))
    done = s["ended"].gather(1, beam) | (tok == s["end"])
    rows = beam + K * torch.arange(G, device=x.device)[:, None]
    return tok.to(torch.int32), rows.to(torch.int32), score.float(), done


def _plain_reorder(s):
    s["state"].copy_(s["state"][:, s["rows"].long()])
    return s["state"]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(state):
    case, s = state["case"], state
    op = case["op"]
    if own:
        import gated_delta_rule_24_amd as gdr
        gen = gdr.generation
        if op == "select":
            return gen.beam_select(s["logits"], s["scores"], case["M"], ended=s["ended"], end_token=s["end"],
                                   keep_slots=case["keep"])
        if op == "reorder":
            return gen.state_reorder(s["state"], s["rows"], case["K"], dim=1)
        cache = gdr.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if op == "shared":
            return gen.attn_decode_shared(s["q"], cache, s["table"], s["len"], s["groups"], s["pages"],
                                          window=case["window"],
                                          out_dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
        if op == "fork":
            table, length, missing = gen.kv_fork(cache, s["table"], s["len"], s["rows"], room=case["room"], held=s["held"])
            return dict(_cache_outputs(s), table=table, len=length, missing=missing)
        table, used = gen.kv_compact(cache, s["table"], s["len"], held=s["held"])
        return dict(_cache_outputs(s), table=table, used=used)
    return {"shared": _plain_shared, "fork": _plain_fork, "compact": _plain_compact, "select": _plain_select,
            "reorder": _plain_reorder}[op](s)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _exact_shared(s):
    """Each sequence for itself, over its own row of the table."""
    c, rows = s["case"], []
    kc, vc = s["k"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn)
    for i, n in enumerate(s["len"].tolist()):
        begin = max(0, n - c["window"]) if c["window"] else 0
        t = s["table"][i, begin // PAGE:_pages_of(n)].long()
        a, b = begin % PAGE, n - begin // PAGE * PAGE
        k = (kc[t].double() * s["k_scale"][t].double()[..., None, None]).transpose(0, 1).flatten(1, 2)[:, a:b]
        v = (vc[t].double() * s["v_scale"][t].double()[..., None, None, None]).permute(1, 0, 2, 4, 3).flatten(1, 3)[:, a:b]
        q = s["q"][i].double().view(c["Hkv"], -1, c["d"])
        p = torch.softmax(torch.bmm(q, k.transpose(1, 2).contiguous()) * c["d"] ** -0.5, -1)
        rows.append(torch.bmm(p, v.contiguous()).reshape(c["Hq"], c["d"]))
    return torch.stack(rows)


def _cache_values(s, moves):
    """The cache's values after pages (source, place) were copied, all at once."""
    out = {}
    to = torch.tensor([b for _, b in moves], dtype=torch.long, device="cuda")
    of = torch.tensor([a for a, _ in moves], dtype=torch.long, device="cuda")
    for x in ("k", "v", "k_scale", "v_scale"):
        y = s[x].view(torch.float8_e4m3fn).double() if x in "kv" else s[x].double()
        out[x] = y.index_copy(0, to, y[of])
    return out


def _exact_fork(s):
    """Row by row, as a program on the host would deal out the pages."""
    c, P = s["case"], s["k"].shape[0]
    table, lens, held = s["table"].tolist(), s["len"].tolist(), s["held"].tolist()
    width, out, n, parent = len(table[0]), [], [], s["rows"].tolist()
    for p in parent:
        n.append(lens[p] if p >= 0 else 0)
        out.append((table[p] if p >= 0 else [])[:_pages_of(n[-1])])
    names, writers = {}, {}
    for i, row in enumerate(out):
        for page in row:
            names.setdefault(page, []).append(i)
        if n[i] % PAGE:
            writers.setdefault(row[-1], []).append(i)
    free = iter([page for page in range(P) if page not in names and not held[page]])
    moves, missing = [], []
    for i, row in enumerate(out):
        lacks = 0
        if parent[i] >= 0:
            if n[i] % PAGE:
                page = row[-1]
                if held[page] or writers[page] != names[page] or names[page][0] != i:
                    to = next(free, None)
                    lacks += to is None
                    if to is not None:
                        moves.append((page, to))
                        row = row[:-1] + [to]
            while len(row) < min(width, _pages_of(n[i] + c["room"])):
                to = next(free, None)
                lacks += to is None
                row = row + [-1 if to is None else to]
        out[i] = row
        missing.append(lacks)
    out = [row + [-1] * (width - len(row)) for row in out]
    return dict(_cache_values(s, moves), table=torch.tensor(out), len=torch.tensor(n), missing=torch.tensor(missing))


def _exact_compact(s):
    P, held = s["k"].shape[0], s["held"].tolist()
    rows = [row[:_pages_of(n)] for row, n in zip(s["table"].tolist(), s["len"].tolist())]
    used = {page for row in rows for page in row}
    to, low, high = {}, 0, P - 1
    while True:
        while low < P and (low in used or held[low]):
            low += 1
        while high >= 0 and (high not in used or held[high]):
            high -= 1
        if low >= high:
            break
        to[high] = low
        low, high = low + 1, high - 1
    rows = [[to.get(page, page) for page in row] for row in rows]
    width = s["table"].shape[1]
    most = max([page + 1 for row in rows for page in row] + [page + 1 for page in range(P) if held[page]])
    return dict(_cache_values(s, list(to.items())), table=torch.tensor([row + [-1] * (width - len(row)) for row in rows]),
                used=torch.tensor([most]))


def _exact_select(s):
    """Group by group, all candidates sorted; the tokens and rows follow from the order."""
    c = s["case"]
    K, M, V = c["K"], c["M"], c["V"]
    tokens, rows, scores, ended = [], [], [], []
    for g in range(c["G"]):
        x = torch.log_softmax(s["logits"][g * K:(g + 1) * K].double(), -1)
        x[s["ended"][g]] = -math.inf
        x[s["ended"][g], s["end"]] = 0.0
        x += s["scores"][g].double()[:, None]
        value, at = x.flatten().sort(dim=-1, descending=True, stable=True)
        took = [(float(v), int(i) // V, int(i) % V) for v, i in zip(value[:M], at[:M])]
        if c["keep"]:
            place, rest = [None] * M, []
            for one in took:
                if place[one[1]] is None:
                    place[one[1]] = one
                else:
                    rest.append(one)
            took = [one if one is not None else rest.pop(0) for one in place]
        tokens.append([t for _, _, t in took])
        rows.append([g * K + k for _, k, _ in took])
        scores.append([v for v, _, _ in took])
        ended.append([bool(s["ended"][g, k]) or t == s["end"] for _, k, t in took])
    return torch.tensor(tokens), torch.tensor(rows), torch.tensor(scores, dtype=torch.float64), torch.tensor(ended)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "reorder":
        return torch.stack([s["state"][:, n].double() for n in s["rows"].tolist()], 1)
    return {"shared": _exact_shared, "fork": _exact_fork, "compact": _exact_compact, "select": _exact_select}[case["op"]](s)
