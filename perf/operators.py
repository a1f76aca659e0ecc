"""The attention layer of a hybrid gated-delta-rule stack, operator by operator: the cases that are
timed, the operators' plain forms and their values in 64 bits.

A hybrid stack alternates recurrent layers with causal attention layers (a 2,048-token window, or
the whole past).  The operators here are what such a layer needs next to the recurrence:

* ``rope``        rotary positions of queries and keys, and their inverse (the gradient);
* ``attn_fwd``    causal attention over a window or the whole past, shared key heads, packed documents;
* ``attn_bwd``    its gradients, the probabilities recomputed from the saved log-sum-exp;
* ``kv_append``   keys and values into a paged 8-bit cache, one power-of-two scale per page and head;
* ``attn_decode`` one query token per sequence over that cache.

``run`` computes the plain forms with elementary torch operations in 32 bits, or, where ``own`` is
true, calls the framework.
"""
import math
import random

import torch

own = False

PAGE = 64           # tokens of a cache page: keys [64, d], values [4, d, 16] (16 tokens side by side)
FP8_MAX = 448.0     # largest e4m3 value
SCALE_MIN = 2.0 ** -96


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one token of each of 64 running sequences, far into their contexts: latency
        dict(name="rope 64 tokens", op="rope", B=64, Hq=16, Hk=4, T=1, d=128, rot=64, dtype="bf16",
             interleaved=True, inverse=False, token_major=False, far=200000, scale=1.0),
        # a training batch's queries and keys
        dict(name="rope 2x16x8192", op="rope", B=2, Hq=16, Hk=16, T=8192, d=128, rot=128, dtype="bf16",
             interleaved=False, inverse=False, token_major=False, far=0, scale=1.0),
        # the gradient of a long sequence in 32 bits, projections' layout, scaled frequencies
        dict(name="rope inverse fp32", op="rope", B=1, Hq=32, Hk=8, T=4099, d=64, rot=32, dtype="fp32",
             interleaved=False, inverse=True, token_major=True, far=30000, scale=1.1),
        # a short prompt, odd length, shared key heads: latency
        dict(name="attn fwd 257", op="attn_fwd", B=1, Hq=16, Hkv=4, Tq=257, Tk=257, d=64, window=0,
             docs=0, token_major=False),
        # the hybrid stack's windowed layer on a training batch
        dict(name="attn fwd window", op="attn_fwd", B=2, Hq=16, Hkv=16, Tq=8192, Tk=8192, d=128,
             window=2048, docs=0, token_major=False),
        # 19 packed documents, whole past, shared key heads, projections' layout
        dict(name="attn fwd packed", op="attn_fwd", B=1, Hq=16, Hkv=4, Tq=16384, Tk=16384, d=128,
             window=0, docs=19, token_major=True),
        # a small training call, odd length, whole past, shared key heads
        dict(name="attn bwd 2047", op="attn_bwd", B=1, Hq=16, Hkv=4, Tq=2047, Tk=2047, d=128, window=0,
             docs=0, token_major=False),
        # the windowed layer's gradients on a training batch
        dict(name="attn bwd window", op="attn_bwd", B=2, Hq=16, Hkv=16, Tq=8192, Tk=8192, d=128,
             window=2048, docs=0, token_major=False),
        # one new token of 256 running sequences into their last pages
        dict(name="append 256 tokens", op="kv_append", nseq=256, Hkv=8, d=128, T=0, have=500),
        # 19 prompts of 16,384 tokens together, some behind tokens that are cached already
        dict(name="append 19 prompts", op="kv_append", nseq=19, Hkv=8, d=128, T=16384, have=500),
        # one sequence with a long context: latency
        dict(name="decode 1x50000", op="attn_decode", nseq=1, Hq=32, Hkv=8, d=128, longest=50000,
             window=0, out="fp32"),
        # a full serving batch of ragged lengths
        dict(name="decode 256 ragged", op="attn_decode", nseq=256, Hq=32, Hkv=8, d=128, longest=8192,
             window=0, out="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "kv_append", "attn_decode",
                     "attn_decode"])
    if op == "rope":
        d = rng.choice([32, 64, 128])
        Hk = rng.choice([1, 2, 4, 8, 16])
        Hq = Hk * rng.choice([1, 2, 4])
        B = rng.choice([1, 2, 3, 64])
        T = _log(rng, 1, max(1, 33000000 // (B * (Hq + Hk) * d)))
        return dict(op=op, B=B, Hq=Hq, Hk=Hk, T=min(T, 16384), d=d, rot=rng.choice([16, 32, d]),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.5, token_major=rng.random() < 0.5, far=_log(rng, 1, 1000000),
                    scale=rng.choice([1.0, 1.2]))
    if op in ("attn_fwd", "attn_bwd"):
        d = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8, 16])
        Hq = Hkv * rng.choice([1, 2, 4, 8]) if Hkv < 8 else Hkv * rng.choice([1, 2])
        T = _log(rng, 1, 8192)
        docs = rng.choice([0, 0, rng.randint(1, 24)])
        Tk = T if docs or rng.random() < 0.7 else T + _log(rng, 1, 1024)
        B = 1 if docs else rng.randint(1, 3)
        case = dict(op=op, B=B, Hq=Hq, Hkv=Hkv, Tq=T, Tk=Tk, d=d,
                    window=rng.choice([0, 0, _log(rng, 1, 4096)]), docs=docs, token_major=rng.random() < 0.5)
        # no more work than the largest listed case, and room for the plain forms' score matrices
        while work(case)["flops"] > 6e11 or case["B"] * Hq * case["Tq"] * case["Tk"] > 2 ** 31:
            case["Tq"], case["Tk"] = case["Tq"] * 2 // 3 + 1, case["Tk"] * 2 // 3 + 1
        return case
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "kv_append":
        nseq = _log(rng, 1, 256)
        return dict(op=op, nseq=nseq, Hkv=Hkv, d=d, T=rng.choice([0, _log(rng, nseq, 16384)]),
                    have=_log(rng, 1, 1000))
    nseq = _log(rng, 1, 256)
    longest = _log(rng, 1, min(100000, 1000000 // nseq))
    return dict(op=op, nseq=nseq, Hq=Hkv * rng.choice([1, 3, 4, 8, 16]), Hkv=Hkv, d=d, longest=longest,
                window=rng.choice([0, 0, _log(rng, 1, 4096)]), out=rng.choice(["bf16", "fp32"]))


def _split(total, n, mix):
    """`total` tokens as `n` ragged lengths (some may be zero), the same for every seed."""
    r = random.Random(mix)
    cuts = sorted(r.randint(0, total) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _lengths(case):
    """Cached tokens of each sequence (decode: the new token among them)."""
    r = random.Random(case["nseq"] * 7919 + 17)
    if case["op"] == "kv_append":
        return [r.randint(0, case["have"]) for _ in range(case["nseq"])]
    top = case["longest"]
    return [top] + [r.randint(max(1, top // 4), top) for _ in range(case["nseq"] - 1)]


def _doc_lengths(case):
    return _split(case["Tq"], case["docs"], case["docs"] * 131 + case["Tq"])


def _new_lengths(case):
    return _split(case["T"], case["nseq"], case["nseq"] + case["T"]) if case["T"] else [1] * case["nseq"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------


def _pairs_of(Tq, Tk, window):
    """Query-key pairs of one head: query i stands at i + Tk - Tq and sees the last `window` keys up to it."""
    full = window if window else 1 << 60
    first, last = Tk - Tq + 1, Tk                      # keys up to each row's position, before the window
    first = max(first, 1)
    if last < first:
        return 0
    cut = min(max(full, first - 1), last)              # rows below the cut see all, the others `full`
    return (first + cut) * (cut - first + 1) // 2 + (last - cut) * min(full, last)


def work(case):
    op, d = case["op"], case["d"]
    if op == "rope":
        n = case["B"] * case["T"] * (case["Hq"] + case["Hk"])
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * d * size + case["B"] * case["T"] * 4, "flops": n * case["rot"] * 3}
    if op in ("attn_fwd", "attn_bwd"):
        B, Hq, Hkv, Tq, Tk = (case[x] for x in ("B", "Hq", "Hkv", "Tq", "Tk"))
        if case["docs"]:
            pairs = sum(_pairs_of(n, n, case["window"]) for n in _doc_lengths(case))
        else:
            pairs = B * _pairs_of(Tq, Tk, case["window"])
        rows, keys = B * Hq * Tq, B * Hkv * Tk
        if op == "attn_fwd":
            return {"bytes": 2 * d * (2 * rows + 2 * keys) + 4 * rows, "flops": 4 * d * Hq * pairs}
        return {"bytes": 2 * d * (4 * rows + 4 * keys) + 4 * rows, "flops": 10 * d * Hq * pairs}
    if op == "kv_append":
        n = sum(_new_lengths(case)) * case["Hkv"] * d
        return {"bytes": 2 * n * 2 + 2 * n, "flops": 4 * n}
    seen = sum(min(n, case["window"]) if case["window"] else n for n in _lengths(case))
    size = 2 if case["out"] == "bf16" else 4
    return {"bytes": seen * case["Hkv"] * d * 2 + case["nseq"] * case["Hq"] * d * (2 + size),
            "flops": 4 * d * case["Hq"] * seen}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _shape(case, H, T):
    """[B, H, T, d], packed documents without the batch; projections' layout: tokens before heads."""
    s = (T, H, case["d"]) if case["token_major"] else (H, T, case["d"])
    return s if case.get("docs") else (case["B"],) + s


def _tables(case, g, lens):
    """Shuffled pages, each sequence's in its own row of the block table."""
    need = [(n + PAGE - 1) // PAGE for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    width = max(max(need), 1)
    table = torch.zeros((len(lens), width), dtype=torch.int32, device="cuda")
    row = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(need))
    col = torch.cat([torch.arange(n) for n in need]) if sum(need) else torch.zeros(0, dtype=torch.long)
    table[row.cuda(), col.cuda()] = order[:sum(need)]
    return pages, table


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, d, dev = case["op"], case["d"], "cuda"

    def normal(shape, dtype=torch.bfloat16, by=1.0):
        return (torch.randn(shape, generator=g, device=dev) * by).to(dtype)

    s = {"case": case}
    if op == "rope":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["q"] = normal(_shape(case, case["Hq"], case["T"]), dt)
        s["k"] = normal(_shape(case, case["Hk"], case["T"]), dt)
        i = torch.arange(case["rot"] // 2, dtype=torch.float64, device=dev)
        s["inv_freq"] = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=dev), -2 * i / case["rot"]).float()
        first = torch.randint(0, case["far"] + 1, (case["B"], 1), generator=g, device=dev)
        s["positions"] = (first + torch.arange(case["T"], device=dev)).to(torch.int32)
        return s
    if op in ("attn_fwd", "attn_bwd"):
        s["q"] = normal(_shape(case, case["Hq"], case["Tq"]))
        s["k"] = normal(_shape(case, case["Hkv"], case["Tk"]))
        s["v"] = normal(_shape(case, case["Hkv"], case["Tk"]))
        if case["docs"]:
            ends = [0]
            for n in _doc_lengths(case):
                ends.append(ends[-1] + n)
            s["cu"] = torch.tensor(ends, dtype=torch.int32, device=dev)
        if op == "attn_bwd":
            s["dO"] = normal(_shape(case, case["Hq"], case["Tq"]))
            s["o"], s["lse"] = _plain_attn(s)     # the forward's results, kept for the backward
        return s
    lens = _lengths(case)
    if op == "kv_append":
        new = _new_lengths(case)
        pages, s["table"] = _tables(case, g, [a + b for a, b in zip(lens, new)])
        T = sum(new)
        s["k"] = normal((case["nseq"], case["Hkv"], d) if not case["T"] else (case["Hkv"], T, d))
        s["v"] = normal((case["nseq"], case["Hkv"], d) if not case["T"] else (case["Hkv"], T, d), by=0.7)
        if case["T"]:
            ends = [0]
            for n in new:
                ends.append(ends[-1] + n)
            s["cu"] = torch.tensor(ends, dtype=torch.int32, device=dev)
    else:
        pages, s["table"] = _tables(case, g, lens)
        s["q"] = normal((case["nseq"], case["Hq"], d))
    s["len"] = torch.tensor(lens, dtype=torch.int32, device=dev)

    def cache(shape):
        x = torch.randn(shape, generator=g, device=dev) * 80.0
        return x.clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)

    def scales():
        e = torch.randint(-8, -5, (pages, case["Hkv"]), generator=g, device=dev)
        return _pow2(e)

    s["k_cache"], s["v_cache"] = cache((pages, case["Hkv"], PAGE, d)), cache((pages, case["Hkv"], PAGE // 16, d, 16))
    s["k_scale"], s["v_scale"] = scales(), scales()
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------


def _plain_rope(s):
    case = s["case"]
    half = case["rot"] // 2
    turn = s["positions"].double()[..., None] * s["inv_freq"].double()
    cos, sin = turn.cos().float() * case["scale"], turn.sin().float() * case["scale"]
    sin = -sin if case["inverse"] else sin
    cos, sin = (x[:, :, None, :] if case["token_major"] else x[:, None, :, :] for x in (cos, sin))

    def turned(x):
        y = x.float()
        r = y[..., :case["rot"]]
        if case["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = r[..., :half], r[..., half:]
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((r, y[..., case["rot"]:]), -1).to(x.dtype)

    return turned(s["q"]), turned(s["k"])


def _heads_first(case, x):
    """[B, H, T, d] in 32 bits."""
    x = x.float()[None] if case["docs"] else x.float()
    return x.transpose(1, 2).contiguous() if case["token_major"] else x


def _as_given(case, x):
    x = x.to(torch.bfloat16)
    x = x.transpose(1, 2).contiguous() if case["token_major"] else x
    return x[0] if case["docs"] else x


def _hidden(s):
    """True where a query does not see a key."""
    case = s["case"]
    i = torch.arange(case["Tq"], device="cuda")[:, None] + (case["Tk"] - case["Tq"])
    j = torch.arange(case["Tk"], device="cuda")[None, :]
    m = j > i
    if case["window"]:
        m |= j <= i - case["window"]
    if case["docs"]:
        doc = torch.searchsorted(s["cu"], torch.arange(case["Tk"], device="cuda", dtype=torch.int32), right=True)
        m |= doc[:, None] != doc[None, :]
    return m


def _plain_probabilities(s, q, k):
    """The rows' probabilities [B, H, Tq, Tk] and log-sum-exps; a row that sees nothing has zeros and -inf."""
    case = s["case"]
    x = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(1 / math.sqrt(case["d"]))
    x.masked_fill_(_hidden(s), -math.inf)
    top = x.amax(-1, keepdim=True)
    at = top.masked_fill(top == -math.inf, 0.0)
    x = x.sub_(at).exp_()
    total = x.sum(-1, keepdim=True)
    lse = (at + total.log())[..., 0]
    return x.div_(total.masked_fill(total == 0, 1.0)), lse


def _plain_attn(s):
    case = s["case"]
    G = case["Hq"] // case["Hkv"]
    q, k, v = (_heads_first(case, s[x]) for x in "qkv")
    P, lse = _plain_probabilities(s, q, k.repeat_interleave(G, 1))
    o = torch.matmul(P, v.repeat_interleave(G, 1))
    return _as_given(case, o), lse[0] if case["docs"] else lse


def _plain_attn_bwd(s):
    case = s["case"]
    G, by = case["Hq"] // case["Hkv"], 1 / math.sqrt(case["d"])
    q, k, v, dO = (_heads_first(case, s[x]) for x in ("q", "k", "v", "dO"))
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    P, _ = _plain_probabilities(s, q, k)

    def shared(x):      # the sum over the queries' heads that share a key head
        return x.unflatten(1, (case["Hkv"], G)).sum(2)

    dv = shared(torch.matmul(P.transpose(-1, -2).contiguous(), dO))
    dS = torch.matmul(dO, v.transpose(-1, -2).contiguous())
    dS.sub_((P * dS).sum(-1, keepdim=True)).mul_(P).mul_(by)
    dq = torch.matmul(dS, k)
    dk = shared(torch.matmul(dS.transpose(-1, -2).contiguous(), q))
    return {"dq": _as_given(case, dq), "dk": _as_given(case, dk), "dv": _as_given(case, dv)}


def _pow2(e):
    """2^e as a 32-bit float, by its exponent field (-126 <= e <= 127)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _pow2_scale(top):
    """The smallest power of two s >= SCALE_MIN with top <= 448 s, exactly (top = m 2^e, 0.5 <= m < 1)."""
    m, e = torch.frexp(top)
    e = torch.where(m > FP8_MAX / 512, e - 8, e - 9).clamp_min(-96)
    return _pow2(torch.where(top > 0, e, torch.full_like(e, -96)))


def _plain_append_one(cache, scale, x, place, page_of, slot, first, transposed):
    """New tokens x [T, H, d] into the pages `place` [U]; token t goes to touched page page_of[t] at slot[t]."""
    T, H, d = x.shape
    U = place.numel()
    x = x.float()
    top = torch.zeros((U, H), device=x.device).index_reduce_(0, page_of, x.abs().amax(-1), "amax")
    old = torch.where((first > 0)[:, None], scale[place], torch.zeros_like(top))
    s = torch.maximum(old, _pow2_scale(top))
    kept = cache[place].view(torch.float8_e4m3fn).float()
    kept = kept.transpose(3, 4).flatten(2, 3) if transposed else kept         # [U, H, 64, d]
    again = (kept * (old / s)[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    was = kept.to(torch.float8_e4m3fn).view(torch.uint8)
    before = torch.arange(PAGE, device=x.device)[None, :] < first[:, None]
    page = torch.where(before[:, None, :, None], again, was)
    page[page_of, :, slot] = (x / s[page_of][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    cache[place] = page.unflatten(2, (PAGE // 16, 16)).transpose(3, 4).contiguous() if transposed else page
    scale[place] = s


def _plain_append(s):
    case = s["case"]
    if case["T"]:
        t = torch.arange(case["T"], device="cuda", dtype=torch.int32)
        seq = torch.searchsorted(s["cu"], t, right=True) - 1
        at = s["len"][seq].long() + (t - s["cu"][seq]).long()
        k, v = s["k"].transpose(0, 1), s["v"].transpose(0, 1)
    else:
        seq = torch.arange(case["nseq"], device="cuda")
        at, k, v = s["len"].long(), s["k"], s["v"]
    width = s["table"].shape[1]
    touched, page_of = torch.unique(seq * width + at // PAGE, return_inverse=True)
    place = s["table"].flatten()[touched].long()
    slot = at % PAGE
    first = torch.full((touched.numel(),), PAGE, device="cuda").scatter_reduce(0, page_of, slot, "amin")
    _plain_append_one(s["k_cache"], s["k_scale"], k, place, page_of, slot, first, False)
    _plain_append_one(s["v_cache"], s["v_scale"], v, place, page_of, slot, first, True)


def _cache_outputs(s):
    """The cache's values beside their scales."""
    return {"k": s["k_cache"].view(torch.float8_e4m3fn), "v": s["v_cache"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_decode(s):
    case = s["case"]
    N, Hkv, d = case["nseq"], case["Hkv"], case["d"]
    G, t = case["Hq"] // Hkv, s["table"].long()
    k = s["k_cache"].view(torch.float8_e4m3fn)[t].float() * s["k_scale"][t][..., None, None]   # [N, P, H, 64, d]
    v = s["v_cache"].view(torch.float8_e4m3fn)[t].float() * s["v_scale"][t][..., None, None, None]
    k = k.permute(0, 2, 4, 1, 3).flatten(3).contiguous()                                       # [N, H, d, P 64]
    v = v.permute(0, 2, 1, 3, 5, 4).flatten(2, 4).contiguous()                                 # [N, H, P 64, d]
    x = torch.matmul(s["q"].float().view(N, Hkv, G, d), k).mul_(1 / math.sqrt(d))
    j = torch.arange(x.shape[-1], device="cuda")[None, :]
    n = s["len"].long()[:, None]
    hidden = j >= n
    if case["window"]:
        hidden |= j < n - case["window"]
    x.masked_fill_(hidden[:, None, None, :], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(x, v) / x.sum(-1, keepdim=True)
    return o.reshape(N, case["Hq"], d).to(torch.bfloat16 if case["out"] == "bf16" else torch.float32)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(state):
    case, s = state["case"], state
    op = case["op"]
    if own:
        import gated_delta_rule_24_amd as gdr
        if op == "rope":
            return gdr.rope(s["q"], s["k"], s["inv_freq"], s["positions"], interleaved=case["interleaved"],
                            inverse=case["inverse"], scale=case["scale"], token_major=case["token_major"])
        if op == "attn_fwd":
            if case["docs"]:
                return gdr.attn_fwd_varlen(s["q"], s["k"], s["v"], s["cu"], window=case["window"],
                                           token_major=case["token_major"])
            return gdr.attn_fwd(s["q"], s["k"], s["v"], window=case["window"], token_major=case["token_major"])
        if op == "attn_bwd":
            if case["docs"]:
                return gdr.attn_bwd_varlen(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dO"], s["cu"],
                                           window=case["window"], token_major=case["token_major"])
            return gdr.attn_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dO"], window=case["window"],
                                token_major=case["token_major"])
        cache = gdr.KVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        if op == "kv_append":
            gdr.kv_append(s["k"], s["v"], cache, s["table"], s["len"], s.get("cu"))
            return _cache_outputs(s)
        return gdr.attn_decode(s["q"], cache, s["table"], s["len"], window=case["window"],
                               out_dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    if op == "rope":
        return _plain_rope(s)
    if op == "attn_fwd":
        return _plain_attn(s)
    if op == "attn_bwd":
        return _plain_attn_bwd(s)
    if op == "kv_append":
        _plain_append(s)
        return _cache_outputs(s)
    return _plain_decode(s)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _exact_rope(s):
    c = s["case"]
    w = torch.exp(1j * s["positions"].double()[..., None] * s["inv_freq"].double())
    w = (w.conj() if c["inverse"] else w) * c["scale"]
    w = w.unsqueeze(2 if c["token_major"] else 1)
    out = []
    for x in (s["q"], s["k"]):
        y, r = x.double(), c["rot"]
        i = torch.arange(r // 2, device=x.device)
        re, im = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + r // 2)
        z = torch.complex(y[..., re], y[..., im]) * w
        y[..., re], y[..., im] = z.real.contiguous(), z.imag.contiguous()
        out.append(y)
    return tuple(out)


def _exact_attn(s, backward):
    """Row by row of (batch, query head), the softmax's derivative written out."""
    c = s["case"]
    T, U, G, by = c["Tq"], c["Tk"], c["Hq"] // c["Hkv"], c["d"] ** -0.5

    def head(x, b, h):
        x = x if c["docs"] else x[b]
        return (x[:, h] if c["token_major"] else x[h]).double()

    row, col = torch.arange(T, device="cuda") + U - T, torch.arange(U, device="cuda")
    low = torch.zeros_like(row)
    if c["docs"]:
        begin = torch.repeat_interleave(s["cu"][:-1].long(), s["cu"].diff().long())
        low = torch.maximum(low, begin)
    if c["window"]:
        low = torch.maximum(low, row - c["window"] + 1)
    seen = (col[None] >= low[:, None]) & (col[None] <= row[:, None])
    like = {x: torch.zeros(s[x].shape, dtype=torch.float64, device="cuda") for x in "qkv"}
    lse = torch.empty((c["B"], c["Hq"], T), dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        for h in range(c["Hq"]):
            q, k, v = head(s["q"], b, h), head(s["k"], b, h // G), head(s["v"], b, h // G)
            e = torch.where(seen, (q @ k.t().contiguous()) * by, -math.inf)
            z = torch.logsumexp(e, -1)
            lse[b, h] = z
            p = torch.where(seen, torch.exp(e - torch.where(z == -math.inf, 0.0, z)[:, None]), 0.0)

            def view(x):
                x = like[x] if c["docs"] else like[x][b]
                return x.transpose(0, 1) if c["token_major"] else x

            if not backward:
                view("q")[h] = p @ v
                continue
            g = head(s["dO"], b, h)
            t = g @ v.t().contiguous()
            t = p * (t - (p * t).sum(-1, keepdim=True)) * by
            view("q")[h] = t @ k
            view("k")[h // G] += t.t().contiguous() @ q
            view("v")[h // G] += p.t().contiguous() @ g
    if backward:
        return {"dq": like["q"], "dk": like["k"], "dv": like["v"]}
    return like["q"], lse[0] if c["docs"] else lse


def _exact_e4m3(y):
    """y rounded to the nearest e4m3 value, ties to even: steps of 2^(e-3), e >= -6."""
    _, e = torch.frexp(y)
    step = _pow2((e - 1).clamp_min(-6) - 3).double()
    return torch.round(y / step) * step


def _exact_append(s):
    c = s["case"]
    out = {"k": s["k_cache"].view(torch.float8_e4m3fn).double(), "v": s["v_cache"].view(torch.float8_e4m3fn).double(),
           "k_scale": s["k_scale"].double(), "v_scale": s["v_scale"].double()}
    have, new, table = s["len"].tolist(), _new_lengths(c), s["table"].tolist()
    begin = 0
    for i in range(c["nseq"]):
        for name in "kv":
            x = s[name][:, begin:begin + new[i]] if c["T"] else s[name][i][:, None]
            x = x.double()                                                     # [H, n, d]
            done = 0
            while done < new[i]:
                at = have[i] + done
                page, off = table[i][at // PAGE], at % PAGE
                n = min(PAGE - off, new[i] - done)
                part = x[:, done:done + n]
                scale = torch.ceil(torch.log2(part.abs().amax((1, 2)) / 448.0)).clamp_min(-96.0)
                scale = _pow2(scale.long()).double()
                values = out[name][page]                                       # [H, 64, d]
                values = values.transpose(2, 3).flatten(1, 2) if name == "v" else values
                if off:
                    old = out[name + "_scale"][page]
                    scale = torch.maximum(scale, old)
                    values[:, :off] = _exact_e4m3(values[:, :off] * (old / scale)[:, None, None])
                values[:, off:off + n] = _exact_e4m3(part / scale[:, None, None])
                out[name][page] = values if name == "k" else values.unflatten(1, (PAGE // 16, 16)).transpose(2, 3)
                out[name + "_scale"][page] = scale
                done += n
        begin += new[i]
    return out


def _exact_decode(s):
    c = s["case"]
    G, rows = c["Hq"] // c["Hkv"], []
    kc, vc = s["k_cache"].view(torch.float8_e4m3fn), s["v_cache"].view(torch.float8_e4m3fn)
    for i, n in enumerate(s["len"].tolist()):
        t = s["table"][i, :(n + PAGE - 1) // PAGE].long()
        begin = max(0, n - c["window"]) if c["window"] else 0
        k = (kc[t].double() * s["k_scale"][t].double()[..., None, None]).transpose(0, 1).flatten(1, 2)[:, begin:n]
        v = (vc[t].double() * s["v_scale"][t].double()[..., None, None, None])
        v = v.permute(1, 0, 2, 4, 3).flatten(1, 3)[:, begin:n]
        q = s["q"][i].double().view(c["Hkv"], G, c["d"])
        p = torch.softmax(torch.bmm(q, k.transpose(1, 2).contiguous()) * c["d"] ** -0.5, -1)
        rows.append(torch.bmm(p, v.contiguous()).reshape(c["Hq"], c["d"]))
    return torch.stack(rows)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _exact_rope(s)
    if op in ("attn_fwd", "attn_bwd"):
        return _exact_attn(s, op == "attn_bwd")
    return _exact_append(s) if op == "kv_append" else _exact_decode(s)
