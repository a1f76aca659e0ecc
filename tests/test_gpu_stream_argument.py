"""Calls on a stream that is not the current one, while the current one still has work
queued on memory that it has given back: the results are those of the current stream."""
import pytest
import torch

import gated_delta_rule_24_amd as gdr
import gdr_synth as gs
from tests.helpers import to_dev
from tests.test_gpu_attn import _inputs

pytestmark = pytest.mark.gpu


def _parts(out):
    if isinstance(out, torch.Tensor):
        return [out]
    return [t for t in (out.values() if isinstance(out, dict) else out) if t is not None]


def _calls():
    x = {n: t.cuda() for n, t in _inputs(1, 4, 2, 1100, 1100, 64, 1).items()}
    q, k, v, dO = (x[n] for n in ("q", "k", "v", "dO"))
    f, _ = gdr.rope_frequencies(32)
    o, lse = gdr.attn_fwd(q, k, v)
    cache = gdr.kv_cache(40, 2, 64)
    table = torch.randperm(40, device="cuda").to(torch.int32)[:36].view(1, 36).contiguous()
    cu, have = torch.tensor([0, 1100], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    gdr.kv_append(k[0], v[0], cache, table, have, cu)
    q1, full = q[:, :, 0].contiguous(), have + 1100
    r = to_dev(gs.make_inputs(1, 2, 256, 64, 64, seed=3))
    rec = [r[n] for n in ("q", "k", "v", "log_alpha", "b", "w", "S0")]
    return [lambda **s: gdr.rope(q, k, f, **s), lambda **s: gdr.attn_fwd(q, k, v, **s),
            lambda **s: gdr.attn_bwd(q, k, v, o, lse, dO, **s),
            lambda **s: gdr.attn_decode(q1, cache, table, full, **s),
            lambda **s: gdr.chunk_fwd(*rec, **s), lambda **s: gdr.chunk_bwd(*rec, rec[2], **s)]


def test_memory_that_the_current_stream_still_writes():
    calls = _calls()
    want = [[t.clone() for t in _parts(c())] for c in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    work = torch.randn(4096, 4096, device="cuda")
    for i, (c, w) in enumerate(zip(calls, want)):
        torch.cuda.empty_cache()
        # memory of the outputs' and the workspaces' sizes, written behind long work and given back
        held = [torch.empty(t.numel() * t.element_size(), dtype=torch.uint8, device="cuda") for t in w for _ in range(2)]
        held += [torch.empty(1 << n, dtype=torch.uint8, device="cuda") for n in range(12, 27)]
        torch.cuda.synchronize()
        for _ in range(8):
            work = work @ work * 0.01
        for h in held:
            h.fill_(0x7f)
        del held, h
        got = _parts(c(stream=side))
        side.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, w)), i


def test_captured_on_a_stream_beside_the_capturing_one():
    x = {n: t.cuda() for n, t in _inputs(1, 4, 2, 300, 300, 64, 1).items()}
    q, k, v, dO = (x[n] for n in ("q", "k", "v", "dO"))
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    gdr.attn_bwd(q, k, v, *gdr.attn_fwd(q, k, v), dO)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        o, lse = gdr.attn_fwd(q, k, v, stream=side)
        g = gdr.attn_bwd(q, k, v, o, lse, dO, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for seed in (2, 3, 2):
        y = {n: t.cuda() for n, t in _inputs(1, 4, 2, 300, 300, 64, seed).items()}
        for n in x:
            x[n].copy_(y[n])
        graph.replay()
        torch.cuda.synchronize()
        o2, lse2 = gdr.attn_fwd(*(y[n] for n in "qkv"))
        g2 = gdr.attn_bwd(y["q"], y["k"], y["v"], o2, lse2, y["dO"])
        assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(g[n], g2[n]) for n in g)


def test_results_are_kept_for_the_stream_that_goes_on_with_them():
    """Used on the current stream behind long work and dropped: a second call on the other
    stream does not get their memory before that."""
    calls = _calls()
    want = [[t.clone() for t in _parts(c())] for c in calls]
    torch.cuda.synchronize()
    side, work = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    for i, (c, w) in enumerate(zip(calls, want)):
        got = _parts(c(stream=side))
        torch.cuda.current_stream().wait_stream(side)
        for _ in range(8):
            work = work @ work * 0.01
        kept = [t.clone() for t in got]
        del got
        with torch.cuda.stream(side):
            again = [torch.full_like(t, 7.0) for t in w for _ in range(2)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, w)) and again, i
