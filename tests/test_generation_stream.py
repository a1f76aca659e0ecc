"""The calls for several continuations allocate what they use on the stream they are
given, and keep what they return for the caller's (CPU tensors, the library's calls and
torch's streams replaced; no GPU)."""
import contextlib
import inspect

import pytest
import torch

import gated_delta_rule_24_amd as gdr

gen = gdr.generation


class Stream:
    device, cuda_stream = torch.device("cpu"), 1


CALLER, SIDE = Stream(), Stream()


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


CACHE = gdr.kv_cache(5, 2, 64, device="cpu")
CALLS = {
    "attn_decode_shared": lambda **k: gen.attn_decode_shared(torch.zeros((3, 4, 64), dtype=torch.bfloat16), CACHE, _i(3, 2), _i(3), _i(2),
                                                             _i(1), **k),
    "kv_fork": lambda **k: gen.kv_fork(CACHE, _i(3, 2), _i(3), parent=_i(4), **k),
    "kv_compact": lambda **k: gen.kv_compact(CACHE, _i(3, 2), _i(3), **k),
    "beam_select": lambda **k: gen.beam_select(torch.zeros(6, 9), torch.zeros(2, 3), **k),
}


@pytest.fixture
def world(monkeypatch):
    w = dict(now=[CALLER], allocated=[], launched=[], kept=[])

    @contextlib.contextmanager
    def on(stream):
        w["now"].append(stream)
        yield
        w["now"].pop()

    def empty(like, *a, _empty=torch.Tensor.new_empty, **k):
        t = _empty(like, *a, **k)
        w["allocated"].append((t, w["now"][-1]))
        return t

    monkeypatch.setattr(gen, "_launch", lambda fn, gpu, stream, *a: w["launched"].append((fn, stream)))
    monkeypatch.setattr(gen, "_gpu_of", lambda name, t: t.get_device())
    monkeypatch.setattr(torch.Tensor, "new_empty", empty)
    monkeypatch.setattr(torch, "empty", None)         # (not used)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: w["now"][-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: w["kept"].append((t, s)))
    return w


@pytest.mark.parametrize("name", sorted(CALLS))
def test_what_a_call_uses_is_allocated_on_its_stream(name, world):
    out = CALLS[name](stream=SIDE)
    out = [out] if isinstance(out, torch.Tensor) else list(out)
    assert world["launched"] == [("gdr_" + name, SIDE)] and world["now"] == [CALLER]
    assert len(world["allocated"]) > len(out) and all(s is SIDE for _, s in world["allocated"])      # a workspace as well
    for t in out:
        assert any(t is k and s is CALLER for k, s in world["kept"])
    for kw in ({}, {"stream": CALLER}):
        world["allocated"].clear(), world["kept"].clear()
        CALLS[name](**kw)
        assert world["allocated"] and all(s is CALLER for _, s in world["allocated"]) and not world["kept"]


def test_every_call_that_allocates_is_here():
    with_stream = {n for n, f in vars(gen).items() if inspect.isfunction(f) and not n.startswith(("_", "gdr_"))
                   and "stream" in inspect.signature(f).parameters}
    assert with_stream - {"state_reorder"} == set(CALLS)                                             # in place: allocates nothing


def test_state_reorder_on_its_stream(world):
    S = torch.zeros(6, 4)
    assert gen.state_reorder(S, _i(6), 3, stream=SIDE) is S
    assert world["launched"] == [("gdr_state_reorder", SIDE)] and not world["allocated"]


@pytest.mark.parametrize("call", [
    lambda x: gen.beam_select(torch.zeros(6, 9), torch.zeros(2, 3), n_select=x),
    lambda x: gen.beam_select(torch.zeros(6, 9), torch.zeros(2, 3), end_token=x),
    lambda x: gen.state_reorder(torch.zeros(6, 4), _i(6), x),
])
@pytest.mark.parametrize("x", [(1 << 32) + 3, -(1 << 32) + 1, 1 << 31])
def test_numbers_past_32_bits_are_refused(call, x, world):
    with pytest.raises(ValueError, match="32 bits"):
        call(x)
    assert not world["launched"]
