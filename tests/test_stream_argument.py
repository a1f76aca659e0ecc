"""The calls with a `stream` argument allocate what they use on that stream: the
allocator hands memory out in the order of the stream it is asked on, so memory
allocated on another one may still be written there when the kernel starts.  What the
calls return is kept for the caller's own stream too.  (CPU tensors, the library's
calls and torch's streams replaced; no GPU.)"""
import contextlib

import pytest
import torch

import gated_delta_rule_24_amd as gdr

BF16, F32 = torch.bfloat16, torch.float32


class Stream:
    device, cuda_stream = torch.device("cpu"), 1


CALLER, SIDE = Stream(), Stream()


def _x(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


def _gates(*lead):
    return [_x(*lead, 64) for _ in range(3)] + [_x(*lead, 64, dtype=F32)] + [_x(*lead, 64) for _ in range(2)]


def _cache():
    return gdr.kv_cache(3, 2, 64, device="cpu"), _x(2, 1, dtype=torch.int32), _x(2, dtype=torch.int32)


CU = torch.tensor([0, 40, 64], dtype=torch.int32)
CALLS = {
    "chunk_fwd": lambda **k: gdr.chunk_fwd(*_gates(1, 2, 64), **k),
    "chunk_fwd_varlen": lambda **k: gdr.chunk_fwd_varlen(*_gates(2, 64), CU, **k),
    "decode_step": lambda **k: gdr.decode_step(*_gates(2, 2), _x(2, 2, 64, 64, dtype=F32), **k),
    "chunk_bwd": lambda **k: gdr.chunk_bwd(*_gates(1, 2, 64), None, _x(1, 2, 64, 64), **k),
    "chunk_bwd_varlen": lambda **k: gdr.chunk_bwd_varlen(*_gates(2, 64), CU, None, _x(2, 64, 64), **k),
    "mixer_prologue": lambda **k: gdr.mixer_prologue(*[_x(1, 2, 64, 64)] * 3, *[_x(2, 64, 4, dtype=F32)] * 3,
                                                     _x(1, 2, 64, 64, dtype=F32), *[_x(1, 2, 64, 64)] * 2, **k),
    "mixer_epilogue": lambda **k: gdr.mixer_epilogue(_x(1, 2, 64, 64, dtype=F32), _x(1, 2, 64, 64), _x(64, dtype=F32), **k),
    "mixer_prologue_bwd": lambda **k: gdr.mixer_prologue_bwd(*[_x(1, 2, 64, 64)] * 3, *[_x(2, 64, 4, dtype=F32)] * 3,
                                                             *[_x(1, 2, 64, 64, dtype=F32)] * 3, **k),
    "mixer_epilogue_bwd": lambda **k: gdr.mixer_epilogue_bwd(_x(1, 2, 64, 64, dtype=F32), _x(1, 2, 64, 64), _x(64, dtype=F32),
                                                             _x(1, 2, 64, 64), **k),
    "rope": lambda **k: gdr.rope(_x(1, 4, 8, 64), _x(1, 2, 8, 64), _x(16, dtype=F32), **k),
    "attn_fwd": lambda **k: gdr.attn_fwd(_x(1, 4, 64, 64), _x(1, 2, 64, 64), _x(1, 2, 64, 64), **k),
    "attn_fwd_varlen": lambda **k: gdr.attn_fwd_varlen(_x(4, 64, 64), _x(2, 64, 64), _x(2, 64, 64), CU, **k),
    "attn_bwd": lambda **k: gdr.attn_bwd(_x(1, 4, 64, 64), _x(1, 2, 64, 64), _x(1, 2, 64, 64), _x(1, 4, 64, 64),
                                         _x(1, 4, 64, dtype=F32), _x(1, 4, 64, 64), **k),
    "attn_bwd_varlen": lambda **k: gdr.attn_bwd_varlen(_x(4, 64, 64), _x(2, 64, 64), _x(2, 64, 64), _x(4, 64, 64),
                                                       _x(4, 64, dtype=F32), _x(4, 64, 64), CU, **k),
    "attn_decode": lambda **k: gdr.attn_decode(_x(2, 4, 64), *_cache(), **k),
}


@pytest.fixture
def world(monkeypatch):
    """Records each allocation's stream, each launch's, and what is kept for which."""
    w = dict(now=[CALLER], allocated=[], launched=[], kept=[])

    @contextlib.contextmanager
    def on(stream):
        w["now"].append(stream)
        yield
        w["now"].pop()

    def allocating(fn):
        def f(*a, **k):
            t = fn(*a, **k)
            w["allocated"].append((t, w["now"][-1]))
            return t
        return f

    def launch(fn):
        return lambda *a, **k: w["launched"].append(fn)

    for name in [n for n in dir(gdr) if n.startswith("gdr_") and not n.endswith("_bytes")]:
        monkeypatch.setattr(gdr, name, launch(name))
    monkeypatch.setattr(gdr, "_launch", launch("_launch"))
    monkeypatch.setattr(gdr, "_gpu_of", lambda name, t: t.get_device())
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: w["now"][-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: w["kept"].append((t, s)))
    return w, allocating


def _parts(out):
    if isinstance(out, torch.Tensor):
        return [out]
    return [t for t in (out.values() if isinstance(out, dict) else out) if t is not None]


@pytest.mark.parametrize("name", sorted(CALLS))
def test_what_a_call_uses_is_allocated_on_its_stream(name, world, monkeypatch):
    w, allocating = world
    call = CALLS[name]
    for n in ("empty", "empty_like"):
        monkeypatch.setattr(torch, n, allocating(getattr(torch, n)))
    if name == "attn_decode":                         # the caches above are not the call's own
        monkeypatch.setattr(gdr, "kv_cache", lambda *a, **k: gdr.KVCache(
            _x(3, 2, 64, 64, dtype=torch.uint8), _x(3, 2, 4, 64, 16, dtype=torch.uint8), _x(3, 2, dtype=F32), _x(3, 2, dtype=F32)))
    out = _parts(call(stream=SIDE))
    assert w["launched"] and w["allocated"] and w["now"] == [CALLER]
    assert all(s is SIDE for _, s in w["allocated"])
    made = [t for t, _ in w["allocated"]]
    own = [t for t in out if any(t is m for m in made)]
    assert own
    for t in own:                                     # the caller goes on with them on its own stream
        assert any(t is k and s is CALLER for k, s in w["kept"])
    # without the argument, and with the current stream: that one, and nothing to keep
    for kw in ({}, {"stream": CALLER}):
        w["allocated"].clear(), w["kept"].clear()
        call(**kw)
        assert w["allocated"] and all(s is CALLER for _, s in w["allocated"]) and not w["kept"]


def test_the_stream_as_a_positional_argument(world, monkeypatch):
    w, allocating = world
    monkeypatch.setattr(torch, "empty", allocating(torch.empty))
    gdr.mixer_epilogue(_x(1, 2, 64, 64, dtype=F32), _x(1, 2, 64, 64), _x(64, dtype=F32), SIDE)
    assert [s for _, s in w["allocated"]] == [SIDE]


def test_the_calls_with_a_stream_are_all_here():
    import inspect
    with_stream = {n for n, f in vars(gdr).items() if inspect.isfunction(f) and not n.startswith(("_", "gdr_"))
                   and "stream" in inspect.signature(f).parameters}
    assert with_stream - {"kv_append"} == set(CALLS)   # kv_append allocates nothing
