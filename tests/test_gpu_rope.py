"""gdr_rope on the GPU against its definition in 64 bits."""
import pytest
import torch

import gated_delta_rule_24_amd as gdr
from tests import attn_reference as ref

pytestmark = pytest.mark.gpu
F64 = torch.float64


def _make(B, H, T, d, dtype, seed, packed=False, token_major=False):
    x = torch.randn((B, H, T, d), generator=torch.Generator().manual_seed(seed)).to(dtype)
    given = x.transpose(1, 2).contiguous() if token_major else x
    return x, (given[0] if packed else given).cuda()


def _back(y, packed, token_major):
    y = y[None] if packed else y
    return (y.transpose(1, 2) if token_major else y).cpu()


def _check(got, x, f, pos, rot, interleaved, inverse, scale):
    want = ref.rope(x.to(F64), f.cpu(), pos, rot, interleaved, inverse, scale)
    # the pair's other channel bounds the cancelling sum; cosine and sine off by
    # 2^-21 (the fraction of a turn rounded to fp32, the function, the scale)
    y = x.to(F64).abs()
    pair = torch.zeros_like(y)
    if interleaved:
        both = y[..., 0:rot:2] + y[..., 1:rot:2]
        pair[..., 0:rot:2], pair[..., 1:rot:2] = both, both
    else:
        both = y[..., :rot // 2] + y[..., rot // 2:rot]
        pair[..., :rot // 2], pair[..., rot // 2:rot] = both, both
    half = ref.BF16 if x.dtype == torch.bfloat16 else ref.FP32
    tol = half * want.abs() * 1.01 + 2.0 ** -21 * pair * abs(scale)
    assert bool(((got.to(F64) - want).abs() <= tol).all())
    assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,Hq,Hk,T,d,rot", [(1, 1, 1, 1, 16, 16), (2, 5, 1, 33, 32, 16), (3, 4, 4, 17, 64, 48),
                                             (64, 16, 4, 1, 128, 64), (1, 7, 3, 257, 128, 128), (2, 40, 8, 70, 128, 32)])
def test_rope(dtype, interleaved, B, Hq, Hk, T, d, rot):
    token_major, inverse = (T % 2 == 1), (Hq % 2 == 1)
    f, _ = gdr.rope_frequencies(rot)
    pos = torch.randint(0, 2000, (B, T), generator=torch.Generator().manual_seed(T), dtype=torch.int32)
    q, qd = _make(B, Hq, T, d, dtype, 1, token_major=token_major)
    k, kd = _make(B, Hk, T, d, dtype, 2, token_major=token_major)
    qo, ko = gdr.rope(qd, kd, f, pos.cuda(), interleaved=interleaved, inverse=inverse, scale=1.25,
                      token_major=token_major)
    _check(_back(qo, False, token_major), q, f, pos, rot, interleaved, inverse, 1.25)
    _check(_back(ko, False, token_major), k, f, pos, rot, interleaved, inverse, 1.25)


@pytest.mark.parametrize("pos", [0, 1, -5, 999_983, 16_777_217, 2_147_483_647])
def test_far_positions(pos):
    f, _ = gdr.rope_frequencies(64)
    x, xd = _make(1, 2, 1, 64, torch.float32, 3)
    p = torch.tensor([[pos]], dtype=torch.int32)
    y, _ = gdr.rope(xd, None, f, p.cuda())
    _check(y.cpu(), x, f, p, 64, False, False, 1.0)
    y0, none = gdr.rope(xd, None, f, None, position0=pos)
    assert torch.equal(y0, y) and none is None


def test_packed_in_place_and_round_trip():
    f, s = gdr.rope_frequencies(32, scaling="parts", factor=8.0, trained=2048)
    q, qd = _make(1, 3, 50, 64, torch.float32, 4, packed=True)
    k, kd = _make(1, 2, 50, 64, torch.float32, 5, packed=True)
    pos = torch.cat([torch.arange(20), torch.arange(30)]).to(torch.int32)
    q2, k2 = gdr.rope(qd, kd, f, pos.cuda(), scale=s)
    _check(q2.cpu()[None], q, f, pos[None], 32, False, False, s)
    keep = qd.clone()
    a, b = gdr.rope(qd, kd, f, pos.cuda(), scale=s, q_out=qd, k_out=kd)
    assert a is qd and b is kd and torch.equal(qd, q2) and torch.equal(kd, k2)
    back, _ = gdr.rope(qd, kd, f, pos.cuda(), scale=1 / s, inverse=True)
    # two turns of fp32 values, each off by 2^-21 of the pair's magnitudes (at most 2 x 6)
    assert float((back - keep).abs().max()) <= 2 * 2.0 ** -21 * 12 * 1.3


def test_inverse_is_the_gradient():
    """<rope(x), g> has the gradient rope_inverse(g), also against differences."""
    f, _ = gdr.rope_frequencies(32)
    x, xd = _make(1, 1, 9, 32, torch.float32, 6)
    g, gd = _make(1, 1, 9, 32, torch.float32, 7)
    pos = torch.arange(100, 109, dtype=torch.int32)[None]
    dx, _ = gdr.rope(gd, None, f, pos.cuda(), inverse=True, interleaved=True)
    u = torch.randn(x.shape, generator=torch.Generator().manual_seed(8), dtype=F64)
    up = lambda y: float((ref.rope(y, f.cpu(), pos, 32, True, False, 1.0) * g.to(F64)).sum())  # noqa: E731
    diff = (up(x.to(F64) + 1e-3 * u) - up(x.to(F64) - 1e-3 * u)) / 2e-3          # linear: exact but for rounding
    # 288 terms, each off by 2^-21 of |pair| |u| <= 8 * 4
    assert abs(diff - float((dx.cpu().to(F64) * u).sum())) <= 288 * 2.0 ** -21 * 32


def test_empty_and_refusals():
    f, _ = gdr.rope_frequencies(16)
    z = torch.empty((2, 3, 0, 16), dtype=torch.bfloat16, device="cuda")
    assert gdr.rope(z, z, f)[0].shape == z.shape
    x = torch.zeros((2, 3, 4, 16), device="cuda")
    with pytest.raises(ValueError):
        gdr.rope(x.half(), x.half(), f)
    with pytest.raises(ValueError):
        gdr.rope(x, x[:, :, :2].contiguous(), f)
    with pytest.raises(ValueError):
        gdr.rope(x.transpose(1, 2), None, f)                        # not contiguous
    with pytest.raises(ValueError):
        gdr.rope(x, x, f, torch.zeros((2, 4), device="cuda"))       # positions not int32
    with pytest.raises(ValueError):
        gdr.rope(x, x, f.cpu())
    with pytest.raises(gdr.GdrError):
        gdr.rope(x, x, torch.ones(4, device="cuda"))                # rot_dim 8


def test_other_stream_and_graph():
    f, _ = gdr.rope_frequencies(64)
    _, q = _make(2, 4, 100, 64, torch.bfloat16, 9)
    want, _ = gdr.rope(q, None, f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = gdr.rope(q, None, f, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdr.rope(q, None, f, q_out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
