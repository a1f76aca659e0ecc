"""The 64-bit reference of the attention layer against itself: the gradients'
formulas against central differences, the e4m3 rounding against the type's own
table, rotary positions against their inverse (CPU only)."""
import math

import pytest
import torch

import gated_delta_rule_24_amd as gdr
from tests import attn_reference as ref

F64 = torch.float64


@pytest.mark.parametrize("Tq,Tk,window,cu", [(5, 5, 0, None), (5, 9, 3, None), (7, 4, 0, None), (8, 8, 2, [0, 3, 3, 8]),
                                             (6, 6, 0, [0, 2, 5])])
def test_gradient_formulas_match_differences(Tq, Tk, window, cu):
    g = torch.Generator().manual_seed(Tq * 100 + Tk)
    q, dO = (torch.randn(1, 4, Tq, 6, generator=g, dtype=F64) for _ in range(2))
    k, v = (torch.randn(1, 2, Tk, 6, generator=g, dtype=F64) for _ in range(2))
    got = ref.attention_bwd(q, k, v, dO, window, cu=cu)
    loss = lambda q, k, v: float((ref.attention(q, k, v, window, cu=cu)["o"] * dO).sum())  # noqa: E731
    args = dict(q=q, k=k, v=v)
    eps = 1e-5
    for name, x in args.items():
        for _ in range(6):
            u = torch.randn(x.shape, generator=g, dtype=F64)
            up, down = dict(args), dict(args)
            up[name], down[name] = x + eps * u, x - eps * u
            diff = (loss(**up) - loss(**down)) / (2 * eps)
            want = float((got["d" + name] * u).sum())
            # truncation eps^2 times a third derivative of order 10, rounding 1e-16 / eps
            assert abs(diff - want) <= 1e-8 * (1 + abs(want)) + 1e-9


def test_rows_that_see_nothing():
    q, k = torch.randn(1, 1, 4, 8, dtype=F64), torch.randn(1, 1, 2, 8, dtype=F64)
    f = ref.attention(q, k, k)
    assert torch.equal(f["o"][0, 0, :2], torch.zeros(2, 8, dtype=F64))
    assert (f["lse"][0, 0, :2] == -math.inf).all() and torch.isfinite(f["lse"][0, 0, 2:]).all()


def test_e4m3_rounding_is_the_types_own():
    x = torch.cat([torch.randn(20000, generator=torch.Generator().manual_seed(0)) * 60, torch.arange(-448, 449).float(),
                   torch.arange(0, 600).float() * 2.0 ** -11]).clamp(-448, 448)
    assert torch.equal(ref.e4m3(x.to(F64)), x.to(torch.float8_e4m3fn).to(F64))


def test_pow2_scale():
    assert ref.pow2_scale(0.0) == 2.0 ** -96 and ref.pow2_scale(448.0) == 1.0 and ref.pow2_scale(449.0) == 2.0
    assert ref.pow2_scale(1.75) == 2.0 ** -8


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_inverse_turns_back(interleaved):
    x = torch.randn(2, 3, 5, 32, dtype=F64)
    f = torch.rand(8)
    pos = torch.randint(0, 1000, (2, 5))
    y = ref.rope(x, f, pos, 16, interleaved, False, 1.0)
    assert torch.allclose(ref.rope(y, f, pos, 16, interleaved, True, 1.0), x, atol=1e-12)
    assert torch.equal(y[..., 16:], x[..., 16:])


def test_rope_frequencies():
    f, s = gdr.rope_frequencies(64, device="cpu")
    want = torch.tensor([10000.0 ** (-2 * i / 64) for i in range(32)], dtype=F64).float()
    assert s == 1.0 and torch.equal(f, want)
    f2, _ = gdr.rope_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(f2, want / 4, rtol=2e-7)
    f3, _ = gdr.rope_frequencies(64, scaling="base", factor=4.0, device="cpu")
    assert f3[0] == 1.0 and abs(float(f3[-1] * 4 / want[-1]) - 1) < 1e-6
    f4, s4 = gdr.rope_frequencies(64, scaling="parts", factor=4.0, trained=4096, low=1, high=32, device="cpu")
    turns = 4096 * want.double() / (2 * math.pi)
    assert torch.equal(f4[turns >= 32], want[turns >= 32])
    assert torch.allclose(f4[turns <= 1], want[turns <= 1] / 4, rtol=2e-7)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (f4[mid] < want[mid]).all() and (f4[mid] > want[mid] / 4).all()
    assert abs(s4 - (0.1 * math.log(4.0) + 1)) < 1e-12
    for bad in (dict(rot_dim=7), dict(rot_dim=64, scaling="other"), dict(rot_dim=64, scaling="parts"),
                dict(rot_dim=2, scaling="base")):
        with pytest.raises(ValueError):
            gdr.rope_frequencies(device="cpu", **bad)
