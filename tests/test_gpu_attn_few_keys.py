"""Gradients of rows that see few keys, in calls of every size: dO v - D is a small
difference there, and D must not carry the output's rounding."""
import math

import pytest
import torch

from tests import attn_reference as ref
from tests.test_gpu_attn import _back, _backward, _forward, _inputs

pytestmark = pytest.mark.gpu
F64 = torch.float64


def _bounds(x, Tq, off, scale, rows, keys):
    """Gradients of the first `rows` queries (which see at most `keys` keys), and their bounds
    with D in fp32: scores and dO v are dot products of d exact terms, a weight is off by the
    score's error and the log-sum-exp's (twice the score's), dS is rounded to bf16, and so is the
    result.  (4 fp32 roundings beside each; 2^-21 for the exponential.)"""
    q, dO = (x[n][:, :, :rows].to(F64) for n in ("q", "dO"))
    G = q.shape[1] // x["k"].shape[1]
    k, v = (x[n][:, :, :keys].to(F64).repeat_interleave(G, 1) for n in ("k", "v"))
    d = q.shape[-1]
    i, j = torch.arange(rows)[:, None] + off, torch.arange(keys)[None]
    seen = j <= i
    zero = torch.zeros((), dtype=F64)
    s = torch.where(seen, ref._dot(q, k) * scale, torch.tensor(-math.inf, dtype=F64))
    lse = torch.logsumexp(s, -1, keepdim=True)
    P = torch.where(seen, torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)), zero)
    dP = ref._dot(dO, v)
    mean = (P * dP.abs()).sum(-1, keepdim=True)
    dS = P * (dP - (P * dP).sum(-1, keepdim=True))
    dot = (d + 4) * ref.FP32
    weight = 4 * (dot * torch.where(seen, ref._dot(q.abs(), k.abs()) * scale, zero).amax(-1, keepdim=True) + 2.0 ** -21
                  + 4 * ref.FP32 * torch.where(lse == -math.inf, 0.0, lse).abs())
    pair = dot * ref._dot(dO.abs(), v.abs())
    off_dS = P * (weight * (dP.abs() + 2 * mean) + pair + (P * pair).sum(-1, keepdim=True)
                  + (keys + 4) * ref.FP32 * (dP.abs() + mean)) + ref.BF16 * 1.01 * dS.abs()
    terms = 64 * ref.FP32
    tq = torch.matmul(off_dS + terms * dS.abs(), k.abs()) * scale
    tk = torch.matmul((off_dS + G * terms * dS.abs()).transpose(-1, -2).contiguous(), q.abs()) * scale
    dq = torch.matmul(dS, k) * scale
    dk = torch.matmul(dS.transpose(-1, -2).contiguous(), q) * scale
    tk, dk = ref._shared(tk, x["k"].shape[1]), ref._shared(dk, x["k"].shape[1])
    return dq, tq + ref.BF16 * 1.01 * dq.abs() + ref.TINY, dk, tk + ref.BF16 * 1.01 * dk.abs() + ref.TINY


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Tq,Tk,window,Hq,Hkv", [(256, 256, 0, 16, 16), (257, 257, 0, 16, 16), (300, 300, 200, 16, 4), (2047, 2047, 0, 8, 2),
                                                 (2047, 2047, 1024, 4, 4), (290, 300, 0, 8, 8), (320, 300, 0, 8, 8),
                                                 (1500, 1500, 33, 4, 2)])
def test_rows_of_few_keys_in_calls_of_every_size(Tq, Tk, window, Hq, Hkv, d):
    """The queries that see 1 to 32 keys; those behind them have dO = 0, so that dk of the
    first keys is theirs alone."""
    x = _inputs(2, Hq, Hkv, Tq, Tk, d, Tq + window)
    off = Tk - Tq
    rows, keys = 32 - off, 32
    x["dO"][:, :, rows:] = 0
    o, lse = _forward(x, window)
    got = _backward(x, o, lse, window)
    dq, tq, dk, tk = _bounds(x, Tq, off, d ** -0.5, rows, keys)
    over = (_back(got["dq"], False, False)[:, :, :rows] - dq).abs() - tq
    assert float(over.max()) <= 0, f"dq {float(over.max()):.3g} over its bound ({int((over > 0).sum())} elements)"
    over = (_back(got["dk"], False, False)[:, :, :keys] - dk).abs() - tk
    assert float(over.max()) <= 0, f"dk {float(over.max()):.3g} over its bound ({int((over > 0).sum())} elements)"
