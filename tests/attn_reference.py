"""The attention layer's operators in 64 bits, written from their definitions, with
the error bounds the GPU tests hold the kernels to.

Bounds.  A rounding to a type is off by at most eps/2 of the value: 2^-8 in
bf16, 2^-24 in fp32.  A dot product of d exact bf16 products summed in fp32 in
any order is off by at most d 2^-24 of the sum of the terms' magnitudes.  Below
2^-126 neither type has normal numbers and the kernels may give 0: each weight,
each product of one with another value and each result may be off by that much
more, whatever its size."""
import math

import torch

F64 = torch.float64
BF16 = 2.0 ** -8
FP32 = 2.0 ** -24
TINY = 2.0 ** -126


def rope(x, inv_freq, positions, rot, interleaved, inverse, scale):
    """x [B, H, T, d] (64 bits), positions [B, T]."""
    theta = positions.to(F64)[:, None, :, None] * inv_freq.to(F64)
    c, s = torch.cos(theta) * scale, torch.sin(theta) * (-scale if inverse else scale)
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def seen(Tq, Tk, window, cu=None):
    """[Tq, Tk] truth: query i sees key j."""
    i = torch.arange(Tq)[:, None] + (Tk - Tq)
    j = torch.arange(Tk)[None, :]
    m = j <= i
    if window:
        m &= j > i - window
    if cu is not None:
        doc = torch.full((Tk,), -1)
        for n, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
            doc[a:b] = n
        m &= (doc[:, None] == doc[None, :]) & (doc >= 0)[:, None]
    return m


def _dot(x, y):
    return torch.matmul(x, y.transpose(-1, -2).contiguous())


def _weighted(mask, w, v):
    """sum_j w_ij v_j over the pairs of the mask only: a masked NaN adds nothing."""
    if bool(torch.isfinite(v).all()):
        return torch.matmul(w, v)
    # v [B, H, Tk, d]: plain sums over the seen keys of each row
    out = torch.zeros(w.shape[:-1] + (v.shape[-1],), dtype=F64)
    for i in range(w.shape[-2]):
        j = mask[i].nonzero()[:, 0]
        if len(j):
            out[..., i, :] = (w[..., i, j, None] * v[..., j, :]).sum(-2)
    return out


def attention(q, k, v, window=0, scale=None, cu=None):
    """q [B, Hq, Tq, d], k, v [B, Hkv, Tk, d] in 64 bits -> dict with o, lse, P and
    the bounds o_tol, lse_tol."""
    B, Hq, Tq, d = q.shape
    Hkv, Tk = k.shape[1:3]
    scale = d ** -0.5 if scale is None else scale
    k, v = k.repeat_interleave(Hq // Hkv, 1), v.repeat_interleave(Hq // Hkv, 1)
    mask = seen(Tq, Tk, window, cu)
    s = torch.where(mask, _dot(q, k) * scale, torch.tensor(-math.inf, dtype=F64))
    lse = torch.logsumexp(s, -1) if Tk else torch.full((B, Hq, Tq), -math.inf, dtype=F64)
    P = torch.where(mask, torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None]), torch.zeros((), dtype=F64))
    o = _weighted(mask, P, v)
    # scores: the dot product's bound, and three fp32 roundings of values up to |s|
    # and the exponent's 2^-22 (two units of the hardware's base-2 exponential)
    mag = torch.where(mask, _dot(q.abs(), k.abs()) * scale, torch.zeros((), dtype=F64))
    rel = (d + 4) * FP32 * mag.amax(-1) + 2.0 ** -21 if Tk else torch.zeros((B, Hq, Tq), dtype=F64)
    A = _weighted(mask, P, v.abs())
    # weights rounded to bf16; weights and their sum each off by `rel`; the sum of up
    # to Tk products in fp32; the result rounded to bf16
    o_tol = (BF16 + 2.1 * rel[..., None] + Tk * FP32) * A + BF16 * o.abs() * 1.01 + TINY
    o_tol = o_tol + TINY * torch.where(torch.isfinite(v), v, torch.zeros((), dtype=F64)).abs().sum(-2, keepdim=True)
    lse_tol = rel * 1.1 + (Tk + 8) * FP32 + 4 * FP32 * torch.where(lse == -math.inf, 0.0, lse).abs()
    return dict(o=o, lse=lse, P=P, o_tol=o_tol, lse_tol=lse_tol, rel=rel, mask=mask, k=k, v=v, scale=scale)


def _shared(x, Hkv):
    return x.unflatten(1, (Hkv, x.shape[1] // Hkv)).sum(2)


def attention_bwd(q, k, v, dO, window=0, scale=None, cu=None):
    """Gradients of <dO, o> and their bounds, given the forward's rounded o and lse."""
    Hkv, d = k.shape[1], q.shape[-1]
    f = attention(q, k, v, window, scale, cu)
    P, kk, vv, mask, scale = f["P"], f["k"], f["v"], f["mask"], f["scale"]
    zero = torch.zeros((), dtype=F64)
    dP = torch.where(mask, _dot(dO, vv), zero)
    D = torch.where(mask.any(-1)[..., None] if mask.shape[1] else torch.zeros((q.shape[2], 1), dtype=torch.bool),
                    (dO * f["o"]).sum(-1, keepdim=True), zero)
    dS = torch.where(mask, P * (dP - D), zero)
    Pt, dSt, mt = (x.transpose(-1, -2).contiguous() for x in (P, dS, mask))
    out = dict(dq=_weighted(mask, dS, kk) * scale, dk=_shared(_weighted(mt, dSt, q), Hkv) * scale,
               dv=_shared(_weighted(mt, Pt, dO), Hkv))
    # P off by the scores' bound twice (its own and the log-sum-exp's)
    relP = 2.2 * f["rel"][..., None] + f["lse_tol"][..., None]
    errD = (dO.abs() * f["o_tol"]).sum(-1, keepdim=True) + (d + 2) * FP32 * (dO * f["o"]).abs().sum(-1, keepdim=True)
    errdP = (d + 2) * FP32 * torch.where(mask, _dot(dO.abs(), vv.abs()), zero)
    tol = torch.where(mask, P * (relP * (dP.abs() + D.abs()) + errD + errdP) * 1.05 + BF16 * dS.abs() * 1.01
                      + TINY * (1 + dP.abs() + D.abs()), zero)
    n, G = max(mask.shape), P.shape[1] // Hkv
    tolP = torch.where(mask, P * (relP + BF16 * 1.01) + TINY, zero)
    terms = n * G * FP32

    def grow(t, w, x, by=1.0):
        return torch.matmul(t + terms * w.abs(), x.abs()) * by + n * TINY

    out["dq_tol"] = grow(tol, dS, kk, scale) + BF16 * 1.01 * out["dq"].abs()
    out["dk_tol"] = _shared(grow(tol.transpose(-1, -2).contiguous(), dSt, q, scale), Hkv) + BF16 * 1.01 * out["dk"].abs()
    out["dv_tol"] = _shared(grow(tolP.transpose(-1, -2).contiguous(), Pt, dO), Hkv) + BF16 * 1.01 * out["dv"].abs()
    return out


def e4m3(y):
    """Nearest e4m3 value of y (64 bits, |y| <= 448), ties to even; NaN and infinities give NaN."""
    _, e = torch.frexp(torch.where(torch.isfinite(y), y, torch.zeros((), dtype=F64)))
    step = torch.pow(torch.tensor(2.0, dtype=F64), ((e - 1).clamp_min(-6) - 3).to(F64))
    r = torch.round(y / step) * step
    return torch.where(torch.isfinite(y), r, torch.full((), math.nan, dtype=F64))


def pow2_scale(top):
    """Smallest power of two s >= 2^-96 with top <= 448 s."""
    e = -96
    while top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


class Cache:
    """The paged cache in 64 bits: values [n_pages, H, 64, d] as e4m3 * scale kept apart."""

    def __init__(self, k, v, k_scale, v_scale):
        """From the bytes and scales of a cache on any device."""
        self.k = k.cpu().view(torch.float8_e4m3fn).to(F64)
        self.v = v.cpu().view(torch.float8_e4m3fn).to(F64).transpose(3, 4).flatten(2, 3)
        self.ks, self.vs = k_scale.cpu().to(F64).clone(), v_scale.cpu().to(F64).clone()

    def append(self, k, v, table, have):
        """k, v: per sequence [H, n, d] in 64 bits."""
        for val, sc, new in ((self.k, self.ks, k), (self.v, self.vs, v)):
            for i, x in enumerate(new):
                done = 0
                while done < x.shape[1]:
                    at = have[i] + done
                    n = min(64 - at % 64, x.shape[1] - done)
                    if at // 64 < table.shape[1] and 0 <= int(table[i, at // 64]) < val.shape[0]:
                        pg, off = int(table[i, at // 64]), at % 64
                        for h in range(x.shape[0]):
                            part = x[h, done:done + n]
                            fin = part[torch.isfinite(part)].abs()
                            s = pow2_scale(float(fin.max()) if fin.numel() else 0.0)
                            if off:
                                old = float(sc[pg, h])
                                s = max(s, old)
                                val[pg, h, :off] = e4m3(val[pg, h, :off] * (old / s))
                            val[pg, h, off:off + n] = e4m3(part / s)
                            sc[pg, h] = s
                    done += n

    def tokens(self, table_row, n):
        """Keys and values [H, n, d] of one sequence and which of them exist."""
        pages = [int(p) for p in table_row[:(n + 63) // 64]]
        ok = torch.tensor([0 <= p < self.k.shape[0] for p in pages]).repeat_interleave(64)[:n]
        get = lambda x, s: torch.cat([x[p if 0 <= p < x.shape[0] else 0] * s[p if 0 <= p < x.shape[0] else 0][:, None, None]  # noqa: E731
                                      for p in pages], 1)[:, :n]
        return get(self.k, self.ks), get(self.v, self.vs), ok


def decode(q, cache, table, lens, window=0, scale=None):
    """q [N, Hq, d] in 64 bits -> o and its bound for an fp32 result."""
    N, Hq, d = q.shape
    H = cache.k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o, tol = torch.zeros_like(q), torch.zeros_like(q)
    for i in range(N):
        n = min(int(lens[i]), table.shape[1] * 64)
        if n <= 0:
            continue
        lo = max(0, int(lens[i]) - window) if window else 0
        k, v, ok = cache.tokens(table[i], n)
        at = torch.arange(n)
        at = at[ok & (at >= lo)]
        if not len(at):
            continue
        k, v = k[:, at].repeat_interleave(Hq // H, 0), v[:, at].repeat_interleave(Hq // H, 0)
        s = (q[i][:, None] * k).sum(-1) * scale
        p = torch.softmax(s, -1)
        o[i] = (p[..., None] * v).sum(1)
        # scores as in attention(); a weight as two bf16 values keeps 16 bits
        rel = (d + 4) * FP32 * ((q[i].abs()[:, None] * k.abs()).sum(-1) * scale).amax(-1) + 2.0 ** -21
        tol[i] = (2.0 ** -16 + 2.1 * rel[:, None] + (len(at) + 8) * FP32) * (p[..., None] * v.abs()).sum(1) + 4 * FP32 * o[i].abs()
    return o, tol
