"""The attention layer's calls together, as a hybrid stack makes them: a training
step through rotary positions and attention and back; a prompt and generation
over the 8-bit cache; a layer pair with the recurrence."""
import pytest
import torch

import gated_delta_rule_24_amd as gdr
from tests import attn_reference as ref

pytestmark = pytest.mark.gpu
F64 = torch.float64


def _rand(shape, seed, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


@pytest.mark.parametrize("interleaved", [False, True])
def test_training_step_through_positions_and_attention(interleaved):
    """d loss / d (q, k before the positions), against the formulas applied to the
    rounded values that each call was given."""
    B, Hq, Hkv, T, d, W = 1, 4, 2, 150, 64, 60
    q, k, v, dO = _rand((B, Hq, T, d), 1), _rand((B, Hkv, T, d), 2), _rand((B, Hkv, T, d), 3), _rand((B, Hq, T, d), 4)
    f, s = gdr.rope_frequencies(32)
    qr, kr = gdr.rope(q.cuda(), k.cuda(), f, interleaved=interleaved, scale=s)
    o, lse = gdr.attn_fwd(qr, kr, v.cuda(), window=W)
    g = gdr.attn_bwd(qr, kr, v.cuda(), o, lse, dO.cuda(), window=W)
    dq, dk = gdr.rope(g["dq"], g["dk"], f, interleaved=interleaved, inverse=True, scale=s)
    pos = torch.arange(T)[None]
    r = ref.attention_bwd(qr.cpu().to(F64), kr.cpu().to(F64), v.to(F64), dO.to(F64), W)
    for got, name in ((dq, "dq"), (dk, "dk")):
        want = ref.rope(r[name], f.cpu(), pos, 32, interleaved, True, s)
        # the attention's bound on both channels of a pair, then the second rounding
        pair = r[name + "_tol"].clone()
        both = (pair[..., 0:32:2] + pair[..., 1:32:2]) if interleaved else (pair[..., :16] + pair[..., 16:32])
        if interleaved:
            pair[..., 0:32:2], pair[..., 1:32:2] = both, both
        else:
            pair[..., :16], pair[..., 16:32] = both, both
        tol = pair * 1.01 + ref.BF16 * want.abs() * 1.02 + 2.0 ** -20 * r[name].abs().amax()
        assert bool(((got.cpu().to(F64) - want).abs() <= tol).all())


def test_prompts_then_generation_over_the_cache():
    """Two packed prompts through positions, attention and the cache, then generated
    tokens; every output against the definition over what the cache holds."""
    Hq, H, d, W, lens = 8, 2, 64, 100, [130, 70]
    T, width = sum(lens), 4
    f, _ = gdr.rope_frequencies(64)
    cu = torch.tensor([0, lens[0], T], dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
    q, k, v = _rand((Hq, T, d), 5).cuda(), _rand((H, T, d), 6).cuda(), _rand((H, T, d), 7).cuda()
    q, k = gdr.rope(q, k, f, pos)
    cache = gdr.kv_cache(10, H, d)
    table = torch.tensor([[9, 2, 5, 0], [1, 7, 3, 8]], dtype=torch.int32, device="cuda")
    have = torch.zeros(2, dtype=torch.int32, device="cuda")
    o, _ = gdr.attn_fwd_varlen(q, k, v, cu, window=W)
    gdr.kv_append(k, v, cache, table, have, cu)
    have += cu.diff()
    # the prompt's last tokens again, now over the cache: 8-bit keys and values move the
    # scores and the output; a value is off by at most 2^-4 of itself or, below the
    # normal range, half a step: 2^-10 of the page's scale
    last = torch.stack([q[:, n - 1] for n in cu[1:].tolist()]).contiguous()
    got = gdr.attn_decode(last, cache, table, have, window=W).cpu().to(F64)
    for i, (a, b) in enumerate(zip(cu.tolist(), cu.tolist()[1:])):
        lo = max(a, b - W)
        kk, vv = (x[:, lo:b].cpu().to(F64).repeat_interleave(Hq // H, 0) for x in (k, v))
        qq = q[:, b - 1].cpu().to(F64)
        sub = 2.0 ** -10 * float(torch.maximum(cache.k_scale.max(), cache.v_scale.max()))
        s = (qq[:, None] * kk).sum(-1) * d ** -0.5
        ds = ((qq.abs()[:, None] * (kk.abs() * 2.0 ** -4 + sub)).sum(-1) * d ** -0.5).amax(-1)     # each score's error
        p = torch.softmax(s, -1)
        err = (torch.exp(2 * ds) - 1)[:, None] * (p[..., None] * vv.abs()).sum(1) + \
            torch.exp(2 * ds)[:, None] * (p[..., None] * (vv.abs() * 2.0 ** -4 + sub)).sum(1)
        want = (p[..., None] * vv).sum(1)
        assert bool(((got[i] - want).abs() <= err * 1.01).all())
        assert bool(((o[:, b - 1].cpu().to(F64) - want).abs() <= 2.0 ** -6 * (p[..., None] * vv.abs()).sum(1)).all())
    for step in range(3):
        q1, k1, v1 = _rand((2, Hq, d), 50 + step).cuda(), _rand((2, H, d), 60 + step).cuda(), _rand((2, H, d), 70 + step).cuda()
        q1, k1 = (x[:, :, 0] for x in gdr.rope(q1[:, :, None], k1[:, :, None], f, have[:, None]))
        gdr.kv_append(k1.contiguous(), v1, cache, table, have)
        have += 1
        y = gdr.attn_decode(q1.contiguous(), cache, table, have, window=W)
        want, tol = ref.decode(q1.cpu().to(F64), ref.Cache(*cache), table.cpu(), have.tolist(), W)
        assert bool(((y.cpu().to(F64) - want).abs() <= tol).all())


def test_a_recurrent_layer_and_an_attention_layer():
    """The recurrence's output feeds the attention layer on one stream, with the same
    head layout; each against its own call alone."""
    import gdr_synth as gs
    from tests.helpers import to_dev
    x = to_dev(gs.make_inputs(1, 2, 128, 64, 64, seed=3))
    o, _ = gdr.chunk_fwd(x["q"], x["k"], x["v"], x["log_alpha"], x["b"], x["w"], x["S0"], out_dtype=torch.bfloat16)
    f, _ = gdr.rope_frequencies(64)
    q, k = gdr.rope(o, o, f)
    y, _ = gdr.attn_fwd(q, k, o, window=50)
    w = ref.attention(q.cpu().to(F64), k.cpu().to(F64), o.cpu().to(F64), 50)
    assert bool(((y.cpu().to(F64) - w["o"]).abs() <= w["o_tol"]).all())
