"""GPU parity: batches so long that a warp of the router takes several tokens and
computes their weights together.  Every row is compared with the 64-bit
definition, here in one pass over all tokens."""
import math

import pytest
import torch

import moe_ref
from quantized_matmul_03_b200 import binding as qb
from test_gpu_moe_route import W_TOL, bias_of, logits_of


def route_all(logits, top_k, score="softmax", bias=None, n_groups=1, topk_groups=1, group_top=1, renormalize=True,
              scale=1.0):
    """moe_ref.route over all tokens at once (finite, -inf and NaN logits)."""
    l = logits.double()
    T, E = l.shape
    nan = torch.isnan(l)
    if score == "sigmoid":
        s = torch.sigmoid(l)
    else:
        m = l.masked_fill(nan, -math.inf).amax(-1, keepdim=True)
        ex = torch.where(nan | (m == -math.inf), 0.0, torch.exp(l - m))
        s = ex / ex.sum(-1, keepdim=True).clamp_min(1e-300)
    sel = s if bias is None else s + bias.double()
    key = l if bias is None else sel
    low = -1e308                                   # NaN: below every finite key and -inf, above a dropped group
    # (-inf keys lie below `low` otherwise)
    key = torch.where(nan, low, key.clamp_min(-1e307))
    if n_groups > 1:
        gs = torch.where(nan, math.nan, sel).view(T, n_groups, -1)
        best = gs.masked_fill(torch.isnan(gs), -math.inf).sort(-1, descending=True)[0][..., :group_top].sum(-1)
        rank = best.sort(dim=-1, descending=True, stable=True)[1].argsort(-1)
        key = key.masked_fill((rank >= topk_groups).repeat_interleave(E // n_groups, 1), -math.inf)
    idx = key.sort(dim=-1, descending=True, stable=True)[1][:, :top_k]
    w = s.gather(1, idx)
    if renormalize:
        if score == "softmax":
            lc = l.gather(1, idx)
            m = lc.masked_fill(torch.isnan(lc), -math.inf).amax(-1, keepdim=True)
            w = torch.where(torch.isnan(lc) | (m == -math.inf), 0.0, torch.exp(lc - m))
        z = w.sum(-1, keepdim=True)
        w = torch.where(z > 0, w / z.clamp_min(1e-300), 0.0)
    w = torch.where(nan.any(-1, keepdim=True), math.nan, w * scale)
    return idx.to(torch.int32), w


CALLS = [
    dict(k=1, E=8),
    dict(k=3, E=60),
    dict(k=3, E=60, renormalize=False, scale=1.5),
    dict(k=8, E=64, score="sigmoid"),
    dict(k=1, E=33, score="sigmoid", renormalize=False),
    dict(k=5, E=40, bias=0.1),
    dict(k=5, E=40, bias=0.1, renormalize=False),
    dict(k=4, E=64, score="sigmoid", bias=0.1, n_groups=8, topk_groups=3, group_top=2, scale=2.5),
    dict(k=2, E=60, n_groups=4, topk_groups=2, renormalize=False),
]


def special(lg):
    """Masked experts, an empty token and a NaN token beside ordinary ones."""
    T, E = lg.shape
    lg[1, : E // 2] = -math.inf
    lg[2] = -math.inf
    lg[T // 2, E // 3] = math.nan
    lg[T - 2] = -math.inf
    lg[T - 1, E - 1] = 30.0
    return lg


def call_args(c):
    kw = {n: v for n, v in c.items() if n not in ("k", "E")}
    if "bias" in kw:
        kw["bias"] = bias_of(c["E"], 7, kw["bias"])
    return kw


@pytest.mark.parametrize("c", CALLS)
def test_the_one_pass_definition_is_the_one_of_single_tokens(c):
    lg = special(logits_of(41, c["E"], 5))
    kw = call_args(c)
    ri, rw = moe_ref.route(lg, c["k"], **kw)
    i, w = route_all(lg, c["k"], **kw)
    assert torch.equal(i, ri)
    assert torch.equal(torch.isnan(w), torch.isnan(rw))
    ok = ~torch.isnan(rw)
    assert bool(((w - rw).abs()[ok] <= 1e-14 * rw.abs()[ok] + 1e-300).all())


# 148 SMs x 32 warps: a warp takes 2, 4, 8 and 32 tokens from 9472, 18944, 37888 and 151552 on
# (if that many slots fit its lanes).
@pytest.mark.gpu
@pytest.mark.parametrize("T", [9473, 20001, 40003, 151555])
@pytest.mark.parametrize("c", CALLS)
def test_every_token(T, c):
    lg = special(logits_of(T, c["E"], T, torch.float32 if T != 20001 else torch.bfloat16)).cuda()
    kw = call_args(c)
    if "bias" in kw:
        kw["bias"] = kw["bias"].cuda()
    ri, rw = route_all(lg, c["k"], **kw)
    oi = torch.full((T + 1, c["k"]), -7, dtype=torch.int32, device="cuda")
    ow = torch.full((T + 1, c["k"]), -7.0, device="cuda")
    i, w = qb.qmm_moe_route(lg, c["k"], out=(oi[:T], ow[:T]), **kw)
    assert bool((oi[T] == -7).all()) and bool((ow[T] == -7).all())
    assert torch.equal(i, ri)
    w = w.double()
    assert torch.equal(torch.isnan(w), torch.isnan(rw))
    ok = ~torch.isnan(rw)
    assert bool(((w - rw).abs()[ok] <= W_TOL * rw.abs()[ok] + 1e-37).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [9473, 40003])
def test_keys_that_fp32_cannot_tell_apart_among_others(T):
    """Some of a warp's tokens are ordered again in 64 bits."""
    g = torch.Generator().manual_seed(T)
    E = 64
    base = torch.randn((E,), generator=g) * 1e-3
    lg = torch.randn((T, E), generator=g)
    lg[::3] = base + torch.randn((len(lg[::3]), E), generator=g) * 1e-7
    b = (0.75 - torch.sigmoid(base.double())).float()
    for kw in (dict(), dict(n_groups=8, topk_groups=3, group_top=2)):
        ri, _ = route_all(lg, 4, score="sigmoid", bias=b, **kw)
        i, _ = qb.qmm_moe_route(lg.cuda(), 4, score="sigmoid", bias=b.cuda(), **kw)
        assert torch.equal(i.cpu(), ri)
