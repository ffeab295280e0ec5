"""GPU parity: qmm_moe_route against the float64 definition.

Indices must be equal: the kernel's order is that of fp64 keys.  Weights come
from fp64 (softmax sums over all experts from fp32 terms) and are rounded to
fp32 once: half a step 2^-24, plus 2^-22 for expf's few units in each term of
an unnormalised softmax's sum."""
import math

import pytest
import torch

import moe_ref
from quantized_matmul_03_b200 import binding as qb

pytestmark = pytest.mark.gpu

W_TOL = 2.0 ** -24 + 2.0 ** -22


def check(logits, k, **kw):
    ri, rw = moe_ref.route(logits, k, **kw)
    if kw.get("bias") is not None:
        kw["bias"] = kw["bias"].cuda()
    i, w = qb.qmm_moe_route(logits.cuda(), k, **kw)
    assert i.dtype == torch.int32 and w.dtype == torch.float32
    assert torch.equal(i.cpu(), ri)
    w = w.cpu().double()
    assert torch.equal(torch.isnan(w), torch.isnan(rw))
    ok = ~torch.isnan(rw)
    assert bool(((w - rw).abs()[ok] <= W_TOL * rw.abs()[ok] + 1e-37).all())
    return i, w


def logits_of(T, E, seed, dtype=torch.float32, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E), generator=g) * std).to(dtype)


def bias_of(E, seed, std=0.1):
    return torch.randn((E,), generator=torch.Generator().manual_seed(seed)) * std


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 7, 7), (65, 60, 6), (9, 257, 8), (5, 1000, 32)])
def test_plain_routes(dtype, score, T, E, k):
    lg = logits_of(T, E, T + E, dtype)
    check(lg, k, score=score)
    check(lg, k, score=score, renormalize=False, scale=2.5)
    check(lg, k, score=score, bias=bias_of(E, E), scale=-1.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,tg,gt,k", [(256, 8, 4, 2, 8), (160, 8, 3, 1, 6), (32, 32, 8, 2, 8), (60, 4, 1, 2, 15),
                                         (1024, 32, 32, 1, 4), (6, 2, 1, 2, 3)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_groups(score, E, G, tg, gt, k, with_bias):
    lg = logits_of(33, E, E + G, torch.float32)
    b = bias_of(E, 3) if with_bias else None
    check(lg, k, score=score, bias=b, n_groups=G, topk_groups=tg, group_top=gt)
    check(lg.to(torch.bfloat16), k, score=score, bias=b, n_groups=G, topk_groups=tg, group_top=gt,
          renormalize=False)


@pytest.mark.parametrize("with_bias", [False, True])
def test_equal_logits_go_to_the_lower_index(with_bias):
    lg = torch.zeros((4, 40))
    lg[1, 5::7] = 1.0
    lg[2, 3] = -0.0
    lg[3, 39] = 2.0
    b = torch.zeros(40) if with_bias else None
    i, _ = check(lg, 6, score="sigmoid", bias=b)
    assert i[0].tolist() == [0, 1, 2, 3, 4, 5]
    check(lg, 6, bias=b, n_groups=4, topk_groups=2, group_top=2)


def test_keys_that_fp32_cannot_tell_apart():
    """Scores plus bias that differ by less than fp32 resolves: the order has to
    be that of the 64-bit keys, inside groups, across the last place and between
    groups."""
    g = torch.Generator().manual_seed(5)
    T, E = 64, 64
    lg = torch.randn((T, E), generator=g) * 1e-3
    target = 0.75
    b = (target - torch.sigmoid(lg[0].double())).float()          # token 0's keys all near 0.75
    lg[1:] = lg[0] + torch.randn((T - 1, E), generator=g) * 1e-7
    check(lg, 8, score="sigmoid", bias=b)
    check(lg, 8, score="sigmoid", bias=b, n_groups=8, topk_groups=3, group_top=2)
    z = torch.softmax(lg[0].double(), -1)
    b = (0.1 - z).float()
    check(lg, 8, score="softmax", bias=b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts_and_tokens(score):
    inf = math.inf
    lg = logits_of(6, 33, 9)
    lg[0, ::2] = -inf                       # half of the experts masked
    lg[1] = -inf                            # nothing is left
    lg[2] = -inf
    lg[2, 17] = 0.25                        # one is left
    lg[3] = torch.finfo(torch.float32).min  # masked by the type's lowest value
    lg[3, 4] = 1.0
    lg[4, 8] = math.nan
    lg[5, 30] = 80.0
    check(lg, 5, score=score)
    check(lg, 5, score=score, renormalize=False)
    b = bias_of(33, 1)
    b[3] = -inf
    b[7] = -inf
    check(lg[[0, 5]], 5, score=score, bias=b)
    check(lg[[0, 5]], 32, score=score, bias=b)   # all but one: masked experts among them
    if score == "softmax":                  # scores so far below that fp32 loses them: the bias decides
        lg = logits_of(2, 33, 10)
        lg[:, 0] = 200.0
        b = torch.zeros(33)
        b[0] = -inf
        check(lg, 4, score=score, bias=b)


def test_plus_infinity_takes_the_softmax():
    lg = logits_of(2, 16, 11)
    lg[0, 5] = math.inf
    lg[1, [2, 9]] = math.inf
    i, w = qb.qmm_moe_route(lg.cuda(), 3, renormalize=False)
    assert i[0, 0].item() == 5 and i[1, :2].tolist() == [2, 9]
    assert w[0].tolist() == [1.0, 0.0, 0.0] and w[1].tolist() == [0.5, 0.5, 0.0]


def test_empty_and_shapes():
    i, w = qb.qmm_moe_route(torch.empty((0, 8), device="cuda"), 2)
    assert i.shape == (0, 2) and w.shape == (0, 2)
    lg = logits_of(12, 16, 12)
    i, w = qb.qmm_moe_route(lg.reshape(3, 4, 16).cuda(), 4)
    assert i.shape == (3, 4, 4)
    ri, _ = moe_ref.route(lg, 4)
    assert torch.equal(i.reshape(12, 4).cpu(), ri)


def test_rows_behind_the_last_token_stay():
    lg = logits_of(5, 61, 13, torch.bfloat16).cuda()[1:4]       # rows of 122 bytes, odd start
    oi = torch.full((4, 6), -7, dtype=torch.int32, device="cuda")
    ow = torch.full((4, 6), -7.0, device="cuda")
    qb.qmm_moe_route(lg, 6, out=(oi[:3], ow[:3]))
    ri, _ = moe_ref.route(lg.cpu(), 6)
    assert torch.equal(oi[:3].cpu(), ri)
    assert bool((oi[3] == -7).all()) and bool((ow[3] == -7).all())


def test_long_batch_and_graph_on_another_stream():
    lg = logits_of(5000, 64, 14).cuda()
    ref = qb.qmm_moe_route(lg, 8, score="sigmoid")
    out = (torch.empty_like(ref[0]), torch.empty_like(ref[1]))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        qb.qmm_moe_route(lg, 8, score="sigmoid", out=out)
    for _ in range(2):
        out[0].zero_()
        out[1].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
    ri, _ = moe_ref.route(lg[:50].cpu(), 8, score="sigmoid")
    assert torch.equal(ref[0][:50].cpu(), ri)
