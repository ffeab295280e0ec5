"""GPU parity: NaN logits under a softmax whose scores choose (with a bias, with
groups).  A NaN logit ranks below everything and leaves the other experts' scores
as they are; the token's weights are NaN."""
import math

import pytest
import torch

from test_gpu_moe_route import bias_of, check, logits_of

pytestmark = pytest.mark.gpu


def with_nan(T, E, seed):
    lg = logits_of(T, E, seed)
    lg[0, 0] = math.nan                     # would be the lowest index of a tie
    lg[1, [1, 2, E - 1]] = math.nan
    lg[2, ::2] = math.nan
    lg[3] = math.nan                        # nothing but NaN: the lowest indices
    lg[4] = -math.inf
    lg[4, 1] = math.nan                     # a NaN beside nothing
    lg[5, :E // 2] = -math.inf
    lg[5, E // 2] = math.nan
    lg[6] = math.nan
    lg[6, E - 2] = 0.5                      # one expert is left
    return lg                               # (the last row has none)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(8, 3), (33, 5), (300, 8)])
def test_with_a_bias(score, E, k):
    lg = with_nan(8, E, E)
    check(lg, k, score=score, bias=bias_of(E, 1))
    check(lg, k, score=score, bias=bias_of(E, 1), renormalize=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,tg,gt,k", [(64, 8, 3, 2, 8), (60, 4, 2, 1, 6), (33, 3, 2, 2, 5)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_with_groups(score, E, G, tg, gt, k, with_bias):
    lg = with_nan(8, E, E + 1)
    b = bias_of(E, 2) if with_bias else None
    check(lg, k, score=score, bias=b, n_groups=G, topk_groups=tg, group_top=gt)
    check(lg.half(), k, score=score, bias=b, n_groups=G, topk_groups=tg, group_top=gt)


def test_reordered_in_64_bits():
    """Keys that fp32 cannot tell apart, with a NaN among them."""
    g = torch.Generator().manual_seed(3)
    lg = torch.randn((16, 64), generator=g) * 1e-3
    b = (0.1 - torch.softmax(lg[0].double(), -1)).float()
    lg[1:] = lg[0] + torch.randn((15, 64), generator=g) * 1e-7
    lg[::2, 11] = math.nan
    check(lg, 8, bias=b)
    check(lg, 8, bias=b, n_groups=8, topk_groups=3, group_top=2)
