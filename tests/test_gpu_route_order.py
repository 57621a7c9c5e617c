"""w4a8_route_experts where 32 bits do not decide the order of the groups, and where logits lie
far apart."""

import pytest
import torch

from test_gpu_route_experts import check, logits_of

pytestmark = pytest.mark.gpu


def test_group_sums_that_cancel():
    # 64-bit sums 1.08279741 and 1.08279955; in fp32 the addends' roundings, 6e-5, turn them around
    x = torch.tensor([[1.37066650390625, -0.9182745814323425, -1.0656360387802124, 1.5614804029464722]])
    bias = torch.tensor([1000.0, -1000.0, 1000.0, -1000.0])
    rid, _ = check(x, 1, sigmoid=True, top2=True, bias=bias, n_group=2, topk_group=1)
    assert rid.tolist() == [[2]]


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,n_group,topk_group,k", [(4, 2, 1, 1), (16, 8, 3, 4), (64, 32, 9, 8), (384, 32, 8, 8)])
@pytest.mark.parametrize("size", [1.0, 30.0, 1000.0, 1e6])
def test_groups_under_large_biases_of_opposite_sign(sigmoid, E, n_group, topk_group, k, size):
    """Every group holds one bias of +b, one of -b and, behind both, others far below: the
    group's score is what the two largest scores leave of b - b.  The fp32 rounding of b + s
    is 2^-24 b, far above the differences between the groups."""
    T = 200
    g = torch.Generator().manual_seed(E + int(size))
    per = E // n_group
    bias = torch.full((n_group, per), -8 * size)
    b = size * (1 + torch.rand(n_group, generator=g))
    bias[:, 0], bias[:, 1] = b, -b
    x = logits_of(E, T, E, "fp32")
    check(x, k, sigmoid, top2=True, bias=bias.reshape(-1), n_group=n_group, topk_group=topk_group)
    check(x, k, sigmoid, top2=False, bias=bias.reshape(-1), n_group=n_group, topk_group=topk_group)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("std", [3.0, 10.0, 30.0])
@pytest.mark.parametrize("renorm", [False, True])
def test_weights_of_logits_far_below_the_largest(dtype, std, renorm):
    """The 8 chosen logits lie tens below the row's largest one: the difference from it, 30 or
    so, is rounded to 2^-19 by a 32-bit subtraction, and its exponential by as much."""
    for E in (12, 64, 384):
        check(logits_of(E, 300, E, dtype, std), 8, renorm=renorm)
        check(logits_of(E, 300, E, dtype, std), 8, sigmoid=True, renorm=renorm)
    x = logits_of(5, 300, 64, dtype, 1.0)
    x[:, :9] = logits_of(6, 300, 9, dtype, std) - 20.0
    bias = torch.zeros(64)
    bias[:9] = 5.0  # chosen for their bias, weighted without it
    check(x, 9, renorm=renorm, bias=bias)
    check(x, 9, sigmoid=True, renorm=renorm, bias=bias)
