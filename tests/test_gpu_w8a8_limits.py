"""The W8A8 layer where its choices of kernels change over, with many experts and few rows
each: the most slots that one kernel permutes and quantises, and one more token."""

import functools

import pytest

import test_gpu_w8a8
from helpers import assert_bf16_adjacent
from test_gpu_w8a8 import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k,routing", [(256, 384, 8, "zipf"), (257, 384, 8, "zipf"), (2048, 1024, 1, "uniform"), (64, 1024, 32, "uniform"),
                                           (2049, 1024, 1, "zipf")])
def test_moe_of_many_experts(T, E, k, routing, monkeypatch):
    # An expert may have one row, of 40 values of h.  fp32 (some 14 roundings of 2^-24 from sums
    # to h) puts a value on the other side of a bf16 boundary, 2^-8 apart, about once in 2^16 / 14
    # = 4700: a handful of the up to 82240 values, each the one in its row.
    monkeypatch.setattr(test_gpu_w8a8, "assert_bf16_adjacent", functools.partial(assert_bf16_adjacent, max_frac=1 / 40))
    Layer(T, E, k, 136, 40, routing, seed=T + E).run()
