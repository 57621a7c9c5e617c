"""GPU parity of w4a8_route_experts against the 64-bit oracle: ids equal, weights within
the roundings of the final fp32 value (the scores are 64-bit: half a step, 2^-24, plus the
few 1e-16 of the exponentials)."""

import numpy as np
import pytest
import torch

from oracle import w8a8_oracle as W
from w4a8_quantized_moe_token_b200 import binding as B

pytestmark = pytest.mark.gpu

# the weights are fp32 with 32-bit scores allowed: a few operations on top of the half step
# (exp 2 ulp of 2^-23, sum, division, renormalisation, factor: below 16 half steps)
W_TOL = 16 * 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def check(logits, k, sigmoid=False, renorm=False, top2=False, bias=None, n_group=1, topk_group=1, scale=1.0):
    T, E = logits.shape
    ids = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, dtype=torch.float32, device="cuda")
    flags = B.W4A8_ROUTE_SIGMOID * sigmoid | B.W4A8_ROUTE_RENORM * renorm | B.W4A8_ROUTE_GROUP_TOP2 * top2
    b = None if bias is None else bias.cuda()
    B.w4a8_route_experts(logits.cuda(), k, ids[:T], w[:T], flags, b, n_group, topk_group, scale)
    torch.cuda.synchronize()
    rid, rw = W.route_experts(logits.double().numpy(), k, sigmoid, renorm, top2,
                              None if bias is None else bias.double().numpy(), n_group, topk_group, scale)
    assert np.array_equal(ids[:T].cpu().numpy(), rid)
    got = w[:T].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - rw) <= W_TOL * np.abs(rw) + 1e-37), np.abs(got - rw).max()
    assert (ids[T] == -7).all() and (w[T] == -7).all()  # rows behind the last token stay
    return rid, rw


def logits_of(seed, T, E, dtype, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E), generator=g) * std).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,E,k,n_group,topk_group", [
    (1, 1, 1, 1, 1), (1, 384, 8, 8, 4), (3, 7, 7, 1, 1), (33, 64, 6, 1, 1), (65, 160, 6, 8, 3), (17, 256, 8, 8, 4),
    (9, 1024, 32, 32, 5), (5, 1000, 10, 4, 2), (130, 31, 5, 31, 6), (64, 33, 4, 3, 2), (7, 60, 3, 30, 2), (4, 600, 9, 1, 1),
])
@pytest.mark.parametrize("sigmoid,with_bias,top2", [(False, False, False), (True, True, True), (False, True, False),
                                                    (True, False, True)])
def test_matches_oracle(dtype, T, E, k, n_group, topk_group, sigmoid, with_bias, top2):
    seed = T * 1000 + E + k
    bias = torch.randn(E, generator=torch.Generator().manual_seed(seed)) * 0.05 if with_bias else None
    check(logits_of(seed, T, E, dtype), k, sigmoid, renorm=bool(seed & 1), top2=top2, bias=bias, n_group=n_group,
          topk_group=topk_group, scale=2.5)


def test_large_batch():
    check(logits_of(1, 3001, 96, "bf16"), 8, sigmoid=True, renorm=True, top2=True,
          bias=torch.randn(96, generator=torch.Generator().manual_seed(2)) * 0.05, n_group=8, topk_group=4, scale=2.5)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
def test_ties_go_to_the_lower_id(sigmoid, with_bias):
    # few distinct logits and a constant bias: most comparisons are ties
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-2, 3, (50, 128), generator=g).to(torch.bfloat16)
    bias = torch.full((128,), 0.25) if with_bias else None
    check(x, 10, sigmoid, renorm=True, bias=bias)
    check(x, 10, sigmoid, top2=True, bias=bias, n_group=16, topk_group=5)
    check(-0.0 * x.abs(), 4, sigmoid, bias=bias)  # zeros of both signs are equal
    x[:, ::2] = -0.0
    x[:, 1::2] = 0.0
    check(x, 6, sigmoid, bias=bias)


def test_order_below_fp32_resolution():
    # biases that undo the scores up to 2^-30: fp32 sums would tie or turn around
    E = 64
    x = logits_of(11, 40, E, "fp32", std=0.5)
    x[:] = x[0]
    s = 1.0 / (1.0 + np.exp(-x[0].double().numpy()))
    bias = torch.from_numpy((0.75 - s).astype(np.float32))
    for t in range(40):  # tokens move one expert's logit by a few ulps
        e = (7 * t) % E
        x[t, e] = torch.nextafter(x[t, e], torch.tensor(torch.inf))
    check(x, 8, sigmoid=True, renorm=True, bias=bias)
    check(x, 8, sigmoid=True, renorm=True, bias=bias, top2=True, n_group=8, topk_group=3)
    # softmax: many experts with nearly the same probability
    y = 1e-6 * logits_of(12, 60, E, "fp32")
    check(y, 8, renorm=True, bias=torch.full((E,), 0.5))
    check(y, 8, top2=True, n_group=16, topk_group=5)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("grouped", [False, True])
def test_masked_experts_and_empty_rows(dtype, sigmoid, grouped):
    T, E, k = 40, 48, 6
    x = logits_of(21, T, E, dtype)
    g = torch.Generator().manual_seed(22)
    x[torch.rand((T, E), generator=g) < 0.6] = -torch.inf
    x[0] = -torch.inf               # nothing left
    x[1] = torch.nan
    x[2] = -torch.inf
    x[2, 40] = 0.5                  # one expert left
    x[3, 5] = torch.nan
    x[4] = torch.finfo(DT[dtype]).min   # the type's lowest value is a logit like any other
    x[5, 3:9] = torch.finfo(DT[dtype]).min
    x[6, 7] = torch.inf
    x[7, 7] = x[7, 30] = torch.inf
    x[8] = torch.finfo(DT[dtype]).max
    kw = dict(n_group=8, topk_group=3) if grouped else {}
    for bias in (None, torch.randn(E, generator=g) * 0.1):
        for top2 in (False, True):
            for renorm in (False, True):
                rid, rw = check(x, k, sigmoid, renorm, top2, bias, **kw)
                assert (rw[0] == 0).all() and (rw[1] == 0).all()
    bias = torch.randn(E, generator=g) * 0.1
    bias[::3] = -torch.inf          # experts taken out of service
    bias[7] = torch.nan
    bias[8] = torch.inf             # and one forced
    check(x, k, sigmoid, True, grouped, bias, **kw)


def test_extreme_logits_and_scales():
    x = torch.tensor([[-1e38, 1e38, 3.4e38, -3.4e38, 0.0, 90.0, -90.0, 1e-40]])
    for sigmoid in (False, True):
        check(x, 5, sigmoid)
        check(x, 5, sigmoid, renorm=True, scale=-3.0)
        check(x, 5, sigmoid, bias=torch.linspace(-1e30, 1e30, 8), scale=0.0)


def test_renormalised_weights_of_tiny_scores():
    # sigmoid of -100 is 4e-44 and the softmax's share of a masked-off top 1e-44: the ratios hold
    x = logits_of(41, 20, 32, "fp32")
    check(x - 100.0, 5, sigmoid=True, renorm=True)
    check(x - 300.0, 5, sigmoid=True, renorm=True)
    x[:, 9] = 100.0
    bias = torch.zeros(32)
    bias[9] = -torch.inf
    check(x, 5, renorm=True, bias=bias)


def test_empty_batch_and_refused_tensors():
    ids = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    w = torch.empty((0, 4), dtype=torch.float32, device="cuda")
    B.w4a8_route_experts(torch.empty((0, 8), dtype=torch.bfloat16, device="cuda"), 4, ids, w)
    x = torch.zeros((2, 8), device="cuda")
    ids, w = torch.empty((2, 4), dtype=torch.int32, device="cuda"), torch.empty((2, 4), device="cuda")
    bad = [
        (x.double(), ids, w, {}), (x[:, ::2], ids, w, {}), (x, ids[:1], w, {}), (x, ids, w.half(), {}), (x.cpu(), ids, w, {}),
        (x, ids.long(), w, {}), (x, ids, w, {"bias": torch.zeros(7, device="cuda")}),
        (x, ids, w, {"bias": torch.zeros(8, device="cuda", dtype=torch.bfloat16)}), (x, ids, w, {"n_group": 3}),
        (x, ids, w, {"flags": 64}),
    ]
    for a, i, ww, kw in bad:
        with pytest.raises(B.W4A8Error):
            B.w4a8_route_experts(a, 4, i, ww, **kw)


def test_other_stream_and_graph_replay():
    T, E, k = 37, 256, 8
    x = logits_of(31, T, E, "bf16").cuda()
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    bias = torch.zeros(E, device="cuda")

    def call():
        B.w4a8_route_experts(x, k, ids, w, B.W4A8_ROUTE_SIGMOID | B.W4A8_ROUTE_RENORM | B.W4A8_ROUTE_GROUP_TOP2, bias, 8, 4)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        call()
    torch.cuda.current_stream().wait_stream(st)
    with torch.cuda.graph(graph):
        call()
    for seed in (32, 33):
        x.copy_(logits_of(seed, T, E, "bf16"))
        bias.copy_(torch.randn(E, generator=torch.Generator().manual_seed(seed)) * 0.1)
        ids.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        rid, rw = W.route_experts(x.double().cpu().numpy(), k, True, True, True, bias.double().cpu().numpy(), 8, 4)
        assert np.array_equal(ids.cpu().numpy(), rid)
        assert np.all(np.abs(w.cpu().numpy() - rw) <= W_TOL * rw)
