"""GPU parity of the W8A8 epilogues on inputs whose INT32 sums and scales are exact in fp32, so
that the roundings left can be counted one by one, at scales far from 1, and at the largest
sums."""

import numpy as np
import pytest
import torch

from oracle import w4a8_oracle as O
from oracle import w8a8_oracle as W
from test_gpu_w8a8 import HALF_STEP, TINY, dev_bf16, pack, run_gemm
from w4a8_quantized_moe_token_b200 import binding as B
from w4a8_quantized_moe_token_b200 import synth

pytestmark = pytest.mark.gpu


def exact_rows(rng, n, K, step):
    """Integers times a power of two, the first one 127 steps: the scale is the step."""
    v = rng.integers(-127, 128, (n, K))
    v[:, 0] = 127 * rng.choice([-1, 1], n)
    return (v * step).astype(np.float32)


@pytest.mark.parametrize("T,F", [(40, 128), (200, 128), (256, 257), (600, 64)])
def test_swiglu_rounds_the_64_bit_value(T, F):
    """Sums below 2^24 and scales that are powers of two: gate g and up u are exact.  What is
    left of h = g / (1 + exp(-g)) * u in fp32: exp (2 ulp, 4 half steps of 2^-24, and it is at
    most the whole of 1 + exp), the sum, the quotient and the product, a half step each: 7
    half steps, and the rounding to bf16, half a step of 2^-8.  Below g = -87.3 exp(g) is
    subnormal, and 2 ulp of it are 2^-148."""
    H, pg, pu = 128, 2.0 ** -11, 2.0 ** 25
    rng = np.random.default_rng([T, F])
    x = exact_rows(rng, T, H, 1.0)
    up = np.concatenate([exact_rows(rng, F, H, pg), exact_rows(rng, F, H, pu)])
    (qx, sx), (qu, su) = W.quantize(x), W.quantize(up)
    assert (sx == 1.0).all() and (su[:F] == pg).all() and (su[F:] == pu).all()
    a = W.linear(qx, sx, qu, su)
    g, u = a[:, :F], a[:, F:]
    ref = g / (1.0 + np.exp(-g)) * u
    ws = B.empty_aligned(B.w8a8_moe_workspace_bytes(T, 1, 1, H, F))
    B.w8a8_moe_forward(pack(up, B.W4A8_LAYOUT_GATEUP), pack(np.zeros((H, F), np.float32)), 1, H, F, dev_bf16(x),
                       torch.zeros((T, 1), dtype=torch.int32, device="cuda"), torch.ones((T, 1), device="cuda"),
                       torch.empty((T, H), dtype=torch.bfloat16, device="cuda"), ws)
    torch.cuda.synchronize()
    R, Fp = B.w4a8_moe_rows_capacity(T, 1, 1), O.padded_k(F)
    h = synth.bf16_from_bits(B.w4a8_debug_dump(ws, T, 1, 1, H, F, "h").cpu().numpy().view(np.uint16)).reshape(R, Fp)[:T, :F]
    fp32 = 1.0001 * 7 * 2.0 ** -24 * np.abs(ref) + np.where(g < -87.3, 2.0 ** -148 * np.abs(g * u), 0.0)
    # the two ends of what fp32 may have held, rounded to bf16: h lies between them
    lo, hi = (O.round_to_bf16((ref + s * fp32).astype(np.float64)) for s in (-1, 1))
    bad = (h < lo) | (h > hi)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size}, at g = {g[bad][:5]}: {h[bad][:5]} and not {ref[bad][:5]}"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K", [(3, 64, 512), (5, 257, 300), (300, 514, 640), (40, 512, 4096)])
def test_gemm_scales_whose_product_fp32_does_not_hold(dtype, M, N, K):
    """A token's and a channel's scale of about 2^-67 multiply to less than fp32's smallest
    normal value, while the outputs, 2^-134 times sums of about 2^15, lie above it but for the
    smallest sums; in rows with a scale of 2^100 a sum of 0 stays 0 where the scales' product is
    infinite.  Roundings as counted elsewhere, and one more: below 2^-126 the last product is
    rounded to a multiple of 2^-149, by at most 2^-150."""
    rng = np.random.default_rng([M, N, K])
    qa, sa = O.quantize_act(synth.normal_bf16(rng, (M, K)))
    w = synth.normal_bf16(rng, (N, K), 2.0 ** -62)
    w[1::2] *= 2.0 ** 105  # even channels: scales of about 2^-67, odd ones: 2^38
    qa[2::3] = 0
    sa = (sa * 2.0 ** -61).astype(np.float32)
    sa[2::3] = 2.0 ** 100
    qw, sw = W.quantize(w)
    product = np.outer(sa.astype(np.float64), sw)
    assert (product[0, ::2] < 2.0 ** -126).all() and (product[2, 1::2] > 3.5e38).all()
    got = run_gemm(qa, sa, pack(w), N, K, dtype).double().numpy()
    ref = W.linear(qa, sa, qw, sw)
    bound = W.linear_error_bound(qa, sa, qw, sw) + 2.0 ** -150
    bound = bound + HALF_STEP[dtype] * (np.abs(ref) + bound) + TINY[dtype]
    assert np.all(np.abs(got - ref) <= bound), f"{int((np.abs(got - ref) > bound).sum())} of {ref.size} outside"


def test_gemm_largest_sums_with_codes_of_minus_128():
    # activation codes may be -128, weights' are within +-127: 127 * 128 * 2^17 < 2^31
    K, N = 131072, 3
    qa = np.full((2, K), -128, np.int8)
    qa[1, ::2] = 127
    w = np.ones((N, K), np.float32)
    w[1] = -1.0
    w[2, 1::2] = -1.0
    got = run_gemm(qa, None, pack(w), N, K, torch.int32).numpy()
    assert np.array_equal(got, W.int_sums(qa, W.quantize(w)[0]))
    assert np.abs(got).max() == 127 * 128 * K
