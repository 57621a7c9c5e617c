"""Integers beyond 31 bits at the binding: refused, not passed on as their low 32 bits."""

import pytest
import torch

from w4a8_quantized_moe_token_b200 import binding as B

WIDE = 1 << 32


def test_sizes_of_shapes_beyond_31_bits_are_0():
    assert B.w8a8_packed_bytes(1, 256, 512, 0) > 0
    for a in [(WIDE + 1, 256, 512, 0), (1, WIDE + 256, 512, 0), (1, 256, WIDE + 512, 0), (1, 256, 512, WIDE), (1, 256, 512, -WIDE)]:
        assert B.w8a8_packed_bytes(*a) == 0
    for a in [(WIDE + 4, 256, 512), (4, WIDE + 256, 512), (4, 256, WIDE + 512)]:
        assert B.w8a8_gemm_workspace_bytes(*a) == 0
    for i in range(5):
        a = [4, 8, 2, 256, 128]
        assert B.w8a8_moe_workspace_bytes(*a) > 0
        a[i] += WIDE
        assert B.w8a8_moe_workspace_bytes(*a) == 0


@pytest.mark.gpu
def test_calls_with_integers_beyond_31_bits_are_refused():
    x = torch.zeros((2, 8), device="cuda")
    ids, w = torch.zeros((2, 4), dtype=torch.int32, device="cuda"), torch.zeros((2, 4), device="cuda")
    for kw in [{"flags": WIDE}, {"flags": -WIDE}, {"n_group": WIDE + 1}, {"topk_group": WIDE + 1}, {"flags": -1}]:
        with pytest.raises(B.W4A8Error):
            B.w4a8_route_experts(x, 4, ids, w, **kw)
    weights = torch.zeros((1, 128, 128), dtype=torch.bfloat16, device="cuda")
    packed = B.empty_aligned(B.w8a8_packed_bytes(1, 128, 128, 0))
    with pytest.raises(B.W4A8Error):
        B.w8a8_pack_weights(weights, WIDE, packed)
    B.w8a8_pack_weights(weights, 0, packed)
    up = B.empty_aligned(B.w8a8_packed_bytes(1, 256, 128, 1))
    B.w8a8_pack_weights(torch.zeros((1, 256, 128), dtype=torch.bfloat16, device="cuda"), 1, up)
    t = torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    one, out = ids[:, :1].contiguous(), torch.empty_like(t)
    ws = B.empty_aligned(B.w8a8_moe_workspace_bytes(2, 1, 1, 128, 128))
    for E, F in [(1, 128 - WIDE), (1 - WIDE, 128), (1, WIDE + 128)]:
        with pytest.raises(B.W4A8Error):
            B.w8a8_moe_forward(up, packed, E, 128, F, t, one, w[:, :1].contiguous(), out, ws)
    B.w8a8_moe_forward(up, packed, 1, 128, 128, t, one, w[:, :1].contiguous(), out, ws)
    torch.cuda.synchronize()
