"""NaN and infinities in the W8A8 scheme: a row that holds one has a NaN or an infinite scale
and zero codes, so that every output it enters is NaN, and no other output changes."""

import numpy as np
import pytest
import torch

from helpers import untile_act
from oracle import w8a8_oracle as W
from test_gpu_w8a8 import Layer, dev_bf16, pack, unpack
from w4a8_quantized_moe_token_b200 import binding as B
from w4a8_quantized_moe_token_b200 import synth

pytestmark = pytest.mark.gpu


def forward(L, x, up=None, dn=None):
    out = torch.full((L.T, L.H), 7.0, dtype=torch.bfloat16, device="cuda")
    x = x if isinstance(x, torch.Tensor) else dev_bf16(x)
    B.w8a8_moe_forward(up if up is not None else L.packed[0], dn if dn is not None else L.packed[1], L.E, L.H, L.F, x,
                       torch.from_numpy(L.ids).cuda(), torch.from_numpy(L.w).cuda(), out, L.ws)
    torch.cuda.synchronize()
    assert B.w4a8_last_device_error(L.ws) == 0
    return out.float().cpu().numpy()


def dump(L, what, dt):
    return B.w4a8_debug_dump(L.ws, L.T, L.E, L.k, L.H, L.F, what).cpu().numpy().view(dt)


# every kernel that quantises token rows or rows of h: few slots (T * k <= 2048), a warp and a
# CTA per token; rows of h by a warp (F <= 512, <= 1024, <= 2048 with many rows) and by a CTA
# (F > 1024 with few rows, F > 2048); odd lengths; rows longer than the registers hold
SHAPES = [(1, 2, 2, 128, 64), (24, 3, 2, 257, 100), (40, 3, 2, 8200, 16), (1100, 3, 2, 256, 40), (1100, 3, 2, 515, 600),
          (1100, 3, 2, 1100, 40), (1100, 2, 2, 8200, 8), (40, 2, 2, 128, 1100), (1500, 2, 2, 72, 1100), (1300, 2, 2, 72, 2041),
          (20, 2, 2, 64, 2100), (6, 2, 1, 40, 8300)]


@pytest.mark.parametrize("T,E,k,H,F", SHAPES)
def test_tokens_with_nan_or_infinity_are_nan(T, E, k, H, F):
    L = Layer(T, E, k, H, F, "uniform", seed=T + H + F)
    clean = forward(L, L.x)
    assert np.isfinite(clean).all()
    x = dev_bf16(L.x)
    values = [torch.nan, torch.inf, -torch.inf, -torch.nan]
    rows = list(range(0, T, 5))
    for i, t in enumerate(rows):  # one value at a varying place: first, last, inside
        x[t, (0, H - 1, H // 2, min(H - 1, 17))[i // 4 % 4]] = values[i % 4]
    if T > 3:
        x[3] = torch.nan              # nothing else in the row
    if T > 8:
        x[8, :2] = torch.tensor([torch.inf, torch.nan])
    hit = np.zeros(T, bool)
    hit[rows + [t for t in (3, 8) if t < T and (t == 3 or T > 8)]] = True
    got = forward(L, x)
    assert np.isnan(got[hit]).all()
    assert np.array_equal(got[~hit], clean[~hit])
    # the scales: NaN wins over infinity
    slot = np.arange(T * k)
    row, amax = dump(L, "inv", np.int32), x.float().abs().cpu().numpy().max(axis=1)[slot // k]
    s1 = dump(L, "s1", np.float32)[row]
    assert np.array_equal(np.isnan(s1), np.isnan(amax)) and np.array_equal(np.isinf(s1), np.isinf(amax))
    act = untile_act(dump(L, "act1", np.int8), B.w4a8_moe_rows_capacity(T, E, k), B.padded_k(H))[row]
    assert not act[~np.isfinite(amax)].any()


@pytest.mark.parametrize("T,E,k,H,F", SHAPES)
def test_h_beyond_bf16_is_nan(T, E, k, H, F):
    # gate and up of about 2^70 each: their product passes bf16's largest value, h is infinite
    L = Layer(T, E, k, H, F, "uniform", seed=T + H + F)
    clean = forward(L, L.x)
    up = L.up.copy()
    up[0] *= 2.0 ** 80
    got = forward(L, L.x, up=pack(up, B.W4A8_LAYOUT_GATEUP))
    h = synth.bf16_from_bits(dump(L, "h", np.uint16)).reshape(-1, B.padded_k(F))[dump(L, "inv", np.int32), :F]
    wide = ~np.isfinite(h).all(axis=1).reshape(T, k)
    assert wide[L.ids == 0].any() and not wide[L.ids != 0].any()
    assert np.isnan(got[wide.any(axis=1)]).all()
    other = ~(L.ids == 0).any(axis=1)
    assert np.array_equal(got[other], clean[other])


@pytest.mark.parametrize("E,N,K,layout", [(1, 1, 1, 0), (2, 130, 300, 0), (2, 258, 1032, 1), (1, 140, 8300, 0)])
def test_packed_channels_with_nan_or_infinity(E, N, K, layout):
    rng = np.random.default_rng(N + K)
    w = dev_bf16(synth.normal_bf16(rng, (E, N, K), 0.02))
    w[0, 0, 0] = torch.nan
    if N > 4:
        w[0, 2, K - 1], w[E - 1, 3, K // 2], w[0, 4] = torch.inf, -torch.inf, torch.nan
        w[0, 5, :2] = torch.tensor([torch.inf, torch.nan])
    codes = torch.full((E, N, B.padded_k(K)), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((E, N), 99.0, device="cuda")
    packed = B.empty_aligned(B.w8a8_packed_bytes(E, N, K, layout))
    B.w8a8_pack_weights(w, layout, packed, codes=codes, scale=scale)
    got_q, got_s = unpack(packed.cpu().numpy(), E, N, K, layout)
    wf = w.float().cpu().numpy()
    amax = np.abs(wf).max(axis=2)
    fine = np.isfinite(amax)
    for q, s in [(codes.cpu().numpy(), scale.cpu().numpy()), (got_q, got_s)]:
        assert np.array_equal(np.isnan(s), np.isnan(amax)) and np.array_equal(np.isinf(s), np.isinf(amax))
        assert not q[~fine].any()
        for e in range(E):
            if fine[e].any():
                rq, rs = W.quantize(wf[e][fine[e]])
                assert np.array_equal(q[e][fine[e]], rq) and np.array_equal(s[e][fine[e]], rs)


@pytest.mark.parametrize("M,N", [(3, 200), (60, 4096), (300, 514)])
def test_gemm_columns_of_nan_weights_and_rows_of_nan_scales(M, N):
    K = 256
    rng = np.random.default_rng([M, N])
    qa = torch.from_numpy(rng.integers(-127, 128, (M, K)).astype(np.int8)).cuda()
    sa = torch.rand(M, device="cuda") + 0.1
    w = dev_bf16(synth.normal_bf16(rng, (1, N, K), 0.02))
    ws = B.empty_aligned(B.w8a8_gemm_workspace_bytes(M, N, K))

    def run(dtype):
        packed = B.empty_aligned(B.w8a8_packed_bytes(1, N, K, 0))
        B.w8a8_pack_weights(w, 0, packed)
        y = torch.empty((M, N), dtype=dtype, device="cuda")
        B.w8a8_gemm(qa, sa, packed, N, K, y, ws)
        torch.cuda.synchronize()
        return y.float().cpu().numpy()

    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        w[0, 7, 11], w[0, N - 1, 0] = 0.25, 0.25
        clean = run(dtype)
        w[0, 7, 11], w[0, N - 1, 0] = torch.nan, -torch.inf
        col = np.zeros(N, bool)
        col[[7, N - 1]] = True
        got = run(dtype)
        assert np.isnan(got[:, col]).all() and np.array_equal(got[:, ~col], clean[:, ~col])
        sa[1] = torch.nan
        got = run(dtype)
        assert np.isnan(got[1]).all()
        sa[1] = 0.5


@pytest.mark.parametrize("T", [20, 1100])
def test_layer_with_nan_weights(T):
    E, k, H, F = 4, 2, 200, 70
    L = Layer(T, E, k, H, F, "uniform", seed=T)
    clean = forward(L, L.x)
    up, dn = dev_bf16(L.up), dev_bf16(L.dn)
    up[1, 5, 3] = torch.nan         # a gate channel of expert 1: its h has a NaN in every row
    up[2, F + 6, 0] = torch.inf     # an up channel of expert 2
    dn[3, 9, 2] = torch.nan         # one output of expert 3
    pu, pd = (B.empty_aligned(B.w8a8_packed_bytes(*v.shape, lay)) for v, lay in ((up, 1), (dn, 0)))
    B.w8a8_pack_weights(up, 1, pu)
    B.w8a8_pack_weights(dn, 0, pd)
    got = forward(L, L.x, pu, pd)
    whole = np.isin(L.ids, [1, 2]).any(axis=1)
    assert np.isnan(got[whole]).all()
    want = clean[~whole].copy()
    want[(L.ids[~whole] == 3).any(axis=1), 9] = np.nan
    assert np.array_equal(got[~whole], want, equal_nan=True)
