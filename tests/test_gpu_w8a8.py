"""GPU parity of the W8A8 scheme against the oracle: packed codes and scales bit-exact, the
INT32 sums exact, the dense outputs within the counted roundings, the MoE layer within the
layer tolerance, and the operators together as a serving step uses them."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from helpers import assert_bf16_adjacent, untile_act
from oracle import w4a8_oracle as O
from oracle import w8a8_oracle as W
from w4a8_quantized_moe_token_b200 import binding as B
from w4a8_quantized_moe_token_b200 import synth

pytestmark = pytest.mark.gpu

SHORT_WAIT = 2_000_000  # clock cycles, about 1 ms
HALF_STEP = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # half the smallest step


def dev_bf16(a):
    return torch.from_numpy(synth.bf16_bits(np.ascontiguousarray(a, dtype=np.float32)).view(np.int16)).view(torch.bfloat16).cuda()


def pack(w, layout=0, **kw):
    w = w if w.ndim == 3 else w[None]
    packed = B.empty_aligned(B.w8a8_packed_bytes(*w.shape, layout))
    B.w8a8_pack_weights(dev_bf16(w), layout, packed, **kw)
    return packed


def unpack(buf, E, N, K, layout):
    """Tiled packed buffer -> codes int8 [E][N][Kp], scale float32 [E][N]; checks the padding."""
    NT = -(-(N // 2) // 64) if layout == 1 else -(-N // 128)
    G = -(-K // 128)
    a = 256 + E * NT * 512
    scale = buf[256:a].copy().view(np.float32).reshape(E, NT * 128)
    blocks = buf[a:a + E * NT * G * 16384].view(np.int8).reshape(E, NT, G, 128, 8, 16)
    rows = np.zeros((E, NT, 128, G, 8, 16), np.int8)
    r = np.arange(128)
    for c in range(8):
        rows[:, :, :, :, c] = blocks[:, :, :, r, c ^ (r & 7)].transpose(0, 1, 3, 2, 4)
    rows = rows.reshape(E, NT * 128, G * 128)
    i = np.arange(NT * 128)
    if layout == 1:
        f = (i // 128) * 64 + (i % 128) // 2
        src, valid = np.where(i & 1, N // 2 + f, f), f < N // 2
    else:
        src, valid = i, i < N
    assert not rows[:, ~valid].any() and not scale[:, ~valid].any()
    codes, sc = np.zeros((E, N, G * 128), np.int8), np.zeros((E, N), np.float32)
    codes[:, src[valid]], sc[:, src[valid]] = rows[:, valid], scale[:, valid]
    return codes, sc


@pytest.mark.parametrize("E,N,K,layout", [(1, 1, 1, 0), (1, 128, 128, 0), (3, 200, 300, 0), (2, 130, 136, 0), (2, 258, 257, 1),
                                          (2, 2 * 64, 512, 1), (1, 2 * 100, 2048 + 8, 1)])
def test_pack_is_bit_exact(E, N, K, layout):
    w = synth.normal_bf16(np.random.default_rng(N + K), (E, N, K), 0.02)
    w[0, 0] = 0.0                       # an all-zero channel
    w[-1, -1] = 3e38 * np.sign(w[-1, -1])  # and one near the type's limit
    codes = torch.full((E, N, B.padded_k(K)), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((E, N), 99.0, device="cuda")
    w = synth.bf16_round(w)
    buf = pack(w, layout, codes=codes, scale=scale).cpu().numpy()
    got_q, got_s = unpack(buf, E, N, K, layout)
    for e in range(E):
        q, s = W.quantize(w[e])
        assert np.array_equal(codes[e].cpu().numpy(), q) and np.array_equal(scale[e].cpu().numpy(), s)
        assert np.array_equal(got_q[e], q) and np.array_equal(got_s[e], s)


# one row, tile edges of tokens and channels, K below / on / off a plane, many row tiles, a
# long K, odd N (unaligned output rows), more tiles than CTAs
SHAPES = [(1, 1, 1), (1, 128, 128), (1, 4096, 2048), (3, 127, 100), (15, 129, 384), (16, 256, 512), (17, 384, 200),
          (32, 640, 4096), (33, 130, 1024), (64, 2048, 4096), (100, 131, 640), (127, 512, 256), (128, 256, 7168),
          (129, 1411, 1000), (200, 320, 1152), (255, 300, 130), (256, 1024, 1024), (257, 768, 896), (511, 96, 2056),
          (700, 2304, 512), (1500, 1000, 264), (2500, 4104, 136), (5, 20000, 256), (9, 256, 20000),
          # tiles of two halves: full, ragged, with one token in the second, a short and a long K
          (4096, 4864, 384), (5000, 5000, 640), (16385, 1152, 128), (9217, 2432, 1536)]


def dense_case(M, N, K, seed=0, bias=False):
    rng = np.random.default_rng([seed, M, N, K])
    x = synth.normal_bf16(rng, (M, K))
    w = synth.normal_bf16(rng, (N, K), 0.02)
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    return (*O.quantize_act(x), w, *W.quantize(w), b)


def run_gemm(qa, sa, packed, N, K, dtype, bias=None):
    """The output, through a buffer whose rows behind the last one must stay as they were."""
    M = qa.shape[0]
    qa = torch.from_numpy(qa).cuda() if isinstance(qa, np.ndarray) else qa
    sa = torch.from_numpy(sa).cuda() if isinstance(sa, np.ndarray) else sa
    y = torch.full((M + 1, N), 77, dtype=dtype, device="cuda")
    ws = B.empty_aligned(B.w8a8_gemm_workspace_bytes(M, N, K))
    ws.fill_(0xAB)  # a workspace holds anything
    B.w8a8_gemm(qa, sa, packed, N, K, y[:M], ws, bias=None if bias is None else torch.from_numpy(bias).cuda())
    torch.cuda.synchronize()
    assert B.w8a8_gemm_last_error(ws) == 0
    assert (y[M] == 77).all()
    return y[:M].cpu()


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_sums_are_exact(M, N, K):
    qa, sa, w, qw, sw, _ = dense_case(M, N, K)
    got = run_gemm(qa, None, pack(w), N, K, torch.int32).numpy()
    assert np.array_equal(got, W.int_sums(qa, qw))


def assert_rounded(got, dtype, qa, sa, qw, sw, b):
    ref = W.linear(qa, sa, qw, sw, b)
    bound = W.linear_error_bound(qa, sa, qw, sw, b)
    bound = bound + HALF_STEP[dtype] * (np.abs(ref) + bound) + TINY[dtype]
    err = np.abs(got.double().numpy() - ref)
    assert np.all(err <= bound), f"{int((err > bound).sum())} of {err.size} outside, worst {(err / bound).max():.3f} bounds"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K,bias", [(1, 1, 1, True), (1, 4096, 2048, False), (2, 130, 130, True), (31, 129, 384, True),
                                        (64, 2048, 4096, False), (129, 1411, 1000, True), (300, 514, 640, False),
                                        (257, 768, 896, True), (1000, 2304, 256, True)])
def test_gemm_outputs_within_counted_roundings(dtype, M, N, K, bias):
    qa, sa, w, qw, sw, b = dense_case(M, N, K, 1, bias)
    assert_rounded(run_gemm(qa, sa, pack(w), N, K, dtype, b), dtype, qa, sa, qw, sw, b)


def test_gemm_largest_sums_and_zero_rows():
    # every product is +-127 * 127 over K = 131072, the largest K: sums of 2.1e9 fit INT32
    K = 131072
    qa = np.full((3, K), 127, np.int8)
    qa[1] = -127
    qa[2] = 0
    w = np.ones((2, K), np.float32)
    w[1] = -1.0
    got = run_gemm(qa, None, pack(w), 2, K, torch.int32).numpy().astype(np.int64)
    s = 127 * 127 * K
    assert got.tolist() == [[s, -s], [-s, s], [0, 0]]
    sa = np.array([1.0, 1.0, 0.0], np.float32)
    qw, sw = W.quantize(w)
    assert_rounded(run_gemm(qa, sa, pack(w), 2, K, torch.float32), torch.float32, qa, sa, qw, sw, None)


def test_gemm_empty_batch_and_refused_tensors():
    N, K = 256, 200
    qa, sa, w, *_ = dense_case(4, N, K)
    packed = pack(w)
    run_gemm(np.zeros((0, 256), np.int8), np.zeros(0, np.float32), packed, N, K, torch.bfloat16)
    q, s, ws = torch.from_numpy(qa).cuda(), torch.from_numpy(sa).cuda(), B.empty_aligned(4096)
    y = torch.empty((4, N), device="cuda")
    for args, kw in [((q[:, :200], s, packed, N, K, y, ws), {}), ((q, s[:3], packed, N, K, y, ws), {}),
                     ((q, s, packed[:-1], N, K, y, ws), {}), ((q, s, packed, N, K, y[:, :255], ws), {}),
                     ((q, s, packed, N, K, y.double(), ws), {}), ((q.cpu(), s, packed, N, K, y, ws), {}),
                     ((q, None, packed, N, K, y, ws), {}), ((q, s, packed, N, K, y, ws[:16]), {}),
                     ((q, s, packed, N, K, y, ws), {"bias": s})]:
        with pytest.raises(B.W4A8Error):
            B.w8a8_gemm(*args, **kw)


# ---------------------------------------------------------------------- the layer
def check_layer(ws, T, E, k, H, F, x, ids, w, experts, out):
    """Every stage of the layer against the oracle on the stage's own input, as dumped from
    the workspace: permutation, token codes and requantised codes bit-exact; h equal to the
    oracle's bf16 h or one step off (both round a value computed to about 1e-6); y2 within the
    roundings of the fp32 scaling; out within k fp32 multiply-adds (half a step each, of at
    most the sum of the terms' magnitudes) and half a bf16 step."""
    def dump(what, dt):
        return B.w4a8_debug_dump(ws, T, E, k, H, F, what).cpu().numpy().view(dt)

    flat = ids.reshape(-1)
    good = np.nonzero((flat >= 0) & (flat < E))[0]
    R, Hp, Fp = B.w4a8_moe_rows_capacity(T, E, k), O.padded_k(H), O.padded_k(F)
    inv, poffs = dump("inv", np.int32), dump("poffs", np.int32)
    bad = np.setdiff1d(np.arange(T * k), good)
    assert (inv[bad] == -1).all()
    order = good[np.argsort(flat[good], kind="stable")]
    counts = np.bincount(flat[good], minlength=E)
    start = np.concatenate([[0], np.cumsum(-(-counts // 16) * 16)])
    assert np.array_equal(poffs, start)
    first = np.concatenate([[0], np.cumsum(counts)])
    row = inv[order]
    assert np.array_equal(row, start[flat[order]] + np.arange(len(order)) - first[flat[order]])
    qx, sx = W.quantize(x)
    act1, s1 = untile_act(dump("act1", np.int8), R, Hp), dump("s1", np.float32)
    assert np.array_equal(act1[row], qx[order // k]) and np.array_equal(s1[row], sx[order // k])
    h = synth.bf16_from_bits(dump("h", np.uint16)).reshape(R, Fp)[:, :F]
    act2, s2 = untile_act(dump("act2", np.int8), R, Fp), dump("s2", np.float32)
    y2 = dump("y2", np.float32).reshape(R, H)
    for e in range(E):
        rr = row[flat[order] == e]
        if rr.size == 0:
            continue
        ref = O.round_to_bf16(O.swiglu(W.linear(act1[rr], s1[rr], *experts[e].up), F))
        assert_bf16_adjacent(h[rr], ref, what=f"h of expert {e}")
        qh, sh = W.quantize(h[rr])
        assert np.array_equal(act2[rr], qh) and np.array_equal(s2[rr], sh)
        err = np.abs(y2[rr] - W.linear(qh, sh, *experts[e].down))
        assert np.all(err <= W.linear_error_bound(qh, sh, *experts[e].down)), f"y2 of expert {e}"
    terms = np.zeros((T * k, H))
    terms[good] = y2[inv[good]]  # (rows of no slot hold anything)
    terms = terms.reshape(T, k, H) * np.asarray(w, np.float64)[:, :, None]
    ref, size = terms.sum(axis=1), np.abs(terms).sum(axis=1)
    bound = 1.0001 * k * 2.0 ** -24 * size
    bound = bound + 2.0 ** -8 * (np.abs(ref) + bound) + 2.0 ** -134
    assert np.all(np.abs(out - ref) <= bound), "out"


def assert_close_overall(got, ref):
    """The whole layer against the oracle's: two bf16 roundings are at most 2^-8 + 2^-8 of
    the norm apart; the few h values that round to the other side of a bf16 boundary (below
    one in a thousand, see check_layer, which bounds each stage on its own input) move the
    norm by less than the 0.2% left."""
    assert np.linalg.norm(got - ref) <= 1e-2 * np.linalg.norm(ref)


class Layer:
    def __init__(self, T, E, k, H, F, routing, seed):
        self.T, self.E, self.k, self.H, self.F = T, E, k, H, F
        self.x = synth.activations(seed, T, H)
        self.ids, self.w = synth.synthetic_routing(seed, T, E, k, routing, 1.1)
        self.up = np.stack([synth.expert_weight(seed, e, "up", 2 * F, H) for e in range(E)])
        self.dn = np.stack([synth.expert_weight(seed, e, "down", H, F) for e in range(E)])
        self.packed = pack(self.up, B.W4A8_LAYOUT_GATEUP), pack(self.dn)
        self.experts = {e: W.QuantExpert(self.up[e], self.dn[e]) for e in range(E)}
        self.ws = B.empty_aligned(B.w8a8_moe_workspace_bytes(T, E, k, H, F))
        self.ws.fill_(0x7F)  # a workspace holds anything

    def run(self, ids=None, err=0):
        out = torch.full((self.T + 1, self.H), 7.0, dtype=torch.bfloat16, device="cuda")
        ids = self.ids if ids is None else ids
        B.w8a8_moe_forward(*self.packed, self.E, self.H, self.F, dev_bf16(self.x), torch.from_numpy(ids).cuda(),
                           torch.from_numpy(self.w).cuda(), out[:self.T], self.ws)
        torch.cuda.synchronize()
        assert B.w4a8_last_device_error(self.ws) == err
        assert (out[self.T] == 7.0).all()
        out = out[:self.T].double().cpu().numpy()
        check_layer(self.ws, self.T, self.E, self.k, self.H, self.F, self.x, ids, self.w, self.experts, out)
        return out

    def ref(self, ids=None):
        return W.moe_forward(self.x, self.ids if ids is None else ids, self.w, self.experts, self.E, self.F)


LAYERS = [
    (1, 4, 2, 256, 128, "uniform"), (1, 1, 1, 128, 1, "uniform"), (37, 5, 3, 200, 100, "uniform"),
    (3, 8, 2, 1024, 352, "uniform"), (48, 16, 4, 1024, 640, "zipf"), (64, 64, 6, 512, 352, "uniform"),
    (130, 2, 1, 264, 70, "uniform"), (333, 3, 2, 384, 200, "zipf"), (600, 4, 2, 256, 256, "uniform"),
    (900, 4, 3, 520, 130, "zipf"), (2100, 6, 2, 128, 64, "uniform"), (3000, 3, 2, 384, 136, "uniform"),
    (20, 200, 8, 128, 64, "uniform"),
    (1500, 3, 2, 256, 320, "uniform"), (1100, 2, 2, 640, 64, "zipf"), (2500, 4, 2, 136, 96, "zipf"),
]


@pytest.mark.parametrize("T,E,k,H,F,routing", LAYERS)
def test_moe_matches_oracle(T, E, k, H, F, routing):
    L = Layer(T, E, k, H, F, routing, seed=5 * T + E)
    assert_close_overall(L.run(), L.ref())


def test_moe_permutation_in_three_passes():
    # more than 16384 slots take the multi-CTA permutation
    Layer(5000, 5, 4, 128, 64, "zipf", seed=9).run()


def test_moe_all_tokens_to_one_expert_the_same_twice_and_bad_ids():
    L = Layer(150, 6, 2, 256, 192, "uniform", seed=4)
    ids = np.full_like(L.ids, 3)  # the same expert twice
    assert_close_overall(L.run(ids), L.ref(ids))
    ids = L.ids.copy()
    ids[::7, 0] = -1
    ids[3, 1] = 6
    assert_close_overall(L.run(ids, err=2), L.ref(ids))
    ids[:] = -1
    assert (L.run(ids, err=2) == 0).all()  # no slot left: zero rows


def test_moe_zero_rows_and_outliers():
    L = Layer(40, 4, 2, 256, 128, "uniform", seed=6)
    L.x[5] = 0.0
    L.x[:, 17] *= 50.0
    L.x = synth.bf16_round(L.x)
    got, ref = L.run(), L.ref()
    assert (got[5] == 0).all()
    assert_close_overall(got, ref)


# rows longer than a thread's or a warp's registers hold, and both sides of each choice of
# quantisation kernel: H > 8192 and F > 2048; F in (1024, 2048] with few and with many rows;
# more than 2048 slots with H on both sides of 512 and 1024; odd lengths of each
LONG_ROWS = [
    (3, 2, 2, 8200, 16, "uniform"), (2, 2, 1, 8193, 9, "uniform"), (1100, 2, 2, 8200, 8, "uniform"),
    (5, 2, 2, 64, 2100, "uniform"), (3, 2, 1, 40, 2049, "uniform"), (20, 2, 2, 128, 1100, "uniform"),
    (1500, 2, 2, 72, 1100, "uniform"), (1300, 2, 2, 72, 2041, "zipf"), (1100, 3, 2, 513, 40, "uniform"),
    (1100, 3, 2, 1024, 24, "uniform"), (1100, 3, 2, 1031, 513, "uniform"), (700, 3, 3, 1040, 1025, "zipf"),
]


@pytest.mark.parametrize("T,E,k,H,F,routing", LONG_ROWS)
def test_moe_long_rows(T, E, k, H, F, routing):
    L = Layer(T, E, k, H, F, routing, seed=3 * T + H)
    L.run()


@pytest.mark.parametrize("T,H", [(24, 256), (24, 257), (1100, 256), (1100, 1100), (1100, 515)])
def test_moe_codes_next_to_a_rounding_boundary(T, H):
    """Token rows whose quotients lie on or next to n + 1/2, rows of subnormal and of the
    largest values, and rows with one value only: codes and
    scales equal the oracle's bit by bit."""
    L = Layer(T, 3, 2, H, 32, "uniform", seed=H + T)
    rng = np.random.default_rng(T + H)
    step = 2.0 ** rng.integers(-100, 20, (T, 1))
    x = (rng.integers(-64, 64, (T, H)) + 0.5) * step
    x[:, 0] = 127.0 * step[:, 0]  # the scale is the step, within one rounding
    x[0::7] *= 2.0 ** -40         # some further down, into the subnormals
    x[1::7] = np.sign(x[1::7]) * rng.integers(1, 128, x[1::7].shape) * 2.0 ** -133
    x[2::7, 1:] = 0.0
    x[3::7] = x[3::7] * 2.0 ** 100 / step[3::7]
    L.x = synth.bf16_round(x.astype(np.float32))
    L.w = (L.w * 2.0 ** -20).astype(np.float32)
    qx, sx = W.quantize(L.x)
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    B.w8a8_moe_forward(*L.packed, L.E, H, L.F, dev_bf16(L.x), torch.from_numpy(L.ids).cuda(), torch.from_numpy(L.w).cuda(),
                       out, L.ws)
    torch.cuda.synchronize()

    def dump(what, dt):
        return B.w4a8_debug_dump(L.ws, T, L.E, L.k, H, L.F, what).cpu().numpy().view(dt)

    row = dump("inv", np.int32)
    act = untile_act(dump("act1", np.int8), B.w4a8_moe_rows_capacity(T, L.E, L.k), O.padded_k(H))
    slots = np.arange(T * L.k)
    assert np.array_equal(dump("s1", np.float32)[row], sx[slots // L.k])
    assert np.array_equal(act[row], qx[slots // L.k])


@pytest.mark.parametrize("M,N,K", [(16, 256, 640), (300, 256, 640), (1, 512, 4096)])
def test_gemm_wait_timeout_is_reported_and_recovers(M, N, K):
    qa, sa, w, qw, sw, _ = dense_case(M, N, K)
    packed = pack(w)
    q, ws = torch.from_numpy(qa).cuda(), B.empty_aligned(B.w8a8_gemm_workspace_bytes(M, N, K))
    y = torch.empty((M, N), dtype=torch.int32, device="cuda")
    try:
        B.w4a8_debug_inject(B.W4A8_DEBUG_SKIP_FIRST_COPY, SHORT_WAIT)
        B.w8a8_gemm(q, None, packed, N, K, y, ws)
        torch.cuda.synchronize()
        assert B.w8a8_gemm_last_error(ws) & 1, "the wait that ran out must set bit 0"
    finally:
        B.w4a8_debug_inject(0, 0)
    B.w8a8_gemm(q, None, packed, N, K, y, ws)
    torch.cuda.synchronize()
    assert B.w8a8_gemm_last_error(ws) == 0
    assert np.array_equal(y.cpu().numpy(), W.int_sums(qa, qw))


@pytest.mark.parametrize("T,E,k", [(48, 8, 2), (600, 4, 2)])
def test_moe_wait_timeout_is_reported_and_recovers(T, E, k):
    L = Layer(T, E, k, 256, 256, "uniform", seed=T)
    try:
        B.w4a8_debug_inject(B.W4A8_DEBUG_SKIP_FIRST_COPY, SHORT_WAIT)
        B.w8a8_moe_forward(*L.packed, E, 256, 256, dev_bf16(L.x), torch.from_numpy(L.ids).cuda(),
                           torch.from_numpy(L.w).cuda(), torch.empty((T, 256), dtype=torch.bfloat16, device="cuda"), L.ws)
        torch.cuda.synchronize()
        assert B.w4a8_last_device_error(L.ws) & 1
    finally:
        B.w4a8_debug_inject(0, 0)
    assert_close_overall(L.run(), L.ref())


class Step:
    """One serving step: router logits -> experts, the W8A8 expert FFN, and a dense W8A8
    layer beside it (a shared expert's projection), all on one stream."""

    def __init__(self, T, seed):
        E, k, H, F, N = 16, 4, 256, 128, 320
        self.dims = E, k, H, F, N
        self.L = Layer(T, E, k, H, F, "uniform", seed)
        self.T = T
        rng = np.random.default_rng(seed)
        self.wn = synth.normal_bf16(rng, (N, H), 0.02)
        self.packed_n = pack(self.wn)
        d = "cuda"
        self.x = torch.empty((T, H), dtype=torch.bfloat16, device=d)
        self.logits = torch.empty((T, E), dtype=torch.bfloat16, device=d)
        self.bias = torch.from_numpy((rng.standard_normal(E) * 0.05).astype(np.float32)).to(d)
        self.ids, self.w = torch.empty((T, k), dtype=torch.int32, device=d), torch.empty((T, k), device=d)
        self.out, self.y = torch.empty((T, H), dtype=torch.bfloat16, device=d), torch.empty((T, N), dtype=torch.bfloat16, device=d)
        self.q, self.s = torch.empty((T, H), dtype=torch.int8, device=d), torch.empty(T, device=d)
        self.ws1 = B.empty_aligned(B.w8a8_moe_workspace_bytes(T, E, k, H, F))
        self.ws2 = B.empty_aligned(B.w8a8_gemm_workspace_bytes(T, N, H))

    def feed(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.x.copy_(torch.randn(self.x.shape, generator=g))
        self.logits.copy_(torch.randn(self.logits.shape, generator=g) * 1.5)

    def run(self):
        E, k, H, F, N = self.dims
        B.w4a8_route_experts(self.logits, k, self.ids, self.w, B.W4A8_ROUTE_SIGMOID | B.W4A8_ROUTE_RENORM |
                             B.W4A8_ROUTE_GROUP_TOP2, self.bias, 4, 2, 2.5)
        B.w8a8_moe_forward(*self.L.packed, E, H, F, self.x, self.ids, self.w, self.out, self.ws1)
        B.w4a8_quant_act(self.x, self.q, self.s)
        B.w8a8_gemm(self.q, self.s, self.packed_n, N, H, self.y, self.ws2)

    def check(self):
        E, k, H, F, N = self.dims
        x = self.x.float().cpu().numpy()
        ids, w = W.route_experts(self.logits.double().cpu().numpy(), k, True, True, True, self.bias.double().cpu().numpy(), 4, 2, 2.5)
        assert np.array_equal(self.ids.cpu().numpy(), ids)
        check_layer(self.ws1, self.T, E, k, H, F, x, ids, self.w.cpu().numpy(), self.L.experts, self.out.double().cpu().numpy())
        qa, sa = O.quantize_act(x)
        assert_rounded(self.y.cpu(), torch.bfloat16, qa, sa, *W.quantize(self.wn), None)


@pytest.mark.parametrize("T", [1, 33, 700])
def test_operators_together_eager_and_replayed(T):
    st = Step(T, 40 + T)
    st.feed(1)
    st.run()
    torch.cuda.synchronize()
    st.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.run()
    for seed in (2, 3):
        st.feed(seed)
        graph.replay()
        torch.cuda.synchronize()
        st.check()


def test_two_streams_at_once():
    a, b = Step(90, 50), Step(200, 51)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a.feed(4), b.feed(5)
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a.run()
        with torch.cuda.stream(s2):
            b.run()
    torch.cuda.synchronize()
    a.check(), b.check()


FIRST_CALL = """
import sys
import torch
from w4a8_quantized_moe_token_b200 import binding as B

def buf(n):
    return B.empty_aligned(n)

torch.manual_seed(0)
E, H, F, k, T = 8, 256, 128, 2, {T}
def pack(E, N, K, layout):
    p = buf(B.w8a8_packed_bytes(E, N, K, layout))
    B.w8a8_pack_weights(torch.randn(E, N, K, device="cuda").bfloat16(), layout, p)
    return p
up, dn, wn = pack(E, 2 * F, H, 1), pack(E, H, F, 0), pack(1, 256, H, 0)
x = torch.randn(T, H, device="cuda").bfloat16()
logits = torch.randn(T, E, device="cuda")
ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
out, y = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, 256, device="cuda")
qa, sa = torch.empty(T, H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
B.w4a8_quant_act(x, qa, sa)
ws, wd = buf(B.w8a8_moe_workspace_bytes(T, E, k, H, F)), buf(B.w8a8_gemm_workspace_bytes(T, 256, H))
def run():
    B.w4a8_route_experts(logits, k, ids, w)
    B.w8a8_moe_forward(up, dn, E, H, F, x, ids, w, out, ws)
    B.w8a8_gemm(qa, sa, wn, 256, H, y, wd)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (ids, w, out, y)]
run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (ids, w, out, y))) and out.abs().sum() > 0 and y.abs().sum() > 0
"""


@pytest.mark.parametrize("T", [1, 1100])
def test_first_call_of_a_process_inside_a_capture(T):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.replace("{T}", str(T))], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_last_error_refuses_other_buffers():
    with pytest.raises(B.W4A8Error):
        B.w8a8_gemm_last_error(B.empty_aligned(2048))
    with pytest.raises(B.W4A8Error):
        B.w8a8_gemm_last_error(torch.zeros(4096, dtype=torch.uint8))
