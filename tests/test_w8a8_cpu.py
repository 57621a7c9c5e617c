"""CPU checks of the W8A8 scheme and the expert routing: the oracle against closed forms
and independent formulations, and every refusal of the entry points before a GPU is used."""

import ctypes
import os
import re

import numpy as np
import pytest

from oracle import w4a8_oracle as O
from oracle import w8a8_oracle as W
from w4a8_quantized_moe_token_b200 import binding as B
from w4a8_quantized_moe_token_b200 import synth

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EALIGN, ENOSPACE, EUNSUPPORTED = -1, -2, -3, -5
vp = ctypes.c_void_p
FAKE = vp(1 << 20)  # aligned, never dereferenced: validation fails first
ODD = vp((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from w4a8_quantized_moe_token_b200 import build
        build.build()
    return B.lib()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "w8a8.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(w8a8_\w+)\s*\(", text))
    assert names == set(B.exported_symbols_w8a8())
    for n in names:
        assert hasattr(lib, n), n


def test_packed_bytes(lib):
    blk = 128 * 128
    assert lib.w8a8_packed_bytes(1, 256, 512, 0) == 256 + 2 * 512 + 2 * 4 * blk
    assert lib.w8a8_packed_bytes(3, 100, 200, 0) == 256 + 3 * 512 + 3 * 2 * blk
    assert lib.w8a8_packed_bytes(8, 2048, 2048, 1) == 256 + 8 * 16 * 512 + 8 * 16 * 16 * blk
    assert lib.w8a8_packed_bytes(1, 66, 1, 1) == 256 + 512 + blk
    for E, N, K in [(1, 256, 512), (3, 100, 200), (2, 2, 1)]:  # what the binding checks against
        assert B._w8_packed_size(E, -(-N // 128), K) == lib.w8a8_packed_bytes(E, N, K, 0)
        assert B._w8_packed_size(E, -(-(N // 2) // 64), K) == lib.w8a8_packed_bytes(E, N, K, 1)
    assert lib.w8a8_packed_bytes(1, 3, 128, 1) == 0   # odd N for gate|up
    assert lib.w8a8_packed_bytes(1, 4, 128, 2) == 0   # unknown layout
    assert lib.w8a8_packed_bytes(1, 4, 128, 0x100) == 0  # W4A8 scheme flags do not apply
    assert lib.w8a8_packed_bytes(0, 4, 128, 0) == 0


def test_pack_refusals(lib):
    big = 1 << 60
    f = lib.w8a8_pack_weights
    assert f(None, 1, 4, 4, 0, FAKE, big, None, None, None) == EINVAL
    assert f(FAKE, 1, 4, 4, 0, None, big, None, None, None) == EINVAL
    assert f(FAKE, 1, 4, 0, 0, FAKE, big, None, None, None) == EINVAL
    assert f(ODD, 1, 4, 4, 0, FAKE, big, None, None, None) == EALIGN
    assert f(FAKE, 1, 4, 4, 0, vp((1 << 20) + 16), big, None, None, None) == EALIGN
    assert f(FAKE, 1, 4, 4, 0, FAKE, big, ODD, None, None) == EALIGN
    assert f(FAKE, 1, 4, 4, 0, FAKE, 256 + 512 + 16383, None, None, None) == ENOSPACE
    assert f(FAKE, 1, 4, 131073, 0, FAKE, big, None, None, None) == EUNSUPPORTED  # INT32 sum
    assert f(FAKE, 1 << 20, 128, 4096, 0, FAKE, big, None, None, None) == EUNSUPPORTED  # 2^32 packed rows


def test_gemm_refusals(lib):
    def call(qa=FAKE, sa=FAKE, M=4, packed=FAKE, N=256, K=512, bias=None, y=FAKE, t=0, ws=FAKE, n=1 << 20):
        return lib.w8a8_gemm(qa, sa, M, packed, N, K, bias, y, t, ws, n, None)

    assert lib.w8a8_gemm_workspace_bytes(4, 256, 512) > 0
    assert lib.w8a8_gemm_workspace_bytes(-1, 256, 512) == 0
    assert call(M=-1) == EINVAL and call(N=0) == EINVAL and call(K=0) == EINVAL
    assert call(t=4) == EINVAL and call(t=-1) == EINVAL
    assert call(qa=None) == EINVAL and call(sa=None) == EINVAL and call(y=None) == EINVAL
    assert call(packed=None) == EINVAL and call(ws=None) == EINVAL
    assert call(qa=vp((1 << 20) + 8)) == EALIGN and call(packed=vp((1 << 20) + 16)) == EALIGN
    assert call(y=ODD) == EALIGN and call(y=vp((1 << 20) + 1), t=1) == EALIGN and call(bias=ODD) == EALIGN
    assert call(ws=vp((1 << 20) + 16)) == EALIGN
    assert call(n=16) == ENOSPACE and lib.w8a8_gemm_last_error(None, None) == EINVAL
    assert call(K=1 << 18) == EUNSUPPORTED
    assert call(M=(1 << 31) - 1, N=1 << 20) == EUNSUPPORTED


def test_moe_refusals(lib):
    def call(up=FAKE, dn=FAKE, E=8, H=256, F=128, x=FAKE, T=4, ids=FAKE, w=FAKE, k=2, out=FAKE, ws=FAKE, n=1 << 40):
        return lib.w8a8_moe_forward(up, dn, E, H, F, x, T, ids, w, k, out, ws, n, None)

    assert lib.w8a8_moe_workspace_bytes(4, 8, 2, 256, 128) > 0
    assert lib.w8a8_moe_workspace_bytes(4, 8, 9, 256, 128) == 0
    assert call(k=9) == EINVAL and call(k=0) == EINVAL and call(T=-1) == EINVAL and call(F=0) == EINVAL
    assert call(up=None) == EINVAL and call(x=None) == EINVAL and call(ids=None) == EINVAL and call(out=None) == EINVAL
    assert call(dn=vp((1 << 20) + 16)) == EALIGN and call(w=vp((1 << 20) + 4)) == EALIGN
    assert call(n=16) == ENOSPACE
    assert call(E=2048) == EUNSUPPORTED and call(E=64, k=33) == EUNSUPPORTED and call(H=1 << 18) == EUNSUPPORTED
    assert call(T=1 << 30, k=4) == EUNSUPPORTED


def test_route_refusals(lib):
    def call(x=FAKE, typ=0, T=4, E=64, k=4, flags=0, bias=None, n_group=1, topk_group=1, scale=1.0, ids=FAKE, w=FAKE):
        return lib.w4a8_route_experts(x, typ, T, E, k, flags, bias, n_group, topk_group, scale, ids, w, None)

    assert call(T=0, x=None) == 0  # nothing to do
    assert call(T=-1) == EINVAL and call(k=0) == EINVAL and call(k=65) == EINVAL
    assert call(n_group=5) == EINVAL and call(n_group=0) == EINVAL
    assert call(n_group=8, topk_group=9) == EINVAL and call(n_group=8, topk_group=0) == EINVAL
    assert call(n_group=32, topk_group=1, k=3) == EINVAL  # two experts in the only group kept
    assert call(flags=8) == EINVAL and call(typ=3) == EINVAL and call(typ=-1) == EINVAL
    assert call(scale=float("nan")) == EINVAL and call(scale=float("inf")) == EINVAL
    assert call(x=None) == EINVAL and call(ids=None) == EINVAL and call(w=None) == EINVAL
    assert call(x=ODD) == EALIGN and call(bias=ODD) == EALIGN and call(w=vp((1 << 20) + 4)) == EALIGN
    assert call(E=2048) == EUNSUPPORTED and call(k=33) == EUNSUPPORTED and call(n_group=64, topk_group=4) == EUNSUPPORTED


# ------------------------------------------------------------------- the oracle
def test_linear_closed_form_and_dequantised_product():
    # one channel of weights 127 * 2^-7, tokens of 1: codes 127, sums K * 127^2
    x, w = np.ones((2, 5), np.float32), np.full((1, 5), 127 / 128, np.float32)
    qa, sa = O.quantize_act(x)
    qw, sw = W.quantize(w)
    assert (W.int_sums(qa, qw) == 5 * 127 * 127).all()
    np.testing.assert_allclose(W.linear(qa, sa, qw, sw, [0.5]), 5 * 127 / 128 + 0.5, rtol=1e-6)
    x, w = synth.dense_gemm_inputs(3, 7, 200, 33)
    qa, sa = O.quantize_act(x)
    qw, sw = W.quantize(w)
    deq = (qa * sa[:, None].astype(np.float64)) @ (qw * sw[:, None].astype(np.float64)).T
    np.testing.assert_allclose(W.linear(qa, sa, qw, sw), deq, rtol=1e-12, atol=1e-12)
    assert np.all(np.abs(w - qw[:, :200] * sw[:, None]) <= 0.5001 * sw[:, None])  # half a step


def test_moe_oracle_against_a_per_token_formulation():
    T, E, k, H, F = 9, 4, 2, 96, 40
    x = synth.activations(1, T, H)
    ids, w = synth.synthetic_routing(2, T, E, k, "uniform")
    wu = [synth.expert_weight(3, e, "up", 2 * F, H) for e in range(E)]
    wd = [synth.expert_weight(3, e, "down", H, F) for e in range(E)]
    got = W.moe_forward(x, ids, w, {e: W.QuantExpert(wu[e], wd[e]) for e in range(E)}, E, F)

    def deq(v):
        q, s = W.quantize(v)
        return q[:, :v.shape[1]].astype(np.float64) * s[:, None].astype(np.float64)

    for t in range(T):
        out = np.zeros(H)
        for j in range(k):
            e = ids[t, j]
            a = deq(wu[e]) @ deq(x[t:t + 1])[0]
            h = O.round_to_bf16(a[:F] / (1 + np.exp(-a[:F])) * a[F:])
            out += w[t, j] * (deq(wd[e]) @ deq(h[None].astype(np.float32))[0])
        # both are rounded from fp64 sums that agree to 1e-12: half a bf16 step at most between them
        np.testing.assert_allclose(got[t], out, rtol=2.0 ** -8, atol=1e-9)


def test_route_oracle_closed_forms():
    lg = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    ids, w = W.route_experts(lg, 2)
    assert ids.tolist() == [[2, 1]] and np.allclose(w, [[0.5, 0.25]])
    ids, w = W.route_experts(lg, 2, renorm=True, scale=3.0)
    assert np.allclose(w, [[2.0, 1.0]])
    ids, w = W.route_experts(lg, 1, sigmoid=True, bias=[1.0, 0, 0, 0])  # chosen by the bias, weighted without it
    assert ids.tolist() == [[0]] and np.allclose(w, [[0.5]])
    # groups {0,1} and {2,3}: best member 4 against 2, sum of two 5 (4/8 + 1/8) against 3/8
    assert W.route_experts(lg, 2, n_group=2, topk_group=1)[0].tolist() == [[2, 3]]
    assert W.route_experts(np.log([[3.0, 3.0, 4.0, 1.0]]), 2, top2=True, n_group=2, topk_group=1)[0].tolist() == [[0, 1]]
    # masks: -inf and NaN rank last and weigh nothing; a row with nothing left weighs nothing
    x = np.array([[-np.inf, 0.0, np.nan, 0.0], [-np.inf] * 4])
    ids, w = W.route_experts(x, 3, renorm=True)
    assert ids.tolist() == [[1, 3, 0], [0, 1, 2]] and np.allclose(w, [[0.5, 0.5, 0], [0, 0, 0]])
    assert np.allclose(W.route_experts([[np.inf, 0.0, np.inf]], 2)[1], [[0.5, 0.5]])
    # the plain softmax gating is the existing oracle's
    lg = synth.router_logits(5, 20, 24)
    for a, b in zip(W.route_experts(lg, 3), O.route_topk(lg, 3)):
        np.testing.assert_allclose(a, b, rtol=1e-12)
