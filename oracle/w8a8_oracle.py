"""CPU oracle of the W8A8 scheme and of the expert routing with bias and groups.

Plain numpy, step by step from the definitions in include/w8a8.h and include/w4a8.h:
fp64 for what is compared within a tolerance, IEEE fp32 for the quantisation decisions,
exact integers for the INT32 sums.  Shares SwiGLU, the bf16 rounding and the combine with
the W4A8 oracle, and nothing with the CUDA path.
"""

from __future__ import annotations

import numpy as np

from . import w4a8_oracle as O


def quantize(v: np.ndarray):
    """Symmetric INT8 per row of v [N][K]: codes int8 [N][Kp] (K padded to 128 with zeros)
    and scale float32 [N] = max|v| * (1 / 127), both fp32; codes from the fp32 quotient."""
    v = np.asarray(v, dtype=np.float32)
    s = (np.abs(v).max(axis=1) * (np.float32(1.0) / np.float32(127.0))).astype(np.float32)
    q = np.zeros(v.shape, np.int8)
    nz = s > 0
    q[nz] = np.clip(np.rint(v[nz] / s[nz][:, None]), -127, 127).astype(np.int8)
    return O.pad_k(q), s


def int_sums(qa: np.ndarray, qw: np.ndarray) -> np.ndarray:
    """sum_k qa[m][k] * qw[n][k], exact (fp64 products of integers, sums < 2^53), int64."""
    return np.rint(qa.astype(np.float64) @ qw.astype(np.float64).T).astype(np.int64)


def linear(qa, sa, qw, sw, bias=None) -> np.ndarray:
    """y[m][n] = sa[m] * sw[n] * sum_k qa * qw (+ bias[n]), fp64."""
    y = int_sums(qa, qw) * (np.asarray(sa, np.float64)[:, None] * np.asarray(sw, np.float64)[None, :])
    return y if bias is None else y + np.asarray(bias, np.float64)[None, :]


def linear_error_bound(qa, sa, qw, sw, bias=None) -> np.ndarray:
    """Largest error of the fp32 evaluation of linear(): the integer sum, the product of the
    scales and their product are rounded once each and the bias is added with one rounding,
    each by at most half a step, 2^-24 of its value (1.0001 covers their products)."""
    y = np.abs(linear(qa, sa, qw, sw))
    e = 3 * 2.0 ** -24 * y
    if bias is not None:
        e = e + 2.0 ** -24 * (y + np.abs(np.asarray(bias, np.float64))[None, :])
    return 1.0001 * e


class QuantExpert:
    """Quantised weights of one expert: up [2F][Hp] (gate|up rows) and down [H][Fp]."""

    def __init__(self, w_up, w_down):
        self.up = quantize(w_up)
        self.down = quantize(w_down)


def moe_forward(x, ids, w, experts: dict, E: int, F: int, stages: dict | None = None):
    """The W8A8 MoE expert FFN [T][H], rounded to bf16 (as fp64 values).  Slots whose id is
    out of range contribute nothing."""
    x = np.asarray(x, dtype=np.float32)
    T, H = x.shape
    k = ids.shape[1]
    qx, sx = quantize(x)
    y2 = np.zeros((T * k, H))
    flat = np.asarray(ids).reshape(-1)
    hs = np.zeros((T * k, F))
    for e in range(E):
        slots = np.nonzero(flat == e)[0]
        if slots.size == 0:
            continue
        t = slots // k
        h = O.round_to_bf16(O.swiglu(linear(qx[t], sx[t], *experts[e].up), F))
        hs[slots] = h
        qh, sh = quantize(h.astype(np.float32))
        y2[slots] = linear(qh, sh, *experts[e].down)
    if stages is not None:
        stages.update(h=hs, y2=y2)
    return O.round_to_bf16(O.combine(y2, w, np.arange(T * k), T, k))


def route_experts(logits, k, sigmoid=False, renorm=False, top2=False, bias=None, n_group=1, topk_group=1, scale=1.0):
    """Expert ids int32 [T][k] and weights float64 [T][k], one token at a time."""
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    size = E // n_group
    ids = np.zeros((T, k), np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        v = x[t]
        live = v > -np.inf  # false for NaN
        if sigmoid:
            with np.errstate(over="ignore"):
                s = np.where(live, 1.0 / (1.0 + np.exp(-np.where(live, v, 0.0))), 0.0)
        else:
            top = v[live].max() if live.any() else 0.0
            d = np.full(E, -np.inf)
            for e in range(E):
                if live[e]:
                    d[e] = 0.0 if v[e] == top else v[e] - top
            p = np.exp(d)
            s = p / p.sum() if live.any() else p
        usable = live.copy()
        if bias is not None:
            usable &= np.asarray(bias) > -np.inf
        if bias is None and not top2:
            c = np.where(usable, v, -np.inf)
        else:
            b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
            c = np.where(usable, s + np.where(usable, b, 0.0), -np.inf)
        eligible = list(range(E))
        if n_group > 1:
            gs = []
            for g in range(n_group):
                best = sorted((c[e] for e in range(g * size, (g + 1) * size) if usable[e]), reverse=True)
                gs.append(-np.inf if not best else sum(best[:2]) if top2 else best[0])
            kept = sorted(range(n_group), key=lambda g: (-gs[g], g))[:topk_group]
            eligible = [e for e in eligible if e // size in kept]
        chosen = sorted(eligible, key=lambda e: (-c[e], e))[:k]
        ids[t] = chosen
        wt = np.array([s[e] if usable[e] else 0.0 for e in chosen])
        if renorm:
            # s_j / sum s_i over the chosen; the scores relative to the largest one's exponential,
            # so that neither a common factor (the softmax's sum) nor underflow enters
            got = [e for e in chosen if usable[e]]
            z = [min(v[e], 0.0) if sigmoid else v[e] for e in got]
            rel = {e: (1.0 if z[i] == max(z) else np.exp(z[i] - max(z))) / (1.0 + np.exp(-abs(v[e])) if sigmoid else 1.0)
                   for i, e in enumerate(got)}
            wt = np.array([rel[e] / sum(rel.values()) if e in rel else 0.0 for e in chosen])
        w[t] = wt * scale
    return ids, w
