"""Workloads of the library's expert routing, W8A8 linear layer and W8A8 expert FFN.

Three operators, each in a plain form (elementary torch operations) and, where `own` is
true, as the calls that a user makes of the library:

  route  token t's k experts out of E and their gate weights, from router logits: softmax
         or sigmoid scores, an optional per-expert bias that enters the choice but not the
         weights, an optional restriction to the best groups of experts, an optional
         renormalisation of the chosen scores and a factor;
  gemm   y = sa[m] * sw[n] * sum_k qa[m][k] * qw[n][k] (+ bias[n]): the product of INT8
         activations and INT8 weights with one scale per token and one per output channel;
  moe    out[t] = sum_j w[t][j] * Down_e(SwiGLU(Up_e(x[t]))), e = ids[t][j], both
         projections of every expert W8A8, activations quantised per token.

INT8 quantisation is symmetric: s = max|v| / 127 (fp32), q = round-half-even(v / s); it
decides whole numbers, so its fp32 arithmetic is part of the operators' definition, as is
the rounding of SwiGLU's result to bf16.
"""

import math

import torch

own = False

SOFTMAX, SIGMOID, RENORM, GROUP_TOP2 = 0, 1, 2, 4  # the flags of the routing call
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------- the cases
def _route(T, E, k, dtype, score, bias, groups=1, kept=1, renorm=True, scale=1.0):
    return {"op": "route", "T": T, "E": E, "k": k, "dtype": dtype, "score": score, "bias": bias, "groups": groups,
            "kept": kept, "renorm": renorm, "scale": scale}


def _gemm(M, N, K, dtype, bias):
    return {"op": "gemm", "M": M, "N": N, "K": K, "dtype": dtype, "bias": bias}


def _moe(T, E, k, H, F, skew):
    return {"op": "moe", "T": T, "E": E, "k": k, "H": H, "F": F, "skew": skew}


def listed():
    return [
        # one token of a decode step of a 384-expert layer: latency alone
        {"name": "route_one_token", **_route(1, 384, 8, "bf16", "sigmoid", True, 8, 4, True, 2.5)},
        # the decode layer's batch, softmax gating as the library had it, renormalised
        {"name": "route_decode", **_route(64, 64, 6, "bf16", "softmax", False)},
        # an odd batch, groups limited by their best expert, fp16 logits, weights as they are
        {"name": "route_ragged", **_route(1999, 160, 6, "fp16", "softmax", False, 8, 3, False, 16.0)},
        # the prefill layer's batch with balance bias and groups, fp32 logits
        {"name": "route_prefill", **_route(16384, 384, 8, "fp32", "sigmoid", True, 8, 4, True, 2.5)},
        # one token through a 2048 -> 7168 linear layer: the weights are read once
        {"name": "gemm_one_token", **_gemm(1, 7168, 2048, "bf16", False)},
        # a decode batch through a square layer of the decode layer's width
        {"name": "gemm_decode", **_gemm(64, 4096, 4096, "bf16", True)},
        # odd everything: rows, channels (below a tile, unaligned rows), a K that is padded
        {"name": "gemm_ragged", **_gemm(777, 1411, 1000, "fp32", True)},
        # the prefill batch through a 7168 -> 4096 linear layer
        {"name": "gemm_prefill", **_gemm(16384, 4096, 7168, "bf16", False)},
        # one token through the decode layer's experts
        {"name": "moe_one_token", **_moe(1, 64, 6, 4096, 1408, 0.0)},
        # the decode layer
        {"name": "moe_decode", **_moe(64, 64, 6, 4096, 1408, 0.0)},
        # skewed routing, odd batch: some experts get hundreds of rows, most a few
        {"name": "moe_skewed", **_moe(1021, 48, 8, 7168, 2048, 1.1)},
        # the prefill layer: 384 experts, 16384 tokens
        {"name": "moe_prefill", **_moe(16384, 384, 8, 7168, 2048, 0.0)},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["route", "gemm", "moe"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, max(2, 8 // groups), 384 // groups)
        kept = rng.randint(max(1, groups // 2), groups)
        k = rng.randint(1, min(10, kept * (E // groups)))
        return _route(_log(rng, 1, 16384), E, k, rng.choice(sorted(TYPES)), rng.choice(["softmax", "sigmoid"]),
                      rng.random() < 0.5, groups, kept, rng.random() < 0.7, rng.choice([1.0, 2.5, 16.0]))
    if op == "gemm":
        N, K = _log(rng, 64, 8192), _log(rng, 64, 8192)
        if rng.random() < 0.5:  # a model's own widths are multiples of 128; others are odd
            N, K = -(-N // 128) * 128, -(-K // 128) * 128
        return _gemm(_log(rng, 1, 8192), N, K, rng.choice(sorted(TYPES)), rng.random() < 0.5)
    E = rng.choice([4, 8, 16, 48, 64])
    H, F = 64 * _log(rng, 4, 112), 32 * _log(rng, 4, 64)
    if rng.random() < 0.25:
        H, F = H + 8 * rng.randint(1, 7), F + rng.randint(1, 31)
    return _moe(_log(rng, 1, 8192), E, rng.randint(1, min(E, 8)), H, F, rng.choice([0.0, 1.1]))


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "fp32" else 2
        # logits and bias in, ids and weights out; a score and a comparison or so per logit
        return {"bytes": T * E * size + (4 * E if case["bias"] else 0) + T * k * 8, "flops": 4 * T * E}
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": M * K + N * K + M * N * size + 4 * (M + N) + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    T, E, k, H, F = (case[n] for n in ("T", "E", "k", "H", "F"))
    touched = E * (1 - (1 - k / E) ** T) if case["skew"] == 0 else min(E, T * k)
    return {"bytes": int(touched * (3 * H * F + 4 * (2 * F + H)) + 4 * T * H + 8 * T * k), "flops": 6 * T * k * H * F}


# ------------------------------------------------------------------ the inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(g, shape, std, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _quantise(v):
    """Symmetric INT8 codes and fp32 scales of the rows of v."""
    v = v.float()
    s = v.abs().amax(dim=-1) / 127.0
    q = torch.where(s[..., None] > 0, torch.round(v / s[..., None]), torch.zeros_like(v))
    return q.clamp_(-127, 127).to(torch.int8), s


def _pad_k(q):
    """INT8 rows padded with zeros to a multiple of 128, as the library keeps them."""
    out = torch.zeros((q.shape[0], -(-q.shape[1] // 128) * 128), dtype=torch.int8, device=q.device)
    out[:, :q.shape[1]] = q
    return out


def _weights(g, E, N, K, layout):
    """E random bf16 matrices [N][K], one after the other: packed by the library, or their INT8 codes and scales."""
    if own:
        from w4a8_quantized_moe_token_b200 import binding as B
        w = torch.empty((E, N, K), dtype=torch.bfloat16, device="cuda")
        for e in range(E):
            w[e] = _normal(g, (N, K), 0.02, torch.bfloat16)
        packed = B.empty_aligned(B.w8a8_packed_bytes(E, N, K, layout))
        B.w8a8_pack_weights(w, layout, packed)
        return packed
    q = torch.empty((E, N, K), dtype=torch.int8, device="cuda")
    s = torch.empty((E, N), dtype=torch.float32, device="cuda")
    for e in range(E):
        q[e], s[e] = _quantise(_normal(g, (N, K), 0.02, torch.bfloat16))
    return q, s


def _choice(g, T, E, k, skew):
    """k distinct experts per token (expert e with probability ~ 1 / rank(e)^skew) and gate weights that sum to 1."""
    rank = torch.randperm(E, generator=g, device="cuda").float()
    u = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    keys = -skew * torch.log1p(rank) - torch.log(-torch.log(u))
    ids = keys.sort(dim=1, descending=True).indices[:, :k].to(torch.int32).contiguous()
    w = torch.randn((T, k), generator=g, device="cuda").exp()
    return ids, (w / w.sum(dim=1, keepdim=True)).contiguous()


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _normal(g, (T, E), 1.5, TYPES[case["dtype"]])
        s["bias"] = _normal(g, (E,), 0.05, torch.float32) if case["bias"] else None
        if own:
            s["ids"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
            s["w"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
    elif case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        qa, s["sa"] = _quantise(_normal(g, (M, K), 1.0, torch.bfloat16))
        s["qa"] = _pad_k(qa)  # as w4a8_quant_act writes them
        s["bias"] = _normal(g, (N,), 0.5, torch.float32) if case["bias"] else None
        s["weights"] = _weights(g, 1, N, K, 0)
        if own:
            from w4a8_quantized_moe_token_b200 import binding as B
            s["y"] = torch.empty((M, N), dtype=TYPES[case["dtype"]], device="cuda")
            s["ws"] = B.empty_aligned(B.w8a8_gemm_workspace_bytes(M, N, K))
    else:
        T, E, k, H, F = (case[n] for n in ("T", "E", "k", "H", "F"))
        s["x"] = _normal(g, (T, H), 1.0, torch.bfloat16)
        s["ids"], s["w"] = _choice(g, T, E, k, case["skew"])
        s["up"] = _weights(g, E, 2 * F, H, 1)
        s["down"] = _weights(g, E, H, F, 0)
        if own:
            from w4a8_quantized_moe_token_b200 import binding as B
            s["out"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
            s["ws"] = B.empty_aligned(B.w8a8_moe_workspace_bytes(T, E, k, H, F))
    return s


# -------------------------------------------------------------- the operators
def _first(v, n):
    """The n largest along the last axis, largest first, ties to the lower index."""
    return v.sort(dim=-1, descending=True, stable=True).indices[..., :n]


def _run_route(s):
    c = s["case"]
    T, E, k, n = c["T"], c["E"], c["k"], c["groups"]
    x = s["logits"].double()  # scores of neighbouring experts may differ by less than 32 bits hold
    if c["score"] == "softmax":
        p = (x - x.amax(dim=1, keepdim=True)).exp()
        p = p / p.sum(dim=1, keepdim=True)
    else:
        p = 1.0 / (1.0 + (-x).exp())
    # without a bias the scores rank as the logits do
    choice = x if s["bias"] is None else p + s["bias"].double()
    if n > 1:
        inside = choice.view(T, n, E // n)
        best = inside.sort(dim=2, descending=True).values
        score = best[:, :, 0] if s["bias"] is None else best[:, :, :2].sum(dim=2)
        kept = torch.zeros((T, n), dtype=torch.bool, device=x.device).scatter_(1, _first(score, c["kept"]), True)
        choice = torch.where(kept[:, :, None], inside, torch.full_like(inside, -math.inf)).view(T, E)
    ids = _first(choice, k)
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), (w * c["scale"]).float()


def _run_gemm(s):
    c = s["case"]
    q, sw = s["weights"]
    y = s["qa"][:, :c["K"]].float() @ q[0].float().T
    y = y * s["sa"][:, None] * sw[0][None, :]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(TYPES[c["dtype"]])


def _run_moe(s):
    c = s["case"]
    T, E, k, H, F = (c[n] for n in ("T", "E", "k", "H", "F"))
    (qu, su), (qd, sd) = s["up"], s["down"]
    qx, sx = _quantise(s["x"])
    slots = s["ids"].reshape(-1).sort(stable=True)
    counts = torch.bincount(slots.values, minlength=E).tolist()
    y = torch.empty((T * k, H), dtype=torch.float32, device=s["x"].device)
    at = 0
    for e, n in enumerate(counts):
        if n == 0:
            continue
        slot = slots.indices[at:at + n]
        at += n
        t = slot // k
        a = qx[t].float() @ qu[e].float().T * sx[t][:, None] * su[e]
        gate, up = a[:, :F], a[:, F:]
        h = (gate / (1.0 + (-gate).exp()) * up).bfloat16()
        qh, sh = _quantise(h)
        y[slot] = qh.float() @ qd[e].float().T * sh[:, None] * sd[e]
    return (y.view(T, k, H) * s["w"][:, :, None]).sum(dim=1).bfloat16()


def run(s):
    c = s["case"]
    if not own:
        return {"route": _run_route, "gemm": _run_gemm, "moe": _run_moe}[c["op"]](s)
    from w4a8_quantized_moe_token_b200 import binding as B
    if c["op"] == "route":
        flags = (SIGMOID if c["score"] == "sigmoid" else SOFTMAX) | (RENORM if c["renorm"] else 0)
        if c["groups"] > 1 and s["bias"] is not None:
            flags |= GROUP_TOP2
        B.w4a8_route_experts(s["logits"], c["k"], s["ids"], s["w"], flags, bias=s["bias"], n_group=c["groups"],
                             topk_group=c["kept"], scale=c["scale"])
        return s["ids"], s["w"]
    if c["op"] == "gemm":
        B.w8a8_gemm(s["qa"], s["sa"], s["weights"], c["N"], c["K"], s["y"], s["ws"], bias=s["bias"])
        return s["y"]
    B.w8a8_moe_forward(s["up"], s["down"], c["E"], c["H"], c["F"], s["x"], s["ids"], s["w"], s["out"], s["ws"])
    return s["out"]


# ----------------------------------------------------- the definitions, 64 bits
def _exact_route(case, g):
    T, E, k, n = case["T"], case["E"], case["k"], case["groups"]
    x = _normal(g, (T, E), 1.5, TYPES[case["dtype"]]).double()
    b = _normal(g, (E,), 0.05, torch.float32).double() if case["bias"] else None
    p = torch.softmax(x, dim=1) if case["score"] == "softmax" else torch.sigmoid(x)
    c = x if b is None else p + b
    ids = []
    allowed = torch.ones_like(c, dtype=torch.bool)
    if n > 1:
        size = E // n
        total = torch.stack([c[:, i * size:(i + 1) * size].topk(1 if b is None else min(2, size), dim=1).values.sum(dim=1)
                             for i in range(n)], dim=1)
        # a group stays if fewer than `kept` groups beat it (a tie goes to the lower index)
        lower = torch.arange(n, device=x.device)[None, :] < torch.arange(n, device=x.device)[:, None]
        beats = (total[:, None, :] > total[:, :, None]) | ((total[:, None, :] == total[:, :, None]) & lower[None])
        allowed = (beats.sum(dim=2) < case["kept"]).repeat_interleave(size, dim=1)
    c = c.masked_fill(~allowed, -math.inf)
    number = torch.arange(E, device=x.device)[None, :]
    for _ in range(k):
        best = c.amax(dim=1, keepdim=True)
        e = torch.where(c == best, number, E).amin(dim=1, keepdim=True)
        ids.append(e)
        c = c.scatter(1, e, -math.inf)
    ids = torch.cat(ids, dim=1)
    w = p.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), w * case["scale"]


def _exact_gemm(case, g):
    M, N, K = case["M"], case["N"], case["K"]
    q, sa = _quantise(_normal(g, (M, K), 1.0, torch.bfloat16))
    b = _normal(g, (N,), 0.5, torch.float32) if case["bias"] else None
    qw, sw = _quantise(_normal(g, (N, K), 0.02, torch.bfloat16))
    y = torch.matmul(q.double(), qw.double().t()).mul_(torch.outer(sa.double(), sw.double()))
    return y if b is None else y + b.double()


def _exact_moe(case, g):
    T, E, k, H, F = (case[n] for n in ("T", "E", "k", "H", "F"))
    q, s = _quantise(_normal(g, (T, H), 1.0, torch.bfloat16))
    ids, w = _choice(g, T, E, k, case["skew"])
    up = []
    for e in range(E):
        up.append(_quantise(_normal(g, (2 * F, H), 0.02, torch.bfloat16)))
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        qd, sd = _quantise(_normal(g, (H, F), 0.02, torch.bfloat16))
        chosen = ids == e
        t = chosen.any(dim=1).nonzero()[:, 0]
        if t.numel() == 0:
            continue
        qu, su = up[e]
        up[e] = None
        a = torch.matmul(q[t].double(), qu.double().t()).mul_(torch.outer(s[t].double(), su.double()))
        h = (torch.nn.functional.silu(a[:, :F]) * a[:, F:]).to(torch.bfloat16)
        qh, sh = _quantise(h)
        y = torch.matmul(qh.double(), qd.double().t()).mul_(torch.outer(sh.double(), sd.double()))
        out[t] += y * (w[t].double() * chosen[t]).sum(dim=1, keepdim=True)
    return out


def exact(case, seed):
    return {"route": _exact_route, "gemm": _exact_gemm, "moe": _exact_moe}[case["op"]](case, _generator(seed))
