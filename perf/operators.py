"""The 8-bit integer operators as measurable cases: per-row quantisation, the int8 matrix
product with token and channel scales, and the whole mixture-of-experts layer for a few tokens.

A case names an operator (``op``) and its sizes. ``own = False`` computes the plain forms in
elementary torch operations; ``own = True`` makes the package's calls on the same state.
"""
import math

import torch

own = False


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode token's hidden state: latency of a single small launch
        dict(name="quantize 1x5120", op="quantize", M=1, K=5120),
        # a prefill batch's hidden states
        dict(name="quantize 4096x5120", op="quantize", M=4096, K=5120),
        # decode, one token: the dense layer's gate and up projections with SwiGLU
        dict(name="gemm 1 gate_up", op="gemm", M=1, N=34816, K=5120, act="swiglu", out="bf16"),
        # decode, eight sequences: the down projection into the fp32 residual stream
        dict(name="gemm 8 down", op="gemm", M=8, N=5120, K=17408, act="none", out="fp32"),
        # odd sizes throughout: a ragged batch, an odd number of channels, K not a multiple of a tile
        dict(name="gemm 37 ragged", op="gemm", M=37, N=2051, K=2064, act="none", out="fp32"),
        # a chunk of prefill, or many decoding sequences: the down projection, bf16 out
        dict(name="gemm 300 down", op="gemm", M=300, N=5120, K=17408, act="none", out="bf16"),
        # prefill: gate and up with SwiGLU
        dict(name="gemm 512 gate_up", op="gemm", M=512, N=34816, K=5120, act="swiglu", out="bf16"),
        # a long prefill: one projection, fp32 out
        dict(name="gemm 4096", op="gemm", M=4096, N=17408, K=5120, act="none", out="fp32"),
        # mixture-of-experts decode: one token, eight and thirty-two sequences
        dict(name="moe 1", op="moe", M=1, E=128, topk=8, H=2048, F=768, residual=True),
        dict(name="moe 8", op="moe", M=8, E=128, topk=8, H=2048, F=768, residual=True),
        dict(name="moe 32", op="moe", M=32, E=128, topk=8, H=2048, F=768, residual=False),
        # a small layer of odd sizes
        dict(name="moe 5 ragged", op="moe", M=5, E=40, topk=3, H=1040, F=336, residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "moe"])
    if op == "quantize":
        K = 16 * _log(rng, 1, 1088)
        return dict(op=op, M=min(_log(rng, 1, 8192), 4096 * 5120 // K), K=K)
    if op == "gemm":
        act = rng.choice(["none", "none", "swiglu"])
        M, K = _log(rng, 1, 4096), 16 * _log(rng, 4, 1088)
        N = _log(rng, 32, 34816)
        N = max(1, min(N, 4096 * 17408 * 5120 // (M * K), 34816 * 5120 // K))
        if act == "swiglu":
            return dict(op=op, M=M, N=2 * max(1, N // 2), K=K, act=act, out="bf16")
        return dict(op=op, M=M, N=N, K=K, act=act, out=rng.choice(["fp32", "bf16"]))
    E = _log(rng, 4, 160)
    H, F = 16 * _log(rng, 8, 256), 16 * _log(rng, 4, 128)
    E = max(2, min(E, 128 * 2048 * 768 // (H * F)))
    return dict(op=op, M=_log(rng, 1, 32), E=E, topk=rng.randint(1, min(E, 8)), H=H, F=F,
                residual=rng.random() < 0.5)


# --------------------------------------------------------------------------- inputs

def _codes(g, rows, K):
    """int8 rows as a per-row quantiser leaves them: near normal, the largest at 127."""
    q = torch.empty(rows, K, dtype=torch.int8, device="cuda")
    step = max(1, (1 << 26) // K)
    for r in range(0, rows, step):
        q[r:r + step] = torch.randn(q[r:r + step].shape, generator=g, device="cuda").mul_(32).round_().clamp_(-127, 127)
    return q


def _scales(g, shape, size):
    return size * torch.exp(0.3 * torch.randn(shape, generator=g, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "quantize":
        # activations of a transformer: normal, rows of their own size, a few channels far larger
        x = torch.randn(case["M"], case["K"], generator=g, device="cuda")
        x *= torch.exp(torch.randn(case["M"], 1, generator=g, device="cuda"))
        x[:, ::97] *= 12
        s["X"] = x.to(torch.bfloat16)
        s["Q"] = torch.empty(case["M"], case["K"], dtype=torch.int8, device="cuda")
        s["scale"] = torch.empty(case["M"], dtype=torch.float32, device="cuda")
    elif case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        s["W"], s["w_scale"] = _codes(g, N, K), _scales(g, (N,), 0.01 / math.sqrt(K))
        s["X"], s["x_scale"] = _codes(g, M, K), _scales(g, (M,), 0.03)
        wide = N // 2 if case["act"] == "swiglu" else N
        s["Y"] = torch.empty(M, wide, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device="cuda")
    else:
        M, E, H, F = case["M"], case["E"], case["H"], case["F"]
        s["logits"] = 2 * torch.randn(M, E, generator=g, device="cuda")
        s["X"] = torch.randn(M, H, generator=g, device="cuda").to(torch.bfloat16)
        s["W_gate_up"] = _codes(g, E * 2 * F, H).view(E, 2 * F, H)
        s["s_gate_up"] = _scales(g, (E, 2 * F), 1 / (32 * math.sqrt(H)))
        s["W_down"] = _codes(g, E * H, F).view(E, H, F)
        s["s_down"] = _scales(g, (E, H), 1 / (32 * math.sqrt(F)))
        s["R"] = torch.randn(M, H, generator=g, device="cuda") if case["residual"] else None
        s["Y"] = torch.empty(M, H, dtype=torch.float32, device="cuda")
        # the scratch buffer that a program keeps for all its layers
        s["ws"] = torch.empty(16 << 20, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------- the plain forms

def _quantize(X):
    # the code is 127 x / amax rounded to nearest, ties to even: next to a tie 32 bits would not decide it
    x = X.to(torch.float64)
    amax = x.abs().amax(dim=1, keepdim=True)
    q = torch.where(amax > 0, torch.round(127 * x / amax), 0 * x).to(torch.int8)
    return q, (amax[:, 0].to(torch.float32) / 127)


def _swiglu(gu):
    gate, up = gu.chunk(2, dim=-1)
    return gate / (1 + torch.exp(-gate)) * up


def _gemm(s):
    y = (s["X"].float() @ s["W"].float().T) * s["x_scale"][:, None] * s["w_scale"]
    return (_swiglu(y) if s["act"] == "swiglu" else y).to(s["Y"].dtype)


def _topk(logits, topk):
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    v, ids = order.values[:, :topk], order.indices[:, :topk]
    e = torch.exp(v - v[:, :1])
    return ids, e / e.sum(dim=1, keepdim=True)


def _moe(s, real=torch.float32):
    # every expert on every token, then the selected ones weighted
    ids, w = _topk(s["logits"].to(real), s["topk"])
    gates = torch.zeros(s["M"], s["E"], dtype=real, device="cuda").scatter_(1, ids, w)
    gu = torch.matmul(s["X"].to(real), s["W_gate_up"].to(real).transpose(1, 2)) * s["s_gate_up"].to(real)[:, None]
    o = torch.matmul(_swiglu(gu), s["W_down"].to(real).transpose(1, 2)) * s["s_down"].to(real)[:, None]
    y = (gates.T[:, :, None] * o).sum(dim=0)
    return y if s["R"] is None else s["R"].to(real) + y


# ------------------------------------------------------------------------- one pass

def run(s):
    if own:
        import q4_weight_only_super_b200 as q
        if s["op"] == "quantize":
            return q.i8_quantize(s["X"], Q=s["Q"], scale=s["scale"])
        if s["op"] == "gemm":
            return q.i8_gemm(s["W"], s["w_scale"], s["X"], s["x_scale"],
                             act=q.ACT_SWIGLU if s["act"] == "swiglu" else q.ACT_NONE, Y=s["Y"])
        return q.moe_i8_layer(s["logits"], s["topk"], s["W_gate_up"], s["s_gate_up"], s["W_down"], s["s_down"],
                              s["X"], residual=s["R"], Y=s["Y"], ws=s["ws"])
    if s["op"] == "quantize":
        return _quantize(s["X"])
    return _gemm(s) if s["op"] == "gemm" else _moe(s)


def exact(case, seed):
    """The same outputs from the definitions in 64 bits, written for one thing at a time."""
    s = prepare(case, seed)
    real = torch.float64
    if case["op"] == "quantize":
        X = s["X"].to(real)
        scale = X.abs().max(dim=1).values / 127
        # x / (amax / 127): (x / amax) * 127 would round twice before the tie is decided
        n, d = X * 127, X.abs().max(dim=1, keepdim=True).values.clamp_min(1e-300)
        low = torch.floor(n / d)
        twice = 2 * (n - low * d)  # exact: 15-bit numerators over 8-bit denominators
        up = (twice > d) | ((twice == d) & (low % 2 != 0))
        return (low + up).to(torch.int8), scale
    if case["op"] == "gemm":
        w = s["W"].to(real)
        y = torch.einsum("mk,nk->mn", s["X"].to(real), w).mul_(s["w_scale"].to(real)).mul_(s["x_scale"].to(real)[:, None])
        if case["act"] == "swiglu":
            half = case["N"] // 2
            y = y[:, half:] * y[:, :half] * torch.sigmoid(y[:, :half])
        return y
    # token by token, slot by slot
    y = torch.zeros(case["M"], case["H"], dtype=real, device="cuda") if s["R"] is None else s["R"].to(real)
    for t in range(case["M"]):
        row = s["logits"][t].tolist()
        ids = sorted(range(case["E"]), key=lambda e: (-row[e], e))[:case["topk"]]
        p = torch.softmax(torch.tensor([row[e] for e in ids], dtype=real), dim=0).tolist()
        x = s["X"][t].to(real)
        for e, pe in zip(ids, p):
            gu = (s["W_gate_up"][e].to(real) @ x) * s["s_gate_up"][e].to(real)
            h = gu[:case["F"]] * torch.sigmoid(gu[:case["F"]]) * gu[case["F"]:]
            y[t] += pe * ((s["W_down"][e].to(real) @ h) * s["s_down"][e].to(real))
    return y


def work(case):
    M, K = case["M"], case.get("K")
    if case["op"] == "quantize":
        return dict(bytes=3 * M * K + 4 * M, flops=3 * M * K)
    if case["op"] == "gemm":
        N = case["N"]
        wide = N // 2 if case["act"] == "swiglu" else N
        out = M * wide * (2 if case["out"] == "bf16" else 4)
        return dict(bytes=N * K + M * K + 4 * (M + N) + out, flops=2 * M * N * K)
    E, H, F, k = case["E"], case["H"], case["F"], case["topk"]
    # experts that at least one of M tokens selects, with tokens choosing alike and independently
    hit = E * (1 - (1 - k / E) ** M)
    wide = M * H * (2 + 4 + (4 if case["residual"] else 0)) + 4 * M * E
    return dict(bytes=hit * (3 * F * H + 4 * (2 * F + H)) + wide, flops=2 * M * k * 3 * F * H)
