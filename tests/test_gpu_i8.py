"""The 8-bit integer lane on the GPU against plain 64-bit implementations.

Tolerances. i8_quantize and the integer sums are exact: codes compare equal, and
i8_gemm's fp32 result is RN(RN(RN(acc) * sx) * sw) of an exact int32 acc, three roundings of
at most 2^-24 each, so it is compared for equality with the same three fp32 operations and
within 3 * 2^-24 (+ second order) of the 64-bit value. A bf16 result adds 2^-8 / 2 ... half a
bf16 step, 2^-9 relative of a value in [1, 2) at the top and 2^-8 at the bottom: eps/2 = 2^-8.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

q = pytest.importorskip("q4_weight_only_super_b200")

F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_ok):
    q.lib()
    q.q4k_last_device_status()
    yield
    assert q.q4k_last_device_status() == 0


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def codes(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int32).to(torch.int8)


def scales(g, *shape):
    return torch.rand(shape, generator=g, device="cuda") * 0.02 + 1e-4


# ------------------------------------------------------------------ i8_quantize

def quantize_ref(X):
    """Exact rounding of 127 x / amax in integers: the remainder decides, ties to even."""
    x = X.to(F64)
    amax = x.abs().amax(dim=1, keepdim=True)
    d = amax.clamp_min(1e-300)
    low = torch.floor(127 * x / d)
    twice = 2 * (127 * x - low * d)
    codes = low + ((twice > d) | ((twice == d) & (low % 2 != 0)))
    codes = torch.where(amax > 0, codes, torch.zeros_like(codes))
    # divided in 64 bits: an 8-bit value over 127 lies nowhere near a 24-bit midpoint, so the
    # second rounding changes nothing (torch divides 32-bit tensors by a number as x * (1/127))
    return codes.to(torch.int8), (amax[:, 0] / 127).to(torch.float32)


@pytest.mark.parametrize("M,K", [(1, 16), (1, 5120), (7, 48), (33, 1024), (3, 1040), (9, 4096), (5, 4112), (4, 8192),
                                 (3, 8208), (2, 16384), (2, 17408), (2, 32768), (3, 40000), (1000, 256), (1, 131056)])
def test_quantize_matches_the_definition(M, K):
    g = _gen(M * 1000 + K)
    X = torch.randn(M, K, generator=g, device="cuda") * torch.exp(3 * torch.randn(M, 1, generator=g, device="cuda"))
    X = X.to(torch.bfloat16)
    Q, s = q.i8_quantize(X)
    Qr, sr = quantize_ref(X)
    assert torch.equal(Q, Qr)
    assert torch.equal(s, sr)


def test_quantize_ties_and_every_bf16_ratio():
    # amax fixed at 1 and at 254 (127 x / amax = x / 2: every odd x is a tie), every other value below
    for top in (1.0, 254.0, 1.9921875):
        bits = torch.arange(0, 0x4380, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
        vals = bits[bits.float() <= top]
        K = 4096
        n = (vals.numel() + K - 2) // (K - 1)
        X = torch.zeros(n, K, dtype=torch.bfloat16, device="cuda")
        X[:, 0] = top
        for r in range(n):
            part = vals[r * (K - 1):(r + 1) * (K - 1)]
            X[r, 1:1 + part.numel()] = part
        X[:, 1::2] = -X[:, 1::2]
        Q, s = q.i8_quantize(X)
        Qr, sr = quantize_ref(X)
        assert torch.equal(Q, Qr) and torch.equal(s, sr)


@pytest.mark.parametrize("size", [2.0 ** -130, 2.0 ** -100, 2.0 ** -64, 2.0 ** -63, 2.0 ** 99, 2.0 ** 100, 2.0 ** 127])
def test_quantize_extreme_magnitudes(size):
    X = (torch.rand(4, 96, generator=_gen(5), device="cuda", dtype=F64) * 2 - 1) * size
    X = X.to(torch.float32).to(torch.bfloat16)
    Q, s = q.i8_quantize(X)
    Qr, sr = quantize_ref(X)
    assert torch.equal(Q, Qr) and torch.equal(s, sr)


def test_quantize_zero_rows_and_non_finite_rows():
    X = torch.randn(6, 48, generator=_gen(6), device="cuda").to(torch.bfloat16)
    X[1] = 0
    X[2, 5] = float("inf")
    X[3, 7] = float("nan")
    X[4, 0] = -float("inf")
    Q, s = q.i8_quantize(X)
    for r in (0, 5):
        Qr, sr = quantize_ref(X[r:r + 1])
        assert torch.equal(Q[r:r + 1], Qr) and torch.equal(s[r:r + 1], sr)
    assert s[1] == 0 and torch.count_nonzero(Q[1:5]) == 0
    assert torch.isnan(s[2:5]).all()


def test_quantize_leaves_its_surroundings():
    """Rows before and behind the outputs stay as they were."""
    X = torch.randn(3, 80, generator=_gen(7), device="cuda").to(torch.bfloat16)
    Qb = torch.full((5, 80), 99, dtype=torch.int8, device="cuda")
    sb = torch.full((12,), 7.0, device="cuda")
    q.i8_quantize(X, Q=Qb[1:4], scale=sb[4:7])
    Qr, sr = quantize_ref(X)
    assert torch.equal(Qb[1:4], Qr) and torch.equal(sb[4:7], sr)
    assert (Qb[[0, 4]] == 99).all() and (sb[:4] == 7).all() and (sb[7:] == 7).all()


# ---------------------------------------------------------------------- i8_gemm

def acc_ref(W, X):
    return torch.round(X.to(F64) @ W.to(F64).T)  # integers below 2^31: exact in fp64


def gemm_ref32(W, sw, X, sx):
    """The three fp32 roundings of the definition."""
    return acc_ref(W, X).to(torch.float32) * sx[:, None] * sw


SHAPES = [(1, 1, 16), (1, 128, 128), (1, 300, 80), (2, 129, 144), (5, 64, 2064), (8, 5120, 1024), (15, 33, 4096),
          (16, 257, 384), (17, 1000, 272), (31, 515, 640), (32, 2048, 2048), (33, 200, 1040), (37, 2051, 2064),
          (64, 640, 512), (100, 130, 17408), (128, 1024, 656), (129, 384, 256), (200, 999, 1024), (255, 128, 4096),
          (256, 512, 512), (257, 640, 400), (300, 1283, 2048), (512, 768, 1024), (513, 4096, 128), (700, 100, 16),
          (1025, 2048, 208), (2048, 1536, 512)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out_bf16", [False, True])
def test_gemm_matches_the_definition(M, N, K, out_bf16):
    g = _gen(M * 7 + N * 3 + K)
    W, X, sw, sx = codes(g, N, K), codes(g, M, K), scales(g, N), scales(g, M)
    Y = q.i8_gemm(W, sw, X, sx, out_bf16=out_bf16)
    ref = gemm_ref32(W, sw, X, sx)
    if out_bf16:
        assert torch.equal(Y, ref.to(torch.bfloat16))
        return
    assert torch.equal(Y, ref)
    exact = acc_ref(W, X) * sx.to(F64)[:, None] * sw.to(F64)
    assert ((Y.to(F64) - exact).abs() <= 3.0000002 * 2.0 ** -24 * exact.abs()).all()


@pytest.mark.parametrize("M,F,K", [(1, 1, 16), (1, 64, 128), (1, 17408, 512), (3, 63, 144), (8, 65, 2048), (16, 768, 2048),
                                   (17, 100, 1040), (33, 200, 272), (64, 1000, 512), (130, 129, 4096), (256, 512, 384),
                                   (300, 320, 1024), (512, 1027, 256), (1100, 448, 128)])
def test_gemm_swiglu(M, F, K):
    g = _gen(M + F * 5 + K)
    W, X = codes(g, 2 * F, K), codes(g, M, K)
    # gate and up values of a few units, as in a model
    sw, sx = scales(g, 2 * F) / (80 * K ** 0.5), scales(g, M) * 80
    Y = q.i8_gemm(W, sw, X, sx, act=q.ACT_SWIGLU)
    y = acc_ref(W, X) * sx.to(F64)[:, None] * sw.to(F64)
    gate, up = y[:, :F], y[:, F:]
    exact = gate * torch.sigmoid(gate) * up
    # bf16 rounding 2^-8 of the value; before it: g and u 3 roundings each, the exponential
    # (argument off by 3 * 2^-24 * |g|, 2 ulp of its own), sum, quotient, two products
    assert Y.dtype == torch.bfloat16
    tol = exact.abs() * (2.0 ** -8 + (16 + 3 * gate.abs()) * 2.0 ** -24 * (1 + 2.0 ** -8)) + 1e-38
    assert ((Y.to(F64) - exact).abs() <= tol).all()


def test_gemm_extreme_codes_and_longest_k():
    """-128 x -128 over the longest K: the largest sum, 2147221504, fits int32."""
    K = 131056
    W = torch.full((130, K), -128, dtype=torch.int8, device="cuda")
    X = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    X[1] = 127
    X[2] = 0
    one = torch.ones(130, device="cuda")
    Y = q.i8_gemm(W, one, X, one[:3].clone())
    ref = torch.tensor([128.0 * 128 * K, -128.0 * 127 * K, 0.0], dtype=F64).to(torch.float32)
    assert torch.equal(Y.cpu(), ref[:, None].expand(3, 130))


def test_gemm_rows_do_not_depend_on_the_batch():
    g = _gen(11)
    W, sw = codes(g, 700, 1024), scales(g, 700)
    X, sx = codes(g, 600, 1024), scales(g, 600)
    whole = q.i8_gemm(W, sw, X, sx)
    for M in (1, 8, 9, 16, 17, 40, 130, 300):
        assert torch.equal(q.i8_gemm(W, sw, X[:M], sx[:M]), whole[:M])


def test_gemm_special_scales():
    g = _gen(12)
    W, sw, X, sx = codes(g, 200, 256), scales(g, 200), codes(g, 40, 256), scales(g, 40)
    sx[3], sx[4], sw[7] = float("nan"), 0.0, float("inf")
    for M in (2, 40):
        Y = q.i8_gemm(W, sw, X[:M], sx[:M])
        ref = gemm_ref32(W, sw, X[:M], sx[:M])
        assert torch.equal(torch.isnan(Y), torch.isnan(ref))
        assert torch.equal(torch.nan_to_num(Y, 0.0), torch.nan_to_num(ref, 0.0))


@pytest.mark.parametrize("M", [1, 8, 20, 130, 300])
@pytest.mark.parametrize("act", [0, 1])
def test_gemm_leaves_its_surroundings(M, act):
    g = _gen(13)
    N, K = 202, 272
    W, sw, X, sx = codes(g, N, K), scales(g, N), codes(g, M, K), scales(g, M)
    wide = N // 2 if act else N
    big = torch.full(((M + 16) * wide,), 5.0, dtype=torch.bfloat16 if act else torch.float32, device="cuda")
    Y = big[8 * wide:(8 + M) * wide].view(M, wide)
    q.i8_gemm(W, sw, X, sx, act=act, Y=Y)
    assert torch.equal(Y, q.i8_gemm(W, sw, X, sx, act=act))
    assert (big[:8 * wide] == 5).all() and (big[(8 + M) * wide:] == 5).all()


# ----------------------------------------------------------------- moe_i8_layer

def route_ref(logits, topk):
    ids, ws = [], []
    for row in logits.tolist():
        order = sorted(range(len(row)), key=lambda e: (-row[e], e))[:topk]
        v = np.array([row[e] for e in order], dtype=np.float64)
        p = np.exp(v - v[0])
        ids.append(order)
        ws.append(p / p.sum())
    return ids, ws


def moe_ref(L, topk, Wg, sg, Wd, sd, X, residual=None):
    """(value, sum of magnitudes of its terms, sum of the down weights' magnitudes) per output, in
    64 bits."""
    M, E = L.shape
    F, H = Wd.shape[2], Wd.shape[1]
    ids, ws = route_ref(L, topk)
    y = torch.zeros(M, H, dtype=F64, device="cuda") if residual is None else residual.to(F64).clone()
    S, A = y.abs().clone(), torch.zeros_like(y)
    for t in range(M):
        x = X[t].to(F64)
        for e, p in zip(ids[t], ws[t]):
            wg, wd = Wg[e].to(F64) * sg[e].to(F64)[:, None], Wd[e].to(F64) * sd[e].to(F64)[:, None]
            gu = wg @ x
            a = wg.abs() @ x.abs()
            gate, up = gu[:F], gu[F:]
            sig = torch.sigmoid(gate)
            h = gate * sig * up
            # how far h may be off per unit of relative error in the sums: d h <= a_g |up| * 1.1 + a_u |silu|
            hm = 1.1 * a[:F] * up.abs() + a[F:] * (gate * sig).abs() + h.abs()
            y[t] += p * (wd @ h)
            S[t] += p * (wd.abs() @ hm)
            A[t] += p * wd.abs().sum(1)
    return y, S, A


def moe_inputs(seed, M, E, H, F):
    g = _gen(seed)
    L = 2 * torch.randn(M, E, generator=g, device="cuda")
    X = torch.randn(M, H, generator=g, device="cuda").to(torch.bfloat16)
    Wg, Wd = codes(g, E, 2 * F, H), codes(g, E, H, F)
    sg, sd = scales(g, E, 2 * F) / H ** 0.5, scales(g, E, H) / F ** 0.5
    return L, Wg, sg, Wd, sd, X


def check_moe(Y, L, topk, Wg, sg, Wd, sd, X, residual=None):
    y, S, A = moe_ref(L, topk, Wg, sg, Wd, sd, X, residual)
    H, F = X.shape[1], Wd.shape[2]
    # fp32 sums of exact products: at most one rounding (2^-23, truncation allowed for) per
    # 16-term MMA step and per later addition, of a partial sum below the sum of magnitudes
    u = 2.0 ** -23
    tol = ((H / 16 + F / 16 * 3 + 64 + topk) * u + 1e-6) * S  # 1e-6: the routing weights' own bound
    tol += 2.0 ** -123 * A  # the resolution of h where it is below 2^-100 throughout a row
    err = (Y.to(F64) - y).abs()
    assert (err <= tol).all(), float((err / tol.clamp_min(1e-300)).max())


MOE = [(1, 128, 8, 2048, 768), (1, 4, 1, 16, 16), (1, 1, 1, 64, 64), (2, 8, 2, 128, 64), (3, 33, 5, 80, 48),
       (5, 40, 3, 1040, 336), (8, 128, 8, 2048, 768), (9, 3, 3, 256, 128), (16, 64, 16, 512, 80), (32, 2, 2, 272, 144),
       (32, 128, 8, 512, 256), (31, 200, 6, 528, 208), (32, 1, 1, 1024, 512), (7, 600, 4, 64, 32), (4, 1024, 16, 48, 16),
       (1, 16, 2, 4096, 2048)]


@pytest.mark.parametrize("M,E,topk,H,F", MOE)
@pytest.mark.parametrize("with_residual", [False, True])
def test_moe_layer(M, E, topk, H, F, with_residual):
    L, Wg, sg, Wd, sd, X = moe_inputs(M + 10 * E + H, M, E, H, F)
    R = torch.randn(M, H, generator=_gen(3), device="cuda") if with_residual else None
    Y = q.moe_i8_layer(L, topk, Wg, sg, Wd, sd, X, residual=R)
    check_moe(Y, L, topk, Wg, sg, Wd, sd, X, R)


def test_moe_equal_logits_go_to_the_lower_id():
    L, Wg, sg, Wd, sd, X = moe_inputs(21, 6, 24, 128, 64)
    L[0] = 0.0
    L[1, ::2] = 1.5
    L[2] = torch.where(torch.arange(24, device="cuda") % 3 == 0, 0.0, -0.0)  # +0 and -0 are equal
    L[3, 5:] = -float("inf")
    check_moe(q.moe_i8_layer(L, 4, Wg, sg, Wd, sd, X), L, 4, Wg, sg, Wd, sd, X)


def test_moe_equal_logits_of_many_experts():
    L, Wg, sg, Wd, sd, X = moe_inputs(27, 32, 1000, 32, 16)
    L[:30] = 0.25
    L[1, 960:] = 0.5  # the larger ones behind
    L[2] = torch.arange(1000, device="cuda") // 100  # ties at the last selected one
    check_moe(q.moe_i8_layer(L, 16, Wg, sg, Wd, sd, X), L, 16, Wg, sg, Wd, sd, X)


def test_moe_token_with_every_expert_masked_stays_alone():
    L, Wg, sg, Wd, sd, X = moe_inputs(28, 5, 12, 64, 48)
    L[2] = -float("inf")
    L[3, 1:] = -float("inf")  # one expert left: the others weigh nothing
    L[4] = torch.finfo(torch.float32).min  # the lowest value is a value: equal weights
    Y = q.moe_i8_layer(L, 4, Wg, sg, Wd, sd, X)
    assert torch.isnan(Y[2]).all()
    rest = [0, 1, 3, 4]
    check_moe(Y[rest], L[rest], 4, Wg, sg, Wd, sd, X[rest])


def test_moe_nan_logits_rank_last():
    L, Wg, sg, Wd, sd, X = moe_inputs(22, 3, 12, 64, 48)
    L[1, [0, 4, 7]] = float("nan")
    clean = L.clone()
    clean[1, [0, 4, 7]] = -1e30
    Y = q.moe_i8_layer(L, 4, Wg, sg, Wd, sd, X)
    assert torch.equal(Y, q.moe_i8_layer(clean, 4, Wg, sg, Wd, sd, X))
    L[1] = float("nan")  # nothing left to rank: this token alone is NaN
    Y2 = q.moe_i8_layer(L, 4, Wg, sg, Wd, sd, X)
    assert torch.isnan(Y2[1]).all()
    # the others' sums are taken in an order that depends on the whole routing: equal to fp32
    # rounding, not bit for bit
    check_moe(Y2[[0, 2]], L[[0, 2]], 4, Wg, sg, Wd, sd, X[[0, 2]])


def test_moe_non_finite_token_stays_alone():
    L, Wg, sg, Wd, sd, X = moe_inputs(23, 8, 4, 128, 64)
    Y = q.moe_i8_layer(L, 4, Wg, sg, Wd, sd, X)
    X2 = X.clone()
    X2[3, 17], X2[6, 2] = float("nan"), float("inf")
    Y2 = q.moe_i8_layer(L, 4, Wg, sg, Wd, sd, X2)
    rest = [0, 1, 2, 4, 5, 7]
    assert torch.equal(Y2[rest], Y[rest])
    assert torch.isnan(Y2[3]).all() and not torch.isfinite(Y2[6]).any()


def test_moe_all_tokens_on_the_same_experts():
    """32 rows per expert: four groups of eight."""
    L, Wg, sg, Wd, sd, X = moe_inputs(24, 32, 16, 256, 128)
    L[:, 3] += 20
    L[:, 11] += 30
    check_moe(q.moe_i8_layer(L, 2, Wg, sg, Wd, sd, X), L, 2, Wg, sg, Wd, sd, X)


def test_moe_residual_in_place_and_dirty_workspace():
    L, Wg, sg, Wd, sd, X = moe_inputs(25, 6, 20, 192, 96)
    R = torch.randn(6, 192, generator=_gen(4), device="cuda")
    Y = q.moe_i8_layer(L, 3, Wg, sg, Wd, sd, X, residual=R)
    need = q.q4k_workspace_bytes(q.OP_MOE_I8, 6, 192, 96, 20, 3)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    buf = R.clone()
    q.moe_i8_layer(L, 3, Wg, sg, Wd, sd, X, residual=buf, Y=buf, ws=ws[:need])
    assert torch.equal(buf, Y)
    assert (ws[need:] == 0xFF).all()


def test_moe_is_deterministic_and_rows_independent():
    L, Wg, sg, Wd, sd, X = moe_inputs(26, 32, 64, 512, 256)
    a = q.moe_i8_layer(L, 8, Wg, sg, Wd, sd, X)
    for _ in range(3):
        assert torch.equal(a, q.moe_i8_layer(L, 8, Wg, sg, Wd, sd, X))
