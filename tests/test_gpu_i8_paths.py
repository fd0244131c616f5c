"""The 8-bit integer lane as a program uses it: a feed-forward block from Q4_K weights, graphs,
streams, shared workspaces, waits that run out, and the routes that the sizes of the other
tests do not take."""
import numpy as np
import pytest
import torch

import synth
from oracle import i8 as OI
from oracle import q4k as O
from tests.gpu_util import dev, host
from tests.test_gpu_i8 import check_moe, codes, gemm_ref32, moe_inputs, scales, _gen

pytestmark = pytest.mark.gpu

q = pytest.importorskip("q4_weight_only_super_b200")

F64 = torch.float64
TIMEOUT = 7  # Q4K_ERR_DEVICE_TIMEOUT


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_ok):
    q.lib()
    q.q4k_test_wait_fault(-1, 0)
    assert q.q4k_last_device_status() == 0
    yield
    q.q4k_test_wait_fault(-1, 0)
    assert q.q4k_last_device_status() == 0


# ------------------------------------------------------------------ against the oracle

def test_against_the_numpy_oracle():
    rng = np.random.default_rng(5)
    x = synth.bf16_normal(rng, (9, 272))
    Q, s = q.i8_quantize(dev(x))
    Qr, sr = OI.quantize_rows(x)
    assert np.array_equal(host(Q), Qr) and np.array_equal(host(s), sr)
    W, sw = rng.integers(-128, 128, (77, 272)).astype(np.int8), rng.random(77).astype(np.float32)
    y = host(q.i8_gemm(dev(W), dev(sw), Q, s))
    assert np.array_equal(y, OI.matmul_ref(W, sw, Qr, sr)[1])
    E, H, Fw = 6, 272, 80
    wg, wd = rng.integers(-127, 128, (E, 2 * Fw, H)).astype(np.int8), rng.integers(-127, 128, (E, H, Fw)).astype(np.int8)
    sg, sd = (rng.random((E, 2 * Fw)) / 1000).astype(np.float32), (rng.random((E, H)) / 1000).astype(np.float32)
    L = rng.standard_normal((9, E)).astype(np.float32)
    y = host(q.moe_i8_layer(dev(L), 3, dev(wg), dev(sg), dev(wd), dev(sd), dev(x)))
    ref = OI.moe_layer_ref(L, 3, wg, sg, wd, sd, x)
    assert np.linalg.norm(y - ref) <= 2e-6 * np.linalg.norm(ref)  # 24-bit operands and fp32 sums


# ------------------------------------------------------------- a feed-forward block

def ffn(Wgu, sgu, Wd, sd, x):
    """int8 FFN: quantise, gate and up with SwiGLU, quantise, down."""
    Xq, sx = q.i8_quantize(x)
    h = q.i8_gemm(Wgu, sgu, Xq, sx, act=q.ACT_SWIGLU)
    Hq, sh = q.i8_quantize(h)
    return h, Hq, sh, q.i8_gemm(Wd, sd, Hq, sh)


@pytest.mark.parametrize("M", [1, 7, 40, 300])
def test_ffn_from_q4k_weights(M):
    """Q4_K weights dequantised to bf16 rows, quantised per channel at load, then the block;
    each stage against 64 bits from its own inputs, and the whole against the Q4_K product."""
    H, Fw = 512, 768
    rng = np.random.default_rng(M)
    Wgu4, Wd4 = synth.q4k_random_blocks(rng, 2 * Fw, H), synth.q4k_random_blocks(rng, H, Fw)
    bgu, bd = q.q4k_dequant(dev(Wgu4), out_bf16=True).view(2 * Fw, H), q.q4k_dequant(dev(Wd4), out_bf16=True).view(H, Fw)
    (Wgu, sgu), (Wd, sd) = q.i8_quantize(bgu), q.i8_quantize(bd)
    # a code is off by at most half a step s = amax / 127 of its row, and the scale by 2^-24 of
    # itself, which 127 codes make 127 * 2^-24 s
    assert ((bgu.to(F64) - Wgu.to(F64) * sgu.to(F64)[:, None]).abs() <= (0.5 + 128 * 2.0 ** -24) * sgu.to(F64)[:, None]).all()
    x = dev(synth.bf16_normal(rng, (M, H))).view(torch.bfloat16)
    h, Hq, sh, y = ffn(Wgu, sgu, Wd, sd, x)
    Xq, sx = q.i8_quantize(x)
    gu = gemm_ref32(Wgu, sgu, Xq, sx).to(F64)
    exact = gu[:, :Fw] * torch.sigmoid(gu[:, :Fw]) * gu[:, Fw:]
    assert ((h.to(F64) - exact).abs() <= exact.abs() * (2.0 ** -8 + 2.0 ** -18) + 1e-38).all()
    assert torch.equal(y, gemm_ref32(Wd, sd, Hq, sh))
    # the int8 gate and up product against the Q4_K one: the quantisation's own bound
    g4 = q.q4k_gemm(dev(Wgu4), x, 2 * Fw, H).to(F64)
    xa, wa = x.to(F64), bgu.to(F64)
    bound = 0.5 * sx.to(F64)[:, None] * wa.abs().sum(1) + 0.5 * sgu.to(F64) * xa.abs().sum(1)[:, None] \
        + 0.25 * H * sx.to(F64)[:, None] * sgu.to(F64) + 1e-4 * (xa.abs() @ wa.abs().T)
    assert ((gu - g4).abs() <= bound).all()


# ------------------------------------------------------------- graphs and streams

def moe_case(seed, M, E, topk, H, Fw):
    L, Wg, sg, Wd, sd, X = moe_inputs(seed, M, E, H, Fw)
    return (L, topk, Wg, sg, Wd, sd, X)


def test_captured_and_replayed():
    g0 = _gen(1)
    H, Fw = 256, 320
    Wgu, sgu, Wd, sd = codes(g0, 2 * Fw, H), scales(g0, 2 * Fw) / 30, codes(g0, H, Fw), scales(g0, H)
    x = torch.randn(12, H, generator=g0, device="cuda").to(torch.bfloat16)
    moe = moe_case(2, 12, 16, 3, H, 128)
    q.moe_i8_layer(*moe), ffn(Wgu, sgu, Wd, sd, x)  # first calls outside the capture
    ws = torch.empty(q.q4k_workspace_bytes(q.OP_MOE_I8, 12, H, 128, 16, 3), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = ffn(Wgu, sgu, Wd, sd, x)[3]
        z = q.moe_i8_layer(*moe, residual=y, ws=ws)
        z = q.moe_i8_layer(*moe, residual=z, Y=z, ws=ws)  # the same workspace, in order
    for seed in (3, 4, 5):
        x.copy_(torch.randn(12, H, generator=_gen(seed), device="cuda"))
        moe[0].copy_(torch.randn(12, 16, generator=_gen(seed + 10), device="cuda"))
        g.replay()
        ye = ffn(Wgu, sgu, Wd, sd, x)[3]
        ze = q.moe_i8_layer(*moe, residual=ye)
        ze = q.moe_i8_layer(*moe, residual=ze)
        torch.cuda.synchronize()
        assert torch.equal(y, ye) and torch.equal(z, ze)


@pytest.mark.parametrize("raw", [False, True])
def test_on_a_given_stream(raw):
    g0 = _gen(6)
    W, sw = codes(g0, 300, 512), scales(g0, 300)
    x = torch.randn(20, 512, generator=g0, device="cuda").to(torch.bfloat16)
    moe = moe_case(7, 5, 12, 2, 128, 64)
    expect = q.i8_gemm(W, sw, *q.i8_quantize(x)), q.moe_i8_layer(*moe)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    st = s.cuda_stream if raw else s
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)  # what runs on another stream would read too early
        x2 = x * 1
    Q, sx = q.i8_quantize(x2, stream=st)
    y = q.i8_gemm(W, sw, Q, sx, stream=st)
    z = q.moe_i8_layer(*moe, stream=st)
    s.synchronize()
    assert torch.equal(y, expect[0]) and torch.equal(z, expect[1])


def test_two_streams_at_once():
    cases = [moe_case(20 + i, 9, 24, 4, 256, 192) for i in range(2)]
    g0 = _gen(8)
    prods = [(codes(g0, 700, 1024), scales(g0, 700), codes(g0, m, 1024), scales(g0, m)) for m in (3, 260)]
    expect = [(q.moe_i8_layer(*c), q.i8_gemm(*p)) for c, p in zip(cases, prods)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((q.moe_i8_layer(*cases[i]), q.i8_gemm(*prods[i])))
    torch.cuda.synchronize()
    for i in range(2):
        for m, y in got[i]:
            assert torch.equal(m, expect[i][0]) and torch.equal(y, expect[i][1])


# ------------------------------------------------------------------ other routes

@pytest.mark.parametrize("M,E,topk,H,F", [(32, 300, 16, 144, 80), (29, 1024, 11, 64, 48), (12, 257, 1, 272, 16),
                                          (32, 40, 16, 1040, 208), (32, 8, 8, 128, 64), (2, 3, 3, 4096, 32),
                                          (3, 5, 2, 32, 3104), (11, 129, 9, 16, 1040), (32, 130, 4, 20000, 16)])
def test_moe_more_shapes(M, E, topk, H, F):
    case = moe_case(M + E + H, M, E, topk, H, F)
    L, k, Wg, sg, Wd, sd, X = case
    check_moe(q.moe_i8_layer(*case), L, k, Wg, sg, Wd, sd, X)


def test_moe_rows_of_very_different_size():
    """A token, and a row of h, far above the others: each row has its own scale."""
    L, Wg, sg, Wd, sd, X = moe_inputs(31, 8, 6, 256, 128)
    X = (X.float() * torch.tensor([1e-20, 1.0, 1e15, 3.0, 1e-30, 1e3, 0.0, 2.0], device="cuda")[:, None]).to(torch.bfloat16)
    sg, sd = sg * 1e-3, sd
    Y = q.moe_i8_layer(L, 2, Wg, sg, Wd, sd, X)
    for t in range(8):
        check_moe(Y[t:t + 1], L[t:t + 1], 2, Wg, sg, Wd, sd, X[t:t + 1])
    assert torch.count_nonzero(Y[6]) == 0


def test_moe_one_hot_activations():
    """All of a row in one value: one column of the weights, exact to fp32 rounding."""
    L, Wg, sg, Wd, sd, X = moe_inputs(32, 4, 4, 192, 64)
    X = torch.zeros_like(X)
    for t, (k, v) in enumerate(((0, 1.0), (191, -3.5), (64, 0.0078125), (17, 250.0))):
        X[t, k] = v
    check_moe(q.moe_i8_layer(L, 2, Wg, sg, Wd, sd, X), L, 2, Wg, sg, Wd, sd, X)


def test_moe_leaves_its_surroundings():
    case = moe_case(33, 5, 9, 3, 144, 48)
    big = torch.full((9, 144), 7.0, device="cuda")
    q.moe_i8_layer(*case, Y=big[2:7])
    assert torch.equal(big[2:7], q.moe_i8_layer(*case))
    assert (big[:2] == 7).all() and (big[7:] == 7).all()


@pytest.mark.parametrize("M,N,K", [(1, 40000, 64), (3, 16, 131056), (2500, 130, 48), (257, 33, 8192), (1000, 16, 16384),
                                   (511, 2064, 144), (48, 5000, 2064), (96, 300, 30000)])
@pytest.mark.parametrize("act", [0, 1])
def test_gemm_more_shapes(M, N, K, act):
    if act and N % 2:  # refused: as many gate as up rows
        N += 1
    g = _gen(M + N + K)
    W, X, sw, sx = codes(g, N, K), codes(g, M, K), scales(g, N) / K ** 0.5, scales(g, M)
    Y = q.i8_gemm(W, sw, X, sx, act=act)
    ref = gemm_ref32(W, sw, X, sx)
    if not act:
        assert torch.equal(Y, ref)
        return
    y = ref.to(F64)
    exact = y[:, :N // 2] * torch.sigmoid(y[:, :N // 2]) * y[:, N // 2:]
    assert ((Y.to(F64) - exact).abs() <= exact.abs() * (2.0 ** -8 + 2.0 ** -18) + 1e-38).all()


def test_gemm_swiglu_extremes():
    """Gates far out on both sides: silu(g) = g and silu(g) = 0, never an overflow."""
    W = torch.tensor([[127] * 16, [-127] * 16, [1] * 16, [1] * 16], dtype=torch.int8, device="cuda")
    X = torch.full((2, 16), 127, dtype=torch.int8, device="cuda")
    sw, sx = torch.tensor([1e3, 1e3, 1e-6, 1e-6], device="cuda"), torch.tensor([1.0, 1e20], device="cuda")
    Y = q.i8_gemm(W, sw, X, sx, act=q.ACT_SWIGLU).float()
    y = gemm_ref32(W, sw, X, sx)
    for m in range(2):
        up = (y[m, 0].to(F64) * y[m, 2].to(F64)).to(torch.float32).to(torch.bfloat16).float()
        assert Y[m, 0] == up or abs(Y[m, 0] / up - 1) <= 2.0 ** -7
        assert Y[m, 1] == 0


@pytest.mark.parametrize("K", [16, 4096])
@pytest.mark.parametrize("g", [-60.0, -88.5, -100.0, -150.0])
def test_gemm_swiglu_small_gate_times_large_up(K, g):
    """exp(g) below fp32's range, silu(g) * u well within it."""
    W = torch.zeros(2, K, dtype=torch.int8, device="cuda")
    W[0, :16], W[1, :16] = -127, 1
    X = torch.full((3, K), 127, dtype=torch.int8, device="cuda")
    u = 1e4 * 10.0 ** (-g / 2.5)
    if u > 1e38:
        u = 1e38
    sw = torch.tensor([-g / (127 * 127 * 16), u / (127 * 16)], dtype=torch.float32, device="cuda")
    Y = q.i8_gemm(W, sw, X, torch.ones(3, device="cuda"), act=q.ACT_SWIGLU)
    gate, up = -127.0 * 127 * 16 * float(sw[0]), 127.0 * 16 * float(sw[1])
    exact = gate * np.exp(gate) / (1 + np.exp(gate)) * up
    # the gate's two roundings move the exponential by 2 * 2^-24 |g|, ex2 of half of it, squared, by
    # 2 * (2 + 0.6 |g|) ulp of 2^-23; a few roundings more: below 2^-14 together; then bf16
    assert (abs(Y.double().cpu() / exact - 1) <= 2.0 ** -8 + 2.0 ** -14).all()


# ------------------------------------------------------------ refusals on the GPU

def test_binding_refusals():
    g = _gen(40)
    W, sw, X, sx = codes(g, 32, 64), scales(g, 32), codes(g, 4, 64), scales(g, 4)
    bad = [dict(W=W.t()), dict(W=codes(g, 32, 128)[:, ::2]), dict(w_scale=sw[:31]), dict(w_scale=sw.double()),
           dict(X=X[:, :48]), dict(X=X.to(torch.int32)), dict(x_scale=sx.cpu()), dict(x_scale=sx[::2]),
           dict(Y=torch.empty(4, 31, device="cuda")), dict(Y=torch.empty(4, 32, device="cuda", dtype=torch.float16)),
           dict(X=X.cpu())]
    for change in bad:
        with pytest.raises(ValueError):
            q.i8_gemm(**{**dict(W=W, w_scale=sw, X=X, x_scale=sx), **change})
    with pytest.raises(ValueError):
        q.i8_gemm(W, sw, X, sx, act=q.ACT_SWIGLU, Y=torch.empty(4, 16, device="cuda"))  # fp32 for SwiGLU
    with pytest.raises(q.Q4KError):
        q.i8_quantize(torch.zeros(2, 24, dtype=torch.bfloat16, device="cuda"))  # K % 16
    with pytest.raises(ValueError):
        q.i8_quantize(torch.zeros(2, 32, device="cuda"))
    case = list(moe_case(41, 3, 6, 2, 64, 32))
    for i, wrong in ((0, case[0][:, :5]), (2, case[2][:, :48]), (3, case[3][:5]), (4, case[4].transpose(1, 2)),
                     (5, case[5].half()), (6, case[6].float())):
        with pytest.raises(ValueError):
            q.moe_i8_layer(*case[:i], wrong, *case[i + 1:])
    with pytest.raises(q.Q4KError):
        q.moe_i8_layer(*case, ws=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(q.Q4KError):
        q.moe_i8_layer(case[0], 7, *case[2:])  # topk > E
    empty = q.moe_i8_layer(case[0][:0], 2, *case[2:6], case[6][:0])
    assert empty.shape == (0, 64) and q.i8_gemm(W, sw, X[:0], sx[:0]).shape == (0, 32)
    assert q.i8_quantize(torch.zeros(0, 32, dtype=torch.bfloat16, device="cuda"))[0].shape == (0, 32)


# ------------------------------------------------------------- waits that run out

@pytest.mark.parametrize("op", ["gemm_lone", "gemm_split", "gemm_pair", "moe"])
def test_bounded_wait_expires_and_recovers(op):
    g = _gen(50)
    if op == "moe":
        case = moe_case(51, 6, 10, 3, 256, 192)
        call = lambda: q.moe_i8_layer(*case)
    else:
        # many tiles of few tokens: lone CTAs; one tile with a long K: a cluster splits it; many
        # tokens: pairs
        M, N, K = {"gemm_lone": (4, 30000, 1024), "gemm_split": (4, 128, 16384), "gemm_pair": (1024, 17408, 1024)}[op]
        W, sw, X, sx = codes(g, N, K), scales(g, N), codes(g, M, K), scales(g, M)
        call = lambda: q.i8_gemm(W, sw, X, sx)
    good = call()
    assert q.q4k_last_device_status() == 0
    try:
        q.q4k_test_wait_fault(0, 200_000)  # skip stage 0 everywhere; 200 us limit
        call()
        assert q.q4k_last_device_status() == TIMEOUT
    finally:
        q.q4k_test_wait_fault(-1, 0)
    assert q.q4k_last_device_status() == 0
    assert torch.equal(call(), good)
    assert q.q4k_last_device_status() == 0
