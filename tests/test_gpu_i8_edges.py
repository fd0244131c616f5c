"""moe_i8_layer within the bound that its number formats allow, and the 8-bit lane at the edges
of what its entry points accept: masked experts, NaN logits, gates far below zero."""
import math

import pytest
import torch

from tests.i8_bound import moe_ref_and_bound
from tests.test_gpu_i8 import MOE, codes, moe_inputs, scales, _gen

pytestmark = pytest.mark.gpu

q = pytest.importorskip("q4_weight_only_super_b200")

F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_ok):
    q.lib()
    q.q4k_last_device_status()
    yield
    assert q.q4k_last_device_status() == 0


def within(Y, *case, residual=None):
    y, tol = moe_ref_and_bound(*case, residual=residual)
    bad = ~((Y.to(F64) - y).abs() <= tol)  # (a NaN is bad)
    assert not bad.any(), float(((Y.to(F64) - y).abs() / tol.clamp_min(1e-300)).max())


# ------------------------------------------------------------ the layer's precision

@pytest.mark.parametrize("M,E,topk,H,F", MOE + [(32, 128, 8, 2048, 768), (32, 300, 16, 144, 80), (32, 40, 16, 1040, 208),
                                                (3, 5, 2, 32, 3104), (29, 1024, 11, 64, 48), (6, 20, 4, 4096, 6400)])
@pytest.mark.parametrize("with_residual", [False, True])
def test_moe_keeps_24_bits(M, E, topk, H, F, with_residual):
    L, Wg, sg, Wd, sd, X = moe_inputs(M + 7 * E + H, M, E, H, F)
    R = 0.01 * torch.randn(M, H, generator=_gen(9), device="cuda") if with_residual else None
    within(q.moe_i8_layer(L, topk, Wg, sg, Wd, sd, X, residual=R), L, topk, Wg, sg, Wd, sd, X, residual=R)


def test_moe_rows_of_wide_range_keep_24_bits():
    """A few activations thousands of times the others."""
    L, Wg, sg, Wd, sd, X = moe_inputs(61, 9, 8, 1024, 256)
    X[:, ::97] *= 3000
    X[2, 5] *= 1e6
    sg = sg / 300
    within(q.moe_i8_layer(L, 3, Wg, sg, Wd, sd, X), L, 3, Wg, sg, Wd, sd, X)


def test_moe_tokens_do_not_touch_each_other():
    """With the routing as it is, other tokens' values change nothing, across groups of 8 rows."""
    L, Wg, sg, Wd, sd, X = moe_inputs(62, 32, 4, 320, 144)
    Y = q.moe_i8_layer(L, 2, Wg, sg, Wd, sd, X)
    X2 = X.clone()
    X2[1::2] *= torch.tensor([1e4, -1e-6, 0.0, 1e12] * 4, device="cuda")[:, None].to(torch.bfloat16)
    Y2 = q.moe_i8_layer(L, 2, Wg, sg, Wd, sd, X2)
    assert torch.equal(Y2[::2], Y[::2]) and not torch.equal(Y2[1::2], Y[1::2])


# ------------------------------------------------- masked experts and NaN logits

@pytest.mark.parametrize("E", [6, 140, 300])
def test_moe_fewer_numbers_than_topk_among_the_logits(E):
    """A NaN logit ranks below all others; selected for want of others it weighs nothing."""
    L, Wg, sg, Wd, sd, X = moe_inputs(63, 4, E, 64, 48)
    nan = float("nan")
    L[0, 2:] = nan
    L[1, :] = nan
    L[1, E - 1] = -3.0
    L[2, 1:] = nan
    L[2, 3] = -float("inf")
    L[3, 1] = float("inf")  # no softmax with it
    Y = q.moe_i8_layer(L, 4, Wg, sg, Wd, sd, X)
    within(Y[:3], L[:3], 4, Wg, sg, Wd, sd, X[:3])
    assert torch.isnan(Y[3]).all()


def test_moe_masked_expert_weighs_nothing_whatever_it_holds():
    """An expert masked by -inf that is selected for want of others: its NaN scales, or an
    overflow in its product, stay out of the token."""
    L, Wg, sg, Wd, sd, X = moe_inputs(64, 5, 6, 64, 48)
    L[:4, 2:] = -float("inf")
    L[4] = torch.tensor([0.0, 1.0, -9.0, -9.0, -9.0, -9.0])
    bg, bd = sg.clone(), sd.clone()
    bg[2], bd[3] = float("nan"), float("inf")
    bg[4], bd[5] = 1e30, float("nan")
    within(q.moe_i8_layer(L, 4, Wg, bg, Wd, bd, X)[:4], L[:4], 4, Wg, sg, Wd, sd, X[:4])
    # an expert that does weigh in brings its NaN
    assert torch.isnan(q.moe_i8_layer(L, 4, Wg, bg, Wd, bd, X)[4]).all()


# --------------------------------------------------------- gates far below zero

@pytest.mark.parametrize("K", [16, 4096])
@pytest.mark.parametrize("g", [-165.0, -174.0, -176.0, -178.0, -180.0])
def test_gemm_swiglu_gate_far_below_zero(K, g):
    """u near the largest there is: silu(g) * u is a normal number down to g = -181."""
    W = torch.zeros(2, K, dtype=torch.int8, device="cuda")
    W[0, :16], W[1, :16] = -127, 1
    X = torch.full((3, K), 127, dtype=torch.int8, device="cuda")
    sw = torch.tensor([-g / (127 * 127 * 16), 3.3e38 / (127 * 16)], dtype=torch.float32, device="cuda")
    Y = q.i8_gemm(W, sw, X, torch.ones(3, device="cuda"), act=q.ACT_SWIGLU)
    gate, up = -127.0 * 127 * 16 * float(sw[0]), 127.0 * 16 * float(sw[1])
    exact = gate * math.exp(gate) / (1 + math.exp(gate)) * up
    assert abs(exact) > 2.0 ** -126
    # the gate's two roundings move the exponential by 2 * 2^-24 |g|; that of half the gate is off by
    # (|g| + 8) * 2^-22 squared, and, below the normal numbers, by half a step of 2^-149, as the
    # product with the reciprocal is: of 2^-130 at least, 2^-20 each, the first squared; then bf16
    tol = 2.0 ** -8 + abs(gate) * 2.0 ** -23 + (abs(gate) + 8) * 2.0 ** -22 + 3 * 2.0 ** -20
    assert (abs(Y.double().cpu() / exact - 1) <= 1.01 * tol).all()


@pytest.mark.parametrize("g,u", [(-60.0, 1e3), (-86.0, 1e6), (-95.0, 1e12), (-103.0, 1e16), (-110.0, 1e20),
                                 (-150.0, 1e38)])
def test_moe_gates_far_below_zero(g, u):
    """exp(g) below fp32's range in a whole row of h, h itself well within it."""
    L, Wg, sg, Wd, sd, X = moe_inputs(65, 3, 2, 32, 48)
    F = 48
    Wg[:] = 0
    X[:, 3] = 1.0
    Wg[:, :F, 3], Wg[:, F:, 3] = -127, 127
    sg[:, :F], sg[:, F:] = -g / 127 * (1 + 0.01 * torch.rand(F, generator=_gen(1), device="cuda")), u / 127
    sd[:] = 1e20
    case = (L, 1, Wg, sg, Wd, sd, X)
    Y = q.moe_i8_layer(*case)
    assert torch.count_nonzero(Y) > 0
    within(Y, *case)


# ----------------------------------------------------------------- large sizes

def test_k_beyond_int_is_refused():
    """Passed on as int, 2^32 + 32 would be 32."""
    K = 2 ** 32 + 32
    W, one = torch.zeros(1, K, dtype=torch.int8, device="cuda"), torch.ones(1, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        q.i8_gemm(W, one, W, one)
    with pytest.raises(ValueError, match="2\\^31"):
        q.i8_quantize(torch.zeros(1, K, dtype=torch.bfloat16, device="cuda"))


def test_gemm_most_tokens():
    """M at its limit: 34 GB of codes, in rows that repeat every 1024 under scales that do not."""
    M, K = 2 ** 31 - 1024, 16
    if torch.cuda.mem_get_info()[0] < 70 * 2 ** 30:
        pytest.skip("not enough free memory")
    g = _gen(70)
    W, sw, block = codes(g, 1, K), scales(g, 1), codes(g, 1024, K)
    X = torch.empty(M, K, dtype=torch.int8, device="cuda")
    X.view(-1, 1024, K).copy_(block.expand(M // 1024, 1024, K))
    sx = torch.empty(M, device="cuda")
    sx.view(-1, 1024).copy_((1 + torch.arange(M // 1024, device="cuda") % 4093 / 4096).expand(1024, -1).t())
    Y = q.i8_gemm(W, sw, X, sx)
    acc = (block.to(F64) @ W.to(F64).T).to(torch.float32)[:, 0]
    for c in range(0, M // 1024, 1 << 16):
        rows = slice(1024 * c, 1024 * (c + (1 << 16)))
        assert torch.equal(Y[rows].view(-1, 1024), acc * sx[rows].view(-1, 1024) * sw)
    del X, sx, Y
    torch.cuda.empty_cache()


# ------------------------------------------------------------ waits that run out

@pytest.mark.parametrize("drop", [1, 3, 5, 9])
def test_moe_waits_run_out_part_of_the_way(drop):
    """A later stage never arrives in either kernel, with copies ahead of it and products behind."""
    L, Wg, sg, Wd, sd, X = moe_inputs(66, 12, 24, 1040, 784)
    case = (L, 4, Wg, sg, Wd, sd, X)
    good = q.moe_i8_layer(*case)
    assert q.q4k_last_device_status() == 0
    try:
        q.q4k_test_wait_fault(drop, 200_000)
        q.moe_i8_layer(*case)
        assert q.q4k_last_device_status() == 7  # Q4K_ERR_DEVICE_TIMEOUT
    finally:
        q.q4k_test_wait_fault(-1, 0)
    assert torch.equal(q.moe_i8_layer(*case), good)
    assert q.q4k_last_device_status() == 0
