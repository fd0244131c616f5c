"""The 8-bit integer lane on the CPU: its oracle pinned by brute force, and every refusal of
its entry points and their binding, none of which reaches a GPU."""
import numpy as np
import pytest
import torch

from oracle import i8 as O
from oracle import q4k as Q


@pytest.fixture(scope="module")
def L():
    from q4_weight_only_super_b200 import build
    build.build()
    import q4_weight_only_super_b200 as q
    return q.lib()


# ----------------------------------------------------------------------- oracle

def test_codes_equal_rational_rounding_for_every_mantissa_pair():
    for ma in (128, 131, 150, 171, 200, 233, 254, 255):
        amax = float(ma)
        x = np.array([0.0, amax] + [m * 2.0 ** -s for m in range(1, 256) for s in range(0, 10) if m * 2.0 ** -s <= amax])
        bits = Q.f64_to_bf16_bits(x)[None, :]
        codes, scale = O.quantize_rows(bits)
        exact = [O.code_exact(v, amax) for v in Q.bf16_to_f64(bits)[0]]
        assert codes[0].tolist() == exact
        assert scale[0] == np.float32(amax / 127)


def test_matmul_ref_is_the_integer_product():
    rng = np.random.default_rng(0)
    W, X = rng.integers(-128, 128, (5, 48)).astype(np.int8), rng.integers(-128, 128, (3, 48)).astype(np.int8)
    one = np.ones(5, np.float32)
    y, y32 = O.matmul_ref(W, one, X, one[:3])
    for m in range(3):
        for n in range(5):
            assert y[m, n] == y32[m, n] == sum(int(a) * int(b) for a, b in zip(X[m], W[n]))


def test_moe_ref_of_one_expert_is_its_two_products():
    rng = np.random.default_rng(1)
    H, F = 32, 16
    x = Q.f64_to_bf16_bits(rng.standard_normal((2, H)))
    wg, wd = rng.integers(-9, 10, (1, 2 * F, H)).astype(np.int8), rng.integers(-9, 10, (1, H, F)).astype(np.int8)
    sg, sd = np.full((1, 2 * F), 0.01, np.float32), np.full((1, H), 0.5, np.float32)
    y = O.moe_layer_ref(np.zeros((2, 1), np.float32), 1, wg, sg, wd, sd, x)
    gu = Q.bf16_to_f64(x) @ (wg[0] * np.float64(np.float32(0.01))).T
    h = O.silu(gu[:, :F]) * gu[:, F:]
    np.testing.assert_allclose(y, h @ (wd[0] * 0.5).T, rtol=1e-12)


# -------------------------------------------------------------------- refusals

FAKE, BIG = 4096, 1 << 30  # never dereferenced: every call fails its checks first


def test_quantize_refusals(L):
    f = L.i8_quantize
    assert f(FAKE, 1, 24, FAKE, FAKE, None) == 3 and f(FAKE, 1, 0, FAKE, FAKE, None) == 3
    assert f(FAKE, -1, 32, FAKE, FAKE, None) == 3
    assert f(None, 1, 32, FAKE, FAKE, None) == 1 and f(FAKE, 1, 32, None, FAKE, None) == 1
    assert f(FAKE, 1, 32, FAKE, None, None) == 1
    assert f(FAKE + 8, 1, 32, FAKE, FAKE, None) == 2 and f(FAKE, 1, 32, FAKE + 2, FAKE, None) == 2
    assert f(None, 0, 32, None, None, None) == 0


def test_gemm_refusals(L):
    def f(M=4, N=32, K=64, act=0, bf16=0, **at):
        p = dict(W=FAKE, ws=FAKE, X=FAKE, xs=FAKE, Y=FAKE)
        p.update(at)
        return L.i8_gemm(p["W"], p["ws"], p["X"], p["xs"], p["Y"], M, N, K, act, bf16, None)
    assert f(K=40) == 3 and f(K=0) == 3 and f(M=-1) == 3 and f(N=-1) == 3
    assert f(act=7) == 4
    assert f(act=1, N=33, bf16=1) == 3     # an odd number of gate and up rows
    assert f(act=1, bf16=0) == 4           # SwiGLU is bf16
    assert f(K=131072) == 4                # sums beyond int32
    assert f(M=2 ** 31 - 1) == 4 and f(N=2 ** 31 - 1) == 4
    for name in ("W", "ws", "X", "xs", "Y"):
        assert f(**{name: None}) == 1
        assert f(**{name: FAKE + 4}) == 2
    assert f(M=0, W=None) == 0 and f(N=0, Y=None) == 0


def test_moe_refusals(L):
    def f(M=2, E=8, topk=2, H=64, F=32, nbytes=BIG, **at):
        p = dict(logits=FAKE, Wg=FAKE, sg=FAKE, Wd=FAKE, sd=FAKE, X=FAKE, R=None, Y=FAKE, ws=FAKE)
        p.update(at)
        return L.moe_i8_layer(p["logits"], M, E, topk, p["Wg"], p["sg"], p["Wd"], p["sd"], H, F, p["X"], p["R"], p["Y"],
                              p["ws"], nbytes, None)
    assert f(H=72) == 3 and f(F=40) == 3 and f(E=0) == 3 and f(topk=0) == 3 and f(M=-1) == 3 and f(H=0) == 3
    assert f(M=33) == 4 and f(E=1025) == 4 and f(topk=9) == 4 and f(E=32, topk=17) == 4
    assert f(H=131072) == 4 and f(F=131072) == 4
    for name in ("logits", "Wg", "sg", "Wd", "sd", "X", "Y", "ws"):
        assert f(**{name: None}) == 1
        assert f(**{name: FAKE + 4}) == 2
    assert f(R=FAKE + 4) == 2
    assert f(nbytes=64) == 5
    assert f(M=0, X=None) == 0


def test_moe_workspace(L):
    # per row of h F values and 4 magnitudes per 64
    def want(M, H, F, topk):
        return M * topk * 4 * (F + 4 * -(-F // 64))
    for M, H, F, topk in ((1, 2048, 768, 8), (32, 2048, 768, 8), (5, 1040, 336, 3)):
        assert L.q4k_workspace_bytes(5, M, H, F, 128, topk) == want(M, H, F, topk)
    assert L.q4k_workspace_bytes(5, 0, 2048, 768, 128, 8) == 0


def test_binding_refuses_what_it_cannot_pass_on():
    import q4_weight_only_super_b200 as q
    x = torch.zeros(2, 32, dtype=torch.bfloat16)
    w, s = torch.zeros(4, 32, dtype=torch.int8), torch.ones(4)
    with pytest.raises(ValueError, match="CUDA"):
        q.i8_quantize(x)
    with pytest.raises(ValueError, match="two dimensions"):
        q.i8_quantize(x[0])
    with pytest.raises(ValueError, match="CUDA"):
        q.i8_gemm(w, s, w[:2], s[:2])
    with pytest.raises(ValueError, match="CUDA"):
        q.moe_i8_layer(torch.zeros(1, 2), 1, torch.zeros(2, 32, 32, dtype=torch.int8), torch.ones(2, 32),
                       torch.zeros(2, 32, 16, dtype=torch.int8), torch.ones(2, 32), x[:1])
