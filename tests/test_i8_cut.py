"""The forms that i8_gemm chooses between, on the CPU: every cut fits what it has to fit, for
devices on which few or many clusters are resident at once."""
import random

import pytest


@pytest.fixture(scope="module")
def q():
    from q4_weight_only_super_b200 import build
    build.build()
    import q4_weight_only_super_b200 as q
    q.lib()
    return q


# clusters of 1..8 CTAs resident at once on 148 SMs, one CTA per SM
FITS = [[0, 148, 74, 48, 36, 28, 24, 20, 16], [0, 148, 74, 44, 33, 26, 22, 18, 14], [0, 148, 74, 0, 0, 0, 0, 0, 0]]


def check(q, M, N, K, act, fit):
    c = q.q4k_test_i8_cut(M, N, K, act, 148, fit)
    P, rows, tile = 1 + c["pair"], N // 2 if act else N, 64 if act else 128
    assert c["m_tiles"] * c["nt"] >= M and c["n_tiles"] * tile * P >= rows
    assert c["nt"] % (16 * P) == 0 and 16 <= c["nt"] <= 256
    assert 1 <= c["stages"] <= 12 and 1 <= c["ksplit"] * P <= 8 and c["ksplit"] <= -(-K // 128)
    smem = 233472 // c["ctas_per_sm"] - 1024  # an SM's, less the 1024 bytes that each CTA costs
    stage = 128 * 128 + c["nt"] // P * 128
    assert c["stages"] * stage + 1024 + 256 + 32 * c["nt"] <= smem
    # accumulators of the CTAs that share an SM's 512 TMEM columns
    assert c["ctas_per_sm"] * (2 if c["ksplit"] == 1 else 1) * c["nt"] <= 512
    if c["ksplit"] > 1:
        per = (-(-c["nt"] // c["ksplit"]) + 3) // 4 * 4
        assert c["ksplit"] * 128 * per * 4 <= c["stages"] * stage
        assert c["m_tiles"] * c["n_tiles"] <= fit[P * c["ksplit"]] * c["ctas_per_sm"]
    return c


@pytest.mark.parametrize("fit", FITS)
def test_cuts_fit(q, fit):
    rng = random.Random(1)
    for _ in range(3000):
        M, N, K = int(2 ** rng.uniform(0, 13)), int(2 ** rng.uniform(1, 16)), 16 * int(2 ** rng.uniform(0, 13))
        act = rng.random() < 0.5
        check(q, M, N // 2 * 2 if act else N, K, int(act), fit)


def test_hook_refusals(q):
    for M, N, K, act in ((0, 32, 64, 0), (4, 0, 64, 0), (4, 32, 40, 0), (4, 33, 64, 1), (4, 32, 64, 2),
                       (4, 32, 131072, 0), (2 ** 31 - 1, 32, 64, 0), (4, 2 ** 31 - 1, 64, 0)):
        with pytest.raises(q.Q4KError):
            q.q4k_test_i8_cut(M, N, K, act, 148, FITS[0])
    with pytest.raises(q.Q4KError):
        q.q4k_test_i8_cut(4, 32, 64, 0, 148, None)


@pytest.mark.parametrize("M", [2 ** 31 - 1024, 2 ** 31 - 1025, 2139130000, 2 ** 31 - 2 ** 24])
@pytest.mark.parametrize("N,K,act", [(1, 16, 0), (4, 16, 1), (100, 144, 0)])
@pytest.mark.parametrize("fit", FITS)
def test_cuts_of_the_most_tokens(q, M, N, K, act, fit):
    c = check(q, M, N, K, act, fit)
    # the first token of every tile, and of a pair's second half of it, stays an int
    assert (c["m_tiles"] - 1) * c["nt"] + c["nt"] // 2 < 2 ** 31


@pytest.mark.parametrize("N", [2 ** 31 - 1024, 2 ** 31 - 1026])
@pytest.mark.parametrize("act", [0, 1])
def test_cuts_of_the_most_channels(q, N, act):
    for M in (1, 300):
        c = check(q, M, N, 16, act, FITS[0])
        assert c["n_tiles"] * (1 + c["pair"]) * 128 < 2 ** 31
