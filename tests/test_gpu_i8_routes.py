"""i8_gemm in each of its forms (lone CTAs or CTA pairs, walking their tiles or splitting K, one
or two CTAs per SM) against plain 64-bit products. Every case asserts the form that its sizes
take, so that a change of the rule that chooses cannot quietly drop one from the tests.

Tolerances. Without an activation the result equals the three fp32 roundings of the definition,
and its bf16 rounding. SwiGLU: of the exact fp32 g and u (the same three roundings), the
exponential exp(-|g| / 2) has an argument rounded twice (|g| / 2 * 2 * 2^-24) and an error of
2^-22 of its own, and enters twice; the reciprocal 2^-23, the sum and four products 2^-24 each:
below (|g| + 8) * 2^-22 of the result; then bf16, half a step, 2^-8; below the normal numbers half
the subnormal step, 2^-134."""
import pytest
import torch

from tests.test_gpu_i8 import codes, gemm_ref32, scales, _gen

pytestmark = pytest.mark.gpu

q = pytest.importorskip("q4_weight_only_super_b200")

F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _gpu(cuda_ok):
    q.lib()
    q.q4k_last_device_status()
    yield
    assert q.q4k_last_device_status() == 0


def form(M, N, K, act):
    """(pair, CTAs per SM, shares of K > 1, most tiles that one CTA or pair computes)."""
    c = q.q4k_test_i8_cut(M, N, K, act)
    places = torch.cuda.get_device_properties(0).multi_processor_count * c["ctas_per_sm"] // (1 + c["pair"])
    return c["pair"], c["ctas_per_sm"], c["ksplit"] > 1, 1 if c["ksplit"] > 1 else -(-c["m_tiles"] * c["n_tiles"] // places)


def check(M, N, K, act, seed):
    """All outputs, fp32 and bf16, and what lies around them."""
    g = _gen(seed)
    W, X = codes(g, N, K), codes(g, M, K)
    # with SwiGLU, gates and ups of a few units
    sw, sx = (scales(g, N) / (80 * K ** 0.5), scales(g, M) * 80) if act else (scales(g, N), scales(g, M))
    ref = gemm_ref32(W, sw, X, sx)
    wide = N // 2 if act else N
    for dtype in (torch.bfloat16,) if act else (torch.float32, torch.bfloat16):
        big = torch.full(((M + 16) * wide,), 5.0, dtype=dtype, device="cuda")
        Y = big[8 * wide:(8 + M) * wide].view(M, wide)
        q.i8_gemm(W, sw, X, sx, act=act, Y=Y)
        assert (big[:8 * wide] == 5).all() and (big[(8 + M) * wide:] == 5).all()
        if not act:
            assert torch.equal(Y, ref.to(dtype))
            continue
        gate, up = ref[:, :wide].to(F64), ref[:, wide:].to(F64)
        exact = gate * torch.sigmoid(gate) * up
        tol = exact.abs() * (2.0 ** -8 + (gate.abs() + 8) * 2.0 ** -22 * (1 + 2.0 ** -8)) + 2.0 ** -134
        assert ((Y.to(F64) - exact).abs() <= tol).all()


# (M, N, K, activation, CTAs per SM, fewest tiles of the busiest pair; 0: K split). K is never a
# multiple of a stage, the last token tile is never full, and of the last pair's rows the odd
# CTA's lie wholly or partly past the end.
PAIRS = [
    (2060, 591, 1440, 0, 1, 1), (2987, 401, 1632, 0, 1, 1), (1455, 3539, 688, 0, 1, 2), (2545, 1862, 816, 0, 1, 2),
    (1694, 10989, 144, 0, 1, 3), (1277, 15452, 144, 0, 1, 3), (18, 22138, 8528, 0, 2, 1), (226, 31031, 544, 0, 2, 2),
    (605, 20980, 304, 0, 2, 3), (583, 19989, 304, 0, 2, 3),
    (1889, 666, 2864, 0, 1, 0), (1897, 529, 3904, 0, 1, 0), (271, 3486, 4240, 0, 2, 0), (267, 3349, 5424, 0, 2, 0),
    # SwiGLU, as many gate rows as fill 16-row groups (one box brings a tile) ...
    (1534, 1088, 1424, 1, 1, 1), (2976, 1600, 800, 1, 1, 2), (1508, 29376, 64, 1, 1, 3), (1457, 30048, 64, 1, 1, 3),
    (482, 25248, 320, 1, 2, 3), (628, 19232, 272, 1, 2, 3), (2064, 480, 4464, 1, 1, 0), (1499, 832, 3120, 1, 1, 0),
    (52, 14528, 8496, 1, 2, 0), (487, 2368, 3312, 1, 2, 0),
    # ... and not
    (1506, 838, 1456, 1, 1, 1), (1673, 2708, 704, 1, 1, 2), (1652, 26002, 64, 1, 1, 3), (2767, 17966, 64, 1, 1, 3),
    (457, 25752, 320, 1, 2, 3), (605, 20322, 480, 1, 2, 3), (1896, 490, 4416, 1, 1, 0), (1458, 848, 4032, 1, 1, 0),
    (347, 3204, 5744, 1, 2, 0), (356, 3170, 4704, 1, 2, 0),
]


@pytest.mark.parametrize("M,N,K,act,per_sm,tiles", PAIRS)
def test_pairs(M, N, K, act, per_sm, tiles):
    pair, got_per_sm, split, most = form(M, N, K, act)
    assert pair and got_per_sm == per_sm
    assert split if tiles == 0 else not split and most >= tiles
    check(M, N, K, act, M + N + K)


# the framework's own dense layer
@pytest.mark.parametrize("M,N,K,act,split", [(300, 5120, 17408, 0, True), (512, 34816, 5120, 1, False),
                                             (2048, 17408, 5120, 0, False)])
def test_pairs_of_the_dense_layer(M, N, K, act, split):
    assert form(M, N, K, act)[::2] == (1, split)
    check(M, N, K, act, 7)


LONE = [(535, 3996, 80, 0, 1, 2), (167, 15035, 64, 0, 1, 3), (17, 29916, 64, 0, 2, 2), (35, 32250, 112, 0, 2, 3),
        (5, 300, 2064, 0, 1, 0), (464, 4832, 80, 1, 1, 2), (135, 14762, 80, 1, 1, 3), (47, 32408, 112, 1, 2, 3),
        (3, 34, 784, 1, 1, 0), (9, 96, 2064, 1, 1, 0)]


@pytest.mark.parametrize("M,N,K,act,per_sm,tiles", LONE)
def test_lone_ctas(M, N, K, act, per_sm, tiles):
    pair, got_per_sm, split, most = form(M, N, K, act)
    assert not pair and got_per_sm == per_sm
    assert split if tiles == 0 else not split and most >= tiles
    check(M, N, K, act, M + N + K)


def test_pairs_on_two_streams_and_replayed():
    """A walking and a splitting product at once, and both captured one after the other."""
    cases = [(605, 20980, 304), (271, 3486, 4240)]
    g = _gen(3)
    args = [(codes(g, N, K), scales(g, N), codes(g, M, K), scales(g, M)) for M, N, K in cases]
    assert [form(*c, 0)[::2] for c in cases] == [(1, False), (1, True)]
    ref = [gemm_ref32(a[0], a[1], a[2], a[3]) for a in args]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cases], [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(q.i8_gemm(*args[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, ref[i]) for y in got[i])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ys = [q.i8_gemm(*a) for a in args]
    for a in args:
        a[2].copy_(codes(g, *a[2].shape))
    graph.replay()
    for a, y in zip(args, ys):
        assert torch.equal(y, gemm_ref32(a[0], a[1], a[2], a[3]))


@pytest.mark.parametrize("M,N,K,act", [(605, 20980, 304, 0), (457, 25752, 320, 1), (271, 3486, 4240, 0), (1499, 832, 3120, 1)])
def test_waits_of_pairs_run_out_and_recover(M, N, K, act):
    """A stage that never arrives: pairs at two CTAs per SM, walking and splitting K."""
    assert form(M, N, K, act)[0] == 1
    g = _gen(5)
    args = (codes(g, N, K), scales(g, N) / 100, codes(g, M, K), scales(g, M))
    good = q.i8_gemm(*args, act=act)
    assert q.q4k_last_device_status() == 0
    try:
        q.q4k_test_wait_fault(0, 200_000)  # every producer skips its first stage; 200 us limit
        q.i8_gemm(*args, act=act)
        assert q.q4k_last_device_status() == 7  # Q4K_ERR_DEVICE_TIMEOUT
    finally:
        q.q4k_test_wait_fault(-1, 0)
    assert torch.equal(q.i8_gemm(*args, act=act), good)
    assert q.q4k_last_device_status() == 0


@pytest.mark.parametrize("drop", [1, 5, 9])
@pytest.mark.parametrize("M,N,K,act", [(605, 20980, 304, 0), (457, 25752, 320, 1), (2048, 17408, 5120, 0), (271, 3486, 4240, 0),
                                       (35, 32250, 112, 0), (5, 300, 2064, 0)])
def test_waits_run_out_part_of_the_way(M, N, K, act, drop):
    """A later stage never arrives, with tiles behind and copies ahead of it."""
    g = _gen(6)
    args = (codes(g, N, K), scales(g, N) / 100, codes(g, M, K), scales(g, M))
    good = q.i8_gemm(*args, act=act)
    assert q.q4k_last_device_status() == 0
    try:
        q.q4k_test_wait_fault(drop, 200_000)
        q.i8_gemm(*args, act=act)
        late = q.q4k_last_device_status()
    finally:
        q.q4k_test_wait_fault(-1, 0)
    assert late in (0, 7)  # (0: no CTA has that many stages)
    assert torch.equal(q.i8_gemm(*args, act=act), good)
    assert q.q4k_last_device_status() == 0
