"""Sizes that the int8 lane's binding cannot pass on as int are refused, not cut off (by shape
alone: the tensors hold no memory)."""
import pytest
import torch


@pytest.fixture(scope="module")
def q():
    from q4_weight_only_super_b200 import build
    build.build()
    import q4_weight_only_super_b200 as q
    q.lib()
    return q


def empty(*shape, dtype=torch.int8):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32 + 8])
def test_sizes_beyond_int(q, n):
    f32, bf16 = torch.float32, torch.bfloat16
    with pytest.raises(ValueError, match="2\\^31"):
        q.i8_quantize(empty(n, 16, dtype=bf16))
    for W, X in (((n, 16), (3, 16)), ((8, 16), (n, 16)), ((8, n), (3, n))):
        with pytest.raises(ValueError, match="2\\^31"):
            q.i8_gemm(empty(*W), empty(W[0], dtype=f32), empty(*X), empty(X[0], dtype=f32))

    def layer(M=2, E=4, topk=2, H=32, F=16):
        q.moe_i8_layer(empty(M, E, dtype=f32), topk, empty(E, 2 * F, H), empty(E, 2 * F, dtype=f32), empty(E, H, F),
                       empty(E, H, dtype=f32), empty(M, H, dtype=bf16))
    for change in (dict(M=n), dict(E=n), dict(topk=n), dict(H=n), dict(F=n)):
        with pytest.raises(ValueError, match="2\\^31"):
            layer(**change)
    with pytest.raises(ValueError, match="CUDA"):
        layer()
