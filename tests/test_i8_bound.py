"""The bound that the GPU tests put on moe_i8_layer, on the CPU: a model of the layer with
activations in three base-256 digits keeps it, with two digits it does not."""
import pytest
import torch

from tests.i8_bound import F64, moe_ref_and_bound, route

TOP = 8355711.0  # the largest that three digits hold


def model(L, topk, Wg, sg, Wd, sd, X, digits):
    """The layer with its activations as fixed point of three digits, or with the lowest cut off."""
    def hold(x, S):
        v = torch.round((x * S).clamp(-TOP, TOP))
        return (v if digits == 3 else torch.round(v / 256) * 256) / S
    M, F = X.shape[0], Wd.shape[2]
    y = torch.zeros(M, Wd.shape[1], dtype=torch.float32)
    for t in range(M):
        x = X[t].to(F64)
        S = 2.0 ** (21 - torch.floor(torch.log2(x.abs().max())))
        ids, ps, _ = route(L[t], topk)
        for e, p in zip(ids, ps):
            gu = ((Wg[e].to(F64) @ hold(x, S)).float() * sg[e]).float()
            h = gu[:F] / (1 + torch.exp(-gu[:F])) * gu[F:]
            o = (Wd[e].to(F64) @ hold(h.to(F64), TOP / h.abs().max().to(F64))).float() * sd[e]
            y[t] += torch.tensor(p, dtype=torch.float32) * o
    return y


@pytest.mark.parametrize("M,E,topk,H,F", [(2, 3, 2, 2048, 768), (2, 2, 1, 4096, 2048), (3, 5, 3, 1040, 336),
                                          (4, 4, 2, 64, 32), (6, 3, 3, 256, 128)])
def test_the_bound_tells_three_digits_from_two(M, E, topk, H, F):
    g = torch.Generator().manual_seed(H + F)
    codes = lambda *s: torch.randint(-127, 128, s, generator=g).to(torch.int8)
    L, X = 2 * torch.randn(M, E, generator=g), torch.randn(M, H, generator=g).to(torch.bfloat16)
    Wg, Wd = codes(E, 2 * F, H), codes(E, H, F)
    sg = (torch.rand(E, 2 * F, generator=g) * 0.02 + 1e-4) / H ** 0.5
    sd = (torch.rand(E, H, generator=g) * 0.02 + 1e-4) / F ** 0.5
    y, tol = moe_ref_and_bound(L, topk, Wg, sg, Wd, sd, X)
    case = (L, topk, Wg, sg, Wd, sd, X)
    assert ((model(*case, 3).to(F64) - y).abs() <= tol).all()
    assert ((model(*case, 2).to(F64) - y).abs() > tol).any(dim=1).all()  # in every token
