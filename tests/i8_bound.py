"""The mixture-of-experts layer over int8 experts in 64 bits, and how far moe_i8_layer may be
from it (no method arithmetic of the kernels beyond their documented number formats).

u = 2^-24 is half a step of fp32. Sums over K are exact, so what remains is:
  x    held to 2^-22 of its row's largest, exactly if it is within 2^14 of it;
  g, u three int32 digit sums made fp32, two fused adds, one scale: u times |sum| or the digit sums'
       magnitudes, which exceed |sum| by the lower digits, 2^-6 of the row's largest;
  h    the exponential of -|g| / 2 (4 u of its own) twice, sum, quotient, products: 16 u;
       then held to 2^-23 of its row's largest, its scale and the inverse rounded apart;
  o    as g, with the scale's inverse not a power of two, the lower digits 2^-7.9;
  p    twice the exponent's rounding and 4 u, the sum of 16 and a quotient;
  y    topk products and additions, those of up to 8 CTAs, the residual's.
All of it first order, and 1% for the rest."""
import torch

F64 = torch.float64
U = 2.0 ** -24


def route(row, topk):
    """Experts and weights of one token: higher logit first, equal logits by the lower id, a NaN
    below them all and without weight."""
    v = [float("-inf") if x != x else x for x in row.tolist()]
    ids = sorted(range(len(v)), key=lambda e: (row[e].item() != row[e].item(), -v[e], e))[:topk]
    z = torch.tensor([v[e] for e in ids], dtype=F64)
    p = torch.exp(z - z.max())
    spread = max([float(z.max() - x) for x in z if x > -200 + z.max()] + [0.0])
    return ids, (p / p.sum()).tolist(), spread


def moe_ref_and_bound(L, topk, Wg, sg, Wd, sd, X, residual=None):
    M, F = X.shape[0], Wd.shape[2]
    y = torch.zeros(M, Wd.shape[1], dtype=F64, device=X.device) if residual is None else residual.to(F64).clone()
    total, tol = y.abs(), torch.zeros_like(y)
    host = L.cpu()
    for t in range(M):
        x = X[t].to(F64)
        top = x.abs().max()
        dx = ((x != 0) & (x.abs() * 2.0 ** 14 < top)).to(F64) * 2.0 ** -22 * top
        ids, ps, spread = route(host[t], topk)
        for e, p in zip(ids, ps):
            if p == 0:
                continue
            wg, wd, s, r = Wg[e].to(F64), Wd[e].to(F64), sg[e].to(F64), sd[e].to(F64)
            acc, mag = wg @ x, wg.abs()
            gu = acc * s
            d = s * (mag @ dx + U * (4 * acc.abs() + 4 * 2.0 ** -6 * top * mag.sum(1)))
            gate, up = gu[:F], gu[F:]
            silu = gate * torch.sigmoid(gate)
            h = silu * up
            # the slope of silu is below 1.1, and far out below (1 + |g|) e^-|g|
            slope = torch.where(gate < -4, (1 + gate.abs()) * torch.exp(gate), 1.1)
            dh = slope * d[:F] * up.abs() + silu.abs() * d[F:] + 16 * U * h.abs()
            high = (h.abs() + dh).max()
            dh = dh + 2.0 ** -23 * (high.clamp_min(2.0 ** -100) + h.abs())
            acc, mag = wd @ h, wd.abs()
            o = acc * r
            do = r * (mag @ dh + U * (6 * acc.abs() + 4 * 2.0 ** -7.9 * high * mag.sum(1)))
            y[t] += p * o
            total[t] += p * o.abs()
            tol[t] += p * do + (2 * spread + 16) * U * p * o.abs()
    return y, 1.01 * (tol + (topk + 10) * U * total)
