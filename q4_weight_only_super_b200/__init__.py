"""Q4_K weight-only matrix products for NVIDIA B200 (sm_100a).

Thin ctypes binding over ``libq4k.so`` (C ABI in ``include/q4k.h``). Every
function here only marshals arguments: tensors are passed as raw device
pointers, the current torch CUDA stream is passed as the stream, and any
non-zero status raises :class:`Q4KError`. All computation happens in the
library's CUDA kernels; there is no CPU path.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "Q4KError", "lib", "q4k_dequant", "q4k_gemv", "q4k_gemv_q8", "q5k_gemv", "q80_gemv", "q6k_gemv", "q4k_repack", "q4k_gemv_repacked", "q4k_gemm", "bf16w_gemm",
    "moe_route_permute",
    "moe_route_permute_noalloc", "moe_route_permute_hidden", "moe_route_gate_up",
    "moe_q4k_grouped", "moe_combine", "moe_combine_residual", "q4k_workspace_bytes", "q4k_last_device_status",
    "i8_quantize", "i8_gemm", "moe_i8_layer",
    "q4k_test_wait_fault", "q4k_test_i8_cut",
    "ACT_NONE", "ACT_SWIGLU", "OP_GEMM", "OP_ROUTE", "OP_GROUPED", "OP_GEMV", "OP_MOE_I8", "EXPORTS",
]

ACT_NONE, ACT_SWIGLU = 0, 1
OP_GEMM, OP_ROUTE, OP_GROUPED, OP_GEMV, OP_MOE_I8 = 1, 2, 3, 4, 5
BLOCK_BYTES = 144
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libq4k.so")

_p, _i, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
# name -> (restype, argtypes); mirrors include/q4k.h
EXPORTS = {
    "q4k_dequant": (_i, [_p, _i64, _i, _p, _p]),
    "q4k_gemv": (_i, [_p, _p, _p, _i, _i, _i, _p, _sz, _p]),
    "q5k_gemv": (_i, [_p, _p, _p, _i, _i, _i, _p, _sz, _p]),
    "q80_gemv": (_i, [_p, _p, _p, _i, _i, _i, _p, _sz, _p]),
    "q6k_gemv": (_i, [_p, _p, _p, _i, _i, _i, _p, _sz, _p]),
    "q4k_gemv_q8": (_i, [_p, _p, _p, _i, _i, _i, _p, _sz, _p]),
    "q4k_repacked_bytes": (_i64, [_i, _i]),
    "q4k_repack": (_i, [_p, _i, _i, _p, _p]),
    "q4k_gemv_repacked": (_i, [_p, _p, _p, _i, _i, _i, _p, _sz, _p]),
    "q4k_gemm": (_i, [_p, _p, _p, _i, _i, _i, _p, _sz, _p]),
    "bf16w_gemm": (_i, [_p, _p, _p, _i, _i, _i, _p]),
    "moe_route_permute": (_i, [_p, _i, _i, _i, _p, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "moe_route_permute_noalloc": (_i, [_p, _i, _i, _i, _p, _p, _p, _p, _p, _p, _p]),
    "moe_route_permute_hidden": (_i, [_p, _p, _i, _i, _i, _i, _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "moe_q4k_grouped": (_i, [_p, _i, _i, _i, _p, _p, _p, _i, _i, _i, _p, _p, _sz, _p]),
    "moe_route_gate_up": (_i, [_p, _i, _i, _i, _p, _p, _p, _p, _p, _p, _p, _i, _i, _p, _p, _p]),
    "moe_combine": (_i, [_p, _p, _p, _i, _i, _i, _p, _p]),
    "moe_combine_residual": (_i, [_p, _p, _p, _p, _i, _i, _i, _p, _p]),
    "i8_quantize": (_i, [_p, _i, _i, _p, _p, _p]),
    "i8_gemm": (_i, [_p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _p]),
    "moe_i8_layer": (_i, [_p, _i, _i, _i, _p, _p, _p, _p, _i, _i, _p, _p, _p, _p, _sz, _p]),
    "q4k_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i]),
    "q4k_last_device_status": (_i, [_p]),
    "q4k_test_wait_fault": (_i, [_i, ctypes.c_uint64]),
    "q4k_test_i8_cut": (_i, [_i, _i, _i, _i, _i, ctypes.POINTER(_i), ctypes.POINTER(_i)]),
    "q4k_status_string": (ctypes.c_char_p, [_i]),
}

_LIB = None


class Q4KError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: status {status} ({lib().q4k_status_string(status).decode()})")


def lib() -> ctypes.CDLL:
    """Load libq4k.so (fails loudly if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing; build it with `python -m q4_weight_only_super_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _LIB = L
    return _LIB


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn, st):
    if st != 0:
        raise Q4KError(fn, st)


def _bits16(x):
    """bf16 activations may be given as bfloat16 or as their int16 bit patterns."""
    assert x.dtype in (torch.bfloat16, torch.int16, torch.uint16), x.dtype
    return x


def q4k_dequant(W, out_bf16: bool = False, out=None, stream=None):
    """W: uint8 [..., 144] Q4_K blocks on the GPU -> fp32 (or bf16) weights [nblocks*256]."""
    nb = W.numel() // BLOCK_BYTES
    if out is None:
        out = torch.empty(nb * 256, dtype=torch.bfloat16 if out_bf16 else torch.float32, device=W.device)
    _check("q4k_dequant", lib().q4k_dequant(_ptr(W), nb, int(out_bf16), _ptr(out), _stream(stream)))
    return out


def _scratch(nbytes: int, device, ws=None):
    if ws is not None:
        return ws
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def q4k_gemv(W, X, N: int, K: int, Y=None, ws=None, stream=None):
    """Y[M][N] = X[M][K] @ W^T for 1 <= M <= 32 (W: Q4_K [N][K/256][144])."""
    M = X.shape[0]
    if Y is None:
        Y = torch.empty(M, N, dtype=torch.float32, device=X.device)
    ws = _scratch(q4k_workspace_bytes(OP_GEMV, M, N, K), X.device, ws)
    _check("q4k_gemv", lib().q4k_gemv(_ptr(W), _ptr(_bits16(X)), _ptr(Y), M, N, K, _ptr(ws), ws.numel(),
                                      _stream(stream)))
    return Y


def q4k_gemv_q8(W, X, N: int, K: int, Y=None, ws=None, stream=None):
    """The Q8 activation lane of q4k_gemv (int8 activations per 256-wide column; accuracy traded)."""
    M = X.shape[0]
    if Y is None:
        Y = torch.empty(M, N, dtype=torch.float32, device=X.device)
    ws = _scratch(q4k_workspace_bytes(OP_GEMV, M, N, K), X.device, ws)
    _check("q4k_gemv_q8", lib().q4k_gemv_q8(_ptr(W), _ptr(_bits16(X)), _ptr(Y), M, N, K, _ptr(ws), ws.numel(),
                                            _stream(stream)))
    return Y


def q5k_gemv(W, X, N: int, K: int, Y=None, ws=None, stream=None):
    """q4k_gemv over Q5_K weights W [N][K/256][176]."""
    M = X.shape[0]
    if Y is None:
        Y = torch.empty(M, N, dtype=torch.float32, device=X.device)
    ws = _scratch(q4k_workspace_bytes(OP_GEMV, M, N, K), X.device, ws)
    _check("q5k_gemv", lib().q5k_gemv(_ptr(W), _ptr(_bits16(X)), _ptr(Y), M, N, K, _ptr(ws), ws.numel(),
                                      _stream(stream)))
    return Y


def q80_gemv(W, X, N: int, K: int, Y=None, ws=None, stream=None):
    """q4k_gemv over Q8_0 weights W [N][K/32][34]."""
    M = X.shape[0]
    if Y is None:
        Y = torch.empty(M, N, dtype=torch.float32, device=X.device)
    ws = _scratch(q4k_workspace_bytes(OP_GEMV, M, N, K), X.device, ws)
    _check("q80_gemv", lib().q80_gemv(_ptr(W), _ptr(_bits16(X)), _ptr(Y), M, N, K, _ptr(ws), ws.numel(),
                                      _stream(stream)))
    return Y


def q6k_gemv(W, X, N: int, K: int, Y=None, ws=None, stream=None):
    """Decode GEMV over Q6_K weights [N][K/256][210]: Y[M][N] = X @ W^T."""
    M = X.shape[0]
    if Y is None:
        Y = torch.empty(M, N, dtype=torch.float32, device=X.device)
    need = q4k_workspace_bytes(OP_GEMV, M, N, K)
    ws = _scratch(need, X.device, ws)
    _check("q6k_gemv", lib().q6k_gemv(_ptr(W), _ptr(_bits16(X)), _ptr(Y), M, N, K, _ptr(ws), ws.numel(),
                                      _stream(stream)))
    return Y


def q4k_repack(W, N: int, K: int, Wr=None, stream=None):
    """Repacked copy of Q4_K weights W [N][K/256][144] for q4k_gemv_repacked (uint8, flat)."""
    nb = lib().q4k_repacked_bytes(N, K)
    if nb <= 0:
        raise ValueError(f"q4k_repack: bad shape N={N} K={K}")
    if Wr is None:
        Wr = torch.empty(nb, dtype=torch.uint8, device=W.device)
    _check("q4k_repack", lib().q4k_repack(_ptr(W), N, K, _ptr(Wr), _stream(stream)))
    return Wr


def q4k_gemv_repacked(Wr, X, N: int, K: int, Y=None, ws=None, stream=None):
    """q4k_gemv on weights from q4k_repack (bit-identical results)."""
    M = X.shape[0]
    if Y is None:
        Y = torch.empty(M, N, dtype=torch.float32, device=X.device)
    ws = _scratch(q4k_workspace_bytes(OP_GEMV, M, N, K), X.device, ws)
    _check("q4k_gemv_repacked", lib().q4k_gemv_repacked(_ptr(Wr), _ptr(_bits16(X)), _ptr(Y), M, N, K, _ptr(ws),
                                                        ws.numel(), _stream(stream)))
    return Y


def q4k_gemm(W, X, N: int, K: int, Y=None, stream=None):
    """Prefill GEMM Y[M][N] = X[M][K] @ W^T on tcgen05 tensor cores."""
    M = X.shape[0]
    if Y is None:
        Y = torch.empty(M, N, dtype=torch.float32, device=X.device)
    _check("q4k_gemm", lib().q4k_gemm(_ptr(W), _ptr(_bits16(X)), _ptr(Y), M, N, K, None, 0,
                                      _stream(stream)))
    return Y


def bf16w_gemm(Wb, X, N: int, K: int, Y=None, stream=None):
    """Y = X @ Wb^T with bf16 weights Wb [N][K] (the unfused chain's GEMM)."""
    M = X.shape[0]
    if Y is None:
        Y = torch.empty(M, N, dtype=torch.float32, device=X.device)
    _check("bf16w_gemm", lib().bf16w_gemm(_ptr(_bits16(Wb)), _ptr(_bits16(X)), _ptr(Y), M, N, K, _stream(stream)))
    return Y


def q4k_workspace_bytes(op: int, M: int, N: int = 0, K: int = 0, E: int = 0, topk: int = 0) -> int:
    return lib().q4k_workspace_bytes(op, M, N, K, E, topk)


def moe_route_permute_hidden(X, W_router, topk: int, out=None, ws=None, stream=None):
    """Router logits X @ W_router^T (bf16 in, fp32 out) then moe_route_permute. Returns
    the routing dict plus "logits"."""
    M, H = X.shape
    E = W_router.shape[0]
    dev = X.device
    if out is None:
        rows = M * topk
        out = {"logits": torch.empty(M, E, dtype=torch.float32, device=dev),
               "topk_ids": torch.empty(M, topk, dtype=torch.int32, device=dev),
               "topk_w": torch.empty(M, topk, dtype=torch.float32, device=dev),
               "expert_offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
               "perm": torch.empty(rows, dtype=torch.int32, device=dev),
               "inv_perm": torch.empty(rows, dtype=torch.int32, device=dev),
               "row_token": torch.empty(rows, dtype=torch.int32, device=dev)}
    ws = _scratch(q4k_workspace_bytes(OP_ROUTE, M, 0, 0, E, topk), dev, ws)
    st = lib().moe_route_permute_hidden(
        _ptr(_bits16(X)), _ptr(_bits16(W_router)), M, E, H, topk, _ptr(out["logits"]), _ptr(out["topk_ids"]),
        _ptr(out["topk_w"]), _ptr(out["expert_offsets"]), _ptr(out["perm"]), _ptr(out["inv_perm"]),
        _ptr(out["row_token"]), _ptr(ws), ws.numel(), _stream(stream))
    _check("moe_route_permute_hidden", st)
    return out


def moe_route_permute(logits, topk: int, out=None, ws=None, stream=None):
    """Top-k routing + stable permutation by expert. Returns a dict of device tensors:
    topk_ids, topk_w, expert_offsets, perm, inv_perm, row_token."""
    M, E = logits.shape
    dev = logits.device
    if out is None:
        out = dict(
            topk_ids=torch.empty(M, topk, dtype=torch.int32, device=dev),
            topk_w=torch.empty(M, topk, dtype=torch.float32, device=dev),
            expert_offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
            perm=torch.empty(M * topk, dtype=torch.int32, device=dev),
            inv_perm=torch.empty(M * topk, dtype=torch.int32, device=dev),
            row_token=torch.empty(M * topk, dtype=torch.int32, device=dev),
        )
    need = q4k_workspace_bytes(OP_ROUTE, M, E=E, topk=topk)
    if ws is None:
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    st = lib().moe_route_permute(
        _ptr(logits), M, E, topk, _ptr(out["topk_ids"]), _ptr(out["topk_w"]),
        _ptr(out["expert_offsets"]), _ptr(out["perm"]), _ptr(out["inv_perm"]),
        _ptr(out["row_token"]), _ptr(ws), ws.numel(), _stream(stream))
    _check("moe_route_permute", st)
    return out


def moe_route_permute_noalloc(logits, topk: int, out=None, stream=None):
    """moe_route_permute with the library's fixed scratch instead of a workspace
    (for callers that cannot allocate device memory at call time; see q4k.h)."""
    M, E = logits.shape
    dev = logits.device
    if out is None:
        out = dict(
            topk_ids=torch.empty(M, topk, dtype=torch.int32, device=dev),
            topk_w=torch.empty(M, topk, dtype=torch.float32, device=dev),
            expert_offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
            perm=torch.empty(M * topk, dtype=torch.int32, device=dev),
            inv_perm=torch.empty(M * topk, dtype=torch.int32, device=dev),
            row_token=torch.empty(M * topk, dtype=torch.int32, device=dev),
        )
    st = lib().moe_route_permute_noalloc(
        _ptr(logits), M, E, topk, _ptr(out["topk_ids"]), _ptr(out["topk_w"]),
        _ptr(out["expert_offsets"]), _ptr(out["perm"]), _ptr(out["inv_perm"]),
        _ptr(out["row_token"]), _stream(stream))
    _check("moe_route_permute_noalloc", st)
    return out


def moe_q4k_grouped(W_experts, E: int, N: int, K: int, A, expert_offsets, rows: int,
                    max_rows_hint: int, act: int = ACT_NONE, row_gather=None, out=None, ws=None,
                    stream=None):
    """Grouped expert matmul over rows sorted by expert (see include/q4k.h)."""
    if out is None:
        if act == ACT_SWIGLU:
            out = torch.empty(rows, N // 2, dtype=torch.bfloat16, device=A.device)
        else:
            out = torch.empty(rows, N, dtype=torch.float32, device=A.device)
    if ws is None and 0 < max_rows_hint <= 32:  # only the decode kernel uses scratch
        ws = _scratch(q4k_workspace_bytes(OP_GROUPED, rows, N, K, E), A.device)
    st = lib().moe_q4k_grouped(_ptr(W_experts), E, N, K, _ptr(_bits16(A)), _ptr(row_gather),
                               _ptr(expert_offsets), rows, max_rows_hint, act, _ptr(out), _ptr(ws),
                               0 if ws is None else ws.numel(), _stream(stream))
    _check("moe_q4k_grouped", st)
    return out


def moe_route_gate_up(logits, topk: int, W_gate_up, N: int, K: int, X, out=None, h=None, stream=None):
    """Routing + permutation and the grouped gate_up SwiGLU GEMV in one launch (decode,
    M <= 32; see include/q4k.h). Returns (routing dict as moe_route_permute's, h)."""
    M, E = logits.shape
    dev = logits.device
    if out is None:
        out = dict(
            topk_ids=torch.empty(M, topk, dtype=torch.int32, device=dev),
            topk_w=torch.empty(M, topk, dtype=torch.float32, device=dev),
            expert_offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
            perm=torch.empty(M * topk, dtype=torch.int32, device=dev),
            inv_perm=torch.empty(M * topk, dtype=torch.int32, device=dev),
            row_token=torch.empty(M * topk, dtype=torch.int32, device=dev),
        )
    if h is None:
        h = torch.empty(M * topk, N // 2, dtype=torch.bfloat16, device=dev)
    st = lib().moe_route_gate_up(_ptr(logits), M, E, topk, _ptr(out["topk_ids"]), _ptr(out["topk_w"]),
                                 _ptr(out["expert_offsets"]), _ptr(out["perm"]), _ptr(out["inv_perm"]),
                                 _ptr(out["row_token"]), _ptr(W_gate_up), N, K, _ptr(_bits16(X)), _ptr(h),
                                 _stream(stream))
    _check("moe_route_gate_up", st)
    return out, h


def moe_combine(O, inv_perm, topk_w, M: int, topk: int, H: int, Y=None, stream=None):
    """y[t] = sum_j topk_w[t,j] * O[inv_perm[t*topk+j]]."""
    if Y is None:
        Y = torch.empty(M, H, dtype=torch.float32, device=O.device)
    _check("moe_combine", lib().moe_combine(_ptr(O), _ptr(inv_perm), _ptr(topk_w), M, topk, H,
                                            _ptr(Y), _stream(stream)))
    return Y


def moe_combine_residual(O, inv_perm, topk_w, residual, M: int, topk: int, H: int, Y=None, stream=None):
    """y[t] = residual[t] + sum_j topk_w[t,j] * O[inv_perm[t*topk+j]] (Y may be residual)."""
    if Y is None:
        Y = torch.empty(M, H, dtype=torch.float32, device=O.device)
    _check("moe_combine_residual", lib().moe_combine_residual(_ptr(O), _ptr(inv_perm), _ptr(topk_w), _ptr(residual),
                                                              M, topk, H, _ptr(Y), _stream(stream)))
    return Y


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_int8, _float32, _bfloat16 = torch.int8, torch.float32, torch.bfloat16
_I8, _F32 = (_int8,), (_float32,)


def _need(fn, name, t, dtypes, shape, dev):
    """An operand of the int8 lane: contiguous, of the right type and shape, on CUDA device `dev`."""
    if t.shape == shape and t.dtype in dtypes and t.get_device() == dev >= 0 and t.is_contiguous():
        return
    raise ValueError(f"{fn}: {name} must be a contiguous {' or '.join(str(d) for d in dtypes)} tensor of shape "
                     f"{tuple(shape)} on {'the CUDA device of the others' if dev >= 0 else 'a CUDA device'}; got "
                     f"{t.dtype} {tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")


def _dims(fn, name, t, n):
    """The n sizes of an operand; they are passed on as int, which would cut a larger one off."""
    if t.dim() != n:
        raise ValueError(f"{fn}: {name} must have {'two' if n == 2 else 'three'} dimensions; got shape {tuple(t.shape)}")
    if max(t.shape) > 0x7fffffff:
        raise ValueError(f"{fn}: {name} has a size beyond 2^31 - 1: {tuple(t.shape)}")
    return t.shape


# (torch.cuda.current_stream() builds a Stream object: 3 us of a small call)
_current_device, _raw_stream = torch.cuda.current_device, torch._C._cuda_getCurrentRawStream


def _empty(shape, dtype, dev, stream):
    """An output or scratch buffer from the pool of the stream that the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", dev))
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", dev))


def i8_quantize(X, Q=None, scale=None, stream=None):
    """bf16 rows X [M][K] -> (int8 codes [M][K], fp32 scales [M]); see include/q4k.h."""
    fn, dev = "i8_quantize", X.get_device()
    shape = M, K = _dims(fn, "X", X, 2)
    _need(fn, "X", X, _BF16, shape, dev)
    if Q is None:
        Q = _empty((M, K), torch.int8, dev, stream)
    else:
        _need(fn, "Q", Q, _I8, shape, dev)
    if scale is None:
        scale = _empty((M,), torch.float32, dev, stream)
    else:
        _need(fn, "scale", scale, _F32, (M,), dev)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return i8_quantize(X, Q, scale, stream)
    st = lib().i8_quantize(X.data_ptr(), M, K, Q.data_ptr(), scale.data_ptr(),
                           _raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise Q4KError(fn, st)
    return Q, scale


def i8_gemm(W, w_scale, X, x_scale, act: int = ACT_NONE, out_bf16: bool = False, Y=None, stream=None):
    """Y[m][n] = x_scale[m] * w_scale[n] * (X[m] . W[n]) from int8 W [N][K] and X [M][K];
    fp32, or bf16 with out_bf16 (or a bf16 Y). ACT_SWIGLU: bf16 [M][N/2], SiLU of the first
    N/2 channels times the others."""
    dev, swiglu = W.get_device(), act == ACT_SWIGLU
    shape, x_shape = W.shape, X.shape
    # one pass over what has to hold (a fifth of a small call's time); which of it does not is
    # found out only then
    if not (len(shape) == len(x_shape) == 2 and shape[1] == x_shape[1]
            and shape[0] <= 0x7fffffff >= shape[1] and x_shape[0] <= 0x7fffffff
            and W.dtype is X.dtype is _int8 and w_scale.dtype is x_scale.dtype is _float32
            and w_scale.shape == shape[:1] and x_scale.shape == x_shape[:1]
            and dev == X.get_device() == w_scale.get_device() == x_scale.get_device() >= 0
            and W.is_contiguous() and X.is_contiguous() and w_scale.is_contiguous() and x_scale.is_contiguous()):
        N, K = _dims("i8_gemm", "W", W, 2)
        M = _dims("i8_gemm", "X", X, 2)[0]
        _need("i8_gemm", "W", W, _I8, (N, K), dev)
        _need("i8_gemm", "w_scale", w_scale, _F32, (N,), dev)
        _need("i8_gemm", "X", X, _I8, (M, K), dev)
        _need("i8_gemm", "x_scale", x_scale, _F32, (M,), dev)
    N, K = shape
    M = x_shape[0]
    if Y is None:
        Y = _empty((M, N // 2 if swiglu else N), _bfloat16 if swiglu or out_bf16 else _float32, dev, stream)
    else:
        _need("i8_gemm", "Y", Y, (_bfloat16,) if swiglu or out_bf16 else (_float32, _bfloat16),
              (M, N // 2 if swiglu else N), dev)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return i8_gemm(W, w_scale, X, x_scale, act, out_bf16, Y, stream)
    st = lib().i8_gemm(W.data_ptr(), w_scale.data_ptr(), X.data_ptr(), x_scale.data_ptr(), Y.data_ptr(), M, N, K, act,
                       Y.dtype is _bfloat16, _raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise Q4KError("i8_gemm", st)
    return Y


def moe_i8_layer(logits, topk: int, W_gate_up, s_gate_up, W_down, s_down, X, residual=None, Y=None, ws=None,
                 stream=None):
    """A whole mixture-of-experts layer for up to 32 tokens over int8 experts, in two launches
    (see include/q4k.h): logits fp32 [M][E], W_gate_up int8 [E][2F][H], W_down int8 [E][H][F]
    with fp32 scales [E][2F] and [E][H], X bf16 [M][H]; returns Y fp32 [M][H]."""
    fn, dev = "moe_i8_layer", W_gate_up.get_device()
    M, E = _dims(fn, "logits", logits, 2)
    _, H, F = _dims(fn, "W_down", W_down, 3)
    if topk > 0x7fffffff:
        raise ValueError(f"{fn}: topk {topk} is beyond 2^31 - 1")
    _need(fn, "logits", logits, _F32, (M, E), dev)
    _need(fn, "W_gate_up", W_gate_up, _I8, (E, 2 * F, H), dev)
    _need(fn, "s_gate_up", s_gate_up, _F32, (E, 2 * F), dev)
    _need(fn, "W_down", W_down, _I8, (E, H, F), dev)
    _need(fn, "s_down", s_down, _F32, (E, H), dev)
    _need(fn, "X", X, _BF16, (M, H), dev)
    if residual is not None:
        _need(fn, "residual", residual, _F32, (M, H), dev)
    if Y is None:
        Y = _empty((M, H), torch.float32, dev, stream)
    else:
        _need(fn, "Y", Y, _F32, (M, H), dev)
    if ws is None:
        ws = _empty((max(16, q4k_workspace_bytes(OP_MOE_I8, M, H, F, E, topk)),), torch.uint8, dev, stream)
    else:
        _need(fn, "ws", ws, (torch.uint8,), (ws.numel(),), dev)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return moe_i8_layer(logits, topk, W_gate_up, s_gate_up, W_down, s_down, X, residual, Y, ws, stream)
    st = lib().moe_i8_layer(logits.data_ptr(), M, E, topk, W_gate_up.data_ptr(), s_gate_up.data_ptr(),
                            W_down.data_ptr(), s_down.data_ptr(), H, F, X.data_ptr(),
                            None if residual is None else residual.data_ptr(), Y.data_ptr(), ws.data_ptr(),
                            ws.numel(), _raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise Q4KError(fn, st)
    return Y


def q4k_last_device_status(stream=None) -> int:
    """Synchronise the stream, return and clear the device status word (0 = ok)."""
    return lib().q4k_last_device_status(_stream(stream))


def q4k_test_wait_fault(drop_stage: int = -1, wait_limit_ns: int = 0) -> None:
    """Test hook: make the weight producers skip stage `drop_stage` (-1: off) and set the
    bounded-wait limit (0: the 2 s default). Synchronous; see include/q4k.h."""
    _check("q4k_test_wait_fault", lib().q4k_test_wait_fault(int(drop_stage), int(wait_limit_ns)))


def q4k_test_i8_cut(M: int, N: int, K: int, act: int = ACT_NONE, sms: int = 0, fit=None) -> dict:
    """Test hook: the form in which i8_gemm computes a product of these sizes, on the current
    device or on one of `sms` SMs with room for fit[c] clusters of c CTAs; see include/q4k.h."""
    cut = (_i * 7)()
    _check("q4k_test_i8_cut", lib().q4k_test_i8_cut(M, N, K, act, sms, None if fit is None else (_i * 9)(*fit), cut))
    return dict(zip(("pair", "ctas_per_sm", "m_tiles", "nt", "n_tiles", "ksplit", "stages"), cut))
