"""Operators of a mixture-of-experts layer on torch tensors: tokens sorted by
expert and back, the experts' products over the sorted rows, and products with
4-bit weights for single tokens.

As the rest of the package this is a thin binding of ``include/tg_gemm.h``:
pointers, shapes and strides are read off the tensors, and all arithmetic
happens in the CUDA library.  Calls are asynchronous on ``stream`` (default:
torch's current stream).
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import ACTIVATIONS, TgError, _operand, _operand_geometry, _stream_ptr, _with_layout
from ._abi import TG_BF16, TG_F32, TG_OK, TG_W4_E2M1, TG_W4_INT4, load, tg_epilogue

__all__ = ["ExpertOrder", "expert_sort", "expert_dispatch", "expert_gather", "expert_combine", "expert_combine_grad",
           "gemm_grouped", "gemm_grouped_wgrad", "gemv_w4", "W4_FORMATS"]

W4_FORMATS = {"int4": TG_W4_INT4, "e2m1": TG_W4_E2M1}
_DTYPES = {torch.float32: TG_F32, torch.bfloat16: TG_BF16}


class ExpertOrder(NamedTuple):
    """The stable order of T x k assignments by expert, int32 CUDA tensors:
    ``offsets`` [E + 1] (expert e's rows), ``source`` [T * k] (the flat
    assignment of each sorted row, -1 behind the last) and ``slot`` [T, k]
    (the sorted row of each assignment, -1 if dropped)."""

    offsets: torch.Tensor
    source: torch.Tensor
    slot: torch.Tensor

    @classmethod
    def empty(cls, tokens: int, k: int, num_experts: int, device="cuda") -> "ExpertOrder":
        """An uninitialised order, to be filled by expert_sort or
        expert_dispatch."""
        n = dict(dtype=torch.int32, device=device)
        return cls(torch.empty(num_experts + 1, **n), torch.empty(tokens * k, **n), torch.empty(tokens, k, **n))


def _check(st: int, what: str) -> None:
    if st != TG_OK:
        raise TgError(st, what)


def _rows(t, what, shape=None):
    """(ptr, ld, tg_dtype) of a 2-D fp32 or bf16 CUDA tensor with unit
    stride in its rows."""
    dt = _DTYPES.get(t.dtype)
    if dt is None or not t.is_cuda:
        raise TypeError(f"{what} must be an fp32 or bf16 CUDA tensor")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{what} must have shape {tuple(shape) if shape is not None else '[rows, D]'}")
    rows, cols = t.shape
    ld, inner = t.stride()
    if inner != 1 and cols > 1 and rows:
        raise ValueError(f"{what} must have unit stride in its last dimension")
    return t.data_ptr(), (ld if rows > 1 and ld > cols else cols), dt


def _weights(w, shape, what="weights"):
    if w is None:
        return None, 0
    if w.dtype != torch.float32 or not w.is_cuda:
        raise TypeError(f"{what} must be an fp32 CUDA tensor")
    if w.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}")
    T, k = shape
    if k > 1 and T and w.stride(1) != 1:
        raise ValueError(f"{what} must have unit stride in its last dimension")
    return w.data_ptr(), (max(w.stride(0), k) if T > 1 else k)


def _order(order, T=None, k=None, E=None):
    offsets, source, slot = order
    for t, name in ((offsets, "offsets"), (source, "source"), (slot, "slot")):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise TypeError(f"order.{name} must be a contiguous int32 CUDA tensor")
    if slot.dim() != 2 or offsets.dim() != 1 or source.shape != (slot.numel(),) or offsets.numel() < 2:
        raise ValueError("order must hold offsets [E + 1], source [T * k] and slot [T, k]")
    if T is not None and (slot.shape != (T, k) or offsets.numel() != E + 1):
        raise ValueError(f"order does not fit {T} x {k} assignments to {E} experts")
    return offsets, source, slot


def _ids(ids):
    if ids.dtype not in (torch.int32, torch.int64) or not ids.is_cuda:
        raise TypeError("ids must be an int32 or int64 CUDA tensor")
    if ids.dim() != 2 or ids.shape[1] < 1:
        raise ValueError("ids must have shape [T, k], k >= 1")
    T, k = ids.shape
    if k > 1 and T and ids.stride(1) != 1:
        raise ValueError("ids must have unit stride in their last dimension")
    return T, k, (max(ids.stride(0), k) if T > 1 else k), ids.element_size()


def expert_sort(ids, num_experts: int, *, order: ExpertOrder | None = None, stream=None) -> ExpertOrder:
    """The order of ids [T, k] (int32 or int64; ids outside [0, num_experts)
    drop their assignment) by expert, stable: equal ids keep their order."""
    T, k, ld, size = _ids(ids)
    if order is None:
        order = ExpertOrder.empty(T, k, num_experts, ids.device)
    offsets, source, slot = _order(order, T, k, num_experts)
    _check(load().tg_expert_sort(ids.data_ptr(), size, ld, T, k, num_experts, offsets.data_ptr(), source.data_ptr(),
                                 slot.data_ptr(), _stream_ptr(stream)), "tg_expert_sort")
    return order


def expert_dispatch(x, ids, num_experts: int, *, xs=None, order: ExpertOrder | None = None, stream=None):
    """(xs, order): the order of ids [T, k] and the rows of x [T, D] (fp32 or
    bf16) in it - xs [T * k, D], xs[s] = x[order.source[s] // k], rows behind
    the last expert zero.  Its gradient is expert_combine(dxs, order)."""
    T, k, ld, size = _ids(ids)
    px, ld_x, dt = _rows(x, "x")
    if x.shape[0] != T:
        raise ValueError(f"x must have {T} rows")
    D = x.shape[1]
    if xs is None:
        xs = torch.empty(T * k, D, dtype=x.dtype, device=x.device)
    pxs, ld_xs, dxs = _rows(xs, "xs", (T * k, D))
    if dxs != dt:
        raise TypeError("xs must have x's dtype")
    if order is None:
        order = ExpertOrder.empty(T, k, num_experts, ids.device)
    offsets, source, slot = _order(order, T, k, num_experts)
    _check(load().tg_expert_dispatch(ids.data_ptr(), size, ld, T, k, num_experts, offsets.data_ptr(),
                                     source.data_ptr(), slot.data_ptr(), px, ld_x, D, dt, pxs, ld_xs,
                                     _stream_ptr(stream)), "tg_expert_dispatch")
    return xs, order


def expert_gather(x, order: ExpertOrder, xs=None, *, stream=None):
    """xs [T * k, D]: the rows of x [T, D] in an order made before."""
    offsets, _, slot = _order(order)
    T, k = slot.shape
    px, ld_x, dt = _rows(x, "x")
    if x.shape[0] != T:
        raise ValueError(f"x must have {T} rows")
    D = x.shape[1]
    if xs is None:
        xs = torch.empty(T * k, D, dtype=x.dtype, device=x.device)
    pxs, ld_xs, dxs = _rows(xs, "xs", (T * k, D))
    if dxs != dt:
        raise TypeError("xs must have x's dtype")
    _check(load().tg_expert_gather(px, ld_x, D, dt, T, k, offsets.numel() - 1, offsets.data_ptr(), slot.data_ptr(),
                                   pxs, ld_xs, _stream_ptr(stream)), "tg_expert_gather")
    return xs


def expert_combine(ys, order: ExpertOrder, weights=None, *, y=None, out_dtype=None, stream=None):
    """y [T, D]: y[t] = sum_j weights[t, j] * ys[order.slot[t, j]] for ys
    [T * k, D] (fp32 or bf16) and fp32 weights [T, k] (None: ones, the
    gradient of expert_dispatch's rows), summed in fp32 and rounded once;
    dropped assignments add nothing.  y: out_dtype, by default ys's."""
    _, _, slot = _order(order)
    T, k = slot.shape
    pys, ld_ys, dt = _rows(ys, "ys")
    S, D = ys.shape
    pw, ld_w = _weights(weights, slot.shape)
    if y is None:
        y = torch.empty(T, D, dtype=out_dtype if out_dtype is not None else ys.dtype, device=ys.device)
    py, ld_y, dty = _rows(y, "y", (T, D))
    _check(load().tg_expert_combine(pys, ld_ys, dt, S, slot.data_ptr(), pw, ld_w, T, k, D, py, ld_y, dty,
                                    _stream_ptr(stream)), "tg_expert_combine")
    return y


def expert_combine_grad(dy, ys, order: ExpertOrder, weights, *, dys=None, dweights=None, out_dtype=None, stream=None):
    """(dys, dweights), the gradient of expert_combine for dy [T, D]:
    dys[order.slot[t, j]] = weights[t, j] * dy[t] (rows of no assignment
    zero; out_dtype, by default ys's) and dweights[t, j] = <dy[t],
    ys[order.slot[t, j]]> (fp32; dropped: zero)."""
    offsets, _, slot = _order(order)
    T, k = slot.shape
    pdy, ld_dy, t_dy = _rows(dy, "dy")
    D = dy.shape[1]
    if dy.shape[0] != T:
        raise ValueError(f"dy must have {T} rows")
    pys, ld_ys, t_ys = _rows(ys, "ys", (T * k, D))
    pw, ld_w = _weights(weights, slot.shape)
    if dys is None:
        dys = torch.empty(T * k, D, dtype=out_dtype if out_dtype is not None else ys.dtype, device=dy.device)
    if dweights is None:
        dweights = torch.empty(T, k, dtype=torch.float32, device=dy.device)
    pdys, ld_dys, t_dys = _rows(dys, "dys", (T * k, D))
    pdw, ld_dw = _weights(dweights, slot.shape, "dweights")
    _check(load().tg_expert_combine_grad(pdy, ld_dy, t_dy, pys, ld_ys, t_ys, offsets.data_ptr(), slot.data_ptr(), pw,
                                         ld_w, T, k, offsets.numel() - 1, D, pdys, ld_dys, t_dys, pdw, ld_dw,
                                         _stream_ptr(stream)), "tg_expert_combine_grad")
    return dys, dweights


def _offsets(offsets, what="offsets"):
    if offsets.dtype != torch.int32 or not offsets.is_cuda or not offsets.is_contiguous():
        raise TypeError(f"{what} must be a contiguous int32 CUDA tensor")
    if offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError(f"{what} must have shape [groups + 1]")
    return offsets.data_ptr(), offsets.numel() - 1


def _bf16_rows(t, what):
    if t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError(f"{what} must be a bf16 CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{what} must have shape [rows, columns]")
    p, rows, cols, ld, _, _ = _operand_geometry(t, -2, what)
    return p, rows, cols, ld


def _epilogue(D, alpha, activation="none", bias=None, groups=0, N=0):
    ep = tg_epilogue()
    ep.alpha = float(alpha)
    ep.activation = ACTIVATIONS[activation]
    ep.out_type = TG_BF16 if D.dtype == torch.bfloat16 else TG_F32
    if bias is not None:
        if bias.dtype != torch.float32 or not bias.is_cuda or (bias.shape[-1] > 1 and bias.stride(-1) != 1):
            raise TypeError("bias must be an fp32 CUDA tensor with unit stride in its last dimension")
        if bias.shape not in ((N,), (groups, N)):
            raise ValueError(f"bias must have shape [{N}] or [{groups}, {N}]")
        ep.bias = bias.data_ptr()
        ep.bias_stride = bias.stride(0) if bias.dim() == 2 and groups > 1 else 0
    return ep


def _out(D, shape, out_dtype, device):
    if D is None:
        return torch.empty(shape, dtype=out_dtype if out_dtype is not None else torch.float32, device=device)
    if D.dtype not in (torch.float32, torch.bfloat16) or not D.is_cuda:
        raise TypeError("D must be an fp32 or bf16 CUDA tensor")
    if D.shape != shape:
        raise ValueError(f"D must have shape {tuple(shape)}")
    return D


def gemm_grouped(A, B, offsets, D=None, *, alpha: float = 1.0, bias=None, activation: str = "none", out_dtype=None,
                 options=None, stream=None):
    """D [S, N] = act(alpha * A @ B[g] + bias[g]) for the rows s of A [S, K]
    with offsets[g] <= s < offsets[g + 1] (int32 [groups + 1] on the GPU, an
    order's), zero for rows in no group.  A and B [groups, K, N] are bf16; a
    transposed view of B is taken as it is, so the gradient of A is
    gemm_grouped(dD, B.transpose(1, 2), offsets).  bias: fp32 [N] or
    [groups, N]; D: fp32 (default) or bf16."""
    po, groups = _offsets(offsets)
    pa, S, K, lda = _bf16_rows(A, "A")
    if B.dtype != torch.bfloat16 or not B.is_cuda:
        raise TypeError("B must be a bf16 CUDA tensor")
    if B.dim() != 3 or B.shape[0] != groups:
        raise ValueError(f"B must have shape [{groups}, K, N]")
    pb, K2, N, ldb, _, strideB, b_cm = _operand(B, "B")
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    D = _out(D, (S, N), out_dtype, A.device)
    pd, _, _, ldd, _, _ = _operand_geometry(D, -2, "D")
    options = _with_layout(options, False, b_cm)
    ep = _epilogue(D, alpha, activation, bias, groups, N)
    _check(load().tg_gemm_grouped(pa, pb, pd, po, groups, S, N, K, lda, ldb, strideB, ldd, ctypes.byref(ep),
                                  _stream_ptr(stream), ctypes.byref(options) if options is not None else None),
           "tg_gemm_grouped")
    return D


def gemm_grouped_wgrad(A, B, offsets, D=None, *, alpha: float = 1.0, out_dtype=None, options=None, stream=None):
    """D [groups, M, N]: D[g] = alpha * A[rows g]^T @ B[rows g] for bf16 A
    [S, M] and B [S, N], rows g = offsets[g] .. offsets[g + 1] - 1; zero for
    an empty group.  With the forward call's A and dL/dD for B this is the
    gradient of its weights.  D: fp32 (default) or bf16."""
    po, groups = _offsets(offsets)
    pa, S, M, lda = _bf16_rows(A, "A")
    pb, S2, N, ldb = _bf16_rows(B, "B")
    if S2 != S:
        raise ValueError(f"A and B have {S} and {S2} rows")
    D = _out(D, (groups, M, N), out_dtype, A.device)
    pd, _, _, ldd, _, strideD = _operand_geometry(D, -2, "D")
    ep = _epilogue(D, alpha)
    _check(load().tg_gemm_grouped_wgrad(pa, pb, pd, po, groups, S, M, N, lda, ldb, ldd, strideD, ctypes.byref(ep),
                                        _stream_ptr(stream), ctypes.byref(options) if options is not None else None),
           "tg_gemm_grouped_wgrad")
    return D


def gemv_w4(x, W, scales, *, zeros=None, offsets=None, y=None, format: str = "int4", group: int | None = None,
            out_dtype=None, stream=None):
    """y [S, N] = x @ w^T for a few bf16 rows x [S, K] and 4-bit weights: W
    [N, K / 2] or [groups, N, K / 2] uint8, two codes a byte (element k in
    byte k // 2, the low nibble for even k).  With offsets (int32 [groups + 1],
    an order's) rows offsets[g] .. offsets[g + 1] - 1 meet group g's weights
    and rows of no group give zeros.  Every ``group`` codes of a row share a
    scale:

    - format "int4": w = (code - z) * scale, scales bf16 [.., N, ceil(K /
      group)], z from zeros (uint8, the scales' shape; None: 8), group 32, 64
      or 128 (the default);
    - format "e2m1": w = e2m1(code) * 2^(e - 127), scales uint8 E8M0 codes,
      group 32: the operands of gemm_mxfp4.

    y: fp32 (default) or bf16."""
    fmt = W4_FORMATS.get(format)
    if fmt is None:
        raise ValueError(f"format must be one of {sorted(W4_FORMATS)}")
    if group is None:
        group = 32 if fmt == TG_W4_E2M1 else 128
    px, S, K, ldx = _bf16_rows(x, "x")
    if W.dtype != torch.uint8 or not W.is_cuda:
        raise TypeError("W must be a uint8 CUDA tensor (two codes a byte)")
    if W.dim() not in (2, 3) or 2 * W.shape[-1] != K:
        raise ValueError(f"W must have shape [.., N, {K // 2}] for x of {K} columns")
    pW, N, _, ldw, groups, strideW = _operand_geometry(W, -2, "W")
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    shape = (*W.shape[:-1], -(-K // group))
    geo = []
    want = torch.uint8 if fmt == TG_W4_E2M1 else torch.bfloat16
    for t, dt, name in ((scales, want, "scales"), (zeros, torch.uint8, "zeros")):
        if t is None:
            geo.append((None, 0, 0))
            continue
        if t.dtype != dt or not t.is_cuda:
            raise TypeError(f"{name} must be a {dt} CUDA tensor")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {list(shape)}")
        p, _, _, ld, _, st = _operand_geometry(t, -2, name)
        geo.append((p, ld, st))
    po = None
    if offsets is not None:
        po, n = _offsets(offsets)
        if n != groups:
            raise ValueError(f"offsets must have shape [{groups + 1}]")
    elif groups != 1:
        raise ValueError("weights of several groups need offsets")
    y = _out(y, (S, N), out_dtype, x.device)
    py, _, _, ldy, _, _ = _operand_geometry(y, -2, "y")
    (ps, ld_s, st_s), (pz, ld_z, st_z) = geo
    _check(load().tg_gemv_w4(px, ldx, pW, 2 * ldw, 2 * strideW, ps, ld_s, st_s, pz, ld_z, st_z, fmt, group, po, groups, S, N, K,
                             py, ldy, TG_BF16 if y.dtype == torch.bfloat16 else TG_F32, _stream_ptr(stream)), "tg_gemv_w4")
    return y
