"""Operators of a mixture-of-experts layer on torch tensors: tokens sorted by
expert and back, the experts' products over the sorted rows, and products with
4-bit weights for single tokens.

As the rest of the package this is a thin binding of ``include/tg_gemm.h``:
pointers, shapes and strides are read off the tensors, and all arithmetic
happens in the CUDA library.  Calls are asynchronous on ``stream`` (default:
torch's current stream).  A row starts behind the one before it: tensors whose
rows share memory, as ``expand`` makes them (the gradient of a sum over
tokens, uniform weights), are refused and go in as a copy (``contiguous()``);
the matrices of a stack may share theirs.  As the rest of the package the
calls record no gradients (``examples/moe_layer.py`` makes an autograd function
of them), and outputs that they make belong to torch's current stream.
"""
from __future__ import annotations

import ctypes

import torch

from . import ACTIVATIONS, TgError, _pitch, _stream_ptr, _with_layout
from ._abi import TG_BF16, TG_F32, TG_OK, TG_W4_E2M1, TG_W4_INT4, load, tg_epilogue, tg_options

__all__ = ["ExpertOrder", "expert_sort", "expert_dispatch", "expert_gather", "expert_combine", "expert_combine_grad",
           "gemm_grouped", "gemm_grouped_wgrad", "gemv_w4", "W4_FORMATS"]

W4_FORMATS = {"int4": TG_W4_INT4, "e2m1": TG_W4_E2M1}
_DTYPES = {torch.float32: TG_F32, torch.bfloat16: TG_BF16}
_BF16, _U8 = torch.bfloat16, torch.uint8

# A call for a few tokens costs the GPU 2-3 us, so these wrappers read each
# property of a tensor once and keep nothing but the library's handle.
_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        _LIB = load()
    return _LIB


def _stream(t, stream):
    """The stream's handle; by default the current one of t's device."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(t.get_device())
    return _stream_ptr(stream)


class ExpertOrder:
    """The stable order of T x k assignments by expert: int32 tensors
    ``offsets`` [E + 1] (expert e's rows), ``source`` [T * k] (the flat
    assignment of each sorted row, -1 behind the last) and ``slot`` [T, k]
    (the sorted row of each assignment, -1 if dropped).  Unpacks as the
    three of them, which stay the ones it was made of."""

    __slots__ = ("_tensors", "shape", "_on_gpu")

    def __init__(self, offsets, source, slot):
        for t, name in ((offsets, "offsets"), (source, "source"), (slot, "slot")):
            if t.dtype != torch.int32 or not t.is_contiguous():
                raise TypeError(f"{name} must be a contiguous int32 tensor")
        if slot.dim() != 2 or slot.shape[1] < 1 or offsets.dim() != 1 or source.shape != (slot.numel(),) or offsets.numel() < 2:
            raise ValueError("an order holds offsets [E + 1], source [T * k] and slot [T, k]")
        self._tensors = (offsets, source, slot)
        self.shape = (*slot.shape, offsets.numel() - 1)  # T, k, E
        self._on_gpu = offsets.is_cuda and source.is_cuda and slot.is_cuda

    offsets = property(lambda self: self._tensors[0])
    source = property(lambda self: self._tensors[1])
    slot = property(lambda self: self._tensors[2])

    def __iter__(self):
        return iter(self._tensors)

    @classmethod
    def empty(cls, tokens: int, k: int, num_experts: int, device="cuda") -> "ExpertOrder":
        """An uninitialised order, to be filled by expert_sort or
        expert_dispatch."""
        n = dict(dtype=torch.int32, device=device)
        return cls(torch.empty(num_experts + 1, **n), torch.empty(tokens * k, **n), torch.empty(tokens, k, **n))


def _check(st: int, what: str) -> None:
    if st != TG_OK:
        raise TgError(st, what)


def _order(order, shape=None):
    """((T, k, E), pointers) of an order on the GPU."""
    if not order._on_gpu:
        raise TypeError("the order's tensors must be on the GPU")
    if shape is not None and order.shape != shape:
        raise ValueError(f"the order is one of {order.shape[0]} x {order.shape[1]} assignments to {order.shape[2]} experts, "
                         f"not {shape[0]} x {shape[1]} to {shape[2]}")
    offsets, source, slot = order._tensors
    return order.shape, (offsets.data_ptr(), source.data_ptr(), slot.data_ptr())


def _rows(t, what, rows=None, cols=None):
    """(ptr, rows, columns, ld, tg_dtype) of a 2-D fp32 or bf16 CUDA tensor
    with unit stride in its rows."""
    dt = _DTYPES.get(t.dtype)
    if dt is None or not t.is_cuda:
        raise TypeError(f"{what} must be an fp32 or bf16 CUDA tensor")
    shape, st = t.shape, t.stride()
    if len(shape) != 2 or (rows is not None and shape[0] != rows) or (cols is not None and shape[1] != cols):
        raise ValueError(f"{what} must have shape [{'rows' if rows is None else rows}, {'columns' if cols is None else cols}]")
    n, c = shape
    if st[1] != 1 and c > 1 and n:
        raise ValueError(f"{what} must have unit stride in its last dimension")
    return t.data_ptr(), n, c, _pitch(st[0], n, c, what), dt


def _weights(w, T, k, what="weights"):
    if w is None:
        return None, 0
    if w.dtype != torch.float32 or not w.is_cuda:
        raise TypeError(f"{what} must be an fp32 CUDA tensor")
    if w.shape != (T, k):
        raise ValueError(f"{what} must have shape [{T}, {k}]")
    st = w.stride()
    if k > 1 and T and st[1] != 1:
        raise ValueError(f"{what} must have unit stride in its last dimension")
    return w.data_ptr(), _pitch(st[0], T, k, what)


def _ids(ids):
    dt = ids.dtype
    if (dt != torch.int64 and dt != torch.int32) or not ids.is_cuda:
        raise TypeError("ids must be an int32 or int64 CUDA tensor")
    shape, st = ids.shape, ids.stride()
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError("ids must have shape [T, k], k >= 1")
    T, k = shape
    if k > 1 and T and st[1] != 1:
        raise ValueError("ids must have unit stride in their last dimension")
    return ids.data_ptr(), (8 if dt == torch.int64 else 4), _pitch(st[0], T, k, "ids"), T, k


def expert_sort(ids, num_experts: int, *, order: ExpertOrder | None = None, stream=None) -> ExpertOrder:
    """The order of ids [T, k] (int32 or int64; ids outside [0, num_experts)
    drop their assignment) by expert, stable: equal ids keep their order."""
    pid, size, ld, T, k = _ids(ids)
    if order is None:
        order = ExpertOrder.empty(T, k, num_experts, ids.device)
    _, (po, pso, psl) = _order(order, (T, k, num_experts))
    _check(_lib().tg_expert_sort(pid, size, ld, T, k, num_experts, po, pso, psl, _stream(ids, stream)), "tg_expert_sort")
    return order


def expert_dispatch(x, ids, num_experts: int, *, xs=None, order: ExpertOrder | None = None, stream=None):
    """(xs, order): the order of ids [T, k] and the rows of x [T, D] (fp32 or
    bf16) in it - xs [T * k, D], xs[s] = x[order.source[s] // k], rows behind
    the last expert zero.  Its gradient is expert_combine(dxs, order)."""
    pid, size, ld, T, k = _ids(ids)
    px, _, D, ld_x, dt = _rows(x, "x", T)
    if xs is None:
        xs = torch.empty(T * k, D, dtype=x.dtype, device=x.device)
    pxs, _, _, ld_xs, dxs = _rows(xs, "xs", T * k, D)
    if dxs != dt:
        raise TypeError("xs must have x's dtype")
    if order is None:
        order = ExpertOrder.empty(T, k, num_experts, ids.device)
    _, (po, pso, psl) = _order(order, (T, k, num_experts))
    _check(_lib().tg_expert_dispatch(pid, size, ld, T, k, num_experts, po, pso, psl, px, ld_x, D, dt, pxs, ld_xs,
                                     _stream(x, stream)), "tg_expert_dispatch")
    return xs, order


def expert_gather(x, order: ExpertOrder, xs=None, *, stream=None):
    """xs [T * k, D]: the rows of x [T, D] in an order made before."""
    (T, k, E), (po, _, psl) = _order(order)
    px, _, D, ld_x, dt = _rows(x, "x", T)
    if xs is None:
        xs = torch.empty(T * k, D, dtype=x.dtype, device=x.device)
    pxs, _, _, ld_xs, dxs = _rows(xs, "xs", T * k, D)
    if dxs != dt:
        raise TypeError("xs must have x's dtype")
    _check(_lib().tg_expert_gather(px, ld_x, D, dt, T, k, E, po, psl, pxs, ld_xs, _stream(x, stream)), "tg_expert_gather")
    return xs


def expert_combine(ys, order: ExpertOrder, weights=None, *, y=None, out_dtype=None, stream=None):
    """y [T, D]: y[t] = sum_j weights[t, j] * ys[order.slot[t, j]] for ys
    [T * k, D] (fp32 or bf16) and fp32 weights [T, k] (None: ones, the
    gradient of expert_dispatch's rows), summed in fp32 and rounded once;
    dropped assignments add nothing.  y: out_dtype, by default ys's."""
    (T, k, _), (_, _, psl) = _order(order)
    pys, S, D, ld_ys, dt = _rows(ys, "ys")
    pw, ld_w = _weights(weights, T, k)
    if y is None:
        y = torch.empty(T, D, dtype=out_dtype if out_dtype is not None else ys.dtype, device=ys.device)
    py, _, _, ld_y, dty = _rows(y, "y", T, D)
    _check(_lib().tg_expert_combine(pys, ld_ys, dt, S, psl, pw, ld_w, T, k, D, py, ld_y, dty, _stream(ys, stream)),
           "tg_expert_combine")
    return y


def expert_combine_grad(dy, ys, order: ExpertOrder, weights, *, dys=None, dweights=None, out_dtype=None, stream=None):
    """(dys, dweights), the gradient of expert_combine for dy [T, D]:
    dys[order.slot[t, j]] = weights[t, j] * dy[t] (rows of no assignment
    zero; out_dtype, by default ys's) and dweights[t, j] = <dy[t],
    ys[order.slot[t, j]]> (fp32; dropped: zero)."""
    (T, k, E), (po, _, psl) = _order(order)
    pdy, _, D, ld_dy, t_dy = _rows(dy, "dy", T)
    pys, _, _, ld_ys, t_ys = _rows(ys, "ys", T * k, D)
    pw, ld_w = _weights(weights, T, k)
    if dys is None:
        dys = torch.empty(T * k, D, dtype=out_dtype if out_dtype is not None else ys.dtype, device=dy.device)
    if dweights is None:
        dweights = torch.empty(T, k, dtype=torch.float32, device=dy.device)
    pdys, _, _, ld_dys, t_dys = _rows(dys, "dys", T * k, D)
    pdw, ld_dw = _weights(dweights, T, k, "dweights")
    _check(_lib().tg_expert_combine_grad(pdy, ld_dy, t_dy, pys, ld_ys, t_ys, po, psl, pw, ld_w, T, k, E, D, pdys, ld_dys, t_dys,
                                         pdw, ld_dw, _stream(dy, stream)), "tg_expert_combine_grad")
    return dys, dweights


def _offsets(offsets):
    if offsets.dtype != torch.int32 or not offsets.is_cuda or not offsets.is_contiguous():
        raise TypeError("offsets must be a contiguous int32 CUDA tensor")
    shape = offsets.shape
    if len(shape) != 1 or shape[0] < 2:
        raise ValueError("offsets must have shape [groups + 1]")
    return offsets.data_ptr(), shape[0] - 1


def _bf16_rows(t, what):
    if t.dtype != _BF16:
        raise TypeError(f"{what} must be a bf16 CUDA tensor")
    return _rows(t, what)[:4]


def _matrices(t, what):
    """(ptr, groups, rows, columns, ld, group stride, column-major) of a 3-D
    CUDA tensor whose matrices are row-major or transposed views."""
    shape, st = t.shape, t.stride()
    if len(shape) != 3:
        raise ValueError(f"{what} must have shape [groups, rows, columns]")
    g, r, c = shape
    sg = st[0] if g > 1 else 0
    if c > 1 and st[2] != 1 and (st[1] == 1 or r == 1):
        return t.data_ptr(), g, r, c, _pitch(st[2], c, max(r, 1), what), sg, True
    if st[2] != 1 and c > 1 and t.numel():
        raise ValueError(f"{what} must have unit stride in one of its last two dimensions")
    return t.data_ptr(), g, r, c, _pitch(st[1], r, c, what), sg, False


def _plain_epilogue(out_type):
    ep = tg_epilogue()
    ep.alpha = 1.0
    ep.out_type = out_type
    return ctypes.byref(ep)


_PLAIN = {torch.float32: _plain_epilogue(TG_F32), torch.bfloat16: _plain_epilogue(TG_BF16)}
_B_COL_MAJOR = ctypes.byref(tg_options(b_col_major=1))


def _epilogue(dtype, alpha, activation="none", bias=None, groups=0, N=0):
    """The epilogue, by reference."""
    if alpha == 1.0 and activation == "none" and bias is None:
        return _PLAIN[dtype]
    ep = tg_epilogue()
    ep.alpha = float(alpha)
    ep.activation = ACTIVATIONS[activation]
    ep.out_type = _DTYPES[dtype]
    if bias is not None:
        if bias.dtype != torch.float32 or not bias.is_cuda or (bias.shape[-1] > 1 and bias.stride(-1) != 1):
            raise TypeError("bias must be an fp32 CUDA tensor with unit stride in its last dimension")
        if bias.shape not in ((N,), (groups, N)):
            raise ValueError(f"bias must have shape [{N}] or [{groups}, {N}]")
        ep.bias = bias.data_ptr()
        ep.bias_stride = bias.stride(0) if bias.dim() == 2 and groups > 1 else 0
    return ctypes.byref(ep)


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
    if B.dtype != _BF16 or not B.is_cuda:
        raise TypeError("B must be a bf16 CUDA tensor")
    pb, gb, K2, N, ldb, strideB, b_cm = _matrices(B, "B")
    if gb != groups:
        raise ValueError(f"B must have shape [{groups}, K, N]")
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if D is None:
        D = torch.empty(S, N, dtype=out_dtype if out_dtype is not None else torch.float32, device=A.device)
    pd, _, _, ldd, _ = _rows(D, "D", S, N)
    if options is not None:
        options = ctypes.byref(_with_layout(options, False, b_cm))
    elif b_cm:
        options = _B_COL_MAJOR
    _check(_lib().tg_gemm_grouped(pa, pb, pd, po, groups, S, N, K, lda, ldb, strideB, ldd,
                                  _epilogue(D.dtype, alpha, activation, bias, groups, N), _stream(A, stream), options),
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
    if D is None:
        D = torch.empty(groups, M, N, dtype=out_dtype if out_dtype is not None else torch.float32, device=A.device)
    if D.dtype not in _DTYPES or not D.is_cuda:
        raise TypeError("D must be an fp32 or bf16 CUDA tensor")
    pd, gd, Md, Nd, ldd, strideD, d_cm = _matrices(D, "D")
    if (gd, Md, Nd) != (groups, M, N) or d_cm:
        raise ValueError(f"D must be row-major with shape [{groups}, {M}, {N}]")
    _check(_lib().tg_gemm_grouped_wgrad(pa, pb, pd, po, groups, S, M, N, lda, ldb, ldd, strideD, _epilogue(D.dtype, alpha),
                                        _stream(A, stream), ctypes.byref(options) if options is not None else None),
           "tg_gemm_grouped_wgrad")
    return D


def _per_row(t, what, dtype, lead, cols):
    """(ptr, ld, group stride) of scales or zeros [*lead, cols]."""
    if t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{what} must be a {dtype} CUDA tensor")
    if t.shape != (*lead, cols):
        raise ValueError(f"{what} must have shape {[*lead, cols]}")
    st = t.stride()
    if cols > 1 and st[-1] != 1:
        raise ValueError(f"{what} must have unit stride in its last dimension")
    return t.data_ptr(), _pitch(st[-2], lead[-1], cols, what), (st[0] if len(lead) == 2 and lead[0] > 1 else 0)


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
    elif group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    px, S, K, ldx = _bf16_rows(x, "x")
    if W.dtype != _U8 or not W.is_cuda:
        raise TypeError("W must be a uint8 CUDA tensor (two codes a byte)")
    lead = tuple(W.shape[:-1])
    if len(lead) not in (1, 2) or 2 * W.shape[-1] != K:
        raise ValueError(f"W must have shape [.., N, {K // 2}] for x of {K} columns")
    groups, N = (lead if len(lead) == 2 else (1, lead[0]))
    pW, ldw, strideW = _per_row(W, "W", _U8, lead, K // 2)
    runs = -(-K // group)
    ps, ld_s, st_s = _per_row(scales, "scales", _U8 if fmt == TG_W4_E2M1 else _BF16, lead, runs)
    pz, ld_z, st_z = _per_row(zeros, "zeros", _U8, lead, runs) if zeros is not None else (None, 0, 0)
    po = None
    if offsets is not None:
        po, n = _offsets(offsets)
        if n != groups:
            raise ValueError(f"offsets must have shape [{groups + 1}]")
    elif groups != 1:
        raise ValueError("weights of several groups need offsets")
    if y is None:
        y = torch.empty(S, N, dtype=out_dtype if out_dtype is not None else torch.float32, device=x.device)
    py, _, _, ldy, ty = _rows(y, "y", S, N)
    _check(_lib().tg_gemv_w4(px, ldx, pW, 2 * ldw, 2 * strideW, ps, ld_s, st_s, pz, ld_z, st_z, fmt, group, po, groups, S, N, K,
                             py, ldy, ty, _stream(x, stream)), "tg_gemv_w4")
    return y
