"""Refusals of the expert operators: every argument check of the C entry points
runs before any CUDA call, so it is tested without a GPU; and the Python
wrappers' checks of types and shapes on CPU tensors."""
from __future__ import annotations

import pytest
import torch

import tiled_gemm_codegen_gb300 as tg
from tiled_gemm_codegen_gb300 import _abi

INVALID, UNSUPPORTED = tg.TG_ERR_INVALID_ARG, tg.TG_ERR_UNSUPPORTED
# placeholder addresses, far apart
X, XS, IDS, OFF, SRC, SLOT, W, DW, DY = (0x1000000000 * i for i in range(1, 10))


@pytest.fixture(scope="module")
def lib():
    return _abi.load(build_if_missing=True)


def _dispatch(lib, **kw):
    a = dict(ids=IDS, id_bytes=8, ld_ids=4, T=10, k=4, E=8, offsets=OFF, source=SRC, slot=SLOT, x=X, ld_x=64, D=64,
             dtype=tg.TG_BF16 if hasattr(tg, "TG_BF16") else 1, xs=XS, ld_xs=64)
    a.update(kw)
    return lib.tg_expert_dispatch(*a.values(), None)


def test_dispatch_refusals(lib):
    for kw in (dict(T=-1), dict(k=0), dict(E=0), dict(id_bytes=2), dict(ids=None), dict(ids=IDS + 4), dict(offsets=None),
               dict(source=None), dict(slot=None), dict(ld_ids=3), dict(x=None), dict(xs=None), dict(ld_x=63),
               dict(ld_xs=63), dict(x=X + 1), dict(xs=XS + 1), dict(dtype=2), dict(D=-1), dict(T=1 << 30),
               dict(xs=X), dict(xs=X + 64), dict(slot=SRC), dict(offsets=XS + 100), dict(source=IDS), dict(T=1 << 40)):
        assert _dispatch(lib, **kw) == INVALID, kw
    assert _dispatch(lib, E=1025) == UNSUPPORTED
    assert _dispatch(lib, D=(1 << 22) + 1, ld_x=1 << 23, ld_xs=1 << 23) == UNSUPPORTED


def test_sort_and_gather_refusals(lib):
    assert lib.tg_expert_sort(IDS, 4, 4, 10, 4, 1025, OFF, SRC, SLOT, None) == UNSUPPORTED
    assert lib.tg_expert_sort(IDS, 4, 4, 10, 4, 8, OFF, SRC, SRC + 100, None) == INVALID
    good = [X, 64, 64, 1, 10, 4, 8, OFF, SLOT, XS, 64]
    for at, v in ((0, None), (1, 63), (2, -1), (3, 7), (5, 0), (7, None), (8, None), (9, None), (9, X + 128), (10, 3)):
        args = list(good)
        args[at] = v
        assert lib.tg_expert_gather(*args, None) == INVALID, at
    args = list(good)
    args[4] = 0  # no tokens: nothing to do
    assert lib.tg_expert_gather(*args, None) == tg.TG_OK


def test_combine_refusals(lib):
    good = [X, 64, 1, 40, SLOT, W, 4, 10, 4, 64, XS, 64, 1]
    for at, v in ((0, None), (1, 63), (2, 5), (3, -1), (4, None), (6, 3), (7, -1), (8, 0), (9, -2), (10, None), (10, X),
                  (11, 60), (12, 9), (10, XS + 1), (10, W)):
        args = list(good)
        args[at] = v
        assert lib.tg_expert_combine(*args, None) == INVALID, (at, v)
    args = list(good)
    args[7] = 0
    assert lib.tg_expert_combine(*args, None) == tg.TG_OK


def test_combine_grad_refusals(lib):
    good = [DY, 64, 1, X, 64, 1, OFF, SLOT, W, 4, 10, 4, 8, 64, XS, 64, 1, DW, 4]
    for at, v in ((0, None), (1, 63), (2, 5), (3, None), (4, 63), (5, 5), (6, None), (7, None), (9, 3), (11, 0), (12, 0),
                  (13, -1), (14, None), (14, DY), (14, X), (15, 63), (16, 3), (17, XS), (17, W), (18, 3)):
        args = list(good)
        args[at] = v
        assert lib.tg_expert_combine_grad(*args, None) == INVALID, (at, v)


def test_python_checks():
    ids = torch.zeros(4, 2, dtype=torch.int64)
    with pytest.raises(TypeError):
        tg.expert_sort(ids, 3)  # not on the GPU
    with pytest.raises(TypeError):
        tg.expert_dispatch(torch.zeros(4, 8), ids, 3)
    order = tg.ExpertOrder.empty(4, 2, 3, "cpu")
    assert [tuple(t.shape) for t in order] == [(4,), (8,), (4, 2)]
    with pytest.raises(TypeError):
        tg.expert_combine(torch.zeros(8, 8), order)
    with pytest.raises(AttributeError):
        tg.no_such_name


def _ep(**kw):
    ep = tg.tg_epilogue()
    ep.alpha = 1.0
    for k, v in kw.items():
        setattr(ep, k, v)
    return ep


def test_grouped_refusals(lib):
    import ctypes

    def rows(opt=None, ep=None, **kw):
        a = dict(A=X, B=XS, D=DY, offsets=OFF, groups=4, S=100, N=64, K=32, lda=32, ldb=64, strideB=2048, ldd=64)
        a.update(kw)
        return lib.tg_gemm_grouped(*a.values(), ctypes.byref(ep) if ep else None, None, ctypes.byref(opt) if opt else None)

    def wgrad(opt=None, ep=None, **kw):
        a = dict(A=X, B=XS, D=DY, offsets=OFF, groups=4, S=100, M=32, N=64, lda=32, ldb=64, ldd=64, strideD=2048)
        a.update(kw)
        return lib.tg_gemm_grouped_wgrad(*a.values(), ctypes.byref(ep) if ep else None, None, ctypes.byref(opt) if opt else None)

    for kw in (dict(groups=0), dict(S=-1), dict(N=-1), dict(K=-1), dict(lda=31), dict(ldb=63), dict(ldd=63), dict(strideB=-1),
               dict(A=None), dict(B=None), dict(D=None), dict(offsets=None), dict(D=X), dict(D=XS + 64), dict(D=OFF),
               dict(A=X + 1), dict(D=DY + 2), dict(S=2 ** 31 - 1), dict(ep=_ep(residual=W)), dict(ep=_ep(activation=9)),
               dict(ep=_ep(out_type=7)), dict(ep=_ep(bias=W, bias_stride=-1)), dict(opt=tg.make_options(split_k=2)),
               dict(opt=tg.make_options(cta_pair=3)), dict(opt=tg.make_options(a_col_major=1)),
               dict(opt=tg.make_options(b_col_major=1), ldb=31)):
        assert rows(**kw) == INVALID, kw
    for kw in (dict(groups=0), dict(S=-1), dict(M=-1), dict(N=-1), dict(lda=31), dict(ldb=63), dict(ldd=63), dict(strideD=100),
               dict(A=None), dict(B=None), dict(D=None), dict(offsets=None), dict(D=X), dict(D=XS), dict(D=OFF),
               dict(ep=_ep(bias=W)), dict(ep=_ep(activation=1)), dict(opt=tg.make_options(b_col_major=1)),
               dict(opt=tg.make_options(direct=2))):
        assert wgrad(**kw) == INVALID, kw
    assert rows(S=0) == tg.TG_OK and rows(N=0, ldb=1, ldd=1) == tg.TG_OK and wgrad(M=0) == tg.TG_OK


def test_w4_refusals(lib):
    def call(**kw):
        a = dict(x=X, ldx=128, W=XS, ldw=128, strideW=128 * 64, scales=SRC, ld_s=1, stride_s=64, zeros=None, ld_z=0, stride_z=0,
                 format=0, group=128, offsets=OFF, groups=4, S=10, N=64, K=128, y=DY, ldy=64, y_type=0)
        a.update(kw)
        return lib.tg_gemv_w4(*a.values(), None)

    for kw in (dict(groups=0), dict(S=-1), dict(N=-1), dict(K=-2), dict(K=127), dict(ldx=127), dict(ldw=126), dict(ldw=129),
               dict(strideW=-2), dict(strideW=8191), dict(ld_s=0), dict(group=16), dict(group=48), dict(format=2),
               dict(format=1), dict(format=1, group=32, ld_s=4, zeros=SLOT, ld_z=4), dict(zeros=SLOT, ld_z=0), dict(offsets=None),
               dict(x=None), dict(W=None), dict(scales=None), dict(y=None), dict(y=X), dict(y=XS + 4), dict(y=SRC), dict(y=OFF),
               dict(ldy=63), dict(y_type=2), dict(y=DY + 2), dict(x=X + 1), dict(scales=SRC + 1)):
        assert call(**kw) == INVALID, kw
    assert call(groups=70000, S=70000) == UNSUPPORTED
    assert call(S=0) == tg.TG_OK and call(N=0) == tg.TG_OK


class _OnGpu:
    """A CPU tensor that says it is on the GPU: what the wrappers read off it
    before a call."""

    def __init__(self, t):
        self._t = t

    is_cuda = True

    def __getattr__(self, name):
        return getattr(self._t, name)

    def get_device(self):
        return 0


BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _order(T, k, E):
    n = dict(dtype=I32)
    return tg.ExpertOrder(*(_OnGpu(t) for t in (torch.zeros(E + 1, **n), torch.zeros(T * k, **n), torch.zeros(T, k, **n))))


def _shared_rows(rows, cols, dtype):
    """The ways rows may share memory, the first two made by expand."""
    yield torch.zeros(cols, dtype=dtype).expand(rows, cols)
    yield torch.zeros(1, cols, dtype=dtype).expand(rows, cols)
    yield torch.zeros(rows * cols, dtype=dtype).as_strided((rows, cols), (cols - 1, 1))


def test_rows_that_share_memory_are_refused():
    """Read with the row length for a pitch they would be read, or written,
    past their storage: an expanded gradient, expanded weights, one row of
    scales for all.  The refusal comes before any CUDA call."""
    T, k, E, D = 6, 3, 4, 8
    z = lambda *s, dtype=BF: _OnGpu(torch.zeros(*s, dtype=dtype))  # noqa: E731
    order, ids = _order(T, k, E), z(T, k, dtype=torch.int64)
    off = z(E + 1, dtype=I32)

    def check(call, rows, cols, dtype):
        for t in _shared_rows(rows, cols, dtype):
            with pytest.raises(ValueError, match="contiguous"):
                call(_OnGpu(t))

    for c in (D, 1):
        check(lambda t, c=c: tg.expert_combine_grad(t, z(T * k, c), order, None), T, c, BF)
        check(lambda t, c=c: tg.expert_combine_grad(z(T, c), t, order, None), T * k, c, BF)
        check(lambda t, c=c: tg.expert_combine_grad(z(T, c), z(T * k, c), order, None, dys=t), T * k, c, BF)
        check(lambda t: tg.expert_combine(t, order), T * k, c, F32)
        check(lambda t, c=c: tg.expert_combine(z(T * k, c), order, y=t), T, c, BF)
        check(lambda t: tg.expert_gather(t, order), T, c, BF)
        check(lambda t, c=c: tg.expert_dispatch(z(T, c), ids, E, xs=t, order=order), T * k, c, BF)
        check(lambda t, c=c: tg.gemm_grouped(t, z(E, c, 16), off), 20, c, BF)
        check(lambda t, c=c: tg.gemm_grouped(z(20, 16), z(E, 16, c), off, t), 20, c, F32)
        check(lambda t, c=c: tg.gemm_grouped_wgrad(t, z(20, 16), off), 20, c, BF)
    check(lambda t: tg.expert_combine(z(T * k, D), order, t), T, k, F32)
    check(lambda t: tg.expert_combine_grad(z(T, D), z(T * k, D), order, t), T, k, F32)
    check(lambda t: tg.expert_combine_grad(z(T, D), z(T * k, D), order, None, dys=z(T * k, D), dweights=t), T, k, F32)
    check(lambda t: tg.expert_sort(t, E, order=order), T, k, torch.int64)
    check(lambda t: tg.expert_sort(t, E, order=_order(T, 1, E)), T, 1, I32)
    check(lambda t: tg.gemv_w4(t, z(5, 32, dtype=U8), z(5, 1), group=64), 4, 64, BF)
    check(lambda t: tg.gemv_w4(z(4, 64), t, z(5, 1), group=64), 5, 32, U8)
    check(lambda t: tg.gemv_w4(z(4, 64), z(5, 32, dtype=U8), t, group=32), 5, 2, BF)
    check(lambda t: tg.gemv_w4(z(4, 64), z(5, 32, dtype=U8), t, group=64), 5, 1, BF)
    check(lambda t: tg.gemv_w4(z(4, 64), z(5, 32, dtype=U8), z(5, 2), zeros=t, group=32), 5, 2, U8)
    check(lambda t: tg.gemv_w4(z(4, 64), z(5, 32, dtype=U8), z(5, 2), y=t, group=32), 4, 5, F32)
    # matrices of a stack whose rows (or, stored the other way, columns) lie 0 apart
    for B in (torch.zeros(16, dtype=BF).expand(E, 8, 16), torch.zeros(8, 1, dtype=BF).expand(E, 8, 16),
              torch.zeros(E, 8, 1, dtype=BF).expand(E, 8, 16), torch.zeros(E, 1, 1, dtype=BF).expand(E, 1, 16),
              torch.zeros(E, 1, 1, dtype=BF).expand(E, 8, 1)):
        with pytest.raises(ValueError):
            tg.gemm_grouped(z(20, B.shape[1]), _OnGpu(B), off)
    with pytest.raises(ValueError):
        tg.gemm_grouped_wgrad(z(20, 8), z(20, 16), off, _OnGpu(torch.zeros(E, 1, 16).expand(E, 8, 16)))


def test_pitches_that_are_read_off_tensors():
    """Rows apart by their length or more keep their pitch, single rows and
    columns any; the matrices of a stack may be one."""
    from tiled_gemm_codegen_gb300 import experts as ex

    t = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    rows = lambda v: ex._rows(_OnGpu(v), "x")[1:4]  # noqa: E731
    assert rows(t(5, 8)) == (5, 8, 8) and rows(t(5, 12)[:, 2:10]) == (5, 8, 12) and rows(t(10, 8)[::2]) == (5, 8, 16)
    assert rows(t(8).expand(1, 8)) == (1, 8, 8) and rows(t(5, 7)[:, :1]) == (5, 1, 7) and rows(t(5, 1)) == (5, 1, 1)
    assert rows(t(0, 8)) == (0, 8, 8) and rows(t(5, 0))[:2] == (5, 0)
    mats = lambda v: ex._matrices(_OnGpu(v), "B")[1:]  # noqa: E731
    assert mats(t(3, 4, 6)) == (3, 4, 6, 6, 24, False) and mats(t(3, 6, 4).transpose(1, 2)) == (3, 4, 6, 4, 24, True)
    assert mats(t(4, 6).expand(3, 4, 6)) == (3, 4, 6, 6, 0, False) and mats(t(3, 6, 9).transpose(1, 2)[:, :4]) == (3, 4, 6, 9, 54, True)
    assert mats(t(3, 6, 1).transpose(1, 2)) in ((3, 1, 6, 1, 6, True), (3, 1, 6, 6, 6, False))
    assert mats(t(3, 1, 6)) == (3, 1, 6, 6, 6, False) and mats(t(3, 4, 1)) == (3, 4, 1, 1, 4, False)


def test_gemm_operands_whose_rows_share_memory_are_refused():
    A, B = torch.zeros(8, dtype=BF).expand(4, 8), torch.zeros(8, 16, dtype=BF)
    for a, b, c in ((A, B, None), (B.t().contiguous(), A.contiguous().t()[:, :1].expand(8, 4), None),
                    (torch.zeros(4, 8, dtype=BF), B, torch.zeros(16).expand(4, 16))):
        with pytest.raises(ValueError):
            tg.gemm_host(a, b, c)
    with pytest.raises(ValueError, match="contiguous"):
        tg.gemm(_OnGpu(A), _OnGpu(B))
    with pytest.raises(ValueError, match="contiguous"):  # stored column-major, columns 0 apart
        tg.gemm(_OnGpu(torch.zeros(4, 8, dtype=BF)), _OnGpu(torch.zeros(8, 1, dtype=BF).expand(8, 16)))
    with pytest.raises(ValueError, match="contiguous"):
        tg.gemm(_OnGpu(torch.zeros(4, 8, dtype=BF)), _OnGpu(B), _OnGpu(torch.zeros(16).expand(4, 16)))
    with pytest.raises(ValueError, match="contiguous"):
        tg.gemm_fp8(_OnGpu(torch.zeros(32).to(torch.float8_e4m3fn).expand(4, 32)), _OnGpu(torch.zeros(16, 32).to(torch.float8_e4m3fn)))


def test_an_order_uses_the_tensors_it_shows():
    """Its tensors cannot be replaced, and their addresses are read at each
    call (storage that has moved is found where it is)."""
    from tiled_gemm_codegen_gb300 import experts as ex

    order = _order(4, 2, 3)
    for name in ("offsets", "source", "slot"):
        with pytest.raises(AttributeError):
            setattr(order, name, getattr(order, name))
    order.slot._t.set_(torch.ones(4, 2, dtype=I32))
    assert ex._order(order)[1] == tuple(t.data_ptr() for t in order)
    offsets, source, slot = order
    assert offsets is order.offsets and source is order.source and slot is order.slot


def test_layouts_are_the_tensors_own(monkeypatch):
    """Options tuned on transposed operands, used with row-major ones: the layout
    they hold would have the operands read past their storage."""
    from tiled_gemm_codegen_gb300 import experts as ex

    seen = []
    monkeypatch.setattr(tg, "tg_gemm_ex", lambda *a: seen.append((a[-1] and (a[-1].a_col_major, a[-1].b_col_major, a[-1].stages))) or tg.TG_OK)
    A, B, C = torch.zeros(24, 64, dtype=BF), torch.zeros(64, 40, dtype=BF), torch.zeros(24, 40)
    At, Bt = torch.zeros(64, 24, dtype=BF).t(), torch.zeros(40, 64, dtype=BF).t()
    for o in (None, dict(stages=4), dict(stages=4, a_col_major=1), dict(stages=4, a_col_major=1, b_col_major=1)):
        for a, b, want in ((A, B, (0, 0)), (At, B, (1, 0)), (A, Bt, (0, 1)), (At, Bt, (1, 1))):
            opts = None if o is None else tg.make_options(**o)
            tg.gemm(_OnGpu(a), _OnGpu(b), _OnGpu(C), options=opts, stream=0)
            assert seen[-1] == (None if o is None and want == (0, 0) else (*want, 0 if o is None else 4))
            assert opts is None or (opts.a_col_major, opts.b_col_major) == (o.get("a_col_major", 0), o.get("b_col_major", 0))

    class Lib:
        @staticmethod
        def tg_gemm_grouped(*a):
            seen.append(a[-1] and a[-1]._obj.b_col_major)
            return tg.TG_OK

    monkeypatch.setattr(ex, "_lib", lambda: Lib)
    W, Wt = torch.zeros(4, 64, 40, dtype=BF), torch.zeros(4, 40, 64, dtype=BF).transpose(1, 2)
    off, opts = _OnGpu(torch.zeros(5, dtype=I32)), tg.make_options(cta_pair=1, b_col_major=1)
    for b, o, want in ((W, opts, 0), (Wt, opts, 1), (W, None, None), (Wt, None, 1)):
        tg.gemm_grouped(_OnGpu(A), _OnGpu(b), off, _OnGpu(C), options=o, stream=0)
        assert seen[-1] == want


def test_words_off_their_alignment_are_refused(lib):
    """Bounds, slots, weights and bias are read in 4-byte words: a kernel given
    others would fault."""
    for kw in (dict(offsets=OFF + 2), dict(source=SRC + 1), dict(slot=SLOT + 2)):
        assert _dispatch(lib, **kw) == INVALID, kw
    assert lib.tg_expert_sort(IDS, 4, 4, 10, 4, 8, OFF + 2, SRC, SLOT, None) == INVALID
    for off, slot in ((OFF + 2, SLOT), (OFF, SLOT + 1)):
        assert lib.tg_expert_gather(X, 64, 64, 1, 10, 4, 8, off, slot, XS, 64, None) == INVALID
    for slot, w in ((SLOT + 2, W), (SLOT, W + 2)):
        assert lib.tg_expert_combine(X, 64, 1, 40, slot, w, 4, 10, 4, 64, XS, 64, 1, None) == INVALID
    for off, slot, w, dw in ((OFF + 2, SLOT, W, DW), (OFF, SLOT + 2, W, DW), (OFF, SLOT, W + 1, DW), (OFF, SLOT, W, DW + 2)):
        assert lib.tg_expert_combine_grad(DY, 64, 1, X, 64, 1, off, slot, w, 4, 10, 4, 8, 64, XS, 64, 1, dw, 4, None) == INVALID
    import ctypes

    def grouped(off, ep):
        return lib.tg_gemm_grouped(X, XS, DY, off, 4, 100, 64, 32, 32, 64, 2048, 64, ctypes.byref(ep), None, None)

    assert grouped(OFF + 2, _ep()) == INVALID and grouped(OFF, _ep(bias=W + 2)) == INVALID
    assert lib.tg_gemm_grouped_wgrad(X, XS, DY, OFF + 2, 4, 100, 32, 64, 32, 64, 64, 2048, None, None, None) == INVALID
    assert lib.tg_gemv_w4(X, 128, XS, 128, 128 * 64, SRC, 1, 64, None, 0, 0, 0, 128, OFF + 2, 4, 10, 64, 128, DY, 64, 0, None) == INVALID
