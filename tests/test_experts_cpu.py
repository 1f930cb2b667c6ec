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
