"""Refusals of the projections: every argument check of the C entry points runs
before any CUDA call, so it is tested without a GPU; and the Python wrappers'
checks of types and shapes on CPU tensors."""
from __future__ import annotations

import ctypes

import pytest
import torch

import tiled_gemm_codegen_gb300 as tg
from tiled_gemm_codegen_gb300 import _abi

INVALID, UNSUPPORTED, OK = tg.TG_ERR_INVALID_ARG, tg.TG_ERR_UNSUPPORTED, tg.TG_OK
# placeholder addresses, far apart
X, W, H, Z, OFF, DZ, A, B, Y, U, SC = (0x1000000000 * i for i in range(1, 12))
BAD_OPTIONS = (dict(split_k=2), dict(cta_pair=3), dict(a_col_major=1), dict(stages=4), dict(debug_stall=2), dict(direct=1))


@pytest.fixture(scope="module")
def lib():
    return _abi.load(build_if_missing=True)


def _call(fn, a, opt):
    return fn(*a.values(), None, ctypes.byref(opt) if opt else None)


def _gated(lib, opt=None, **kw):
    a = dict(X=X, W=W, H=H, Z=Z, offsets=OFF, groups=4, S=100, F=64, K=32, ldx=32, ldw=128, strideW=4096, ldh=64, ldz=128, act=3)
    return _call(lib.tg_gemm_gated, {**a, **kw}, opt)


def _grad(lib, opt=None, **kw):
    a = dict(dY=X, V=W, Z=Z, dZ=DZ, H=H, offsets=OFF, groups=4, S=100, F=64, K=32, lddy=32, ldv=64, strideV=2048, ldz=128, lddz=128,
             ldh=64, act=3)
    return _call(lib.tg_gemm_gated_grad, {**a, **kw}, opt)


def _adapted(lib, opt=None, **kw):
    a = dict(X=X, W=W, A=A, B=B, Y=Y, U=U, offsets=OFF, scales=SC, groups=4, S=100, N=64, K=32, R=16, ldx=32, ldw=64, lda=32,
             strideA=512, ldb=64, strideB=1024, ldy=64, ldu=16, y_type=0)
    return _call(lib.tg_gemm_adapted, {**a, **kw}, opt)


def test_gated_refusals(lib):
    for kw in (dict(groups=0), dict(S=-1), dict(F=-1), dict(K=-1), dict(ldx=31), dict(ldw=127), dict(ldh=63), dict(ldz=127),
               dict(strideW=-1), dict(X=None), dict(W=None), dict(H=None), dict(offsets=None), dict(X=X + 1), dict(W=W + 1),
               dict(H=H + 1), dict(Z=Z + 1), dict(offsets=OFF + 2), dict(H=X), dict(H=W + 64), dict(Z=X + 100), dict(Z=H), dict(H=OFF),
               dict(S=2 ** 31 - 1), dict(F=2 ** 30, ldw=2 ** 31, ldh=2 ** 31, ldz=2 ** 31), dict(F=2 ** 62), dict(act=4), dict(act=-1),
               dict(ldx=2 ** 41), dict(opt=tg.make_options(b_col_major=1), ldw=31)):
        assert _gated(lib, **kw) == INVALID, kw
    for o in BAD_OPTIONS:
        assert _gated(lib, opt=tg.make_options(**o)) == INVALID, o
    assert _gated(lib, S=0) == OK and _gated(lib, F=0, ldw=1, ldh=1, ldz=1) == OK
    assert _gated(lib, S=0, Z=None, ldz=0) == OK


def test_gated_grad_refusals(lib):
    for kw in (dict(groups=0), dict(S=-1), dict(F=-1), dict(K=-1), dict(lddy=31), dict(ldv=63), dict(ldh=63), dict(ldz=127),
               dict(lddz=127), dict(strideV=-1), dict(dY=None), dict(V=None), dict(Z=None), dict(dZ=None), dict(offsets=None),
               dict(dY=X + 1), dict(V=W + 1), dict(H=H + 1), dict(Z=Z + 1), dict(dZ=DZ + 1), dict(offsets=OFF + 2), dict(H=X), dict(H=Z),
               dict(dZ=Z), dict(dZ=X + 100), dict(dZ=H), dict(dZ=OFF), dict(S=2 ** 31 - 1), dict(act=4), dict(F=2 ** 62),
               dict(opt=tg.make_options(b_col_major=1), ldv=31)):
        assert _grad(lib, **kw) == INVALID, kw
    for o in BAD_OPTIONS:
        assert _grad(lib, opt=tg.make_options(**o)) == INVALID, o
    assert _grad(lib, S=0) == OK and _grad(lib, S=0, H=None, ldh=0) == OK


def test_adapted_refusals(lib):
    for kw in (dict(groups=0), dict(S=-1), dict(N=-1), dict(K=-1), dict(R=0), dict(ldx=31), dict(ldw=63), dict(lda=31), dict(ldb=63),
               dict(ldy=63), dict(ldu=15), dict(strideA=-1), dict(strideB=-1), dict(X=None), dict(W=None), dict(A=None), dict(B=None),
               dict(Y=None), dict(offsets=None), dict(X=X + 1), dict(W=W + 1), dict(A=A + 1), dict(B=B + 1), dict(Y=Y + 2),
               dict(Y=Y + 1, y_type=1), dict(U=U + 1), dict(offsets=OFF + 2), dict(scales=SC + 1), dict(Y=X), dict(Y=A + 64), dict(Y=B),
               dict(Y=SC), dict(U=W), dict(U=Y), dict(Y=OFF), dict(S=2 ** 31 - 1), dict(y_type=2),
               dict(opt=tg.make_options(b_col_major=1), ldw=31)):
        assert _adapted(lib, **kw) == INVALID, kw
    for o in BAD_OPTIONS:
        assert _adapted(lib, opt=tg.make_options(**o)) == INVALID, o
    assert _adapted(lib, groups=4097) == UNSUPPORTED and _adapted(lib, R=257, ldu=257) == UNSUPPORTED
    assert _adapted(lib, S=0) == OK and _adapted(lib, N=0) == OK and _adapted(lib, S=0, U=None, ldu=0, scales=None) == OK


def test_python_checks():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, 6, dtype=torch.bfloat16)
    for call in (lambda: tg.gemm_gated(x, w), lambda: tg.gemm_gated_grad(x, w, x), lambda: tg.gemm_adapted(x, w, w, w, w)):
        with pytest.raises(TypeError):  # not on the GPU
            call()
    with pytest.raises(ValueError):
        tg.gemm_gated(x, w, activation="tanh")
    with pytest.raises(ValueError):
        tg.gemm_gated_grad(x, w, x, activation="tanh")
