"""The grouped GEMM on the GPU: ragged rows (forward and data gradient) and
ragged contraction (weight gradient) against 64-bit products, over group
sizes from none to several tiles, every tile choice, odd extents and pitches
(the realign pass), the fused epilogue, rows of no group, non-finite values
in other groups' rows, and bounds that are not what they should be.

Integer inputs make every partial sum exact, so those results are compared
bit for bit; random ones within the contract of the library's GEMM
(gpu_helpers), and bf16 outputs within one rounding of that."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import tiled_gemm_codegen_gb300 as tg
from expert_ref import within
from gpu_helpers import PER_ELEM, assert_close, dev

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SIZES = {
    "one": [1],
    "mixed": [0, 3, 129, 64, 0, 1, 300, 0],
    "tiles": [128, 256, 512, 64],
    "empty": [0, 0, 0],
    "many": [i % 5 for i in range(70)],
    "long": [700, 5, 1000],
}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tg.load()
    yield
    assert tg.device_error() == tg.TG_OK


def _offsets(sizes, lead=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]) + lead, dtype=torch.int32, device=dev())


def _rand(shape, seed, ints, pitch=None):
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(-3, 4, shape, generator=g).float() if ints else torch.randn(*shape, generator=g)
    v = v.to(BF)
    if pitch:
        store = torch.full((*shape[:-1], pitch), float("nan"), dtype=BF)
        store[..., :shape[-1]] = v
        return store.to(dev())[..., :shape[-1]], v.double().numpy()
    return v.to(dev()), v.double().numpy()


def _rows_ref(A, B, sizes, lead, S):
    D = np.zeros((S, B.shape[2]))
    at = lead
    for g, n in enumerate(sizes):
        D[at:at + n] = A[at:at + n] @ B[g]
        at += n
    return D


def _wgrad_ref(A, B, sizes, lead):
    out, at = [], lead
    for n in sizes:
        out.append(A[at:at + n].T @ B[at:at + n])
        at += n
    return np.stack(out)


def _np(t):
    return t.detach().cpu().double().numpy()


SHAPES = [(64, 128), (72, 136), (1, 1), (200, 333), (640, 512), (65, 257)]


@pytest.mark.parametrize("name", list(SIZES))
@pytest.mark.parametrize("K,N", SHAPES)
@pytest.mark.parametrize("pair", [0, 1, 2])
@pytest.mark.parametrize("transposed", [False, True])
def test_rows_exact(name, K, N, pair, transposed):
    sizes = SIZES[name]
    S = sum(sizes)
    A, av = _rand((S, K), 1, True)
    B, bv = _rand((len(sizes), N, K) if transposed else (len(sizes), K, N), 2, True)
    if transposed:
        B, bv = B.transpose(1, 2), bv.transpose(0, 2, 1)
    opts = tg.make_options(cta_pair=pair)
    D = tg.gemm_grouped(A, B, _offsets(sizes), options=opts)
    assert np.array_equal(_np(D), _rows_ref(av, bv, sizes, 0, S))


@pytest.mark.parametrize("name", list(SIZES))
@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("pair", [0, 1, 2])
def test_wgrad_exact(name, M, N, pair):
    sizes = SIZES[name]
    S = sum(sizes)
    A, av = _rand((S, M), 3, True)
    B, bv = _rand((S, N), 4, True)
    D = tg.gemm_grouped_wgrad(A, B, _offsets(sizes), options=tg.make_options(cta_pair=pair))
    assert np.array_equal(_np(D), _wgrad_ref(av, bv, sizes, 0))


@pytest.mark.parametrize("pitches", [(None, None, 0), (80, 144, 8), (75, 141, 3), (65, 129, 1)])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("pair", [1, 2])
def test_pitches_rows_of_no_group_and_guard_bands(pitches, dtype, pair):
    pa, pb, pd = pitches
    K, N, sizes, lead, S = 65, 129, [40, 0, 150, 7], 11, 230
    A, av = _rand((S, K), 5, True, pa)
    B, bv = _rand((4, K, N), 6, True, pb)
    store = torch.full((S + 2, N + pd), float("nan"), dtype=dtype, device=dev())
    D = store[1:-1, :N]
    tg.gemm_grouped(A, B, _offsets(sizes, lead), D, options=tg.make_options(cta_pair=pair))
    want = torch.from_numpy(_rows_ref(av, bv, sizes, lead, S)).to(dtype).double().numpy()
    assert np.array_equal(_np(D), want)
    assert bool(torch.isnan(store[0]).all()) and bool(torch.isnan(store[-1]).all()) and bool(torch.isnan(store[:, N:]).all())
    X, xv = _rand((S, K), 7, True, pa)
    Y, yv = _rand((S, N), 8, True, pb)
    store = torch.full((6, K + 1, N + pd), float("nan"), dtype=dtype, device=dev())
    W = store[1:-1, :K, :N]
    tg.gemm_grouped_wgrad(X, Y, _offsets(sizes, lead), W, options=tg.make_options(cta_pair=pair))
    want = torch.from_numpy(_wgrad_ref(xv, yv, sizes, lead)).to(dtype).double().numpy()
    assert np.array_equal(_np(W), want)
    store[1:-1, :K, :N] = float("nan")
    assert bool(torch.isnan(store).all())


@pytest.mark.parametrize("pair", [1, 2])
def test_non_finite_rows_stay_in_their_group(pair):
    """Groups that end inside a k-block or tile next to rows of NaN and
    infinities: the others' results are exact, theirs as the formula's."""
    sizes, K, N = [70, 60, 130, 1, 255], 96, 160
    S = sum(sizes)
    A, av = _rand((S, K), 9, True)
    Y, yv = _rand((S, N), 10, True)
    W, wv = _rand((5, K, N), 11, True)
    bad = slice(70, 130)  # group 1
    A[bad] = float("nan")
    Y[bad] = float("inf")
    A[260] = float("inf")  # group 3, its only row
    off = _offsets(sizes)
    opts = tg.make_options(cta_pair=pair)
    D = _np(tg.gemm_grouped(A, W, off, options=opts))
    G = _np(tg.gemm_grouped_wgrad(A, Y, off, options=opts))
    want_d, want_g = _rows_ref(av, wv, sizes, 0, S), _wgrad_ref(av, yv, sizes, 0)
    good = np.ones(S, bool)
    good[70:130] = good[260] = False
    assert np.array_equal(D[good], want_d[good])
    assert np.isnan(D[70:130]).all()
    for g in (0, 2, 4):
        assert np.array_equal(G[g], want_g[g])
    assert np.isnan(G[1]).all()
    assert not np.isfinite(G[3]).any()


# Few tiles and a long contraction: the tiles are shared between workers
SHARED = [([5000], 130, 70), ([3000, 0, 17, 2500], 64, 128), ([1, 6000], 300, 260), ([64 * 9 - 1], 40, 40)]


@pytest.mark.parametrize("sizes,M,N", SHARED)
@pytest.mark.parametrize("pair", [0, 1, 2])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_shared_tiles_of_wgrad(sizes, M, N, pair, dtype):
    S = sum(sizes)
    A, av = _rand((S, M), 30, True)
    B, bv = _rand((S, N), 31, True)
    off, opts = _offsets(sizes), tg.make_options(cta_pair=pair)
    want = torch.from_numpy(_wgrad_ref(av, bv, sizes, 0)).to(dtype).double().numpy()
    for _ in range(2):  # the arrival counters are left ready for the next call
        assert np.array_equal(_np(tg.gemm_grouped_wgrad(A, B, off, out_dtype=dtype, options=opts)), want)


@pytest.mark.parametrize("sizes", [[1], [3, 0, 2], [0, 40], [130]])
@pytest.mark.parametrize("K,N", [(4096, 64), (5000, 200), (1100, 129)])
@pytest.mark.parametrize("pair", [0, 1, 2])
def test_shared_tiles_of_rows(sizes, K, N, pair):
    S = sum(sizes)
    A, av = _rand((S, K), 32, True)
    B, bv = _rand((len(sizes), K, N), 33, True)
    bias = torch.randint(-4, 5, (len(sizes), N), device=dev()).float()
    want = np.maximum(_rows_ref(av, bv, sizes, 0, S) + np.repeat(_np(bias), sizes, axis=0), 0)
    for _ in range(2):
        D = tg.gemm_grouped(A, B, _offsets(sizes), bias=bias, activation="relu", options=tg.make_options(cta_pair=pair))
        assert np.array_equal(_np(D), want)


RANDOM = [([0, 300, 17, 1000, 256], 1024, 640), ([2000, 96], 512, 1408), ([2] * 40 + [0] * 9, 2048, 200)]


@pytest.mark.parametrize("sizes,K,N", RANDOM)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_random_values(sizes, K, N, dtype):
    S, off = sum(sizes), _offsets(sizes)
    A, av = _rand((S, K), 12, False)
    B, bv = _rand((len(sizes), K, N), 13, False)
    C, cv = _rand((S, N), 14, False)
    for got, want, depth in (
            (tg.gemm_grouped(A, B, off, out_dtype=dtype), _rows_ref(av, bv, sizes, 0, S), K),
            (tg.gemm_grouped(C, B.transpose(1, 2), off, out_dtype=dtype), _rows_ref(cv, bv.transpose(0, 2, 1), sizes, 0, S), N),
            (tg.gemm_grouped_wgrad(A, C, off, out_dtype=dtype), _wgrad_ref(av, cv, sizes, 0), max(sizes))):
        assert got.dtype == dtype
        if dtype == F32:
            assert_close(_np(got), want, depth)
        else:
            assert within(got, want, PER_ELEM * np.sqrt(depth) * np.abs(want).max(), dtype)


@pytest.mark.parametrize("size", [200, 33, 95])
@pytest.mark.parametrize("N", [384, 392, 700])
@pytest.mark.parametrize("pair", [1, 2])
def test_bf16_boxes_stored_plainly_between_boxes_stored_by_tma(size, N, pair):
    """A group's last rows, and a box cut off by the row's end, leave their
    staging box by plain stores, the others by asynchronous ones that may
    still read theirs: short products over many groups, several tiles a
    worker, every element of every call."""
    groups, K = 160, 64
    S, off = groups * size, _offsets([size] * groups)
    A, _ = _rand((S, K), 60, True)
    B, _ = _rand((groups, K, N), 61, True)
    want = torch.bmm(A.float().view(groups, size, K), B.float()).view(S, N).to(BF)  # integers: exact before the rounding
    opts, D = tg.make_options(cta_pair=pair), torch.empty(S, N, dtype=BF, device=dev())
    wrong = torch.zeros((), dtype=torch.int64, device=dev())
    for _ in range(200):
        D.fill_(float("nan"))
        tg.gemm_grouped(A, B, off, D, options=opts)
        wrong += (D != want).sum()
    assert int(wrong) == 0


@pytest.mark.parametrize("activation", ["none", "relu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("per_group", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_epilogue(activation, per_group, dtype):
    """act(alpha A B + bias) against the same formula in 64 bits; the extra
    error is a few fp32 roundings of values below 64 and the activation
    function's own (tanh, exp: a few units)."""
    sizes, K, N = [33, 0, 200], 136, 200
    S = sum(sizes)
    A, av = _rand((S, K), 15, False)
    B, bv = _rand((3, K, N), 16, False)
    bias = torch.randn(3, N + 5, device=dev())[:, :N] if per_group else torch.randn(N, device=dev())
    D = tg.gemm_grouped(A, B, _offsets(sizes), alpha=0.125, bias=bias, activation=activation, out_dtype=dtype)
    z = 0.125 * _rows_ref(av, bv, sizes, 0, S) + np.repeat(_np(bias) if per_group else np.tile(_np(bias), (3, 1)), sizes, axis=0)
    want = {"none": lambda v: v, "relu": lambda v: np.maximum(v, 0), "silu": lambda v: v / (1 + np.exp(-v)),
            "gelu_tanh": lambda v: 0.5 * v * (1 + np.tanh(np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)))}[activation](z)
    bound = 2 * (PER_ELEM * np.sqrt(K) * 0.125 * np.abs(z).max() + 16 * 2.0 ** -24 * (1 + np.abs(z)))
    assert within(D, want, bound, dtype)


def test_no_terms_and_no_rows():
    off = _offsets([3, 2])
    bias = torch.randn(2, 24, device=dev())
    D = tg.gemm_grouped(torch.empty(7, 0, dtype=BF, device=dev()), torch.empty(2, 0, 24, dtype=BF, device=dev()), off, bias=bias)
    want = torch.cat((bias[:1].expand(3, 24), bias[1:].expand(2, 24), torch.zeros(2, 24, device=dev())))
    assert torch.equal(D, want)
    W = tg.gemm_grouped_wgrad(torch.empty(0, 40, dtype=BF, device=dev()), torch.empty(0, 24, dtype=BF, device=dev()), off)
    assert torch.equal(W, torch.zeros(2, 40, 24, device=dev()))
    assert tg.gemm_grouped(torch.empty(0, 8, dtype=BF, device=dev()), torch.empty(2, 8, 24, dtype=BF, device=dev()), off).shape == (0, 24)


def test_bounds_outside_the_rows_are_clamped():
    """Bounds past the rows, negative or falling: nothing out of range is
    touched, and groups whose bounds are sound keep their values."""
    S, K, N = 100, 64, 64
    A, av = _rand((S, K), 17, True)
    B, bv = _rand((3, K, N), 18, True)
    store = torch.full((S + 2, N), float("nan"), device=dev())
    D = store[1:-1]
    for bounds in ([0, 30, 2 ** 31 - 1, 2 ** 31 - 1], [-5, 30, 100, 400], [0, 30, 100, -2 ** 31]):
        off = torch.tensor(bounds, dtype=torch.int32, device=dev())
        tg.gemm_grouped(A, B, off, D)
        assert np.array_equal(_np(D), _rows_ref(av, bv, [30, 70], 0, S))
        assert bool(torch.isnan(store[0]).all()) and bool(torch.isnan(store[-1]).all())
        W = tg.gemm_grouped_wgrad(A, A, off)
        assert np.array_equal(_np(W)[:2], _wgrad_ref(av, av, [30, 70], 0))


def test_one_matrix_for_every_group():
    sizes, K, N = [5, 90], 72, 80
    A, av = _rand((95, K), 19, True)
    B, bv = _rand((1, K, N), 20, True)
    D = tg.gemm_grouped(A, B.expand(2, K, N), _offsets(sizes))
    assert np.array_equal(_np(D), av @ bv[0])


def test_gradients_against_differences():
    """<c, D> is linear in A and in B: its central difference along a
    direction of integers is exact in fp32, as is the gradient's product."""
    sizes, K, N = [13, 0, 70], 40, 56
    S, off = sum(sizes), _offsets(sizes)
    A, _ = _rand((S, K), 21, True)
    B, _ = _rand((3, K, N), 22, True)
    C, _ = _rand((S, N), 23, True)
    dA, _ = _rand((S, K), 24, True)
    dB, _ = _rand((3, K, N), 25, True)
    loss = lambda a, b: float((C.double() * tg.gemm_grouped(a, b, off).double()).sum())  # noqa: E731
    grad_a = tg.gemm_grouped(C, B.transpose(1, 2), off)
    grad_b = tg.gemm_grouped_wgrad(A, C, off)
    assert (loss(A + dA, B) - loss(A - dA, B)) / 2 == float((grad_a.double() * dA.double()).sum())
    assert (loss(A, B + dB) - loss(A, B - dB)) / 2 == float((grad_b.double() * dB.double()).sum())


def test_same_bits_again_graph_and_stream():
    sizes, K, N = [300, 0, 45, 700], 256, 384
    S, off = sum(sizes), _offsets(sizes)
    A, _ = _rand((S, K), 26, False)
    B, _ = _rand((4, K, N), 27, False)
    s = torch.cuda.Stream()
    first = tg.gemm_grouped(A, B, off)
    first_w = tg.gemm_grouped_wgrad(A, A, off)
    s.wait_stream(torch.cuda.current_stream())
    D, W = torch.empty_like(first), torch.empty_like(first_w)
    with torch.cuda.stream(s):
        tg.gemm_grouped(A, B, off, D)
        tg.gemm_grouped_wgrad(A, A, off, W)
    s.synchronize()
    assert torch.equal(D, first) and torch.equal(W, first_w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        tg.gemm_grouped(A, B, off, D)
        tg.gemm_grouped_wgrad(A, A, off, W)
    for moved in ([300, 0, 45, 700], [0, 1045, 0, 0], [1, 2, 3, 4]):
        off.copy_(_offsets(moved))  # the bounds are read at each replay
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(D, tg.gemm_grouped(A, B, _offsets(moved)))
        assert torch.equal(W, tg.gemm_grouped_wgrad(A, A, _offsets(moved)))


@pytest.mark.parametrize("wgrad", [False, True])
@pytest.mark.parametrize("pair", [1, 2])
@pytest.mark.parametrize("sizes", [[300, 5, 170], [6000]])  # whole tiles; shared ones
def test_watchdog(wgrad, pair, sizes):
    """A wait that nothing ends runs out after its limit, is reported by
    tg_device_error, and leaves the device and the next call's counters sound."""
    S, K, N = sum(sizes), 128, 192
    A, av = _rand((S, K), 40, True)
    B, bv = _rand((S, N) if wgrad else (len(sizes), K, N), 41, True)
    off = _offsets(sizes)
    call = tg.gemm_grouped_wgrad if wgrad else tg.gemm_grouped
    call(A, B, off, options=tg.make_options(cta_pair=pair, debug_stall=1, timeout_ns=20_000_000))
    assert tg.device_error() == tg.TG_ERR_TIMEOUT
    assert tg.device_error() == tg.TG_OK
    got = call(A, B, off, options=tg.make_options(cta_pair=pair))
    assert tg.device_error() == tg.TG_OK
    assert np.array_equal(_np(got), _wgrad_ref(av, bv, sizes, 0) if wgrad else _rows_ref(av, bv, sizes, 0, S))


def test_checks_build_gives_the_same_bits():
    """The library built with device-side checks: the same results, and no
    check fails."""
    import ctypes

    lib = tg.load_checks()
    sizes, K, N = [300, 0, 45, 700], 200, 264
    S, off = sum(sizes), _offsets(sizes)
    A, _ = _rand((S, K), 42, False)
    B, _ = _rand((4, K, N), 43, False)
    D, W = tg.gemm_grouped(A, B, off), tg.gemm_grouped_wgrad(A, A, off)
    D2, W2 = torch.empty_like(D), torch.empty_like(W)
    ep = tg.tg_epilogue()
    ep.alpha = 1.0
    s = torch.cuda.current_stream().cuda_stream
    assert lib.tg_gemm_grouped(A.data_ptr(), B.data_ptr(), D2.data_ptr(), off.data_ptr(), 4, S, N, K, K, N, K * N, N,
                               ctypes.byref(ep), s, None) == tg.TG_OK
    assert lib.tg_gemm_grouped_wgrad(A.data_ptr(), A.data_ptr(), W2.data_ptr(), off.data_ptr(), 4, S, K, K, K, K, K, K * K,
                                     ctypes.byref(ep), s, None) == tg.TG_OK
    assert lib.tg_device_error(s) == tg.TG_OK
    assert torch.equal(D, D2) and torch.equal(W, W2)


def test_rows_past_two_billion_elements():
    """A and D of more than 2^31 elements: the last group's rows, and the
    weight gradient of rows that lie behind them all."""
    S, K = 270000, 8192
    A = torch.zeros(S, K, dtype=BF, device=dev())
    tail, tv = _rand((700, K), 50, True)
    A[-700:] = tail
    B, bv = _rand((2, K, 24), 51, True)
    off = torch.tensor([0, S - 700, S], dtype=torch.int32, device=dev())
    D = tg.gemm_grouped(A, B, off)
    assert np.array_equal(_np(D[-700:]), tv @ bv[1])
    assert not bool(D[:-700].any())
    W = tg.gemm_grouped_wgrad(A, A[:, :40], off)
    assert np.array_equal(_np(W[1]), tv.T @ tv[:, :40])
    assert not bool(W[0].any())
    del D, W
    X, xv = _rand((300, 32), 52, True)
    x = torch.zeros(S, 32, dtype=BF, device=dev())
    x[-300:] = X
    V, vv = _rand((1, 32, K), 53, True)
    out = tg.gemm_grouped(x, V, torch.tensor([0, S], dtype=torch.int32, device=dev()), out_dtype=BF)
    assert np.array_equal(_np(out[-300:]), torch.from_numpy(xv @ vv[0]).to(BF).double().numpy())
