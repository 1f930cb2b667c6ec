"""Tokens sorted by expert and back on the GPU against the plain 64-bit forms:
sizes from one token to several sorting blocks, experts with no rows, dropped
and out-of-range ids, rows of every alignment and both types, strided
operands, the gradient (by its formula and by differences), CUDA graphs and
a second stream.

Tolerances: the order and the row copies are exact.  A combined value is a
sum of k products in fp32, each within one rounding of its term, so it lies
within (k + 1) 2^-24 of the sum of the terms' magnitudes, and a bf16 output
between the roundings of that interval's ends; a weight gradient is a sum of
D products in fp32 in some order, within (D + 1) 2^-24 of the magnitudes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import tiled_gemm_codegen_gb300 as tg
from expert_ref import U32, combine_grad_ref, combine_ref, gather_ref, order_ref, within
from gpu_helpers import dev

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tg.load()
    yield
    assert tg.device_error() == tg.TG_OK


def _ids(T, k, E, seed, drop=0.1, skew=False):
    g = np.random.default_rng(seed)
    ids = g.integers(0, E, (T, k))
    if skew:
        ids[g.random((T, k)) < 0.7] = E // 2
    ids[g.random((T, k)) < drop] = -1
    return ids


def _rows(rows, D, seed, dtype, pitch=None, offset=0):
    """A rows x D tensor with the given pitch, `offset` elements into its
    storage, around it NaN; and its values in 64 bits."""
    pitch = D if pitch is None else pitch
    g = torch.Generator().manual_seed(seed)
    vals = torch.randn(rows, D, generator=g).to(dtype)
    store = torch.full((offset + rows * pitch + 8,), float("nan"), dtype=dtype)
    view = store[offset:offset + rows * pitch].view(rows, pitch)[:, :D] if rows else store[:0].view(0, D)
    view.copy_(vals)
    d = store.to(dev())
    return d, (d[offset:offset + rows * pitch].view(rows, pitch)[:, :D] if rows else d[:0].view(0, D)), vals.double().numpy()


def _np(t):
    return t.detach().cpu().double().numpy()


SORT = [(0, 3, 5), (1, 1, 1), (1, 8, 64), (5, 2, 8), (31, 4, 7), (128, 8, 1024), (1024, 1, 3), (1025, 1, 1023),
        (700, 3, 17), (900, 5, 1024), (2048, 8, 60), (5461, 3, 100), (4096, 8, 60), (33333, 2, 256), (70000, 8, 128)]


@pytest.mark.parametrize("T,k,E", SORT)
@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
def test_sort(T, k, E, dtype):
    ids = _ids(T, k, E, 7 * T + k, skew=T % 2 == 1)
    if T > 3:
        ids[2, 0] = E          # out of range: dropped like -1
        ids[3, k - 1] = 2 ** 31 - 1
    order = tg.expert_sort(torch.from_numpy(ids).to(dtype).to(dev()), E)
    if T * k > 20000:  # the same by a stable argsort
        key = np.where((ids >= 0) & (ids < E), ids, E).reshape(-1)
        by = np.argsort(key, kind="stable")
        offsets = np.searchsorted(key[by], np.arange(E + 1))
        slot = np.full(T * k, -1)
        slot[by] = np.arange(T * k)
        slot = np.where(key < E, slot, -1).reshape(T, k)
        source = np.where(key[by] < E, by, -1)
    else:
        offsets, source, slot = order_ref(ids, E)
    assert np.array_equal(_np(order.offsets), offsets)
    assert np.array_equal(_np(order.source), source)
    assert np.array_equal(_np(order.slot), slot)


def test_sort_of_large_ids_and_strided_ids():
    ids = torch.full((6, 9), -5, dtype=torch.int64)
    ids[:, 2:5] = torch.tensor([[0, 1, 2], [2, 1, 0], [2 ** 40, 0, 1], [-2 ** 40, 2, 2], [1, 1, 1], [2 ** 32, 2 ** 32 + 1, 0]])
    view = ids.to(dev())[:, 2:5]
    order = tg.expert_sort(view, 3)
    offsets, source, slot = order_ref(ids[:, 2:5].numpy(), 3)
    assert np.array_equal(_np(order.offsets), offsets)
    assert np.array_equal(_np(order.source), source)
    assert np.array_equal(_np(order.slot), slot)


def test_every_assignment_dropped_and_one_expert_takes_all():
    for fill, E in ((-1, 4), (2, 4)):
        ids = torch.full((2000, 2), fill, dtype=torch.int32, device=dev())
        x = torch.randn(2000, 40, device=dev())
        xs, order = tg.expert_dispatch(x, ids, E)
        offsets, source, slot = order_ref(ids.cpu().numpy(), E)
        assert np.array_equal(_np(order.offsets), offsets)
        assert np.array_equal(_np(order.source), source)
        assert np.array_equal(_np(xs), gather_ref(_np(x), source, 2))


# rows: aligned multiples of 16 bytes, odd widths, pitches and offsets
ROWS = [(64, None, 0), (8, None, 0), (1, None, 0), (7, None, 0), (1001, None, 0), (1000, 1003, 1), (333, 340, 5),
        (16, 24, 8), (2056, None, 0), (129, 129, 3)]


@pytest.mark.parametrize("D,pitch,offset", ROWS)
@pytest.mark.parametrize("T,k,E", [(1, 8, 64), (37, 3, 9), (700, 2, 33), (9000, 2, 5)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_dispatch_and_gather(D, pitch, offset, T, k, E, dtype):
    ids = _ids(T, k, E, D + T)
    _, x, xv = _rows(T, D, 3, dtype, pitch, offset)
    store, xs, _ = _rows(T * k, D, 4, dtype, pitch, offset)
    got, order = tg.expert_dispatch(x, torch.from_numpy(ids).to(dev()), E, xs=xs)
    offsets, source, slot = order_ref(ids, E)
    assert np.array_equal(_np(order.offsets), offsets)
    assert np.array_equal(_np(order.slot), slot)
    want = gather_ref(xv, source, k)
    assert np.array_equal(_np(got), want)
    assert got is xs
    if pitch:  # what lies between the rows stays
        p = D if pitch is None else pitch
        body = store[offset:offset + T * k * p].view(T * k, p)
        assert bool(torch.isnan(body[:, D:]).all())
    assert bool(torch.isnan(store[:offset]).all()) and bool(torch.isnan(store[-8:]).all())
    xs2 = tg.expert_gather(x, order)
    assert np.array_equal(_np(xs2), want)


@pytest.mark.parametrize("D,pitch,offset", ROWS)
@pytest.mark.parametrize("T,k,E", [(1, 1, 2), (5, 2, 8), (67, 4, 9), (40, 11, 16)])
@pytest.mark.parametrize("dtypes", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(D, pitch, offset, T, k, E, dtypes, weighted):
    ids = _ids(T, k, E, D + T, drop=0.3)
    _, _, slot = order_ref(ids, E)
    order = tg.expert_sort(torch.from_numpy(ids).to(dev()), E)
    _, ys, ysv = _rows(T * k, D, 5, dtypes[0], pitch, offset)
    store, y, _ = _rows(T, D, 6, dtypes[1], pitch, offset)
    w = torch.rand(T, k + 3, device=dev())[:, 1:k + 1] if weighted else None
    tg.expert_combine(ys, order, w, y=y)
    want, mag = combine_ref(ysv, slot, _np(w) if weighted else None)
    assert within(y, want, (k + 1) * U32 * mag + 1e-38, dtypes[1])
    assert bool(torch.isnan(store[:offset]).all()) and bool(torch.isnan(store[-8:]).all())


def test_combine_ignores_what_dropped_assignments_hold():
    """Rows of no expert and weights of dropped assignments may hold NaN."""
    ids = torch.tensor([[0, -1], [-1, -1], [1, 0]], device=dev())
    order = tg.expert_sort(ids, 2)
    ys = torch.full((6, 16), float("nan"), device=dev())
    ys[:3] = torch.arange(48.0, device=dev()).view(3, 16)
    w = torch.tensor([[2.0, float("nan")], [float("nan"), float("inf")], [0.5, 1.0]], device=dev())
    y = tg.expert_combine(ys, order, w)
    assert torch.equal(y[0], 2 * ys[0])
    assert torch.equal(y[1], torch.zeros(16, device=dev()))
    assert torch.equal(y[2], 0.5 * ys[2] + ys[1])
    dys, dw = tg.expert_combine_grad(torch.ones(3, 16, device=dev()), ys, order, w)
    assert torch.equal(dys[3:], torch.zeros(3, 16, device=dev()))
    assert torch.equal(dw, torch.tensor([[ys[0].sum(), 0], [0, 0], [ys[2].sum(), ys[1].sum()]], device=dev()))


def test_slots_out_of_range_are_neither_read_nor_written():
    order = tg.ExpertOrder(torch.tensor([0, 4], dtype=torch.int32, device=dev()),
                           torch.arange(4, dtype=torch.int32, device=dev()),
                           torch.tensor([[0, 2 ** 31 - 1], [-7, 1]], dtype=torch.int32, device=dev()))
    ys = torch.ones(4, 24, device=dev())
    y = tg.expert_combine(ys, order)
    assert torch.equal(y, torch.ones(2, 24, device=dev()))
    dys = torch.full((4, 24), 7.0, device=dev())
    _, dw = tg.expert_combine_grad(torch.ones(2, 24, device=dev()), ys, order, None, dys=dys)
    assert torch.equal(dw, torch.tensor([[24.0, 0.0], [0.0, 24.0]], device=dev()))
    assert torch.equal(dys[:2], torch.ones(2, 24, device=dev())) and torch.equal(dys[2:], torch.full((2, 24), 7.0, device=dev()))


@pytest.mark.parametrize("D,pitch,offset", ROWS)
@pytest.mark.parametrize("T,k,E", [(1, 8, 64), (37, 3, 9), (20, 11, 16), (700, 2, 33)])
@pytest.mark.parametrize("dtypes", [(BF, BF, BF), (F32, F32, F32), (F32, BF, BF), (BF, F32, F32)])
def test_combine_grad(D, pitch, offset, T, k, E, dtypes):
    ids = _ids(T, k, E, D + T, drop=0.2)
    _, _, slot = order_ref(ids, E)
    order = tg.expert_sort(torch.from_numpy(ids).to(dev()), E)
    _, dy, dyv = _rows(T, D, 7, dtypes[0], pitch, offset)
    _, ys, ysv = _rows(T * k, D, 8, dtypes[1], pitch, offset)
    store, dys, _ = _rows(T * k, D, 9, dtypes[2], pitch, offset)
    w = torch.rand(T, k, device=dev())
    _, dw = tg.expert_combine_grad(dy, ys, order, w, dys=dys)
    want, want_w, mag = combine_grad_ref(dyv, ysv, slot, _np(w))
    assert within(dys, want, U32 * np.abs(want) + 1e-38, dtypes[2])
    assert np.all(np.abs(_np(dw) - want_w) <= (D + 1) * U32 * mag + 1e-38)
    assert bool(torch.isnan(store[:offset]).all()) and bool(torch.isnan(store[-8:]).all())


def test_gradient_against_differences():
    """The combine is linear in ys and in the weights, so a central
    difference of L = <c, y> along any direction equals <gradient, direction>
    up to rounding: (k + 1) 2^-24 of the magnitudes of y's terms at each end,
    summed over y and divided by the step (here 1)."""
    T, k, E, D = 50, 3, 7, 96
    ids = torch.from_numpy(_ids(T, k, E, 1)).to(dev())
    order = tg.expert_sort(ids, E)
    g = torch.Generator(device=dev()).manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev())  # noqa: E731
    ys, w, c, d_ys, d_w = rnd(T * k, D), rnd(T, k), rnd(T, D), rnd(T * k, D), rnd(T, k)
    dys, dw = tg.expert_combine_grad(c, ys, order, w)
    loss = lambda y: float((c.double() * y.double()).sum())  # noqa: E731
    slot = order.slot.cpu().numpy()
    for (up, down, want) in (
            ((ys + d_ys, w), (ys - d_ys, w), float((dys.double() * d_ys.double()).sum())),
            ((ys, w + d_w), (ys, w - d_w), float((dw.double() * d_w.double()).sum()))):
        got = (loss(tg.expert_combine(up[0], order, up[1])) - loss(tg.expert_combine(down[0], order, down[1]))) / 2
        mags = [combine_ref(np.abs(_np(a)), slot, np.abs(_np(b)))[0] for a, b in (up, down)]
        # rounding of both ends, of the perturbed operands and of the gradient itself
        bound = (k + D + 4) * U32 * float((np.abs(_np(c)) * (mags[0] + mags[1])).sum())
        assert abs(got - want) <= bound, (got, want, bound)


def test_gather_gradient_is_the_unweighted_combine():
    T, k, E, D = 33, 4, 6, 40
    ids = torch.from_numpy(_ids(T, k, E, 3, drop=0.2)).to(dev())
    x = torch.randint(-8, 9, (T, D), device=dev()).float()
    c = torch.randint(-8, 9, (T * k, D), device=dev()).float()
    xs, order = tg.expert_dispatch(x, ids, E)
    dx = tg.expert_combine(c, order)
    # integers: <c, gather(x)> = <dx, x> exactly
    assert float((c * xs).sum()) == float((dx * x).sum())


def test_graph_capture_and_streams():
    T, k, E, D = 9000, 2, 16, 128
    for tokens in (T, 3000, 40):  # three sorting launches; one; one with the copy
        x = torch.randn(tokens, D, device=dev()).to(BF)
        ids = torch.randint(0, E, (tokens, k), device=dev())
        w = torch.rand(tokens, k, device=dev())
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        order = tg.ExpertOrder.empty(tokens, k, E)
        xs = torch.empty(tokens * k, D, dtype=BF, device=dev())
        y = torch.empty(tokens, D, dtype=BF, device=dev())
        with torch.cuda.stream(s):
            tg.expert_dispatch(x, ids, E, xs=xs, order=order)  # sizes the stream's workspace
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            tg.expert_dispatch(x, ids, E, xs=xs, order=order)
            tg.expert_combine(xs, order, w, y=y)
        for seed in range(3):
            ids.copy_(torch.randint(0, E, (tokens, k), device=dev()))
            x.copy_(torch.randn(tokens, D, device=dev()))
            graph.replay()
            torch.cuda.synchronize()
            _, source, _ = order_ref(ids.cpu().numpy(), E)
            assert np.array_equal(_np(order.source), source)
            assert np.array_equal(_np(xs), gather_ref(_np(x), source, k))
            want = _np(x) * _np(w.sum(1, keepdim=True))
            assert within(y, want, 8 * U32 * np.abs(want) + 1e-30, BF)


def test_repeated_calls_give_the_same_bits():
    T, k, E, D = 5000, 4, 32, 264
    ids = torch.from_numpy(_ids(T, k, E, 5)).to(dev())
    x = torch.randn(T, D, device=dev()).to(BF)
    w = torch.rand(T, k, device=dev())
    first = None
    for _ in range(3):
        xs, order = tg.expert_dispatch(x, ids, E)
        y = tg.expert_combine(xs, order, w)
        dys, dw = tg.expert_combine_grad(y, xs, order, w)
        now = (xs, *order, y, dys, dw)
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def test_rows_past_two_billion_elements():
    """Offsets of rows beyond 32 bits: the last tokens and slots of a batch
    whose sorted rows hold 2.3 x 10^9 elements, aligned and not."""
    T, k, E = 140000, 2, 3
    ids = torch.randint(0, E, (T, k), device=dev())
    w = torch.rand(T, k, device=dev())
    for D in (8192, 8193):
        x = torch.zeros(T, D, dtype=BF, device=dev())
        x[:, -16:] = torch.arange(T, device=dev())[:, None] % 251
        xs, order = tg.expert_dispatch(x, ids, E)
        s = torch.arange(T * k - 500, T * k, device=dev())
        src = order.source[s].long()
        assert torch.equal(xs[s], x[src // k])
        y = tg.expert_combine(xs, order, w)
        t = torch.arange(T - 500, T, device=dev())
        want = _np(x[t]) * _np(w[t].sum(1, keepdim=True))
        assert within(y[t], want, 4 * U32 * np.abs(want) + 1e-30, BF)
        del y
        dys, dw = tg.expert_combine_grad(x, xs, order, w)
        assert within(dys[s], _np(x[src // k]) * _np(w.reshape(-1)[src])[:, None], U32 * 300, BF)
        assert torch.equal(dw[t, 0], (x[t].float() ** 2).sum(1))
        del dys, xs, x


@pytest.mark.parametrize("T,k,E", [(1300001, 2, 33), (2 ** 21, 2, 1024)])
def test_sort_of_millions_of_ids(T, k, E):
    """More ids than the largest number of blocks places in one turn each."""
    ids = torch.randint(-1, E + 1, (T, k), generator=torch.Generator().manual_seed(T)).to(dev())
    order = tg.expert_sort(ids, E)
    key = torch.where((ids >= 0) & (ids < E), ids, E).flatten()
    by = torch.argsort(key, stable=True)
    kept = int((key < E).sum())
    assert torch.equal(order.offsets, torch.searchsorted(key[by], torch.arange(E + 1, device=dev())).int())
    assert torch.equal(order.source[:kept], by[:kept].int()) and bool((order.source[kept:] == -1).all())
    slot = torch.full((T * k,), -1, dtype=torch.int32, device=dev())
    slot[by[:kept]] = torch.arange(kept, dtype=torch.int32, device=dev())
    assert torch.equal(order.slot.flatten(), slot)
