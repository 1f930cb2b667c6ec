"""Products with 4-bit weights on the GPU against 64-bit products of the values
the codes stand for: both formats, every group size, zero points, one to
many rows, groups with and without rows, odd and misaligned extents.

A code's value times an activation is exact in fp32 (5 and 8 bits), so a
group's sum and the sum over groups round at most once for each of the K
additions and once for each scale's product: |error| <= (K + runs + 2) 2^-24
times the sum of the magnitudes (any order of summation).  The hardware's
product of a 16-wide k step rounds its intermediate sum toward zero, a factor
of two on that step: 2 (K + runs + 2) 2^-24 covers both.  bf16 outputs lie
within one rounding of that."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import tiled_gemm_codegen_gb300 as tg
from expert_ref import U32, within
from gpu_helpers import dev

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tg.load()
    yield
    assert tg.device_error() == tg.TG_OK


def _weights(groups, N, K, fmt, G, seed, zeros=False, pitch=0):
    """(W, scales, zeros) on the GPU and the values [groups, N, K] in 64 bits."""
    g = np.random.default_rng(seed)
    runs = -(-K // G)
    W = torch.from_numpy(g.integers(0, 256, (groups, N, K // 2 + pitch), dtype=np.uint8)).to(dev())[..., :K // 2]
    w = W.cpu().numpy()
    q = np.stack((w & 15, w >> 4), -1).reshape(groups, N, K)
    z = None
    if fmt == "e2m1":
        sc = torch.from_numpy(g.integers(118, 131, (groups, N, runs + pitch), dtype=np.uint8)).to(dev())[..., :runs]
        v, s = E2M1[q], np.exp2(sc.cpu().double().numpy() - 127)
    else:
        sc = torch.from_numpy(g.random((groups, N, runs + pitch)) * 0.1 + 0.01).to(BF).to(dev())[..., :runs]
        s = sc.cpu().double().numpy()
        if zeros:
            z = torch.from_numpy(g.integers(0, 16, (groups, N, runs + pitch), dtype=np.uint8)).to(dev())[..., :runs]
            v = q - np.repeat(z.cpu().numpy().astype(np.int64), G, -1)[..., :K]
        else:
            v = q - 8.0
    return W, sc, z, v * np.repeat(s, G, -1)[..., :K]


def _x(S, K, seed, pitch=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(S, K + pitch, generator=g).to(BF)
    return x.to(dev())[:, :K], x[:, :K].double().numpy()


def _check(y, xv, wv, offsets, K, G, dtype):
    S, N = y.shape
    want, mag = np.zeros((S, N)), np.zeros((S, N))
    for g in range(len(offsets) - 1):
        r = slice(offsets[g], offsets[g + 1])
        want[r] = xv[r] @ wv[g].T
        mag[r] = np.abs(xv[r]) @ np.abs(wv[g]).T
    assert within(y, want, 2 * (K + -(-K // G) + 2) * U32 * mag, dtype)


def _check_wide(y, xv, wv, K, G):
    """The same near fp32's largest value: where the magnitudes add up to more
    than it, some orders of summation overflow."""
    y, want, mag = y.cpu().double().numpy(), xv @ wv[0].T, np.abs(xv) @ np.abs(wv[0]).T
    top = torch.finfo(F32).max
    assert np.all(~np.isfinite(y[np.abs(want) > top * (1 + U32)]))
    with np.errstate(invalid="ignore"):
        near = np.abs(y - want) <= 2 * (K + -(-K // G) + 2) * U32 * mag
    assert np.all(near | (~np.isfinite(y) & (mag > top)))


FORMATS = [("int4", 32, False), ("int4", 64, True), ("int4", 128, False), ("int4", 128, True), ("int4", 32, True),
           ("e2m1", 32, False)]


@pytest.mark.parametrize("fmt,G,zeros", FORMATS)
@pytest.mark.parametrize("K,N", [(2, 1), (32, 16), (128, 130), (256, 32), (1000, 40), (1024, 33), (2050, 70), (5000, 17), (8192, 48)])
@pytest.mark.parametrize("S", [1, 3, 8, 21])
def test_dense(fmt, G, zeros, K, N, S):
    W, sc, z, wv = _weights(1, N, K, fmt, G, K + N, zeros)
    x, xv = _x(S, K, S)
    dtype = BF if S % 2 else F32
    y = tg.gemv_w4(x, W[0], sc[0], zeros=z[0] if z is not None else None, format=fmt, group=G, out_dtype=dtype)
    assert y.dtype == dtype
    _check(y, xv, wv, [0, S], K, G, dtype)


@pytest.mark.parametrize("fmt,G,zeros", FORMATS)
@pytest.mark.parametrize("sizes", [[1], [0, 1, 0, 2], [9, 0, 0, 1, 17], [0] * 33 + [1] * 5 + [0] * 40 + [2], [0, 0]])
@pytest.mark.parametrize("K,N", [(256, 72), (1100, 50)])
def test_groups(fmt, G, zeros, sizes, K, N):
    groups, tail, lead = len(sizes), 2, 1
    W, sc, z, wv = _weights(groups, N, K, fmt, G, 5 * groups, zeros)
    offsets = np.concatenate([[0], np.cumsum(sizes)]) + lead
    S = int(offsets[-1]) + tail
    x, xv = _x(S, K, 3)
    off = torch.from_numpy(offsets).int().to(dev())
    y = torch.full((S, N), float("nan"), device=dev())
    tg.gemv_w4(x, W, sc, zeros=z, offsets=off, y=y, format=fmt, group=G)
    _check(y, xv, wv, offsets, K, G, F32)


@pytest.mark.parametrize("fmt,G,zeros", FORMATS)
@pytest.mark.parametrize("pitch", [16, 4, 1])
def test_pitches_and_guard_bands(fmt, G, zeros, pitch):
    K, N, S = 480, 40, 5
    W, sc, z, wv = _weights(2, N, K, fmt, G, pitch, zeros, pitch)
    x, xv = _x(S, K, 4, pitch)
    store = torch.full((S + 2, N + pitch), float("nan"), device=dev())
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device=dev())
    y = store[1:-1, :N]
    tg.gemv_w4(x, W, sc, zeros=z, offsets=off, y=y, format=fmt, group=G)
    _check(y, xv, wv, [0, 2, 5], K, G, F32)
    y.fill_(float("nan"))
    assert bool(torch.isnan(store).all())


@pytest.mark.parametrize("skip", [1, 2, 8])
def test_operands_off_their_alignment(skip):
    """Bases that are not 16-byte aligned."""
    K, N, S = 512, 24, 2
    W0, sc0, _, wv = _weights(1, N, K, "int4", 64, 9)
    W = torch.empty(W0.numel() + 32, dtype=torch.uint8, device=dev())[skip:skip + W0.numel()].view(W0.shape[1:])
    W.copy_(W0[0])
    sc = torch.empty(sc0.numel() + 32, dtype=BF, device=dev())[skip:skip + sc0.numel()].view(sc0.shape[1:])
    sc.copy_(sc0[0])
    x0, xv = _x(S, K, 5)
    x = torch.empty(S * K + 32, dtype=BF, device=dev())[skip:skip + S * K].view(S, K)
    x.copy_(x0)
    _check(tg.gemv_w4(x, W, sc, group=64), xv, wv, [0, S], K, 64, F32)


def test_special_scales_and_activations():
    """A NaN scale (E8M0 255) and infinite activations reach the outputs they
    belong to and no others; the smallest scale is 2^-127."""
    K, N = 96, 40
    W, sc, _, wv = _weights(1, N, K, "e2m1", 32, 11)
    W[0, 3] = 0x22  # every code 1
    sc[0, 3] = 0
    sc[0, 5, 1] = 255
    x, xv = _x(3, K, 6)
    x[1].fill_(1.0)
    x[2, 40] = float("inf")
    W[0, 7, 20] = 0x21  # w[7, 40] = 0.5: the infinity stays one
    y = tg.gemv_w4(x, W[0], sc[0], format="e2m1")
    yn = y.cpu().double().numpy()
    assert np.isnan(yn[:, 5]).all()
    good = [n for n in range(N) if n not in (3, 5)]
    want = xv[0] @ wv[0].T
    mag = np.abs(xv[0]) @ np.abs(wv[0]).T
    assert np.all(np.abs(yn[0] - want)[[n for n in good if n != 7]] <= (2 * 105 * U32 * mag)[[n for n in good if n != 7]])
    assert yn[1, 3] == 96 * 2.0 ** -127
    assert np.isinf(yn[2, 7])
    assert not np.isfinite(yn[2]).any()  # an infinity times a zero code is NaN, else infinite


def test_no_terms_and_no_rows():
    y = tg.gemv_w4(torch.empty(3, 0, dtype=BF, device=dev()), torch.empty(5, 0, dtype=torch.uint8, device=dev()),
                   torch.empty(5, 0, dtype=BF, device=dev()))
    assert torch.equal(y, torch.zeros(3, 5, device=dev()))
    W, sc, _, _ = _weights(1, 8, 64, "int4", 64, 1)
    assert tg.gemv_w4(torch.empty(0, 64, dtype=BF, device=dev()), W[0], sc[0], group=64).shape == (0, 8)


def test_bounds_are_clamped():
    K, N, S = 128, 24, 6
    W, sc, _, wv = _weights(2, N, K, "int4", 128, 2)
    x, xv = _x(S, K, 7)
    for bounds in ([0, 2, 2 ** 31 - 1], [-9, 2, 6]):
        off = torch.tensor(bounds, dtype=torch.int32, device=dev())
        _check(tg.gemv_w4(x, W, sc, offsets=off), xv, wv, [0, 2, 6], K, 128, F32)


def test_same_weights_as_the_block_scaled_gemm():
    """gemv_w4 reads the very operands of gemm_mxfp4: activations that E2M1
    holds exactly give equal products from both."""
    K, N, S = 512, 128, 4
    W, sc, _, _ = _weights(1, N, K, "e2m1", 32, 13)
    sc.fill_(127)
    a = torch.randint(0, 256, (S, K // 2), dtype=torch.uint8, device=dev())
    an = a.cpu().numpy()
    x = torch.from_numpy(E2M1[np.stack((an & 15, an >> 4), -1).reshape(S, K)]).to(BF).to(dev())
    ones = torch.full((S, K // 32), 127, dtype=torch.uint8, device=dev())
    assert torch.equal(tg.gemv_w4(x, W[0], sc[0], format="e2m1"), tg.gemm_mxfp4(a, W[0], ones, sc[0]))


def test_same_bits_again_graph_and_stream():
    K, N, groups = 1024, 200, 6
    W, sc, z, _ = _weights(groups, N, K, "int4", 64, 17, True)
    x, _ = _x(9, K, 8)
    off = torch.tensor([0, 1, 1, 4, 4, 9, 9], dtype=torch.int32, device=dev())
    first = tg.gemv_w4(x, W, sc, zeros=z, offsets=off, group=64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(first)
    with torch.cuda.stream(s):
        tg.gemv_w4(x, W, sc, zeros=z, offsets=off, group=64, y=y)
    s.synchronize()
    assert torch.equal(y, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        tg.gemv_w4(x, W, sc, zeros=z, offsets=off, group=64, y=y)
    off.copy_(torch.tensor([0, 0, 3, 3, 7, 7, 8], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, tg.gemv_w4(x, W, sc, zeros=z, offsets=off, group=64))


@pytest.mark.parametrize("fmt,G,zeros", FORMATS)
@pytest.mark.parametrize("S", [5, 9])
def test_activations_that_do_not_fit_shared_memory(fmt, G, zeros, S):
    K, N = 16640, 40
    W, sc, z, wv = _weights(1, N, K, fmt, G, 31, zeros)
    x, xv = _x(S, K, 12)
    y = tg.gemv_w4(x, W[0], sc[0], zeros=z[0] if z is not None else None, format=fmt, group=G)
    _check(y, xv, wv, [0, S], K, G, F32)


def test_one_matrix_for_every_group():
    K, N, G = 512, 48, 64
    W, sc, z, wv = _weights(1, N, K, "int4", G, 32, True)
    x, xv = _x(6, K, 13)
    off = torch.tensor([0, 4, 4, 6], dtype=torch.int32, device=dev())
    y = tg.gemv_w4(x, W.expand(3, N, K // 2), sc.expand(3, N, K // G), zeros=z.expand(3, N, K // G), offsets=off, group=G)
    _check(y, xv, wv, [0, 6], K, G, F32)


def test_infinite_activations_reach_int4_as_the_formula_says():
    """x w is an infinity of w's sign, NaN where the weight is zero; other rows
    of the same pass are untouched."""
    K, N = 1024, 70
    W, sc, _, wv = _weights(1, N, K, "int4", 128, 33)
    x, xv = _x(4, K, 14)
    x[1, 700] = float("inf")
    x[3, 5] = float("nan")
    y = tg.gemv_w4(x, W[0], sc[0]).cpu().double().numpy()
    w = wv[0][:, 700]
    assert np.array_equal(np.isnan(y[1]), w == 0)
    assert np.array_equal(y[1][w != 0], np.where(w > 0, np.inf, -np.inf)[w != 0])
    assert np.isnan(y[3]).all()
    for t in (0, 2):
        want, mag = xv[t] @ wv[0].T, np.abs(xv[t]) @ np.abs(wv[0]).T
        assert np.all(np.abs(y[t] - want) <= 2 * (K + 10) * U32 * mag)


@pytest.mark.parametrize("fmt,G,zeros", FORMATS)
@pytest.mark.parametrize("K,N,sizes", [(512, 28672, [16]), (512, 28672, [64]), (256, 9000, [16, 0, 1, 8, 40]), (9216, 2048, [40])])
def test_infinities_and_large_values_in_the_rows_of_several_passes(fmt, G, zeros, K, N, sizes):
    """Workers go on from one pass of eight rows, or slice of K, to the next:
    infinities and magnitudes from 2^116 in some rows of each, every column
    of every row, several calls alike."""
    S, groups = sum(sizes), len(sizes)
    W, sc, z, wv = _weights(groups, N, K, fmt, G, K + N, zeros)
    x, xv = _x(S, K, 19)
    off = np.concatenate([[0], np.cumsum(sizes)])
    inf, large = list(range(3, S, 8)), list(range(5, S, 16))
    at = [(t * 37) % K for t in range(S)]
    for t in inf:
        x[t, at[t]] = xv[t, at[t]] = float("inf") if t % 3 else float("-inf")
    for t in large:
        x[t, at[t]] = 2.0 ** 116
        xv[t, at[t]] = 2.0 ** 116
    offsets = torch.from_numpy(off).int().to(dev())
    y = tg.gemv_w4(x, W, sc, zeros=z, offsets=offsets, format=fmt, group=G)
    for _ in range(3):
        again = tg.gemv_w4(x, W, sc, zeros=z, offsets=offsets, format=fmt, group=G)
        assert torch.equal(torch.nan_to_num(again, nan=7e30), torch.nan_to_num(y, nan=7e30))
    y = y.cpu().double().numpy()
    bound = 2 * (K + -(-K // G) + 2) * U32
    for g in range(groups):
        for t in range(off[g], off[g + 1]):
            if t in inf:
                w = wv[g][:, at[t]] * np.sign(xv[t, at[t]])
                assert np.array_equal(np.isnan(y[t]), w == 0)
                assert np.array_equal(y[t][w != 0], np.where(w > 0, np.inf, -np.inf)[w != 0])
            else:
                want, mag = xv[t] @ wv[g].T, np.abs(xv[t]) @ np.abs(wv[g]).T
                assert np.all(np.abs(y[t] - want) <= bound * mag)


# K whose rows lie on 16 bytes, 4 bytes and neither
ROWS_ON = [1024, 1000, 1022]


@pytest.mark.parametrize("fmt,G,zeros", FORMATS)
@pytest.mark.parametrize("K", ROWS_ON)
@pytest.mark.parametrize("S", [1, 9])
def test_codes_of_zero_weights_give_zero(fmt, G, zeros, K, S):
    """A code at its zero point is the weight 0: no activation, of whatever size,
    leaves anything of it."""
    N = 70
    W, sc, z, _ = _weights(1, N, K, fmt, G, 41, zeros)
    code = np.zeros((1, N, K), np.uint8) if fmt == "e2m1" else np.repeat(z.cpu().numpy() if zeros else np.full(sc.shape, 8, np.uint8), G, -1)[..., :K]
    W = torch.from_numpy(code[..., 0::2] | code[..., 1::2] << 4).to(dev())
    x, _ = _x(S, K, 21)
    x[:, 5::7] *= 1000
    y = tg.gemv_w4(x, W[0], sc[0], zeros=z[0] if zeros else None, format=fmt, group=G)
    assert torch.equal(y, torch.zeros(S, N, device=dev()))


@pytest.mark.parametrize("fmt,G,zeros", FORMATS)
@pytest.mark.parametrize("K", ROWS_ON)
@pytest.mark.parametrize("power", [20, 40, 100, 117, 125])
def test_large_activations_over_zero_weights(fmt, G, zeros, K, power):
    """A channel of large activations whose weights are zero leaves the others'
    products as they are."""
    N, S, at = 70, 3, 333
    W, sc, z, wv = _weights(1, N, K, fmt, G, 42, zeros)
    code = torch.zeros_like(sc[..., at // G]).to(torch.uint8) if fmt == "e2m1" else z[..., at // G] if zeros else torch.full_like(W[..., 0], 8)
    W[..., at // 2] = (W[..., at // 2] & 15) | code << 4
    x, xv = _x(S, K, 22)
    x[:, at] = 2.0 ** power
    xv[:, at] = 2.0 ** power
    wv[..., at] = 0
    y = tg.gemv_w4(x, W[0], sc[0], zeros=z[0] if zeros else None, format=fmt, group=G)
    _check(y, xv, wv, [0, S], K, G, F32)


@pytest.mark.parametrize("fmt,G,zeros", FORMATS)
@pytest.mark.parametrize("K", ROWS_ON)
@pytest.mark.parametrize("power", [115, 118, 121, 126])
def test_large_activations_with_small_scales(fmt, G, zeros, K, power):
    """A group's codes times its activations may add up to more than fp32's
    largest value where its scale brings them back; rows of usual size and
    a row with an infinity lie beside."""
    N, S = 70, 6
    W, sc, z, wv = _weights(1, N, K, fmt, G, 44, zeros)
    if fmt == "e2m1":
        sc -= 40
    else:
        sc *= 2.0 ** -40
    wv = wv * 2.0 ** -40
    x, xv = _x(S, K, 24)
    for t in (1, 4):
        x[t] = xv[t] = 2.0 ** power
        x[t, ::3] = -1.5 * 2.0 ** power
        xv[t, ::3] = -1.5 * 2.0 ** power
    x[3, 77] = float("inf")
    y = tg.gemv_w4(x, W[0], sc[0], zeros=z[0] if zeros else None, format=fmt, group=G)
    keep = [0, 1, 2, 4, 5]
    _check(y[keep], xv[keep], wv, [0, 5], K, G, F32)
    w = wv[0][:, 77]
    assert torch.equal(torch.isnan(y[3]).cpu(), torch.from_numpy(w == 0))
    assert torch.equal(y[3].cpu()[w != 0], torch.from_numpy(np.where(w > 0, np.inf, -np.inf)[w != 0]).float())


@pytest.mark.parametrize("K", ROWS_ON)
@pytest.mark.parametrize("code", [0, 1, 120, 250, 254])
def test_e2m1_scales_of_any_size(K, code):
    """Scales from 2^-127 to 2^127 with activations that keep the results in
    range; what a product below 2^-126 loses (2^-150 at most, half a unit of
    fp32 there) is allowed for each of them."""
    N, S = 40, 3
    W, sc, _, wv = _weights(1, N, K, "e2m1", 32, 43)
    x, xv = _x(S, K, 23)
    up = 2.0 ** min(100, max(-100, 127 - code))
    x, xv = (x.double() * up).to(BF), xv * up
    wv = wv / np.repeat(np.exp2(sc.cpu().double().numpy() - 127), 32, -1)[..., :K] * 2.0 ** (code - 127)
    sc.fill_(code)
    y = tg.gemv_w4(x, W[0], sc[0], format="e2m1")
    want, mag = xv @ wv[0].T, np.abs(xv) @ np.abs(wv[0]).T
    assert np.all(np.abs(y.cpu().double().numpy() - want) <= 2 * (K + -(-K // 32) + 2) * U32 * mag + 2 * K * 2.0 ** -150)


@pytest.mark.parametrize("power", [-120, -60, 60, 110, 124])
def test_activations_of_any_magnitude(power):
    """Rows scaled by powers of two give results scaled by the same, exactly
    (no step of the product depends on their magnitude); where bf16 cannot hold
    the scaled rows (below 2^-126 it has fewer bits), the product of the rows
    as they were rounded; and from 2^114, where rows are summed in another
    order, the product within its bound."""
    K, N = 768, 40
    W, sc, _, wv = _weights(1, N, K, "int4", 128, 34)
    x, _ = _x(2, K, 15)
    scaled = (x.double() * 2.0 ** power).bfloat16()
    z = tg.gemv_w4(scaled, W[0], sc[0])
    if power < 114 and torch.equal(scaled.double(), x.double() * 2.0 ** power):
        assert torch.equal(z.double(), tg.gemv_w4(x, W[0], sc[0]).double() * 2.0 ** power)
    else:
        _check_wide(z, scaled.cpu().double().numpy(), wv, K, 128)


def test_codes_past_four_gigabytes():
    K, N, groups = 8192, 8192, 140  # 32 MiB a group, 4.7 GB in all
    W = torch.zeros(groups, N, K // 2, dtype=torch.uint8, device=dev())
    sc = torch.ones(groups, N, K // 128, dtype=BF, device=dev())
    last, slc, _, wv = _weights(1, N, K, "int4", 128, 35)
    W[-1], sc[-1] = last[0], slc[0]
    off = torch.zeros(groups + 1, dtype=torch.int32, device=dev())
    off[-1] = 2
    x, xv = _x(2, K, 16)
    y = tg.gemv_w4(x, W, sc, offsets=off)
    _check(y[:, -64:], xv, wv[:, -64:], [0, 2], K, 128, F32)
    _check(y[:, :64], xv, wv[:, :64], [0, 2], K, 128, F32)


@pytest.mark.parametrize("K", [2 ** 30 + 1024, 2 ** 30 + 520, 2 ** 30 + 26])
def test_rows_of_more_than_a_billion_codes(K):
    """Byte counts of a row past 31 bits, for rows on 16, 4 and 1 bytes: few
    activations are not zero, so the sums are exact."""
    N, G = 2, 128
    g = torch.Generator(device=dev()).manual_seed(40)
    W = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, generator=g, device=dev())
    sc = torch.ones(N, -(-K // G), dtype=BF, device=dev())
    x = torch.zeros(1, K, dtype=BF, device=dev())
    at = torch.tensor([0, 1, 300, 513, 2 ** 20 + 7, 2 ** 29, 2 ** 30 - 1, 2 ** 30, K - 1], device=dev())
    x[0, at] = torch.arange(1, 10, device=dev()).to(BF)
    q = (W[:, at // 2].int() >> (4 * (at % 2))) & 15
    want = ((q - 8) * torch.arange(1, 10, device=dev())).sum(1).float()
    assert torch.equal(tg.gemv_w4(x, W, sc)[0], want)


@pytest.mark.parametrize("power", [-120, 116, 125])
def test_e2m1_activations_of_any_magnitude(power):
    K, N = 768, 40
    W, sc, _, wv = _weights(1, N, K, "e2m1", 32, 36)
    x, _ = _x(2, K, 17)
    scaled = (x.double() * 2.0 ** power).clamp(-2.0 ** 127, 2.0 ** 127).bfloat16()
    scaled[0] = x[0]
    s = torch.full_like(sc[0], 123)
    g = np.exp2(123.0 - 127) * wv / np.repeat(np.exp2(sc.cpu().double().numpy() - 127), 32, -1)
    y = tg.gemv_w4(scaled, W[0], s, format="e2m1", group=32)
    assert bool(torch.isinf(y).any()) == (power == 125)  # three values lie past fp32's largest
    _check_wide(y, scaled.cpu().double().numpy(), g, K, 32)


@pytest.mark.parametrize("fmt,G,zeros", FORMATS)
def test_slices_of_the_contraction(fmt, G, zeros):
    """Long rows are cut into slices that a second kernel adds: groups with and
    without rows, rows of no group, infinities in one slice, the same bits again."""
    K, N, S = 9000, 136, 23
    K += K % 32 and 32 - K % 32
    W, sc, z, wv = _weights(4, N, K, fmt, G, 37, zeros)
    x, xv = _x(S, K, 18)
    offsets = [1, 12, 12, 20, 22]
    off = torch.tensor(offsets, dtype=torch.int32, device=dev())
    y = tg.gemv_w4(x, W, sc, zeros=z, offsets=off, format=fmt, group=G)
    _check(y, xv, wv, offsets, K, G, F32)
    assert torch.equal(y, tg.gemv_w4(x, W, sc, zeros=z, offsets=off, format=fmt, group=G))
    assert not bool(y[0].any()) and not bool(y[22].any())
    b = tg.gemv_w4(x, W, sc, zeros=z, offsets=off, format=fmt, group=G, out_dtype=BF)
    assert torch.equal(b, y.to(BF))
    stream, g2 = torch.cuda.Stream(), torch.empty_like(y)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):  # another stream's scratch, then a captured call
        tg.gemv_w4(x, W, sc, zeros=z, offsets=off, format=fmt, group=G, y=g2)
    stream.synchronize()
    assert torch.equal(g2, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        tg.gemv_w4(x, W, sc, zeros=z, offsets=off, format=fmt, group=G, y=g2)
    off.copy_(torch.tensor([0, 3, 15, 15, 23], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    _check(g2, xv, wv, [0, 3, 15, 15, 23], K, G, F32)
    off.copy_(torch.tensor(offsets, dtype=torch.int32))
    x[13, K - 3] = float("inf")
    v = tg.gemv_w4(x, W, sc, zeros=z, offsets=off, format=fmt, group=G)
    w = wv[2][:, K - 3]
    assert torch.equal(torch.isnan(v[13]).cpu(), torch.from_numpy(w == 0))
    keep = [i for i in range(S) if i != 13]
    assert torch.equal(v[keep], y[keep])


@pytest.mark.parametrize("fmt,G,zeros", FORMATS)
@pytest.mark.parametrize("K,N,sizes", [(512, 9000, [16]), (4096, 600, [3, 0, 9]), (9216, 2048, [40])])
def test_watchdog(fmt, G, zeros, K, N, sizes):
    """The checks build, whose first warp's weights are never loaded: the waits
    run out after their limit, whole blocks leave (whoever noticed first),
    tg_device_error says so, and the next call is right."""
    import ctypes

    lib = tg.load_checks()
    lib.tg_gemv_w4_watchdog.argtypes, lib.tg_gemv_w4_watchdog.restype = [ctypes.c_int32, ctypes.c_uint64], None
    S, groups, runs = sum(sizes), len(sizes), -(-K // G)
    W, sc, z, wv = _weights(groups, N, K, fmt, G, 39, zeros)
    x, xv = _x(S, K, 20)
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    off = torch.from_numpy(offsets).int().to(dev())
    y = torch.empty(S, N, device=dev())
    s = torch.cuda.current_stream().cuda_stream

    def call():
        return lib.tg_gemv_w4(x.data_ptr(), K, W.data_ptr(), K, N * K, sc.data_ptr(), runs, N * runs,
                              z.data_ptr() if z is not None else None, runs, N * runs, tg.W4_FORMATS[fmt], G, off.data_ptr(), groups,
                              S, N, K, y.data_ptr(), N, 0, s)

    try:
        for _ in range(10):
            lib.tg_gemv_w4_watchdog(1, 2_000_000)
            assert call() == tg.TG_OK
            assert lib.tg_device_error(s) == tg.TG_ERR_TIMEOUT
    finally:
        lib.tg_gemv_w4_watchdog(0, 0)
    assert lib.tg_device_error(s) == tg.TG_OK
    assert call() == tg.TG_OK
    assert lib.tg_device_error(s) == tg.TG_OK
    _check(y, xv, wv, offsets, K, G, F32)
