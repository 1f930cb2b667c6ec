"""The projections on the GPU against 64-bit forms: the gated projection and the
gradient through it, dense and by group, and the projection with adapters,
over group sizes from none to several tiles, every tile choice, odd extents and
pitches, rows of no group, non-finite values in other groups' operands, and
bounds that are not what they should be.

Integer inputs make every sum exact, so those results are compared bit for
bit; the activations and random values within fp32's error (projection_ref)
and one rounding."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import tiled_gemm_codegen_gb300 as tg
from expert_ref import U32, within
from gpu_helpers import PER_ELEM, dev
from projection_ref import act, act_error, adapted, in_group, products, slope, slope_error

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")
SIZES = {
    "one": [1],
    "mixed": [0, 3, 129, 64, 0, 1, 300, 0],
    "tiles": [128, 256, 512, 64],
    "empty": [0, 0, 0],
    "many": [i % 5 for i in range(70)],
    "long": [700, 5, 1000],
}
SHAPES = [(64, 128), (72, 136), (1, 1), (200, 333), (640, 512), (65, 257)]
ACTS = ["none", "relu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tg.load()
    yield
    assert tg.device_error() == tg.TG_OK


def _offsets(sizes, lead=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]) + lead, dtype=torch.int32, device=dev())


def _rand(shape, seed, ints=True, pitch=None):
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(-3, 4, shape, generator=g).float() if ints else torch.randn(*shape, generator=g)
    v = v.to(BF)
    if pitch:
        store = torch.full((*shape[:-1], pitch), NAN, dtype=BF)
        store[..., :shape[-1]] = v
        return store.to(dev())[..., :shape[-1]], v.double().numpy()
    return v.to(dev()), v.double().numpy()


def _mats(lead, K, N, seed, transposed, ints=True):
    """Weights [*lead, K, N], stored transposed or not."""
    W, wv = _rand((*lead, N, K) if transposed else (*lead, K, N), seed, ints)
    return (W.transpose(-1, -2), np.swapaxes(wv, -1, -2)) if transposed else (W, wv)


def _np(t):
    return t.detach().cpu().double().numpy()


def _bf(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(BF).double().numpy()


def _f32(a):
    return np.asarray(a, np.float32).astype(np.float64)


# ---------------------------------------------------------------- gated
@pytest.mark.parametrize("name", list(SIZES))
@pytest.mark.parametrize("K,F", SHAPES)
@pytest.mark.parametrize("pair", [0, 1, 2])
@pytest.mark.parametrize("transposed", [False, True])
def test_gated_exact(name, K, F, pair, transposed):
    """Integers: z is exact, and a product of two of its values is rounded to
    fp32, then to bf16."""
    sizes = SIZES[name]
    X, xv = _rand((sum(sizes), K), 1)
    W, wv = _mats((len(sizes),), K, 2 * F, 2, transposed)
    H, Z = tg.gemm_gated(X, W, _offsets(sizes), Z=True, activation="relu", options=tg.make_options(cta_pair=pair))
    z = products(xv, wv, sizes)
    assert np.array_equal(_np(Z), _bf(z))
    assert np.array_equal(_np(H), _bf(_f32(np.maximum(z[:, :F], 0) * z[:, F:])))


@pytest.mark.parametrize("S", [1, 2, 31, 33, 128, 300, 1025])
@pytest.mark.parametrize("K,F", [(1, 1), (130, 70), (1000, 200), (2048, 1408)])
@pytest.mark.parametrize("pair", [0, 1, 2])
@pytest.mark.parametrize("transposed", [False, True])
def test_gated_dense(S, K, F, pair, transposed):
    X, xv = _rand((S, K), 3)
    W, wv = _mats((), K, 2 * F, 4, transposed)
    opts = tg.make_options(cta_pair=pair)
    z = xv @ wv
    want = _bf(_f32(z[:, :F] * z[:, F:]))
    for _ in range(2):  # the arrival counters of shared tiles are left ready
        assert np.array_equal(_np(tg.gemm_gated(X, W, activation="none", options=opts)), want)
    H, Z = tg.gemm_gated(X, W, activation="none", Z=True, options=opts)
    assert np.array_equal(_np(H), want) and np.array_equal(_np(Z), _bf(z))


@pytest.mark.parametrize("activation", ACTS)
@pytest.mark.parametrize("pair", [1, 2])
def test_gated_activations(activation, pair):
    sizes, K, F = [33, 0, 200, 1], 136, 200
    X, xv = _rand((sum(sizes), K), 5, False)
    W, wv = _mats((4,), K, 2 * F, 6, False, False)
    W, wv = W * 0.125, wv * 0.125
    H = tg.gemm_gated(X, W, _offsets(sizes), activation=activation, options=tg.make_options(cta_pair=pair))
    z = products(xv, wv, sizes)
    g, u = z[:, :F], z[:, F:]
    ez = PER_ELEM * np.sqrt(K) * np.abs(z).max()
    a = np.abs(act(activation, g))
    # |act'| <= 1.13
    bound = (1.13 * ez + act_error(g)) * (np.abs(u) + ez) + a * ez + U32 * a * np.abs(u)
    assert within(H, act(activation, g) * u, bound, BF)


@pytest.mark.parametrize("pitches", [(None, None, 0), (80, 280, 8), (75, 269, 3), (66, 259, 1)])
@pytest.mark.parametrize("F", [128, 129])
@pytest.mark.parametrize("pair", [1, 2])
def test_gated_pitches_rows_of_no_group_and_guard_bands(pitches, F, pair):
    px, pw, ph = pitches
    K, sizes, lead, S = 65, [40, 0, 150, 7], 11, 230
    X, xv = _rand((S, K), 7, True, px)
    W, wv = _rand((4, K, 2 * F), 8, True, pw)
    hs = torch.full((S + 2, F + ph), NAN, dtype=BF, device=dev())
    zs = torch.full((S + 2, 2 * F + ph), NAN, dtype=BF, device=dev())
    H, Z = hs[1:-1, :F], zs[1:-1, :2 * F]
    tg.gemm_gated(X, W, _offsets(sizes, lead), H, Z=Z, activation="relu", options=tg.make_options(cta_pair=pair))
    z = products(xv, wv, sizes, lead)
    assert np.array_equal(_np(Z), _bf(z))
    assert np.array_equal(_np(H), _bf(_f32(np.maximum(z[:, :F], 0) * z[:, F:])))
    H.fill_(NAN), Z.fill_(NAN)
    assert bool(torch.isnan(hs).all()) and bool(torch.isnan(zs).all())


def test_gated_infinities_follow_the_formula():
    """relu and none have no indeterminate forms but the formula's own; a row's
    infinity stays in its row, a feature's in its feature, a group's in its group."""
    sizes, K, F = [70, 60, 5], 96, 72
    X, xv = _rand((135, K), 9)
    W, wv = _rand((3, K, 2 * F), 10)
    X[3] = float("inf")
    X[70:130] = NAN
    W[2, :, F + 5] = NAN
    W[2, 7, 9] = float("inf")
    xv[3], xv[70:130], wv[2, :, F + 5], wv[2, 7, 9] = np.inf, np.nan, np.nan, np.inf
    for opt in (1, 2):
        H, Z = tg.gemm_gated(X, W, _offsets(sizes), activation="none", Z=True, options=tg.make_options(cta_pair=opt))
        with np.errstate(all="ignore"):
            z = products(xv, wv, sizes)
            h = _f32(z[:, :F] * z[:, F:])
        assert np.array_equal(_np(Z), _bf(z), equal_nan=True) and np.array_equal(_np(H), _bf(h), equal_nan=True)


def test_gated_one_matrix_for_every_group_and_no_terms():
    sizes, K, F = [5, 90], 72, 80
    X, xv = _rand((95, K), 11)
    W, wv = _rand((1, K, 2 * F), 12)
    H = tg.gemm_gated(X, W.expand(2, K, 2 * F), _offsets(sizes), activation="none")
    z = xv @ wv[0]
    assert np.array_equal(_np(H), _bf(_f32(z[:, :F] * z[:, F:])))
    H, Z = tg.gemm_gated(torch.empty(7, 0, dtype=BF, device=dev()), torch.empty(0, 48, dtype=BF, device=dev()), Z=True)
    assert not bool(H.any()) and not bool(Z.any()) and H.shape == (7, 24) and Z.shape == (7, 48)
    assert tg.gemm_gated(torch.empty(0, 8, dtype=BF, device=dev()), torch.empty(8, 48, dtype=BF, device=dev())).shape == (0, 24)


# ---------------------------------------------------------------- gradient
def _grad_ref(activation, dh, z, F, rows):
    g, u = z[:, :F], z[:, F:]
    a, s = act(activation, g), slope(activation, g)
    dz = np.concatenate((dh * u * s, dh * a), 1)
    h = a * u
    dz[~rows], h[~rows] = 0, 0
    return dz, h


@pytest.mark.parametrize("name", list(SIZES))
@pytest.mark.parametrize("K,F", SHAPES)
@pytest.mark.parametrize("pair", [0, 1, 2])
@pytest.mark.parametrize("transposed", [False, True])
def test_gated_grad_exact(name, K, F, pair, transposed):
    sizes = SIZES[name]
    S = sum(sizes)
    dY, yv = _rand((S, K), 20)
    V, vv = _mats((len(sizes),), K, F, 21, transposed)
    Z, zv = _rand((S, 2 * F), 22)
    dZ, H = tg.gemm_gated_grad(dY, V, Z, _offsets(sizes), H=True, activation="relu", options=tg.make_options(cta_pair=pair))
    dz, h = _grad_ref("relu", products(yv, vv, sizes), zv, F, in_group(S, sizes))
    assert np.array_equal(_np(dZ), _bf(_f32(dz))) and np.array_equal(_np(H), _bf(h))


@pytest.mark.parametrize("S", [1, 2, 31, 33, 128, 300, 1025])
@pytest.mark.parametrize("K,F", [(1, 1), (130, 70), (1000, 200), (2048, 1408)])
@pytest.mark.parametrize("pair", [0, 1, 2])
def test_gated_grad_dense(S, K, F, pair):
    dY, yv = _rand((S, K), 23)
    V, vv = _mats((), K, F, 24, True)
    Z, zv = _rand((S, 2 * F), 25)
    want, _ = _grad_ref("none", yv @ vv, zv, F, in_group(S, [S]))
    for _ in range(2):
        dZ = tg.gemm_gated_grad(dY, V, Z, activation="none", options=tg.make_options(cta_pair=pair))
        assert np.array_equal(_np(dZ), _bf(_f32(want)))


@pytest.mark.parametrize("activation", ACTS)
@pytest.mark.parametrize("pair", [1, 2])
def test_gated_grad_activations(activation, pair):
    sizes, lead, S, K, F = [33, 0, 200, 1], 6, 250, 136, 200
    dY, yv = _rand((S, K), 26)
    V, vv = _mats((4,), K, F, 27, True)
    Z, zv = _rand((S, 2 * F), 28, False)
    dZ, H = tg.gemm_gated_grad(dY, V, Z, _offsets(sizes, lead), H=True, activation=activation, options=tg.make_options(cta_pair=pair))
    dh = products(yv, vv, sizes, lead)
    dz, h = _grad_ref(activation, dh, zv, F, in_group(S, sizes, lead))
    g, u = zv[:, :F], zv[:, F:]
    bound = np.concatenate((np.abs(dh * u) * (slope_error(g) + 4 * U32 * np.abs(slope(activation, g))),
                            np.abs(dh) * (act_error(g) + 2 * U32 * np.abs(act(activation, g)))), 1)
    assert within(dZ, dz, bound, BF)
    assert within(H, h, np.abs(u) * (act_error(g) + 2 * U32 * np.abs(act(activation, g))), BF)


@pytest.mark.parametrize("pitches", [(None, None, None, 0), (80, 136, 264, 8), (75, 133, 267, 3), (66, 130, 259, 1)])
@pytest.mark.parametrize("F", [128, 129])
@pytest.mark.parametrize("pair", [1, 2])
def test_gated_grad_pitches_rows_of_no_group_and_guard_bands(pitches, F, pair):
    py, pv, pz, po = pitches
    K, sizes, lead, S = 65, [40, 0, 150, 7], 11, 230
    dY, yv = _rand((S, K), 29, True, py)
    V, vv = _rand((4, K, F), 30, True, pv)
    Z, zv = _rand((S, 2 * F), 31, True, pz)
    hs = torch.full((S + 2, F + po), NAN, dtype=BF, device=dev())
    zs = torch.full((S + 2, 2 * F + po), NAN, dtype=BF, device=dev())
    H, dZ = hs[1:-1, :F], zs[1:-1, :2 * F]
    tg.gemm_gated_grad(dY, V, Z, _offsets(sizes, lead), dZ, H=H, activation="relu", options=tg.make_options(cta_pair=pair))
    dz, h = _grad_ref("relu", products(yv, vv, sizes, lead), zv, F, in_group(S, sizes, lead))
    assert np.array_equal(_np(dZ), _bf(_f32(dz))) and np.array_equal(_np(H), _bf(h))
    H.fill_(NAN), dZ.fill_(NAN)
    assert bool(torch.isnan(hs).all()) and bool(torch.isnan(zs).all())


@pytest.mark.parametrize("size", [200, 33, 95])
@pytest.mark.parametrize("F", [384, 392, 700])
@pytest.mark.parametrize("pair", [1, 2])
def test_boxes_stored_plainly_between_boxes_stored_by_tma(size, F, pair):
    """A group's last rows, and a box cut off by the row's end, leave their
    staging box by plain stores, the others by asynchronous ones that may
    still read theirs: short products over many groups, several tiles a
    worker, every element of every call."""
    groups, K = 160, 64
    S, off = groups * size, _offsets([size] * groups)
    X, _ = _rand((S, K), 32)
    W, _ = _rand((groups, K, 2 * F), 33)
    V, _ = _rand((groups, K, F), 34)
    opts = tg.make_options(cta_pair=pair)
    z = torch.bmm(X.float().view(groups, size, K), W.float()).view(S, 2 * F)  # integers: exact before the rounding
    want_h, want_z = (z[:, :F].clamp(min=0) * z[:, F:]).to(BF), z.to(BF)
    dh = torch.bmm(X.float().view(groups, size, K), V.float()).view(S, F)
    g, u = want_z[:, :F].float(), want_z[:, F:].float()
    want_dz = torch.cat((dh * u * (g > 0), dh * g.clamp(min=0)), 1).to(BF)
    want_h2 = (g.clamp(min=0) * u).to(BF)
    H, Z, dZ = torch.empty_like(want_h), torch.empty_like(want_z), torch.empty_like(want_z)
    wrong = torch.zeros((), dtype=torch.int64, device=dev())
    for _ in range(50):
        H.fill_(NAN), Z.fill_(NAN)
        tg.gemm_gated(X, W, off, H, activation="relu", options=opts)
        wrong += (H != want_h).sum()
        H.fill_(NAN)
        tg.gemm_gated(X, W, off, H, Z=Z, activation="relu", options=opts)
        wrong += (H != want_h).sum() + (Z != want_z).sum()
        H.fill_(NAN), dZ.fill_(NAN)
        tg.gemm_gated_grad(X, V, want_z, off, dZ, H=H, activation="relu", options=opts)
        wrong += (H != want_h2).sum() + (dZ != want_dz).sum()
    assert int(wrong) == 0


@pytest.mark.parametrize("activation", ACTS)
def test_gated_grad_of_huge_gates(activation):
    """Gates whose square (and cube) pass fp32: the slope is 0 or 1 there, the
    activation 0 or the gate."""
    S, K, F = 40, 16, 64
    dY, yv = _rand((S, K), 45)
    V, vv = _mats((), K, F, 46, True)
    Z, zv = _rand((S, 2 * F), 47)
    for r, g in enumerate((2.0 ** 66, -(2.0 ** 66), 2.0 ** 20, -(2.0 ** 20), 2.0 ** 100, -(2.0 ** 100))):
        Z[r, :F], zv[r, :F] = g, g
    dZ, H = tg.gemm_gated_grad(dY, V, Z, H=True, activation=activation)
    with np.errstate(all="ignore"):
        dz, h = _grad_ref(activation, yv @ vv, zv, F, in_group(S, [S]))
        g, u = zv[:, :F], zv[:, F:]
        # (huge gates: s and 1 - s are exact, and what is left are two products' roundings)
        e_act = np.where(np.abs(g) > 1e5, 4 * U32 * np.abs(g) * (g > 0), act_error(g))
        e_slope = np.where(np.abs(g) > 1e5, 4 * U32, slope_error(g))
    dh = yv @ vv
    assert within(dZ, dz, np.concatenate((np.abs(dh * u) * (e_slope + 8 * U32), np.abs(dh) * (e_act + 4 * U32 * np.abs(act(activation, g)))), 1), BF)
    assert within(H, h, np.abs(u) * (e_act + 4 * U32 * np.abs(act(activation, g))), BF)


def test_gradients_of_a_block_against_differences():
    """x -> gated -> down, all gradients: each against the central difference
    of the 64-bit formula along a random direction."""
    S, D, F = 50, 40, 72
    X, xv = _rand((S, D), 35, False)
    W, wv = _mats((), D, 2 * F, 36, True, False)
    Dn, dv = _rand((F, D), 37, False)
    W, wv, Dn, dv = W * 0.125, wv * 0.125, Dn * 0.125, dv * 0.125
    C, cv = _rand((S, D), 38, False)
    H, Z = tg.gemm_gated(X, W, Z=True)
    dZ, H2 = tg.gemm_gated_grad(C, Dn.t(), Z, H=True)
    dX = tg.gemm(dZ, W.t())
    dW = tg.gemm(X.t(), dZ)
    dD = tg.gemm(H2.t(), C)

    def loss(x, w, d):
        z = x @ w
        return float((cv * (act("silu", z[:, :F]) * z[:, F:] @ d)).sum())

    # The operands of the gradient's products were rounded to bf16 (by at most 2^-8): Z, whose
    # error moves dz and h along their slopes (silu'' <= 0.5, silu' <= 1.1), then dZ and H.
    z, dh = xv @ wv, cv @ dv.T
    gate, up = z[:, :F], z[:, F:]
    a, sl = np.abs(act("silu", gate)), np.abs(slope("silu", gate))
    half = 2.0 ** -8
    e_dz = half * np.abs(np.concatenate((dh * up * sl, dh * a), 1)) + half * np.abs(np.concatenate(
        (dh * (np.abs(up) * sl + 0.5 * np.abs(up * gate)), dh * 1.1 * gate), 1))
    e_h = half * (2 * a * np.abs(up) + 1.1 * np.abs(gate * up))
    errors = (e_dz @ np.abs(wv).T, np.abs(xv).T @ e_dz, e_h.T @ np.abs(cv))
    g = np.random.default_rng(0)
    for at, got in enumerate((dX, dW, dD)):
        args = [xv, wv, dv]
        step = g.standard_normal(args[at].shape)
        lo, hi = list(args), list(args)
        lo[at], hi[at] = args[at] - 1e-4 * step, args[at] + 1e-4 * step
        diff = (loss(*hi) - loss(*lo)) / 2e-4
        # (second-order terms of the difference and fp32 sums: far below 1e-4 of the terms)
        bound = float((errors[at] * np.abs(step)).sum()) + 1e-4 * float((np.abs(_np(got)) * np.abs(step)).sum())
        assert abs(float((_np(got) * step).sum()) - diff) <= bound


# ---------------------------------------------------------------- adapters
def _adapters(sizes, K, N, R, seed, ints=True, S=None, transposed=False):
    S = sum(sizes) if S is None else S
    X, xv = _rand((S, K), seed, ints)
    W, wv = _mats((), K, N, seed + 1, transposed, ints)
    A, av = _rand((len(sizes), R, K), seed + 2, ints)
    B, bv = _rand((len(sizes), R, N), seed + 3, ints)
    return (X, W, A, B), (xv, wv, av, bv)


RANKS = [1, 4, 8, 16, 20, 32, 33, 64, 100, 128, 200, 256]


@pytest.mark.parametrize("name", list(SIZES))
@pytest.mark.parametrize("R", RANKS)
@pytest.mark.parametrize("pair", [0, 1, 2])
@pytest.mark.parametrize("transposed", [False, True])
def test_adapted_exact(name, R, pair, transposed):
    """Integers below 2^16 in u: its two parts hold it, and all sums are exact."""
    sizes, K, N = SIZES[name], 40, 200
    t, v = _adapters(sizes, K, N, R, 40, transposed=transposed)
    scales = torch.tensor([(-1.0) ** i * 2.0 ** (i % 3 - 1) for i in range(len(sizes))], device=dev())
    Y, U = tg.gemm_adapted(*t, _offsets(sizes), scales=scales, U=True, options=tg.make_options(cta_pair=pair))
    y, u = adapted(*v, sizes, _np(scales))
    assert np.array_equal(_np(Y), y) and np.array_equal(_np(U), _bf(u))


@pytest.mark.parametrize("K,N", [(1, 1), (64, 64), (65, 257), (200, 333), (640, 512), (0, 40)])
@pytest.mark.parametrize("sizes,lead,S", [([1], 0, 1), ([3, 0, 30], 5, 60), ([100, 1, 1, 300], 77, 500), ([0], 0, 40), ([1] * 300, 3, 310)])
@pytest.mark.parametrize("R", [8, 16, 40])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_adapted_rows_of_no_adapter(K, N, sizes, lead, S, R, dtype):
    t, v = _adapters(sizes, K, N, R, 50, S=S)
    Y, U = tg.gemm_adapted(*t, _offsets(sizes, lead), U=True, out_dtype=dtype)
    y, u = adapted(*v, sizes, lead=lead)
    assert np.array_equal(_np(Y), y if dtype == F32 else _bf(y)) and np.array_equal(_np(U), _bf(u))


@pytest.mark.parametrize("sizes,lead,S", [([1], 0, 1), ([2] * 30, 0, 64), ([200, 100], 0, 300)])
@pytest.mark.parametrize("K,N", [(4096, 64), (5000, 200), (1100, 129)])
@pytest.mark.parametrize("pair", [0, 1, 2])
def test_adapted_shared_tiles(sizes, lead, S, K, N, pair):
    R = 16
    t, v = _adapters(sizes, K, N, R, 60, S=S)
    y, u = adapted(*v, sizes, lead=lead)
    # u has up to 16 bits here, so Y's sums stay below 2^24
    assert np.abs(u).max() < 2 ** 16 and np.abs(y).max() < 2 ** 24
    for _ in range(2):
        Y = tg.gemm_adapted(*t, _offsets(sizes, lead), options=tg.make_options(cta_pair=pair))
        assert np.array_equal(_np(Y), y)


@pytest.mark.parametrize("pitches", [(None, None, None, None, 0, 0), (72, 144, 80, 152, 8, 8), (67, 135, 71, 133, 3, 1)])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("pair", [1, 2])
def test_adapted_pitches_and_guard_bands(pitches, dtype, pair):
    px, pw, pa, pb, py, pu = pitches
    sizes, lead, S, K, N, R = [40, 0, 150, 7], 11, 230, 65, 129, 20
    X, xv = _rand((S, K), 70, True, px)
    W, wv = _rand((K, N), 71, True, pw)
    A, av = _rand((4, R, K), 72, True, pa)
    B, bv = _rand((4, R, N), 73, True, pb)
    ys = torch.full((S + 2, N + py), NAN, dtype=dtype, device=dev())
    us = torch.full((S + 2, R + pu), NAN, dtype=BF, device=dev())
    Y, U = ys[1:-1, :N], us[1:-1, :R]
    tg.gemm_adapted(X, W, A, B, _offsets(sizes, lead), Y, U=U, options=tg.make_options(cta_pair=pair))
    y, u = adapted(xv, wv, av, bv, sizes, lead=lead)
    assert np.array_equal(_np(Y), y if dtype == F32 else _bf(y)) and np.array_equal(_np(U), _bf(u))
    Y.fill_(NAN), U.fill_(NAN)
    assert bool(torch.isnan(ys).all()) and bool(torch.isnan(us).all())


@pytest.mark.parametrize("R", [4, 16, 48, 100])
@pytest.mark.parametrize("K", [96, 3200])  # whole tiles; shared ones
@pytest.mark.parametrize("pair", [1, 2])
def test_adapters_stay_in_their_rows(R, K, pair):
    """Infinities and NaN in one adapter's matrices and rows next to others in
    the same tile: the others exact, its own as the formula's."""
    sizes, N = [3, 5, 2, 40, 1, 100, 2], 160
    t, v = _adapters(sizes, K, N, R, 80, S=160)
    (X, W, A, B), (xv, wv, av, bv) = t, v
    for arr, val in ((B, bv),):
        arr[1, 0, 7], val[1, 0, 7] = float("inf"), np.inf
        arr[3, R - 1, 150], val[3, R - 1, 150] = NAN, np.nan
        arr[5, :, :], val[5, :, :] = float("-inf"), -np.inf
    A[6, 0, 5], av[6, 0, 5] = NAN, np.nan
    X[50], xv[50] = float("inf"), np.inf
    X[155], xv[155] = NAN, np.nan
    Y = _np(tg.gemm_adapted(X, W, A, B, _offsets(sizes), options=tg.make_options(cta_pair=pair)))
    with np.errstate(all="ignore"):
        y, _ = adapted(xv, wv, av, bv, sizes)
    assert np.array_equal(np.isnan(Y), np.isnan(y))
    assert np.array_equal(Y, y, equal_nan=True)


@pytest.mark.parametrize("R", [8, 24])
@pytest.mark.parametrize("pair", [1, 2])
def test_an_infinite_row_beside_infinities_of_its_adapter(R, pair):
    """u of a row is infinite and its B holds an infinity: the other
    features are the formula's infinities, no NaN of a zeroed product."""
    sizes, K, N = [4, 6, 3], 72, 200
    (X, W, A, B), (xv, wv, av, bv) = _adapters(sizes, K, N, R, 87)
    B[B == 0], bv[bv == 0] = 1, 1  # (0 x infinity is the formula's NaN)
    A[1], av[1] = 1, 1
    X[6], xv[6] = 1, 1
    X[6, 3], xv[6, 3] = float("inf"), np.inf
    B[1, 2, 9], bv[1, 2, 9] = NAN, np.nan
    B[1, 5, 140], bv[1, 5, 140] = float("inf"), np.inf
    W[:], wv[:] = 0, 0
    W[3], wv[3] = 1, 1
    B[1], bv[1] = B[1].abs(), np.abs(bv[1])
    Y = _np(tg.gemm_adapted(X, W, A, B, _offsets(sizes), options=tg.make_options(cta_pair=pair)))
    with np.errstate(all="ignore"):
        y, _ = adapted(xv, wv, av, bv, sizes)
    both = np.zeros_like(y, bool)
    both[6, 140] = True  # an infinite u on an infinity of B: NaN here
    assert np.array_equal(np.where(both, 0, Y), np.where(both, 0, y), equal_nan=True)
    assert not np.isfinite(Y[6]).any() and np.isnan(Y[6]).sum() == 2


@pytest.mark.parametrize("R", [8, 16, 40])
@pytest.mark.parametrize("K,N", [(64, 1500), (500, 520), (0, 1500)])
@pytest.mark.parametrize("pair", [1, 2])
def test_adapters_stay_in_their_rows_of_many_tiles(R, K, N, pair):
    """The same over several tiles a worker, one behind another: some have an
    infinity, some none, all are what the formula gives."""
    sizes = [(37 * i) % 450 for i in range(40)]
    S = sum(sizes) + 300
    (X, W, A, B), _ = _adapters(sizes, K, N, R, 85, S=S)
    g = np.random.default_rng(3)
    for val in (float("inf"), NAN, float("-inf")):
        for _ in range(8):
            B[int(g.integers(40)), int(g.integers(R)), int(g.integers(N))] = val
    want = X.double() @ W.double()
    at = 0
    for i, n in enumerate(sizes):
        want[at:at + n] += (X[at:at + n].double() @ A[i].double().t()) @ B[i].double()
        at += n
    for _ in range(3):
        Y = tg.gemm_adapted(X, W, A, B, _offsets(sizes), options=tg.make_options(cta_pair=pair))
        assert torch.equal(torch.isnan(Y), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(Y.double(), 0, 1e30, -1e30), torch.nan_to_num(want, 0, 1e30, -1e30))


@pytest.mark.parametrize("sizes,K,N,R", [([0, 300, 17, 1000, 256], 1024, 640, 16), ([2] * 40 + [0] * 9, 2048, 200, 64), ([700], 520, 392, 100)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_adapted_random_values(sizes, K, N, R, dtype):
    (X, W, A, B), (xv, wv, av, bv) = _adapters(sizes, K, N, R, 90, ints=False)
    A, av = A * 0.125, av * 0.125
    scales = torch.rand(len(sizes), device=dev()) + 0.5
    Y = tg.gemm_adapted(X, W, A, B, _offsets(sizes), scales=scales, out_dtype=dtype)
    y, u = adapted(xv, wv, av, bv, sizes, _np(scales))
    mag = products(np.abs(u), np.abs(bv), sizes)
    # sums as the library's GEMM's; u: its own sum's error, and 2^-17 that its two parts leave
    eu = PER_ELEM * np.sqrt(K) * np.abs(u).max()
    bound = PER_ELEM * np.sqrt(K + 2 * R) * np.abs(y).max() + 2.0 ** -17 * mag + products(np.full_like(u, eu), np.abs(bv), sizes)
    assert within(Y, y, bound, dtype)


def test_adapted_gradients_against_differences():
    """Integers throughout, so central differences along integer directions
    are exact (Y is linear in X, A and B, one at a time)."""
    sizes, K, N, R = [3, 0, 70, 1], 24, 40, 4
    (X, W, A, B), (xv, wv, av, bv) = _adapters(sizes, K, N, R, 95, S=80)
    off = _offsets(sizes, 2)
    C, cv = _rand((80, N), 99)
    scales = torch.tensor([1.0, 2.0, 0.5, 1.0], device=dev())
    _, U = tg.gemm_adapted(X, W, A, B, off, scales=scales, U=True)
    dX, dU = tg.gemm_adapted(C, W.t(), B, A, off, scales=scales, U=True)
    dA = tg.gemm_grouped_wgrad(dU, X, off)
    dB = tg.gemm_grouped_wgrad(U, C, off)
    y = lambda x, a, b: float((cv * adapted(x, wv, a, b, sizes, _np(scales), 2)[0]).sum())  # noqa: E731
    g = np.random.default_rng(1)
    for got, at in ((dX, 0), (dA, 1), (dB, 2)):
        args = [xv, av, bv]
        step = g.integers(-2, 3, args[at].shape).astype(float)
        lo, hi = list(args), list(args)
        lo[at], hi[at] = args[at] - step, args[at] + step
        diff = (y(*hi) - y(*lo)) / 2
        # U and dU are rounded to bf16 on their way out: half a step, 2^-8, of each term
        mag = 0.0 if at == 0 else float((np.abs(step) * _np(tg.gemm_grouped_wgrad((dU if at == 1 else U).abs(), (X if at == 1 else C).abs(), off))).sum())
        assert abs(float((_np(got) * step).sum()) - diff) <= 2.0 ** -8 * mag


@pytest.mark.parametrize("sizes,lead,S", [([3, 0, 1], 500, 1200), ([0, 0], 0, 700), ([2, 40], 33, 75), ([1] * 40, 1900, 2000)])
@pytest.mark.parametrize("K,R", [(64, 16), (1000, 20), (640, 100)])
def test_adapted_mostly_rows_of_no_adapter(sizes, lead, S, K, R):
    t, v = _adapters(sizes, K, 130, R, 160, S=S)
    y, u = adapted(*v, sizes, lead=lead)
    assert np.abs(u).max() < 2 ** 16 and np.abs(y).max() < 2 ** 24
    for _ in range(2):
        U = torch.full((S, R), NAN, dtype=BF, device=dev())
        Y, U = tg.gemm_adapted(*t, _offsets(sizes, lead), U=U)
        assert np.array_equal(_np(Y), y) and np.array_equal(_np(U), _bf(u))


@pytest.mark.parametrize("groups", [511, 512, 513, 1500, 4096])
@pytest.mark.parametrize("R", [8, 64])
def test_adapted_many_adapters(groups, R):
    g = np.random.default_rng(groups)
    sizes = [int(n) for n in g.integers(0, 3, groups)]
    K, N, S = 72, 72, sum(sizes) + 20
    t, v = _adapters(sizes, K, N, R, 170, S=S)
    Y, U = tg.gemm_adapted(*t, _offsets(sizes, 9), U=True)
    y, u = adapted(*v, sizes, lead=9)
    assert np.array_equal(_np(Y), y) and np.array_equal(_np(U), _bf(u))


@pytest.mark.parametrize("sizes,S", [([900, 0, 700, 300, 77], 2000), ([1, 1, 3000], 3100), ([40] * 60, 2500)])
@pytest.mark.parametrize("R", [16, 64])
@pytest.mark.parametrize("pair", [0, 1, 2])
def test_adapted_long_products(sizes, S, R, pair):
    """u by the tensor cores, its contraction shared, in both kinds of tiles."""
    K, N = 2048, 264
    t, v = _adapters(sizes, K, N, R, 180, S=S)
    y, u = adapted(*v, sizes)
    assert np.abs(u).max() < 2 ** 16 and np.abs(y).max() < 2 ** 24
    for _ in range(2):
        Y, U = tg.gemm_adapted(*t, _offsets(sizes), U=True, options=tg.make_options(cta_pair=pair))
        assert np.array_equal(_np(Y), y) and np.array_equal(_np(U), _bf(u))


@pytest.mark.parametrize("sizes", [[3, 1, 0, 7], [300, 500, 20]])
@pytest.mark.parametrize("R", [16, 40])
@pytest.mark.parametrize("which", ["A", "B", "both"])
def test_adapted_one_matrix_for_every_adapter(sizes, R, which):
    (X, W, A, B), (xv, wv, av, bv) = _adapters(sizes, 72, 136, R, 190)
    E = len(sizes)
    if which != "B":
        A, av = A[:1].expand(E, *A.shape[1:]), np.repeat(av[:1], E, 0)
    if which != "A":
        B, bv = B[:1].expand(E, *B.shape[1:]), np.repeat(bv[:1], E, 0)
    scales = torch.tensor([2.0 ** (i % 3) for i in range(E)], device=dev())
    Y, U = tg.gemm_adapted(X, W, A, B, _offsets(sizes), scales=scales, U=True)
    y, u = adapted(xv, wv, av, bv, sizes, _np(scales))
    assert np.array_equal(_np(Y), y) and np.array_equal(_np(U), _bf(u))


# ---------------------------------------------------------------- all of them
def _calls(S, sizes, seed=100):
    """One call of each operator with preallocated outputs, as functions of
    offsets, and their outputs."""
    K, F, R = 192, 200, 16
    X, _ = _rand((S, K), seed, False)
    W, _ = _rand((len(sizes), K, 2 * F), seed + 1, False)
    V, _ = _rand((len(sizes), F, K), seed + 2, False)
    Z, _ = _rand((S, 2 * F), seed + 3, False)
    A, _ = _rand((len(sizes), R, K), seed + 4, False)
    B, _ = _rand((len(sizes), R, F), seed + 5, False)
    out = [torch.empty(S, n, dtype=t, device=dev()) for n, t in ((F, BF), (2 * F, BF), (2 * F, BF), (F, BF), (F, F32), (R, BF))]
    Wd = W[0, :, :F]

    def run(off, opts=None, out=out):
        tg.gemm_gated(X, W, off, out[0], Z=out[1], options=opts)
        tg.gemm_gated_grad(X, V.transpose(1, 2), Z, off, out[2], H=out[3], options=opts)
        tg.gemm_adapted(X, Wd, A, B, off, out[4], U=out[5], options=opts)
        return [t.clone() for t in out]

    return run, out


def test_bounds_outside_the_rows_are_clamped():
    sizes, S = [30, 70, 0], 100
    run, _ = _calls(S, sizes)
    want = run(_offsets(sizes))
    for bounds in ([0, 30, 2 ** 31 - 1, 2 ** 31 - 1], [-5, 30, 100, 400], [0, 30, 100, -2 ** 31]):
        got = run(torch.tensor(bounds, dtype=torch.int32, device=dev()))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_same_bits_again_graph_and_stream():
    sizes, S = [300, 0, 45, 700], 1045
    off = _offsets(sizes)
    run, out = _calls(S, sizes)
    first = run(off)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = run(off)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run(off)
    for moved in ([300, 0, 45, 700], [0, 1045, 0, 0], [1, 2, 3, 4]):
        off.copy_(_offsets(moved))  # the bounds are read at each replay
        for t in out:
            t.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, run(_offsets(moved)))), moved


@pytest.mark.parametrize("S,sizes", [(1045, [300, 0, 45, 700]), (7, [1, 0, 3, 3])])
def test_packed_operands_give_the_same_bits(S, sizes):
    off = _offsets(sizes)
    run, _ = _calls(S, sizes)
    assert all(torch.equal(a, b) for a, b in zip(run(off), run(off, tg.make_options(force_pack=1))))


@pytest.mark.parametrize("bounds", [[0, 30, 30, 100], [0, 0, 0, 100], [5, 30, 2 ** 31 - 1, 2 ** 31 - 1], [-5, 30, 20, 400], [0, 30, 100, -2 ** 31],
                                    [100, 0, 50, 100], [0, 0, 0, 0]])
def test_packed_operands_of_groups_without_rows(bounds):
    """Matrices that meet no rows are not copied: whatever the bounds are, those
    that the product reads are."""
    run, _ = _calls(100, [30, 70, 0])
    off = torch.tensor(bounds, dtype=torch.int32, device=dev())
    assert all(torch.equal(a, b) for a, b in zip(run(off), run(off, tg.make_options(force_pack=1))))


def test_two_streams_at_once():
    runs = [_calls(S, sizes, seed) for S, sizes, seed in ((700, [300, 400], 110), (900, [1, 899], 120))]
    offs = [_offsets([300, 400]), _offsets([1, 899])]
    want = [run(off) for (run, _), off in zip(runs, offs)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(runs[i][0](offs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for g in got[i] for a, b in zip(g, want[i]))


@pytest.mark.parametrize("pair", [1, 2])
@pytest.mark.parametrize("S,sizes", [(475, [300, 5, 170]), (3, [1, 1, 1])])
@pytest.mark.parametrize("K", [128, 4096])  # whole tiles; shared ones
@pytest.mark.parametrize("op", ["gated", "grad", "adapted"])
def test_watchdog(pair, S, sizes, K, op):
    """A wait that nothing ends runs out after its limit, is reported by
    tg_device_error, and leaves the device and the next call's counters sound."""
    F, R = 192, 8
    X, _ = _rand((S, K), 130)
    W, _ = _rand((3, K, 2 * F), 131)
    V, _ = _rand((3, K, F), 132)
    Z, _ = _rand((S, 2 * F), 133)
    A, _ = _rand((3, R, K), 134)
    B, _ = _rand((3, R, F), 135)
    off = _offsets(sizes)
    call = {"gated": lambda **kw: tg.gemm_gated(X, W, off, activation="none", **kw),
            "grad": lambda **kw: tg.gemm_gated_grad(X, V, Z, off, activation="none", **kw),
            "adapted": lambda **kw: tg.gemm_adapted(X, V[0], A, B, off, **kw)}[op]
    want = call(options=tg.make_options(cta_pair=pair))
    call(options=tg.make_options(cta_pair=pair, debug_stall=1, timeout_ns=20_000_000))
    assert tg.device_error() == tg.TG_ERR_TIMEOUT
    assert tg.device_error() == tg.TG_OK
    got = call(options=tg.make_options(cta_pair=pair))
    assert tg.device_error() == tg.TG_OK
    assert torch.equal(got, want)


def test_checks_build_gives_the_same_bits():
    lib = tg.load_checks()
    sizes, S, K, F, R = [300, 0, 45, 700], 1045, 200, 264, 24
    off = _offsets(sizes)
    X, _ = _rand((S, K), 140, False)
    W, _ = _rand((4, K, 2 * F), 141, False)
    V, _ = _rand((4, K, F), 142, False)
    A, _ = _rand((4, R, K), 143, False)
    B, _ = _rand((4, R, F), 144, False)
    H, Z = tg.gemm_gated(X, W, off, Z=True)
    dZ, H2 = tg.gemm_gated_grad(X, V, Z, off, H=True)
    Y, U = tg.gemm_adapted(X, V[0], A, B, off, U=True)
    o = [torch.empty_like(t) for t in (H, Z, dZ, H2, Y, U)]
    p = [t.data_ptr() for t in o]
    s = torch.cuda.current_stream().cuda_stream
    assert lib.tg_gemm_gated(X.data_ptr(), W.data_ptr(), p[0], p[1], off.data_ptr(), 4, S, F, K, K, 2 * F, 2 * K * F, F, 2 * F, 3, s,
                             None) == tg.TG_OK
    assert lib.tg_gemm_gated_grad(X.data_ptr(), V.data_ptr(), Z.data_ptr(), p[2], p[3], off.data_ptr(), 4, S, F, K, K, F, K * F,
                                  2 * F, 2 * F, F, 3, s, None) == tg.TG_OK
    assert lib.tg_gemm_adapted(X.data_ptr(), V.data_ptr(), A.data_ptr(), B.data_ptr(), p[4], p[5], off.data_ptr(), None, 4, S, F, K,
                               R, K, F, K, R * K, F, R * F, F, R, 0, s, None) == tg.TG_OK
    assert lib.tg_device_error(s) == tg.TG_OK
    assert all(torch.equal(a, b) for a, b in zip((H, Z, dZ, H2, Y, U), o))


def test_rows_past_two_billion_elements():
    """Z and dZ of more than 2^31 elements: the last rows; and an adapted Y."""
    S, K, F = 140000, 32, 8192
    X = torch.zeros(S, K, dtype=BF, device=dev())
    tail, tv = _rand((300, K), 150)
    X[-300:] = tail
    W, wv = _rand((K, 2 * F), 151)
    H, Z = tg.gemm_gated(X, W, Z=True, activation="relu")
    z = tv @ wv
    assert np.array_equal(_np(Z[-300:]), _bf(z)) and np.array_equal(_np(H[-300:]), _bf(_f32(np.maximum(z[:, :F], 0) * z[:, F:])))
    assert not bool(H[:-300].any()) and not bool(Z[:-300].any())
    V, vv = _rand((K, F), 152)
    dZ = tg.gemm_gated_grad(X, V, Z, activation="none")
    dz, _ = _grad_ref("none", tv @ vv, _bf(z), F, in_group(300, [300]))
    assert np.array_equal(_np(dZ[-300:]), _bf(_f32(dz))) and not bool(dZ[:-300].any())
    del H, dZ
    A, av = _rand((2, 8, K), 153)
    B, bv = _rand((2, 8, 2 * F), 154)
    Y = tg.gemm_adapted(X, W, A, B, torch.tensor([0, S - 200, S], dtype=torch.int32, device=dev()), Z)
    y, _ = adapted(tv, wv, av, bv, [100, 200])
    assert np.array_equal(_np(Y[-300:]), _bf(y)) and not bool(Y[:-300].any())
