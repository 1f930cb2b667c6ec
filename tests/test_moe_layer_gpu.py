"""The example layer, its operators together: forward and gradients against
the same layer in plain 32-bit torch with its own autograd, dropped assignments
and idle experts included, and the 4-bit experts against the values they
stand for.

The plain layer runs in fp32 on the same bf16 operands; what differs is the
rounding to bf16 of z, h, ys, the row gradients and the result (2^-8 of each
value at most, half that on average).  A value behind m such roundings of the
operands of a sum lies within m 2^-8 of the sum of magnitudes; relative to the
Frobenius norm, where roundings of many values add up like independent errors,
m 2^-8 bounds it with room: m = 4 for y (z, h, ys, y), 7 for the gradients
(z, h and ys or dys, dh, dz, the rows and the result)."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

import tiled_gemm_codegen_gb300 as tg

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")
_spec = importlib.util.spec_from_file_location("moe_layer", _PATH)
moe = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(moe)


def _plain(x, weights, ids, up, down):
    y = torch.zeros(x.shape, device=x.device)
    for e in range(up.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        out = torch.nn.functional.silu(x[t] @ up[e]) @ down[e]
        y = y.index_add(0, t, out * weights[t, j, None])
    return y


def _case(T, E, D, H, k, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = r(T, D).bfloat16()
    up, down = (r(E, D, H) * D ** -0.5).bfloat16(), (r(E, H, D) * H ** -0.5).bfloat16()
    ids, weights = moe.route(x, r(D, E - 1) * D ** -0.5, k)  # (the last expert stays idle)
    ids[::7, 0] = -1
    return x, weights, ids, up, down, r(T, D).bfloat16()


def _off(got, want):
    got, want = got.detach().float(), want.detach().float()
    return float((got - want).norm() / want.norm())


@pytest.mark.parametrize("T,E,D,H,k", [(300, 8, 128, 256, 2), (1, 16, 256, 128, 4), (517, 5, 200, 136, 3)])
def test_training_step(T, E, D, H, k):
    x, weights, ids, up, down, dy = _case(T, E, D, H, k)
    ours = [t.clone().requires_grad_() for t in (x, weights, up, down)]
    y = moe.Experts.apply(ours[0], ours[1], ids, ours[2], ours[3])
    y.backward(dy)
    plain = [t.float().clone().requires_grad_() for t in (x, weights, up, down)]
    want = _plain(plain[0], plain[1], ids, plain[2], plain[3])
    want.backward(dy.float())
    assert tg.device_error() == tg.TG_OK
    assert _off(y, want) <= 4 * 2 ** -8
    for a, b in zip(ours, plain):
        assert _off(a.grad, b.grad) <= 7 * 2 ** -8
    assert bool((ours[2].grad[E - 1] == 0).all())  # no row of its own


@pytest.mark.parametrize("T", [1, 3, 40])
def test_decode_with_4_bit_experts(T):
    E, D, H, k = 12, 256, 384, 4
    x, weights, ids, up, down, _ = _case(T, E, D, H, k, seed=T)
    up4, down4 = moe.quantise_int4(up), moe.quantise_int4(down)

    def values(codes, scales):
        q = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:2], -1).float() - 8
        return (q * scales.float().repeat_interleave(128, -1)).transpose(1, 2)

    y = moe.decode(x, weights, ids, up4, down4)
    want = _plain(x.float(), weights, ids, values(*up4), values(*down4))
    assert tg.device_error() == tg.TG_OK
    assert _off(y, want) <= 4 * 2 ** -8
