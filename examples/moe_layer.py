"""A mixture-of-experts layer on the library's operators: a training step
(forward and backward) with bf16 experts, and decoding of a few tokens with the
same experts in 4 bits.

    python examples/moe_layer.py [--tokens 8192] [--experts 32] [--width 1024] [--hidden 2048] [--top-k 4]

prints the loss of a few steps of plain gradient descent, the time of a step,
and the time of one token through the 4-bit experts beside the bf16 ones.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import tiled_gemm_codegen_gb300 as tg  # noqa: E402

BF16 = torch.bfloat16


class Experts(torch.autograd.Function):
    """y[t] = sum_j weights[t, j] * down_e(silu(up_e(x[t]))) with e = ids[t, j], for
    bf16 x [T, D], up [E, D, H] and down [E, H, D]; an id outside [0, E) drops
    its assignment."""

    @staticmethod
    def forward(ctx, x, weights, ids, up, down):
        xs, order = tg.expert_dispatch(x, ids, up.shape[0])
        z = tg.gemm_grouped(xs, up, order.offsets, out_dtype=BF16)
        h = torch.nn.functional.silu(z)
        ys = tg.gemm_grouped(h, down, order.offsets, out_dtype=BF16)
        ctx.order = order
        ctx.save_for_backward(xs, z, h, ys, weights, up, down)
        return tg.expert_combine(ys, order, weights)

    @staticmethod
    def backward(ctx, dy):
        xs, z, h, ys, weights, up, down = ctx.saved_tensors
        order, off = ctx.order, ctx.order.offsets
        dys, dweights = tg.expert_combine_grad(dy.contiguous(), ys, order, weights)
        dh = tg.gemm_grouped(dys, down.transpose(1, 2), off, out_dtype=BF16)
        ddown = tg.gemm_grouped_wgrad(h, dys, off, out_dtype=BF16)
        s = torch.sigmoid(z.float())
        dz = (dh.float() * s * (1 + z.float() * (1 - s))).to(BF16)
        dxs = tg.gemm_grouped(dz, up.transpose(1, 2), off, out_dtype=BF16)
        dup = tg.gemm_grouped_wgrad(xs, dz, off, out_dtype=BF16)
        return tg.expert_combine(dxs, order), dweights, None, dup, ddown


def route(x, router, k):
    """(ids, weights): the k best experts of each token, their softmax."""
    top, ids = torch.topk(x.float() @ router, k, dim=-1)
    return ids, torch.softmax(top, dim=-1)


def quantise_int4(w, group=128):
    """(codes [E, N, K / 2], scales [E, N, K / group]) of experts w [E, K, N]:
    symmetric codes about 8, a bf16 scale for `group` inputs of an output."""
    t = w.transpose(1, 2).float()
    E, N, K = t.shape
    g = t.reshape(E, N, K // group, group)
    scales = (g.abs().amax(-1) / 7).clamp(min=1e-12).to(BF16)
    q = (torch.round(g / scales.float()[..., None]) + 8).clamp(0, 15).to(torch.uint8).reshape(E, N, K)
    return (q[..., 0::2] | q[..., 1::2] << 4).contiguous(), scales


def decode(x, weights, ids, up4, down4):
    """The same layer for a few tokens on experts quantised by quantise_int4."""
    (up_codes, up_scales), (down_codes, down_scales) = up4, down4
    xs, order = tg.expert_dispatch(x, ids, up_codes.shape[0])
    z = tg.gemv_w4(xs, up_codes, up_scales, offsets=order.offsets, out_dtype=BF16)
    ys = tg.gemv_w4(torch.nn.functional.silu(z), down_codes, down_scales, offsets=order.offsets, out_dtype=BF16)
    return tg.expert_combine(ys, order, weights)


def _us(f, n=50):
    for _ in range(5):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) * 1e3 / n


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 8192), ("experts", 32), ("width", 1024), ("hidden", 2048), ("top-k", 4), ("steps", 5)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    tg.load()
    torch.manual_seed(0)
    dev = "cuda"
    router = torch.randn(a.width, a.experts, device=dev) * a.width ** -0.5
    up = (torch.randn(a.experts, a.width, a.hidden, device=dev) * a.width ** -0.5).to(BF16).requires_grad_()
    down = (torch.randn(a.experts, a.hidden, a.width, device=dev) * a.hidden ** -0.5).to(BF16).requires_grad_()
    x = torch.randn(a.tokens, a.width, device=dev).to(BF16)
    target = torch.randn(a.tokens, a.width, device=dev).to(BF16)
    ids, weights = route(x, router, a.top_k)

    def step():
        y = Experts.apply(x, weights, ids, up, down)
        loss = (y.float() - target.float()).square().mean()
        up.grad = down.grad = None
        loss.backward()
        return loss

    for i in range(a.steps):
        loss = step()
        with torch.no_grad():
            up -= 3e2 * up.grad
            down -= 3e2 * down.grad
        print(f"step {i}: loss {loss.item():.4f}")
    print(f"a step: {_us(step, 10):.0f} us for {a.tokens} tokens x {a.top_k} of {a.experts} experts")
    with torch.no_grad():
        up4, down4 = quantise_int4(up), quantise_int4(down)
        one, one_ids, one_w = x[:1], ids[:1], weights[:1].contiguous()
        y4 = decode(one, one_w, one_ids, up4, down4).float()
        y16 = Experts.apply(one, one_w, one_ids, up, down).float()
        print(f"one token: 4-bit experts {_us(lambda: decode(one, one_w, one_ids, up4, down4)):.1f} us, "
              f"bf16 experts {_us(lambda: Experts.apply(one, one_w, one_ids, up, down)):.1f} us, "
              f"difference {float((y4 - y16).norm() / y16.norm()):.3f}")
    if tg.device_error() != tg.TG_OK:
        raise SystemExit("device error")


if __name__ == "__main__":
    main()
