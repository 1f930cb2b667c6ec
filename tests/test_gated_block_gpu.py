"""The example block, the projections together as they are used: forward and
gradients against the same block in plain 32-bit torch with its own autograd,
rows of no adapter and adapters of no rows included; the step in a captured
graph; and the script.

The plain block runs in fp32 on the same bf16 operands; what differs is the
rounding to bf16 of what is stored between the calls (2^-8 of each value at
most).  A value behind m such roundings of the operands of a sum lies within m
2^-8 of the sum of magnitudes; relative to the Frobenius norm, where roundings of
many values add up like independent errors, m 2^-8 bounds it with room: m = 3 for
y (p, h, y), at most 8 for the gradients (p, z, dy's h or dz, dp, u or du, the
rows and the result)."""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys

import pytest
import torch

import tiled_gemm_codegen_gb300 as tg

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_block.py")
_spec = importlib.util.spec_from_file_location("gated_block", _PATH)
gb = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(gb)


def _plain(x, ids, weights, adapters):
    W, gate_up, down = weights
    A, B, scales = adapters
    p = x @ W.t()
    for g in range(A.shape[0]):
        t = torch.nonzero(ids == g)[:, 0]
        p = p.index_add(0, t, scales[g] * (x[t] @ A[g].t()) @ B[g])
    gate, up = (p @ gate_up.t()).chunk(2, -1)
    return (torch.nn.functional.silu(gate) * up) @ down.t()


def _case(S, D, F, E, R, seed=0):
    torch.manual_seed(seed)
    weights, (A, B, scales) = gb.make(D, F, E, R)
    B = (torch.randn(B.shape, device="cuda") * 0.5).bfloat16()
    x, dy = torch.randn(S, D, device="cuda").bfloat16(), torch.randn(S, D, device="cuda").bfloat16()
    ids = torch.randint(0, max(E - 1, 1), (S,), device="cuda")  # (the last adapter of several stays idle)
    ids[::5] = -1
    if S == 1:
        ids[:] = 0
    return x, ids, weights, (A, B, scales), dy


def _off(got, want):
    got, want = got.detach().float(), want.detach().float()
    return float((got - want).norm() / want.norm())


@pytest.mark.parametrize("S,D,F,E,R", [(300, 256, 512, 6, 16), (1, 512, 384, 3, 8), (517, 200, 328, 40, 20), (2500, 128, 256, 4, 64)])
def test_training_step(S, D, F, E, R):
    x, ids, weights, (A, B, scales), dy = _case(S, D, F, E, R)
    ours = [t.clone().requires_grad_() for t in (x, A, B, *weights[1:])]
    y = gb.block(ours[0], ids, (weights[0], *ours[3:]), (ours[1], ours[2], scales))
    y.backward(dy)
    plain = [t.float().clone().requires_grad_() for t in (x, A, B, *weights[1:])]
    want = _plain(plain[0], ids, (weights[0].float(), *plain[3:]), (plain[1], plain[2], scales))
    want.backward(dy.float())
    assert tg.device_error() == tg.TG_OK
    assert _off(y, want) <= 3 * 2 ** -8
    for a, b in zip(ours, plain):
        assert _off(a.grad, b.grad) <= 8 * 2 ** -8
    idle = [g for g in range(E) if not bool((ids == g).any())]
    assert all(not bool(t.grad[idle].any()) for t in ours[1:3])  # no row of their own


def test_gradient_the_same_for_every_row():
    """A sum's gradient arrives expanded: one row's memory for all."""
    x, ids, weights, (A, B, scales), _ = _case(70, 128, 192, 3, 8)
    grads = []
    for dy in (None, torch.ones(70, 128, device="cuda").bfloat16()):
        t = [v.clone().requires_grad_() for v in (x, A, B)]
        y = gb.block(t[0], ids, weights, (t[1], t[2], scales))
        (y.sum() if dy is None else (y * dy).sum()).backward()
        grads.append([v.grad for v in t])
    assert all(torch.equal(a, b) for a, b in zip(*grads))


def test_block_of_tokens_in_a_graph():
    """A token of each request, captured once: new rows and ids at each replay."""
    x, ids, weights, adapters, _ = _case(12, 256, 384, 5, 16)
    with torch.no_grad():
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            gb.block(x, ids, weights, adapters)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = gb.block(x, ids, weights, adapters)
        for seed in (1, 2):
            x2, _, _, _, _ = _case(12, 256, 384, 5, 16, seed)
            x.copy_(x2), ids.copy_(torch.arange(12, device="cuda") % 7 - seed)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, gb.block(x, ids, weights, adapters))
            want = _plain(x.float(), ids, [w.float() for w in weights], (adapters[0].float(), adapters[1].float(), adapters[2]))
            assert _off(out, want) <= 3 * 2 ** -8


def test_script_runs():
    r = subprocess.run([sys.executable, _PATH, "--tokens", "300", "--width", "256", "--hidden", "384", "--adapters", "4", "--steps", "2"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "a token of each of 4 adapters" in r.stdout and "nan" not in r.stdout
