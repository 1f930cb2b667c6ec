"""Cases of the fused projections of a transformer's feed-forward block: the
gated projection (gate, up, activation and product in one pass), the gradient
through it, and a projection with low-rank adapters of many requests beside
the shared weights.

Every case is one pass through one operator.  With ``own`` false ``run`` is
the operator's plain form (32-bit elementary torch operations, rounded once
at the end); with ``own`` true it is the library's entry point on the same
state.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16
_OUT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
# E = 0: a dense layer; else E groups of consecutive rows (experts, or
# adapters), of which `active` have rows.
def listed():
    return [
        # a handful of decoded tokens through a small block: latency
        {"name": "gated_few", "op": "gated", "S": 5, "E": 0, "active": 0, "K": 640, "F": 384, "act": "silu", "keep": False, "transposed": False},
        # one decoded token through a large block: the weights are the traffic (stored as linear layers store them)
        {"name": "gated_token", "op": "gated", "S": 1, "E": 0, "active": 0, "K": 8192, "F": 14336, "act": "silu", "keep": False, "transposed": True},
        # a training batch: the pre-activations are kept for the backward pass
        {"name": "gated_batch", "op": "gated", "S": 8192, "E": 0, "active": 0, "K": 4096, "F": 8192, "act": "silu", "keep": True, "transposed": False},
        # a prefill batch over gated experts, uneven groups
        {"name": "gated_experts", "op": "gated", "S": 32768, "E": 32, "active": 32, "K": 2048, "F": 2048, "act": "silu", "keep": False, "transposed": False},
        # a few decoded tokens over many experts: two rows an expert, some idle
        {"name": "gated_expert_tokens", "op": "gated", "S": 64, "E": 64, "active": 40, "K": 2048, "F": 1408, "act": "silu", "keep": False, "transposed": False},
        # the backward pass of the training batch, the activations made again for the down weights' gradient
        {"name": "gated_grad_batch", "op": "gated_grad", "S": 8192, "E": 0, "active": 0, "K": 4096, "F": 8192, "act": "silu", "keep": True, "transposed": True},
        # the backward pass over experts, sizes off the tiles
        {"name": "gated_grad_experts", "op": "gated_grad", "S": 5003, "E": 12, "active": 11, "K": 1400, "F": 1000, "act": "silu", "keep": True, "transposed": True},
        # a short odd micro-batch: no row on 16 bytes
        {"name": "gated_grad_odd", "op": "gated_grad", "S": 333, "E": 0, "active": 0, "K": 257, "F": 1001, "act": "gelu_tanh", "keep": False, "transposed": True},
        # one request's token: its adapter beside the shared projection
        {"name": "adapted_token", "op": "adapted", "S": 1, "E": 8, "active": 1, "bare": 0, "K": 4096, "N": 4096, "R": 16, "out": "bf16", "keep": False, "transposed": False},
        # decoding for many requests at once: 40 adapters, a few requests without one
        {"name": "adapted_tokens", "op": "adapted", "S": 64, "E": 64, "active": 40, "bare": 8, "K": 4096, "N": 4096, "R": 16, "out": "bf16", "keep": False, "transposed": False},
        # prompts of a dozen requests, larger adapters
        {"name": "adapted_batch", "op": "adapted", "S": 8192, "E": 16, "active": 12, "bare": 512, "K": 4096, "N": 4096, "R": 64, "out": "bf16", "keep": False, "transposed": False},
        # training adapters: the gradient of the rows (the shared weights read transposed), odd rank, fp32
        {"name": "adapted_grad", "op": "adapted", "S": 1003, "E": 8, "active": 7, "bare": 0, "K": 1400, "N": 1000, "R": 20, "out": "f32", "keep": True, "transposed": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A feature extent: mostly a multiple of 8, as layers have them, now and
    then odd."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.25 else max(8, v // 16 * 16 + 8 * rng.randint(0, 1))


def draw(rng):
    while True:
        op = rng.choice(["gated", "gated_grad", "adapted"])
        S = _log(rng, 1, 32768)
        K = _width(rng, 128, 8192)
        if op == "adapted":
            E = rng.choice([1, 4, 8, 32, 64, 200])
            bare = rng.choice([0, 0, S // 8])
            c = {"op": op, "S": S, "E": E, "active": min(S - bare, max(1, E - rng.randint(0, E // 2))), "bare": bare, "K": K,
                 "N": _width(rng, 128, 8192), "R": rng.choice([4, 8, 16, 16, 20, 32, 64, 128]), "out": rng.choice(["bf16", "bf16", "f32"]),
                 "keep": rng.random() < 0.5, "transposed": rng.random() < 0.5}
            if S * K * c["N"] > 1 << 37 or E * c["R"] * (K + c["N"]) > 1 << 27:
                continue
        else:
            E = rng.choice([0, 0, 4, 8, 12, 32, 64])
            c = {"op": op, "S": S, "E": E, "active": min(S, max(1, E - rng.randint(0, E // 4))) if E else 0, "K": K,
                 "F": _width(rng, 64, 14336), "act": rng.choice(["silu", "silu", "gelu_tanh", "relu", "none"]),
                 "keep": rng.random() < 0.5, "transposed": rng.random() < 0.5}
            if S * K * c["F"] > 1 << 37 or max(1, E) * K * c["F"] > 1 << 28:
                continue
        return c


# ------------------------------------------------------------------ inputs
def _sizes(g, S, E, active):
    """Rows of each group: `active` of the E groups have at least one, the
    rest of the S rows fall on them unevenly."""
    share = torch.rand(active, generator=g, device=DEV).add_(0.25)
    n = torch.ones(active, dtype=torch.long, device=DEV)
    if S > active:
        n += torch.bincount(torch.multinomial(share, S - active, replacement=True, generator=g), minlength=active)
    sizes = torch.zeros(E, dtype=torch.long, device=DEV)
    sizes[torch.randperm(E, generator=g, device=DEV)[:active]] = n
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(sizes, 0)
    return sizes.tolist(), offsets


def _bf16(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device=DEV).mul_(scale).to(BF16)


def _weights(g, lead, K, N, transposed):
    """Weights [*lead, K, N]; transposed: a view of ones stored [*lead, N, K]."""
    if transposed:
        return _bf16(g, *lead, N, K, scale=K ** -0.5).transpose(-1, -2)
    return _bf16(g, *lead, K, N, scale=K ** -0.5)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    S, E, K = case["S"], case["E"], case["K"]
    bare = case.get("bare", 0)
    s["sizes"], s["offsets"] = _sizes(g, S - bare, E, case["active"]) if E else ([S], None)
    s["X"] = _bf16(g, S, K)
    if case["op"] == "adapted":
        N, R = case["N"], case["R"]
        s["W"] = _weights(g, (), K, N, case["transposed"])
        s["A"] = _bf16(g, E, R, K, scale=K ** -0.5)
        s["B"] = _bf16(g, E, R, N, scale=0.3 * R ** -0.5)
        s["scales"] = torch.rand(E, generator=g, device=DEV).add_(0.5)
        s["Y"] = torch.empty(S, N, dtype=_OUT[case["out"]], device=DEV)
        s["U"] = torch.empty(S, R, dtype=BF16, device=DEV) if case["keep"] else None
        return s
    F, lead = case["F"], (E,) if E else ()
    if case["op"] == "gated":
        s["W"] = _weights(g, lead, K, 2 * F, case["transposed"])
        s["Z"] = torch.empty(S, 2 * F, dtype=BF16, device=DEV) if case["keep"] else None
        s["H"] = torch.empty(S, F, dtype=BF16, device=DEV)
    else:
        s["X"] *= 2.0 ** -6  # gradients
        s["W"] = _weights(g, lead, K, F, case["transposed"])
        s["Z"] = _bf16(g, S, 2 * F)
        s["dZ"] = torch.empty(S, 2 * F, dtype=BF16, device=DEV)
        s["H"] = torch.empty(S, F, dtype=BF16, device=DEV) if case["keep"] else None
    return s


# ------------------------------------------------------------------ one pass
def _products(X, W, sizes):
    """X's rows times their group's weights, fp32."""
    if W.dim() == 2:
        return X.float() @ W.float()
    parts = zip(torch.split(X.float(), sizes), W)
    return torch.cat([x @ w.float() for x, w in parts if len(x)])


def _act(act, z):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z.clamp(min=0) if act == "relu" else z


def _slope(act, z):
    """The activation's derivative."""
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return (z > 0).float() if act == "relu" else torch.ones_like(z)


def _run_plain(s):
    op, F = s["op"], s.get("F")
    if op == "gated":
        z = _products(s["X"], s["W"], s["sizes"])
        h = _act(s["act"], z[:, :F]) * z[:, F:]
        return {"H": h.to(BF16), "Z": z.to(BF16)} if s["keep"] else {"H": h.to(BF16)}
    if op == "gated_grad":
        dh = _products(s["X"], s["W"], s["sizes"])
        gate, up = s["Z"][:, :F].float(), s["Z"][:, F:].float()
        a = _act(s["act"], gate)
        out = {"dZ": torch.cat((dh * up * _slope(s["act"], gate), dh * a), 1).to(BF16)}
        if s["keep"]:
            out["H"] = (a * up).to(BF16)
        return out
    S, R, n = s["S"], s["R"], sum(s["sizes"])
    u = torch.zeros(S, R, device=DEV)
    u[:n] = _products(s["X"][:n], s["A"].transpose(1, 2), s["sizes"])
    u[:n] *= torch.repeat_interleave(s["scales"], s["offsets"].diff(), output_size=n)[:, None]
    y = s["X"].float() @ s["W"].float()
    y[:n] += _products(u[:n], s["B"], s["sizes"])
    out = {"Y": y.to(_OUT[s["out"]])}
    if s["keep"]:
        out["U"] = u.to(BF16)
    return out


def _run_own(s):
    import tiled_gemm_codegen_gb300 as tg

    if s["op"] == "gated":
        out = tg.gemm_gated(s["X"], s["W"], s["offsets"], s["H"], Z=s["Z"], activation=s["act"])
        names = ("H", "Z")
    elif s["op"] == "gated_grad":
        out = tg.gemm_gated_grad(s["X"], s["W"], s["Z"], s["offsets"], s["dZ"], H=s["H"], activation=s["act"])
        names = ("dZ", "H")
    else:
        out = tg.gemm_adapted(s["X"], s["W"], s["A"], s["B"], s["offsets"], s["Y"], scales=s["scales"], U=s["U"])
        names = ("Y", "U")
    return dict(zip(names, out)) if s["keep"] else {names[0]: out}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ work
def work(case):
    S, K, used = case["S"], case["K"], case["active"] if case["E"] else 1
    if case["op"] == "adapted":
        N, R = case["N"], case["R"]
        size, rows = 2 if case["out"] == "bf16" else 4, S - case["bare"]
        return {"bytes": 2 * S * K + 2 * K * N + 2 * used * R * (K + N) + size * S * N + (2 * S * R if case["keep"] else 0),
                "flops": 2 * S * K * N + 2 * rows * R * (K + N)}
    F = case["F"]
    if case["op"] == "gated":
        return {"bytes": 2 * S * K + 4 * used * K * F + 2 * S * F + (4 * S * F if case["keep"] else 0), "flops": 4 * S * K * F}
    return {"bytes": 2 * S * K + 2 * used * K * F + 8 * S * F + (2 * S * F if case["keep"] else 0), "flops": 2 * S * K * F}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definitions in 64 bits, a group at a time; None where the 64-bit
    products would take too long."""
    if work(case)["flops"] > 1.2e13:
        return None
    s = prepare(case, seed)
    f64 = torch.float64
    S, E = case["S"], case["E"]
    ends = s["offsets"].tolist() if E else [0, S]
    X = s["X"].to(f64)
    if case["op"] == "adapted":
        Y = X @ s["W"].to(f64)
        U = torch.zeros(S, case["R"], dtype=f64, device=DEV)
        for e in range(E):
            rows = slice(ends[e], ends[e + 1])
            U[rows] = float(s["scales"][e]) * torch.einsum("sk,rk->sr", X[rows], s["A"][e].to(f64))
            Y[rows] += torch.einsum("sr,rn->sn", U[rows], s["B"][e].to(f64))
        return {"Y": Y, "U": U} if case["keep"] else {"Y": Y}
    F = case["F"]
    P = torch.zeros(S, s["W"].shape[-1], dtype=f64, device=DEV)
    for e in range(max(1, E)):
        rows = slice(ends[e], ends[e + 1])
        P[rows] = X[rows] @ (s["W"][e] if E else s["W"]).to(f64)
    gate, up = (P if case["op"] == "gated" else s["Z"].to(f64)).split(F, dim=1)
    act = {"silu": torch.nn.functional.silu, "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh"),
           "relu": torch.relu, "none": lambda z: z}[case["act"]]
    if case["op"] == "gated":
        H = act(gate) * up
        return {"H": H, "Z": P} if case["keep"] else {"H": H}
    with torch.enable_grad():
        leaf = s["Z"].to(f64).requires_grad_()
        H = act(leaf[:, :F]) * leaf[:, F:]
        (dZ,) = torch.autograd.grad(H, leaf, P)
    return {"dZ": dZ, "H": H.detach()} if case["keep"] else {"dZ": dZ}
