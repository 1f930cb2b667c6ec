"""Cases of the mixture-of-experts operators: tokens sorted by expert and back
(with weights, and the gradient), the experts' ragged products in every
direction, and products with 4-bit weights for single tokens.

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
_OUT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token of a layer with many small experts: latency
        {"name": "dispatch_token", "op": "dispatch", "T": 1, "k": 8, "E": 64, "D": 2048, "drop": 0.0},
        # a prefill or training batch; a few assignments over capacity are dropped
        {"name": "dispatch_batch", "op": "dispatch", "T": 16384, "k": 8, "E": 128, "D": 2048, "drop": 0.02},
        # a handful of decoded tokens, hidden size off every vector width
        {"name": "combine_tokens", "op": "combine", "T": 5, "k": 2, "E": 8, "D": 1001, "drop": 0.0},
        # a prefill batch of a wide model
        {"name": "combine_batch", "op": "combine", "T": 16384, "k": 4, "E": 64, "D": 4096, "drop": 0.02},
        # the backward pass of a training batch: row gradients and router-weight gradients
        {"name": "combine_grad_batch", "op": "combine_grad", "T": 8191, "k": 8, "E": 128, "D": 2056, "drop": 0.02},
        # the experts' up projection over a training batch, uneven groups
        {"name": "rows_batch", "op": "rows", "S": 32768, "E": 32, "active": 32, "K": 2048, "N": 4096, "transposed": False},
        # a few decoded tokens: two rows an expert, some experts idle; the weights are the traffic
        {"name": "rows_tokens", "op": "rows", "S": 64, "E": 64, "active": 40, "K": 2048, "N": 1408, "transposed": False},
        # the data gradient of a middling batch (weights read transposed), sizes off the tiles
        {"name": "rows_dgrad", "op": "rows", "S": 5003, "E": 12, "active": 11, "K": 1400, "N": 1000, "transposed": True},
        # the weight gradient of a training batch, in the weights' type
        {"name": "wgrad_batch", "op": "wgrad", "S": 32768, "E": 16, "active": 16, "K": 2048, "N": 2048, "out": "bf16"},
        # the weight gradient of a short ragged micro-batch, an idle expert; fp32, to be summed over micro-batches
        {"name": "wgrad_ragged", "op": "wgrad", "S": 1003, "E": 8, "active": 7, "K": 640, "N": 384, "out": "f32"},
        # one decoded token through a large 4-bit projection
        {"name": "w4_token", "op": "w4", "S": 1, "E": 1, "active": 1, "K": 8192, "N": 28672, "format": "int4", "G": 128},
        # a few decoded tokens through 4-bit experts
        {"name": "w4_experts", "op": "w4", "S": 32, "E": 64, "active": 20, "K": 2048, "N": 1408, "format": "e2m1", "G": 32},
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
        op = rng.choice(["dispatch", "combine", "combine_grad", "rows", "wgrad", "w4"])
        if op in ("dispatch", "combine", "combine_grad"):
            E = rng.choice([8, 16, 60, 64, 128, 256])
            c = {"op": op, "T": _log(rng, 1, 32768), "k": rng.randint(1, min(8, E)), "E": E, "D": _width(rng, 64, 8192),
                 "drop": rng.choice([0.0, 0.0, 0.02, 0.3])}
            cap = 16384 * 8 * 2048 // (2 if op == "combine_grad" else 1)
            if c["T"] * c["k"] * c["D"] > cap:
                continue
        elif op in ("rows", "wgrad"):
            E = rng.choice([1, 4, 8, 12, 32, 64, 128])
            S = _log(rng, 1, 32768)
            c = {"op": op, "S": S, "E": E, "active": min(S, max(1, E - rng.randint(0, E // 4))),
                 "K": _width(rng, 128, 4096), "N": _width(rng, 128, 4096)}
            if op == "rows":
                c["transposed"] = rng.random() < 0.5
            else:  # short micro-batches keep their gradients in fp32, to be summed
                c["out"] = "f32" if S // c["active"] < 256 else "bf16"
            if S * c["K"] * c["N"] > 32768 * 2048 * 4096 or E * c["K"] * c["N"] > 1 << 27:
                continue
        else:
            E = rng.choice([1, 1, 8, 64, 128])
            S = _log(rng, 1, 16 if E == 1 else 64)
            fmt = rng.choice(["int4", "int4_zeros", "e2m1"])
            c = {"op": op, "S": S, "E": E, "active": min(S, E, rng.randint(1, E)), "K": _log(rng, 128, 8192) // 2 * 2,
                 "N": _log(rng, 128, 28672), "format": fmt, "G": 32 if fmt == "e2m1" else rng.choice([32, 64, 128])}
            if rng.random() < 0.75:
                c["K"] = max(128, c["K"] // 128 * 128)
            if E * c["K"] * c["N"] > 1 << 29:
                continue
        if 3 << 10 not in c.values():  # a width that no configuration here has
            return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _route(g, T, k, E, drop):
    """Router logits with popular and unpopular experts, top k of them with
    softmax weights; a dropped assignment has id -1."""
    logits = torch.randn(T, E, generator=g, device=DEV) + 0.7 * torch.randn(E, generator=g, device=DEV)
    top, ids = torch.topk(logits, k, dim=-1)
    weights = torch.softmax(top, dim=-1)
    if drop:
        ids = ids.masked_fill(torch.rand(T, k, generator=g, device=DEV) < drop, -1)
    return ids, weights


def _plain_order(ids, E):
    """(offsets, source, slot) of ids [T, k]: a stable sort by expert,
    dropped assignments behind all experts."""
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    by_expert, source = torch.sort(key, stable=True)
    offsets = torch.searchsorted(by_expert, torch.arange(E + 1, device=ids.device))
    at = torch.arange(flat.numel(), device=ids.device)
    slot = torch.empty_like(source)
    slot[source] = at
    slot = torch.where(key < E, slot, -1)
    source = torch.where(by_expert < E, source, -1)
    return offsets.int(), source.int(), slot.int().reshape(ids.shape)


def _sizes(g, S, E, active):
    """Rows of each group: `active` of the E groups have at least one, the
    rest of the S rows fall on them unevenly."""
    share = torch.rand(active, generator=g, device=DEV).add_(0.25)
    extra = torch.multinomial(share, S - active, replacement=True, generator=g) if S > active else None
    n = torch.ones(active, dtype=torch.long, device=DEV)
    if extra is not None:
        n += torch.bincount(extra, minlength=active)
    sizes = torch.zeros(E, dtype=torch.long, device=DEV)
    sizes[torch.randperm(E, generator=g, device=DEV)[:active]] = n
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(sizes, 0)
    return sizes.tolist(), offsets


def _bf16(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device=DEV).mul_(scale).to(torch.bfloat16)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    if op in ("dispatch", "combine", "combine_grad"):
        T, k, E, D = case["T"], case["k"], case["E"], case["D"]
        s["ids"], s["weights"] = _route(g, T, k, E, case["drop"])
        if op == "dispatch":
            s["x"] = _bf16(g, T, D)
        else:
            s["offsets"], s["source"], s["slot"] = _plain_order(s["ids"], E)
            s["ys"] = _bf16(g, T * k, D)
            if op == "combine_grad":
                s["dy"] = _bf16(g, T, D)
        if own:
            import tiled_gemm_codegen_gb300 as tg

            if op == "dispatch":
                s["order"] = tg.ExpertOrder.empty(T, k, E, DEV)
                s["xs"] = torch.empty(T * k, D, dtype=torch.bfloat16, device=DEV)
            else:
                s["order"] = tg.ExpertOrder(s["offsets"], s["source"], s["slot"])
                if op == "combine":
                    s["y"] = torch.empty(T, D, dtype=torch.bfloat16, device=DEV)
                else:
                    s["dys"] = torch.empty(T * k, D, dtype=torch.bfloat16, device=DEV)
                    s["dweights"] = torch.empty(T, k, device=DEV)
        return s
    S, E, K, N = case["S"], case["E"], case["K"], case["N"]
    s["sizes"], s["offsets"] = _sizes(g, S, E, case["active"])
    if op == "rows":
        s["A"] = _bf16(g, S, K)
        s["B"] = _bf16(g, E, N, K, scale=K ** -0.5).transpose(1, 2) if case["transposed"] else _bf16(g, E, K, N, scale=K ** -0.5)
        s["D"] = torch.empty(S, N, dtype=torch.bfloat16, device=DEV) if own else None
    elif op == "wgrad":
        s["A"] = _bf16(g, S, K)
        s["B"] = _bf16(g, S, N)
        s["D"] = torch.empty(E, K, N, dtype=_OUT[case["out"]], device=DEV) if own else None
    else:
        G = case["G"]
        s["x"] = _bf16(g, S, K)
        groups = -(-K // G)
        s["W"] = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
        s["zeros"] = None
        if case["format"] == "e2m1":
            # powers of two about K**-0.5 / 3
            mid = 127 - int(round(math.log2(3 * K ** 0.5)))
            s["scales"] = torch.randint(mid - 1, mid + 2, (E, N, groups), generator=g, device=DEV, dtype=torch.uint8)
        else:
            s["scales"] = (torch.rand(E, N, groups, generator=g, device=DEV) + 0.5).mul_(0.22 * K ** -0.5).to(torch.bfloat16)
            if case["format"] == "int4_zeros":
                s["zeros"] = torch.randint(5, 11, (E, N, groups), generator=g, device=DEV, dtype=torch.uint8)
        s["y"] = torch.empty(S, N, dtype=torch.bfloat16, device=DEV) if own else None
    return s


# ------------------------------------------------------------------ one pass
def _dequant(s, e, dtype):
    """Group e's weights [N, K] as the values they stand for."""
    W, K, G = s["W"][e], s["K"], s["G"]
    q = torch.stack((W & 15, W >> 4), dim=-1).reshape(W.shape[0], K)
    if s["format"] == "e2m1":
        codes = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=dtype, device=W.device)
        v = torch.cat((codes, -codes))[q.long()]
        sc = torch.exp2(s["scales"][e].to(dtype) - 127)
    else:
        z = s["zeros"][e].repeat_interleave(G, 1)[:, :K].to(dtype) if s["zeros"] is not None else 8
        v = q.to(dtype) - z
        sc = s["scales"][e].to(dtype)
    return v * sc.repeat_interleave(G, 1)[:, :K]


def _run_plain(s):
    op = s["op"]
    if op == "dispatch":
        offsets, source, slot = _plain_order(s["ids"], s["E"])
        xs = s["x"][source.clamp(min=0).long() // s["k"]]
        xs = xs.masked_fill((source < 0)[:, None], 0)
        return {"xs": xs, "offsets": offsets, "source": source, "slot": slot}
    if op == "combine":
        slot = s["slot"].long()
        w = torch.where(slot >= 0, s["weights"], 0.0)
        return {"y": (s["ys"].float()[slot.clamp(min=0)] * w[:, :, None]).sum(1).to(torch.bfloat16)}
    if op == "combine_grad":
        dy, ys, slot, source = s["dy"].float(), s["ys"].float(), s["slot"].long(), s["source"].long()
        f = source.clamp(min=0)
        w = torch.where(source >= 0, s["weights"].reshape(-1)[f], 0.0)
        dys = (dy[f // s["k"]] * w[:, None]).to(torch.bfloat16)
        dot = (dy[:, None] * ys[slot.clamp(min=0)]).sum(-1)
        return {"dys": dys, "dweights": torch.where(slot >= 0, dot, 0.0)}
    if op == "rows":
        out, at = [], 0
        A = s["A"].float()
        for e, n in enumerate(s["sizes"]):
            if n:
                out.append(A[at:at + n] @ s["B"][e].float())
            at += n
        return {"D": torch.cat(out).to(torch.bfloat16)}
    if op == "wgrad":
        out, at = [], 0
        A, B = s["A"].float(), s["B"].float()
        for n in s["sizes"]:
            out.append(A[at:at + n].t() @ B[at:at + n])
            at += n
        return {"D": torch.stack(out).to(_OUT[s["out"]])}
    out, at = [], 0
    x = s["x"].float()
    for e, n in enumerate(s["sizes"]):
        if n:
            out.append(x[at:at + n] @ _dequant(s, e, torch.float32).t())
        at += n
    return {"y": torch.cat(out).to(torch.bfloat16)}


def _run_own(s):
    import tiled_gemm_codegen_gb300 as tg

    op = s["op"]
    if op == "dispatch":
        xs, order = tg.expert_dispatch(s["x"], s["ids"], s["E"], xs=s["xs"], order=s["order"])
        return {"xs": xs, "offsets": order.offsets, "source": order.source, "slot": order.slot}
    if op == "combine":
        return {"y": tg.expert_combine(s["ys"], s["order"], s["weights"], y=s["y"])}
    if op == "combine_grad":
        dys, dw = tg.expert_combine_grad(s["dy"], s["ys"], s["order"], s["weights"], dys=s["dys"], dweights=s["dweights"])
        return {"dys": dys, "dweights": dw}
    if op == "rows":
        return {"D": tg.gemm_grouped(s["A"], s["B"], s["offsets"], s["D"])}
    if op == "wgrad":
        return {"D": tg.gemm_grouped_wgrad(s["A"], s["B"], s["offsets"], s["D"])}
    fmt = "e2m1" if s["format"] == "e2m1" else "int4"
    return {"y": tg.gemv_w4(s["x"], s["W"], s["scales"], zeros=s["zeros"], offsets=s["offsets"], y=s["y"],
                            format=fmt, group=s["G"])}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op in ("dispatch", "combine", "combine_grad"):
        T, k, E, D = case["T"], case["k"], case["E"], case["D"]
        rows, flat = T * k * D * 2, T * k
        kept = rows * (1 - case["drop"])
        if op == "dispatch":  # ids are 8 bytes, as topk gives them
            return {"bytes": 8 * flat + 2 * T * D + rows + 8 * flat + 4 * (E + 1), "flops": 0}
        if op == "combine":
            return {"bytes": 8 * flat + kept + 2 * T * D, "flops": 2 * flat * D}
        return {"bytes": 8 * flat + 2 * T * D + kept + rows + 4 * flat, "flops": 3 * flat * D}
    S, E, K, N, used = case["S"], case["E"], case["K"], case["N"], case["active"]
    if op == "rows":
        return {"bytes": 2 * S * K + 2 * used * K * N + 2 * S * N, "flops": 2 * S * K * N}
    if op == "wgrad":
        size = 2 if case["out"] == "bf16" else 4
        return {"bytes": 2 * S * K + 2 * S * N + size * E * K * N, "flops": 2 * S * K * N}
    per = {"int4": 2, "int4_zeros": 3, "e2m1": 1}[case["format"]]
    return {"bytes": 2 * S * K + used * N * (K // 2 + per * -(-K // case["G"])) + 2 * S * N, "flops": 2 * S * K * N}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definitions in 64 bits: one expert, or one choice of the k, at a
    time, with the order found by counting."""
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "dispatch":
        T, k, E = case["T"], case["k"], case["E"]
        flat = s["ids"].reshape(-1).cpu()
        offsets, source = [0], []
        slot = torch.full((T * k,), -1, dtype=torch.int32)
        for e in range(E):
            mine = torch.nonzero(flat == e).reshape(-1)
            slot[mine] = torch.arange(len(mine), dtype=torch.int32) + offsets[-1]
            source.append(mine)
            offsets.append(offsets[-1] + len(mine))
        source = torch.cat(source)
        xs = torch.zeros(T * k, case["D"], dtype=f64, device=DEV)
        xs[:len(source)] = s["x"].to(f64)[torch.div(source, k, rounding_mode="floor").to(DEV)]
        whole = torch.full((T * k,), -1, dtype=torch.int32)
        whole[:len(source)] = source.int()
        return {"xs": xs, "offsets": torch.tensor(offsets, dtype=torch.int32), "source": whole, "slot": slot.reshape(T, k)}
    if op == "combine":
        y = torch.zeros(case["T"], case["D"], dtype=f64, device=DEV)
        for j in range(case["k"]):
            t = torch.nonzero(s["slot"][:, j] >= 0).reshape(-1)
            y[t] += s["weights"][t, j, None].to(f64) * s["ys"][s["slot"][t, j].long()].to(f64)
        return {"y": y}
    if op == "combine_grad":
        dys = torch.zeros(s["ys"].shape, dtype=f64, device=DEV)
        dw = torch.zeros(s["weights"].shape, dtype=f64, device=DEV)
        for j in range(case["k"]):
            t = torch.nonzero(s["slot"][:, j] >= 0).reshape(-1)
            at = s["slot"][t, j].long()
            d = s["dy"][t].to(f64)
            dys[at] = s["weights"][t, j, None].to(f64) * d
            dw[t, j] = (d * s["ys"][at].to(f64)).sum(-1)
        return {"dys": dys, "dweights": dw}
    ends = s["offsets"].tolist()
    if op == "rows":
        D = torch.zeros(case["S"], case["N"], dtype=f64, device=DEV)
        for e in range(case["E"]):
            rows = slice(ends[e], ends[e + 1])
            D[rows] = s["A"][rows].to(f64) @ s["B"][e].to(f64)
        return {"D": D}
    if op == "wgrad":
        D = torch.zeros(case["E"], case["K"], case["N"], dtype=f64, device=DEV)
        for e in range(case["E"]):
            rows = slice(ends[e], ends[e + 1])
            D[e] = s["A"][rows].to(f64).t() @ s["B"][rows].to(f64)
        return {"D": D}
    K, G = case["K"], case["G"]
    y = torch.zeros(case["S"], case["N"], dtype=f64, device=DEV)
    values = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    for e in range(case["E"]):
        rows = slice(ends[e], ends[e + 1])
        if rows.start == rows.stop:
            continue
        W = s["W"][e]
        w = torch.empty(W.shape[0], K, dtype=f64, device=DEV)
        for half in range(2):  # element k of a row: the low nibble of byte k // 2 for even k
            q = (W >> (4 * half)) & 15
            if case["format"] == "e2m1":
                v = torch.zeros(q.shape, dtype=f64, device=DEV)
                for code, value in enumerate(values):
                    v += value * (q == code) - value * (q == code + 8)
            else:
                v = q.to(f64)
            w[:, half::2] = v
        for at in range(0, K, G):
            sc = s["scales"][e][:, at // G, None].to(f64)
            if case["format"] == "e2m1":
                w[:, at:at + G] *= 2.0 ** (sc - 127)
            else:
                zero = s["zeros"][e][:, at // G, None].to(f64) if s["zeros"] is not None else 8.0
                w[:, at:at + G] = (w[:, at:at + G] - zero) * sc
        y[rows] = s["x"][rows].to(f64) @ w.t()
    return {"y": y}
