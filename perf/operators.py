"""The operators of a layer whose FFN is a mixture of ternary experts: cases, plain forms and calls.

Four operators, as a layer runs them one after the other:

* ``norm``    residual addition, root-mean-square norm, 128-point Hadamard rotation and int8
              quantisation with one fp32 scale per 128-element block (``tq.add_rmsnorm_rotq``);
* ``route``   the router: top-k of the experts' logits with softmax weights, and the slots sorted by
              expert (``tq.moe_route``, ``tq.moe_plan``);
* ``gateup``, ``down``  products grouped by expert, ragged in rows: SiLU(gate) * up as bf16
              (``tq.moe_gateup``) and a single product as fp32 (``tq.moe_gemv``);
* ``layer``   all of it: the norm, the router, both products and the weighted sum of each token's
              experts (``tq.add_rmsnorm_rotq``, ``tq.moe_route``, ``tq.moe_ffn``).

``own`` chooses between the plain torch forms and the library's calls; both take the same state.
Weights are packed as include/tq.h lays them out: 2-bit codes (0 -> 0, 1 -> +1, 2 -> -1) four to a
byte or 1-bit codes (1 -> +1, 0 -> -1) eight to a byte, with one fp16 scale per 128-block and row.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
EPS = float(np.float32(1e-6))     # the calls take it as binary32


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # one decoded token of the dense stack's width; and a prefill block of it
        {"name": "norm_m1", "op": "norm", "m": 1, "hidden": 5120, "res": "f32", "delta": "f32", "gamma": True},
        {"name": "norm_m8192", "op": "norm", "m": 8192, "hidden": 5120, "res": "bf16", "delta": "bf16", "gamma": True},
        # routing of a small decode batch, and of a prefill block over many experts with some masked
        {"name": "route_m8", "op": "route", "m": 8, "experts": 64, "topk": 8, "logits": "f32", "masked": 0.0},
        {"name": "route_m16384", "op": "route", "m": 16384, "experts": 256, "topk": 8, "logits": "bf16", "masked": 0.02},
        # gate/up of one token, of an odd verify block of 1-bit weights, and of a prefill block
        {"name": "gateup_m1", "op": "gateup", "m": 1, "hidden": 2048, "inter": 1024, "experts": 64, "topk": 8, "fmt": 0, "skew": 0.0},
        {"name": "gateup_m33_1bit", "op": "gateup", "m": 33, "hidden": 2048, "inter": 1024, "experts": 64, "topk": 6, "fmt": 1, "skew": 0.5},
        {"name": "gateup_m4096", "op": "gateup", "m": 4096, "hidden": 2048, "inter": 1024, "experts": 64, "topk": 8, "fmt": 0, "skew": 0.5},
        # the second product of a decode batch, and of a ragged middle-sized block
        {"name": "down_m8", "op": "down", "m": 8, "hidden": 5120, "inter": 1536, "experts": 32, "topk": 4, "fmt": 0, "skew": 0.0},
        {"name": "down_m500", "op": "down", "m": 500, "hidden": 2048, "inter": 768, "experts": 128, "topk": 8, "fmt": 0, "skew": 0.7},
        # whole layers: one token, a packed decode batch, and a prefill block (the largest)
        {"name": "layer_m1", "op": "layer", "m": 1, "hidden": 2048, "inter": 1024, "experts": 64, "topk": 8, "fmt": 0, "skew": 0.0},
        {"name": "layer_m64", "op": "layer", "m": 64, "hidden": 5120, "inter": 1536, "experts": 32, "topk": 4, "fmt": 1, "skew": 0.3},
        {"name": "layer_m4096", "op": "layer", "m": 4096, "hidden": 5120, "inter": 1536, "experts": 64, "topk": 8, "fmt": 0, "skew": 0.3},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "route", "gateup", "down", "layer"])
    if op == "norm":
        return {"op": op, "m": _log_int(rng, 1, 8192), "hidden": BLOCK * rng.randint(1, 40),
                "res": rng.choice(["f32", "bf16"]), "delta": rng.choice(["f32", "bf16"]),
                "gamma": rng.random() < 0.7}
    experts = _log_int(rng, 2, 256 if op == "route" else 128)
    topk = rng.randint(1, min(8, experts))
    if op == "route":
        return {"op": op, "m": _log_int(rng, 1, 16384), "experts": experts, "topk": topk,
                "logits": rng.choice(["f32", "bf16"]), "masked": rng.choice([0.0, 0.02, 0.3])}
    hidden, inter = BLOCK * _log_int(rng, 2, 40), BLOCK * _log_int(rng, 1, 12)
    m = _log_int(rng, 1, 4096)
    most = 4096 * 8 * 5120 * 1536
    m = max(1, min(m, most // (topk * hidden * inter)))
    return {"op": op, "m": m, "hidden": hidden, "inter": inter, "experts": experts, "topk": topk,
            "fmt": rng.randint(0, 1), "skew": rng.choice([0.0, 0.3, 0.7, 1.2])}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _codes(g, experts, n, k, fmt):
    """Packed random codes [experts][n][k/4 or k/8]; 2-bit codes 0, 1, 2 in about equal parts."""
    if fmt == 1:
        return torch.randint(0, 256, (experts, n, k // 8), generator=g, device="cuda", dtype=torch.uint8)
    v = torch.arange(81, device="cuda")
    table = (v % 3 + 4 * (v // 3 % 3) + 16 * (v // 9 % 3) + 64 * (v // 27)).to(torch.uint8)
    out = torch.empty((experts, n, k // 4), device="cuda", dtype=torch.uint8)
    step = max(1, (1 << 26) // (n * (k // 4)))
    for e in range(0, experts, step):
        part = out[e:e + step]
        part.copy_(table[torch.randint(0, 81, part.shape, generator=g, device="cuda", dtype=torch.int32)])
    return out


def _experts(g, experts, n, k, fmt):
    scales = (0.01 + 0.04 * torch.rand((experts, n, k // BLOCK), generator=g, device="cuda")).half()
    return {"codes": _codes(g, experts, n, k, fmt), "scales": scales, "experts": experts, "n": n, "k": k, "fmt": fmt}


def _quantised(g, m, k):
    """int8 activations with a scale per block, as a quantiser of normal values leaves them."""
    x = torch.randn((m, k // BLOCK, BLOCK), generator=g, device="cuda")
    s = x.abs().amax(-1, keepdim=True) / 127
    q = torch.round(x / s).clamp(-127, 127).to(torch.int8)
    return q.view(m, k), s.view(m, k // BLOCK).contiguous()


def _logits(g, m, experts, skew, dtype=torch.float32):
    """Router logits; `skew` > 0 makes some experts more popular than others."""
    pop = -skew * torch.log(torch.arange(1, experts + 1, device="cuda", dtype=torch.float32))
    pop = pop[torch.randperm(experts, generator=g, device="cuda")]
    return (torch.randn((m, experts), generator=g, device="cuda") + pop).to(dtype)


def _types(case, key):
    return torch.bfloat16 if case[key] == "bf16" else torch.float32


def prepare(case, seed):
    g, op, m = _gen(seed), case["op"], case["m"]
    st = {"case": case}
    if op in ("norm", "layer"):
        h = case["hidden"]
        res, delta = (_types(case, "res"), _types(case, "delta")) if op == "norm" else (torch.bfloat16, torch.bfloat16)
        st["residual"] = (4 * torch.randn((m, h), generator=g, device="cuda")).to(res)
        st["delta"] = torch.randn((m, h), generator=g, device="cuda").to(delta)
        st["gamma"] = None
        if case.get("gamma", True):
            st["gamma"] = (1 + 0.2 * torch.randn((h,), generator=g, device="cuda")).to(torch.bfloat16)
    if op == "route":
        st["logits"] = _logits(g, m, case["experts"], 0.3, _types(case, "logits"))
        if case["masked"]:
            st["logits"][torch.rand(st["logits"].shape, generator=g, device="cuda") < case["masked"]] = -math.inf
    if op in ("gateup", "down", "layer"):
        e, h, i, f = case["experts"], case["hidden"], case["inter"], case["fmt"]
        logits = _logits(g, m, e, case["skew"])
        if op != "down":
            st["gate"], st["up"] = _experts(g, e, i, h, f), _experts(g, e, i, h, f)
        if op != "gateup":
            st["down"] = _experts(g, e, h, i, f)
        ids, _ = _plain_route(logits, case["topk"])
        offsets, rows, pos = _plain_plan(ids, e)
        # host figures that only the plain form's padding uses
        counts = (offsets[1:] - offsets[:-1]).cpu()
        st["cap"], st["active"] = int(counts.max()), torch.nonzero(counts).flatten().cuda()
        if op == "layer":
            st["logits"] = logits
        else:
            st["offsets"], st["rows"], st["pos"] = offsets, rows, pos
            st["q"], st["s"] = _quantised(g, m if op == "gateup" else m * case["topk"], h if op == "gateup" else i)
    return st


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------

def _weights(w, active):
    """The active experts' weights in fp32, [active][n][k]."""
    c, per = w["codes"][active], 4 if w["fmt"] == 0 else 8
    shift = torch.arange(per, device=c.device, dtype=torch.uint8) * (8 // per)
    c = (c[..., None] >> shift).view(c.shape[0], w["n"], w["k"]) & (3 if per == 4 else 1)
    table = [0.0, 1.0, -1.0, 0.0] if per == 4 else [-1.0, 1.0]
    v = torch.tensor(table, device=c.device)[c.int()].view(c.shape[0], w["n"], -1, BLOCK)
    return v.mul_(w["scales"][active].float()[..., None]).view(c.shape[0], w["n"], w["k"])


def _plain_grouped(w, x, rows, offsets, active, cap):
    """y[r] = W[expert of r] x[rows[r]], the rows of an expert padded to `cap`, fp32."""
    slots = torch.arange(rows.numel(), device=x.device)
    expert = torch.searchsorted(offsets[1:].long(), slots, right=True)
    place = torch.searchsorted(active, expert) * cap + slots - offsets[expert].long()
    padded = torch.zeros((active.numel() * cap, w["k"]), device=x.device)
    padded[place] = x[rows.long()]
    y = torch.bmm(padded.view(active.numel(), cap, -1), _weights(w, active).transpose(1, 2))
    return y.view(-1, w["n"])[place]


def _values(q, s):
    return (q.float().view(q.shape[0], -1, BLOCK) * s[..., None]).view(q.shape)


def _plain_gateup(st, q, s, rows, offsets):
    x = _values(q, s)
    g = _plain_grouped(st["gate"], x, rows, offsets, st["active"], st["cap"])
    u = _plain_grouped(st["up"], x, rows, offsets, st["active"], st["cap"])
    return (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)


def _span(v, h):
    """One stage of the fast Walsh-Hadamard transform over the last axis."""
    p = v.view(*v.shape[:-1], -1, 2, h)
    a, b = p[..., 0, :], p[..., 1, :]
    return torch.stack((a + b, a - b), -2).view(v.shape)


def _plain_rotq(x):
    """bf16 rows -> int8 codes and a scale per block, each step rounded to fp32 in the stated order."""
    v = x.float().view(x.shape[0], -1, BLOCK)
    v = _span(_span(_span(_span(_span(_span(_span(v, 1), 2), 4), 8), 16), 32), 64)
    v = v * float(np.float32(1 / math.sqrt(BLOCK)))
    top = v.abs().amax(-1, keepdim=True)
    s = top / torch.full_like(top, 127.0)
    q = torch.where(s > 0, torch.round(v / s).clamp(-127, 127), torch.zeros_like(v))
    return q.to(torch.int8).view(x.shape), s.squeeze(-1)


def _plain_norm(residual, delta, gamma):
    out = (residual.float() + delta.float()).to(residual.dtype)
    t = out.float()
    # the sum in 64 bits: an ulp in the norm moves codes across a rounding border
    inv = (1 / torch.sqrt(t.double().square().mean(-1, keepdim=True) + EPS)).float()
    x = t * inv
    if gamma is not None:
        x = x * gamma.float()
    return (out, *_plain_rotq(x.to(torch.bfloat16)))


def _plain_route(logits, topk):
    """Ids (-1 where a row has no expert left) and weights that add up to 1 over the chosen."""
    v, ids = torch.sort(logits.float(), dim=-1, descending=True, stable=True)
    v, ids = v[:, :topk], ids[:, :topk].to(torch.int32)
    none = v == -math.inf
    top = torch.where(none[:, :1], torch.zeros_like(v[:, :1]), v[:, :1])
    e = torch.exp(v - top)
    w = e / e.sum(-1, keepdim=True)
    return torch.where(none, torch.full_like(ids, -1), ids), torch.where(none, torch.zeros_like(w), w)


def _plain_plan(ids, experts):
    """The slots (token, choice) sorted by expert: offsets [experts + 1], the token of each sorted slot
    (-1 behind the last) and each slot's place in the order (-1 where it has no expert)."""
    flat = ids.flatten().long()
    key = torch.where(flat < 0, torch.full_like(flat, experts), flat)
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(experts + 1, device=ids.device))
    slots = torch.arange(flat.numel(), device=ids.device)
    rows = torch.where(slots < offsets[-1], order // ids.shape[1], torch.full_like(order, -1))
    pos = torch.empty_like(order)
    pos[order] = torch.where(slots < offsets[-1], slots, torch.full_like(slots, -1))
    return offsets.to(torch.int32), rows.to(torch.int32), pos.to(torch.int32).view(ids.shape)


def _plain_layer(st):
    case = st["case"]
    residual, q, s = _plain_norm(st["residual"], st["delta"], st["gamma"])
    ids, w = _plain_route(st["logits"], case["topk"])
    offsets, rows, pos = _plain_plan(ids, case["experts"])
    hq, hs = _plain_rotq(_plain_gateup(st, q, s, rows, offsets))
    slots = torch.arange(rows.numel(), device=rows.device)
    y = _plain_grouped(st["down"], _values(hq, hs), slots, offsets, st["active"], st["cap"])
    y = (y[pos.long()] * w[..., None]).sum(1)
    return {"residual": residual, "y": y.to(torch.bfloat16)}


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def _held(st):
    """What a program keeps between calls: weight handles, the plan and buffers."""
    from ternary_weight_dp4a_gb300 import tq
    if "held" not in st:
        case, held = st["case"], {}
        for name in ("gate", "up", "down"):
            if name in st:
                held[name] = tq.PackedExperts(**st[name])
        if "offsets" in st:
            held["plan"] = tq.MoePlan(st["offsets"], st["rows"], st["pos"])
        if case["op"] != "norm":
            held["ws"] = tq.moe_workspace(case["m"], case["topk"], case["experts"], case.get("hidden", 0), case.get("inter", 0))
        st["held"] = held
    return tq, st["held"]


def run(st):
    op, case = st["case"]["op"], st["case"]
    if own:
        tq, held = _held(st)
        if op == "norm":
            residual, q, s = tq.add_rmsnorm_rotq(st["residual"], st["delta"], st["gamma"], eps=EPS)
            return {"residual": residual, "values": torch.mul(q.view(*s.shape, BLOCK), s[..., None])}
        if op == "route":
            ids, w = tq.moe_route(st["logits"], case["topk"])
            plan = tq.moe_plan(ids, case["experts"], workspace=held["ws"])
            return {"ids": ids, "weights": w, "offsets": plan.offsets, "rows": plan.rows, "pos": plan.pos}
        if op == "gateup":
            return {"h": tq.moe_gateup(held["gate"], held["up"], st["q"], st["s"], held["plan"], workspace=held["ws"])}
        if op == "down":
            return {"y": tq.moe_gemv(held["down"], st["q"], st["s"], held["plan"], workspace=held["ws"])}
        residual, q, s = tq.add_rmsnorm_rotq(st["residual"], st["delta"], st["gamma"], eps=EPS)
        ids, w = tq.moe_route(st["logits"], case["topk"])
        y = tq.moe_ffn(held["gate"], held["up"], held["down"], q, s, ids, w, dtype=torch.bfloat16, workspace=held["ws"])
        return {"residual": residual, "y": y}
    if op == "norm":
        residual, q, s = _plain_norm(st["residual"], st["delta"], st["gamma"])
        return {"residual": residual, "values": q.view(*s.shape, BLOCK) * s[..., None]}
    if op == "route":
        ids, w = _plain_route(st["logits"], case["topk"])
        offsets, rows, pos = _plain_plan(ids, case["experts"])
        return {"ids": ids, "weights": w, "offsets": offsets, "rows": rows, "pos": pos}
    if op == "gateup":
        return {"h": _plain_gateup(st, st["q"], st["s"], st["rows"], st["offsets"])}
    if op == "down":
        slots = torch.arange(st["rows"].numel(), device="cuda")
        return {"y": _plain_grouped(st["down"], _values(st["q"], st["s"]), slots, st["offsets"], st["active"], st["cap"])}
    return _plain_layer(st)


def work(case):
    m, op = case["m"], case["op"]
    if op == "norm":
        h = case["hidden"]
        size = {"f32": 4, "bf16": 2}
        # residual in and out, delta, gamma, int8 codes and scales (the pass returns the codes' values:
        # four bytes for each)
        return {"bytes": m * h * (2 * size[case["res"]] + size[case["delta"]] + 4 + 4 / BLOCK) + 2 * h * case["gamma"],
                "flops": m * h * 14}
    slots = m * case["topk"]
    if op == "route":
        return {"bytes": m * case["experts"] * (2 if case["logits"] == "bf16" else 4) + slots * 16 + 4 * case["experts"],
                "flops": m * case["experts"] * 4}
    h, i, e = case["hidden"], case["inter"], case["experts"]
    active = e * (1 - (1 - 1 / e) ** slots) if slots > case["topk"] else min(e, slots)   # even routing
    expert = h * i * ((1 / 4 if case["fmt"] == 0 else 1 / 8) + 2 / BLOCK)
    act = 1 + 4 / BLOCK
    if op == "gateup":
        return {"bytes": 2 * active * expert + m * h * act + slots * i * 2, "flops": 4 * slots * h * i}
    if op == "down":
        return {"bytes": active * expert + slots * i * act + slots * h * 4, "flops": 2 * slots * h * i}
    return {"bytes": 3 * active * expert + m * h * (2 + 2 + 2 + 2) + m * e * 4, "flops": 6 * slots * h * i}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_matrix(w, e):
    c = w["codes"][e].to(torch.int64)
    if w["fmt"] == 0:
        c = torch.stack([c % 4, c // 4 % 4, c // 16 % 4, c // 64], -1).reshape(w["n"], w["k"])
        v = (c == 1).double() - (c == 2).double()
    else:
        c = torch.stack([c // 2 ** b % 2 for b in range(8)], -1).reshape(w["n"], w["k"])
        v = 2 * c.double() - 1
    return v * w["scales"][e].double().repeat_interleave(BLOCK, -1)


def _exact_rotq(x):
    n = torch.arange(BLOCK, device=x.device)
    bits = n[:, None] & n[None, :]
    odd = sum((bits >> b) & 1 for b in range(7)) % 2
    v = x.view(x.shape[0], -1, BLOCK) @ ((1 - 2 * odd).double() / math.sqrt(BLOCK))
    s = v.abs().amax(-1, keepdim=True) / 127
    return (torch.where(s > 0, torch.round(v / s.clamp_min(1e-300)), torch.zeros_like(v)) * s).view(x.shape)


def _exact_gateup(st, x, tokens, expert):
    out = torch.empty((len(tokens), st["gate"]["n"]), dtype=torch.float64, device="cuda")
    for e in expert.unique().tolist():
        at = expert == e
        g, u = (x[tokens[at]] @ _exact_matrix(st[n], e).T for n in ("gate", "up"))
        out[at] = g * torch.sigmoid(g) * u
    return out


def _exact_down(st, x, expert):
    out = torch.empty((len(x), st["down"]["n"]), dtype=torch.float64, device="cuda")
    for e in expert.unique().tolist():
        at = expert == e
        out[at] = x[at] @ _exact_matrix(st["down"], e).T
    return out


def exact(case, seed):
    op = case["op"]
    if op in ("gateup", "down", "layer") and work(case)["flops"] > 5e12:
        return None
    st = prepare(case, seed)
    if op in ("norm", "layer"):
        residual = st["residual"].double() + st["delta"].double()
    if op == "norm":
        return {"residual": residual, "values": None}       # a code next to a border has no value in 64 bits
    if op == "route":
        v = st["logits"].double()
        w = torch.zeros((case["m"], case["topk"]), dtype=torch.float64, device="cuda")
        top = torch.topk(v, case["topk"], dim=-1).values
        some = top[:, 0] > -math.inf
        w[some] = torch.softmax(top[some], -1)
        return {"ids": None, "weights": w, "offsets": None, "rows": None, "pos": None}
    if op == "layer":
        ids = torch.topk(st["logits"], case["topk"], dim=-1).indices
        w = torch.softmax(st["logits"].double().gather(1, ids), -1)
        # what is normalised is the residual as it is stored
        t = residual.to(st["residual"].dtype).double()
        x = t / torch.sqrt((t * t).sum(-1, keepdim=True) / t.shape[1] + EPS) * st["gamma"].double()
        x = _exact_rotq(x.to(torch.bfloat16).double())
        expert = ids.flatten()
        tokens = torch.arange(case["m"], device="cuda").repeat_interleave(case["topk"])
        h = _exact_gateup(st, x, tokens, expert)
        y = _exact_down(st, _exact_rotq(h.to(torch.bfloat16).double()), expert)
        return {"residual": residual, "y": (y.view(case["m"], case["topk"], -1) * w[..., None]).sum(1)}
    counts = (st["offsets"][1:] - st["offsets"][:-1]).long()
    expert = torch.repeat_interleave(torch.arange(case["experts"], device="cuda"), counts)
    x = (st["q"].double().view(st["q"].shape[0], -1, BLOCK) * st["s"].double()[..., None]).view(st["q"].shape)
    if op == "gateup":
        return {"h": _exact_gateup(st, x, st["rows"].long(), expert)}
    return {"y": _exact_down(st, x, expert)}
