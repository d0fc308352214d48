"""The operators around a ternary FFN in a decode step: cases, plain forms and calls.

Three operators, as a step runs them where it does not run ternary weights:

* ``gemv``    the product with a matrix of 4-bit weights and a scale (and minimum) for each group of a
              row, for bf16 activations (``tq.q4_gemv``): attention projections, the FFN's second product
              while the ternary copy is not resident, and the head that gives the logits;
* ``gateup``  both projections of a gated FFN over such weights with SiLU(gate) * up, as bf16
              (``tq.q4_gateup``);
* ``sample``  a token for each row of logits by temperature, top-k, min-p and top-p from a given random
              number (``tq.sample``).

``own`` chooses between the plain torch forms and the library's calls; both take the same state.

A weight is ``scale * code - min`` with codes 0 .. 15, or ``scale * (code - 8)`` where a matrix has no
minima; scales and minima are fp16, one for each group of 32, 64 or 128 along k.

Sampling, for a row of logits l, in the order of descending logits with ties to the lowest index (NaN and
-infinity are no candidates, +infinity counts as the largest finite number):
  weights  w_i = exp((l_i - l_max) / temperature); temperature 0: the first of the order, with probability 1
  top-k    the first top_k stay (0: all)
  min-p    of them those with w_i >= min_p; the first always
  top-p    of them the shortest run from the first on with a sum of at least top_p of their sum (1: all); the first always
  draw     the lowest index i with  sum over j <= i of what stayed  >  u * (the sum of what stayed)
and the probability of the drawn token among what stayed.  A row without candidates: -1 and 0.
"""
import math

import torch

own = False

BLOCK = 128
NEG = -math.inf


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # a square projection of one decoded token
        {"name": "gemv_m1", "op": "gemv", "m": 1, "n": 5120, "k": 5120, "group": 128, "mins": False, "out": "f32"},
        # the FFN's second product of a packed decode step
        {"name": "gemv_m8_mins", "op": "gemv", "m": 8, "n": 5120, "k": 17408, "group": 32, "mins": True, "out": "bf16"},
        # a ragged verify block over an odd number of outputs
        {"name": "gemv_m37_odd", "op": "gemv", "m": 37, "n": 6145, "k": 2048, "group": 64, "mins": True, "out": "f32"},
        # the head of one token, and of a decode batch
        {"name": "head_m1", "op": "gemv", "m": 1, "n": 131072, "k": 5120, "group": 128, "mins": False, "out": "f32"},
        {"name": "head_m32", "op": "gemv", "m": 32, "n": 131072, "k": 5120, "group": 32, "mins": False, "out": "bf16"},
        # gate and up of one token, of a small odd batch, and of a prefill block (the largest)
        {"name": "gateup_m1", "op": "gateup", "m": 1, "n": 17408, "k": 5120, "group": 128, "mins": False},
        {"name": "gateup_m13_mins", "op": "gateup", "m": 13, "n": 17408, "k": 5120, "group": 32, "mins": True},
        {"name": "gateup_m512", "op": "gateup", "m": 512, "n": 17408, "k": 5120, "group": 128, "mins": False},
        # one token of a chat with all three cuts
        {"name": "sample_m1", "op": "sample", "m": 1, "vocab": 131072, "logits": "f32", "kind": "mixed", "masked": 0.0, "spread": 3.0},
        # a decode batch whose requests have settings of their own, some tokens banned
        {"name": "sample_m64", "op": "sample", "m": 64, "vocab": 131072, "logits": "bf16", "kind": "mixed", "masked": 0.02, "spread": 3.0},
        # an odd vocabulary, min-p alone
        {"name": "sample_m33_odd", "op": "sample", "m": 33, "vocab": 32003, "logits": "f32", "kind": "min_p", "masked": 0.3, "spread": 2.0},
        # a large batch with top-p over the whole vocabulary
        {"name": "sample_m256", "op": "sample", "m": 256, "vocab": 131072, "logits": "f32", "kind": "top_p", "masked": 0.0, "spread": 2.0},
    ]


KINDS = ("greedy", "plain", "top_k", "top_p", "min_p", "mixed")


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gemv", "gateup", "sample"])
    if op == "sample":
        vocab = _log_int(rng, 50, 160000)
        m = min(_log_int(rng, 1, 256), max(1, 256 * 131072 // vocab))
        return {"op": op, "m": m, "vocab": vocab, "logits": rng.choice(["f32", "bf16"]), "kind": rng.choice(KINDS),
                "masked": rng.choice([0.0, 0.02, 0.3]), "spread": rng.choice([0.5, 2.0, 3.0, 5.0])}
    k = BLOCK * _log_int(rng, 1, 136)
    n = min(_log_int(rng, 16, 131072), 131072 * 5120 // k)
    if op == "gateup":
        n = max(1, n // 2)
    m = max(1, min(_log_int(rng, 1, 512), 512 * 17408 * 5120 // (n * k)))
    case = {"op": op, "m": m, "n": n, "k": k, "group": rng.choice([32, 64, 128]), "mins": rng.random() < 0.5}
    if op == "gemv":
        case["out"] = rng.choice(["f32", "bf16"])
    return case


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _matrix(g, n, k, group, mins):
    """A quantised matrix as a checkpoint holds it: codes [n][k], scales and minima [n][k/group]."""
    shape = (n, k // group)
    scales = ((0.4 + torch.rand(shape, generator=g, device="cuda")) / (5 * math.sqrt(k))).half()
    w = {"codes": torch.randint(0, 16, (n, k), generator=g, device="cuda", dtype=torch.uint8), "scales": scales,
         "mins": None, "group": group}
    if mins:
        # minima that put the codes' middle near zero, as a quantiser of weights around zero leaves them
        w["mins"] = (scales.float() * (7.5 + torch.randn(shape, generator=g, device="cuda"))).half()
    return w


def _settings(g, case):
    """Temperature, top-k, top-p, min-p of each row (None: off) for the kind of case."""
    m, kind = case["m"], case["kind"]

    def rand(lo, hi):
        return lo + (hi - lo) * torch.rand((m,), generator=g, device="cuda")

    st = {"temperature": None, "top_k": None, "top_p": None, "min_p": None}
    if kind == "greedy":
        st["temperature"] = torch.zeros((m,), device="cuda")
        return st
    st["temperature"] = rand(0.6, 1.1)
    if kind in ("top_k", "mixed"):
        st["top_k"] = torch.randint(1, 200, (m,), generator=g, device="cuda", dtype=torch.int32)
    if kind in ("top_p", "mixed"):
        st["top_p"] = rand(0.8, 0.99)
    if kind in ("min_p", "mixed"):
        st["min_p"] = rand(0.001, 0.1)
    if kind == "mixed" and m > 1:
        # requests that turn single settings off, and greedy ones among them
        st["temperature"][torch.rand((m,), generator=g, device="cuda") < 0.1] = 0.0
        st["top_k"][torch.rand((m,), generator=g, device="cuda") < 0.4] = 0
        st["top_p"][torch.rand((m,), generator=g, device="cuda") < 0.3] = 1.0
        st["min_p"][torch.rand((m,), generator=g, device="cuda") < 0.5] = 0.0
    return st


def prepare(case, seed):
    g, m = _gen(seed), case["m"]
    st = {"case": case}
    if case["op"] == "sample":
        logits = case["spread"] * torch.randn((m, case["vocab"]), generator=g, device="cuda")
        if case["masked"]:
            logits[torch.rand(logits.shape, generator=g, device="cuda") < case["masked"]] = NEG
        st["logits"] = logits.to(_dtype(case["logits"]))
        st.update(_settings(g, case))
        st["uniform"] = torch.rand((m,), generator=g, device="cuda")
        return st
    names = ("gate", "up") if case["op"] == "gateup" else ("w",)
    for name in names:
        st[name] = _matrix(g, case["n"], case["k"], case["group"], case["mins"])
    st["x"] = torch.randn((m, case["k"]), generator=g, device="cuda").to(torch.bfloat16)
    return st


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------

def _plain_product(w, x):
    """x W^T in fp32."""
    n, k = w["codes"].shape
    c = w["codes"].float().view(n, -1, w["group"])
    s = w["scales"].float()[..., None]
    v = (c - 8) * s if w["mins"] is None else c * s - w["mins"].float()[..., None]
    return x.float() @ v.view(n, k).T


def _row(st, name, off, like):
    v = st[name]
    return torch.full((like.shape[0], 1), off, dtype=torch.float64, device=like.device) if v is None else v.double()[:, None]


def _plain_sample(st):
    """The rule at the top of the file.  In 64 bits: a sum next to a border decides which token it is."""
    big = torch.finfo(st["logits"].dtype).max
    v = torch.where(torch.isnan(st["logits"]), torch.full_like(st["logits"], NEG), st["logits"]).clamp(max=big).double()
    t, p, floor = _row(st, "temperature", 1.0, v), _row(st, "top_p", 1.0, v), _row(st, "min_p", 0.0, v)
    top = _row(st, "top_k", 0.0, v)
    v, order = torch.sort(v, dim=-1, descending=True, stable=True)
    rank = torch.arange(v.shape[1], device=v.device)[None]
    some = v[:, :1] > NEG
    v0 = torch.where(some, v[:, :1], torch.zeros_like(v[:, :1]))
    w = torch.exp((v - v0) / torch.where(t > 0, t, torch.ones_like(t)))
    w = torch.where(t > 0, w, (rank == 0).double())
    w = torch.where((top > 0) & (rank >= top), torch.zeros_like(w), w)
    w = torch.where((w < floor) & (rank > 0), torch.zeros_like(w), w)
    before = torch.cumsum(w, -1) - w
    w = torch.where((p < 1) & (before >= p * w.sum(-1, keepdim=True)) & (rank > 0), torch.zeros_like(w), w)
    w = torch.where(some, w, torch.zeros_like(w))
    w = torch.zeros_like(w).scatter_(1, order, w)                    # in the order of the indices again
    total = w.sum(-1, keepdim=True)
    hit = (torch.cumsum(w, -1) > st["uniform"].double()[:, None] * total) & (w > 0)
    last = torch.where(w > 0, rank, torch.full_like(rank, -1)).amax(-1)
    ids = torch.where(hit.any(-1), hit.to(torch.uint8).argmax(-1), last)
    probs = w.gather(1, ids.clamp(min=0)[:, None]) / torch.where(total > 0, total, torch.ones_like(total))
    return ids.to(torch.int32), probs.squeeze(1).float()


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def _held(st):
    """The packed matrices, which a program lays out once when it loads a model."""
    from ternary_weight_dp4a_gb300 import tq
    if "held" not in st:
        st["held"] = {name: tq.pack_q4(st[name]["codes"], st[name]["scales"], st[name]["mins"])
                      for name in ("gate", "up", "w") if name in st}
    return tq, st["held"]


def run(st):
    op, case = st["case"]["op"], st["case"]
    if own:
        tq, held = _held(st)
        if op == "gemv":
            return {"y": tq.q4_gemv(held["w"], st["x"], dtype=_dtype(case["out"]))}
        if op == "gateup":
            return {"h": tq.q4_gateup(held["gate"], held["up"], st["x"])}
        ids, probs = tq.sample(st["logits"], st["uniform"], temperature=st["temperature"], top_k=st["top_k"],
                               top_p=st["top_p"], min_p=st["min_p"])
        return {"ids": ids, "probs": probs}
    if op == "gemv":
        return {"y": _plain_product(st["w"], st["x"]).to(_dtype(case["out"]))}
    if op == "gateup":
        g, u = _plain_product(st["gate"], st["x"]), _plain_product(st["up"], st["x"])
        return {"h": (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)}
    ids, probs = _plain_sample(st)
    return {"ids": ids, "probs": probs}


def work(case):
    m = case["m"]
    if case["op"] == "sample":
        entries = m * case["vocab"]
        return {"bytes": entries * (2 if case["logits"] == "bf16" else 4) + m * (5 * 4 + 2 * 4), "flops": 8 * entries}
    n, k = case["n"], case["k"]
    matrix = n * k / 2 + n * (k // case["group"]) * (4 if case["mins"] else 2)
    if case["op"] == "gateup":
        return {"bytes": 2 * matrix + m * k * 2 + m * n * 2, "flops": 4 * m * n * k}
    return {"bytes": matrix + m * k * 2 + m * n * (2 if case["out"] == "bf16" else 4), "flops": 2 * m * n * k}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_product(w, x):
    """Block of rows by block of rows: sum over the groups of scale * sum(code * x) - min * sum(x)."""
    n, k = w["codes"].shape
    group = w["group"]
    xg = x.double().view(x.shape[0], k // group, group)
    low = torch.full_like(w["scales"][:, 0], 8).double() if w["mins"] is None else None
    out = torch.empty((x.shape[0], n), dtype=torch.float64, device=x.device)
    step = max(1, (1 << 27) // k)
    for i in range(0, n, step):
        c = w["codes"][i:i + step].double().view(-1, k // group, group)
        s = w["scales"][i:i + step].double()
        b = s * low[i:i + step, None] if w["mins"] is None else w["mins"][i:i + step].double()
        c.mul_(s[..., None]).sub_(b[..., None])
        out[:, i:i + step] = xg.view(x.shape[0], k) @ c.view(-1, k).T
    return out


def _exact_row(v, u, t, top, p, floor):
    """One row of logits in 64 bits -> (id, probability)."""
    keep = torch.nonzero(v > NEG).flatten()
    if len(keep) == 0:
        return -1, 0.0
    if t == 0:
        return int(keep[v[keep] == v[keep].max()].min()), 1.0
    keep = keep[torch.argsort(-v[keep], stable=True)]
    if top > 0:
        keep = keep[:top]
    w = torch.exp((v[keep] - v[keep[0]]) / t)
    n = max(1, int((w >= floor).sum()))
    keep, w = keep[:n], w[:n]
    if p < 1:
        n = 1 + int((torch.cumsum(w, 0) < p * w.sum()).sum())
        keep, w = keep[:n], w[:n]
    by_index = torch.argsort(keep)
    keep, w = keep[by_index], w[by_index]
    at = min(int((torch.cumsum(w, 0) <= u * w.sum()).sum()), len(w) - 1)
    return int(keep[at]), float(w[at] / w.sum())


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "gemv":
        return {"y": _exact_product(st["w"], st["x"])}
    if case["op"] == "gateup":
        g, u = _exact_product(st["gate"], st["x"]), _exact_product(st["up"], st["x"])
        return {"h": g * torch.sigmoid(g) * u}
    m = case["m"]
    rows = [[st["uniform"].tolist()[r]] + [off if st[name] is None else st[name].tolist()[r] for name, off in
            (("temperature", 1.0), ("top_k", 0), ("top_p", 1.0), ("min_p", 0.0))] for r in range(m)]
    got = [_exact_row(st["logits"][r].double(), *rows[r]) for r in range(m)]
    return {"ids": torch.tensor([g[0] for g in got], dtype=torch.int32, device="cuda"),
            "probs": torch.tensor([g[1] for g in got], dtype=torch.float64, device="cuda")}
