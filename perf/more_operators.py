"""What is measured of the operators around the experts.

Three operators that a served MoE block runs beside its expert products:

``norm``  the residual's addition and the root-mean-square norm in one pass over
          the rows, with the normed rows in their own type, in e4m3 with scales
          (one a row, or one a group of 32, 64 or 128 values), or both:
          ``moe_add_rms_norm``.
``gate``  routing by softmax or sigmoid scores, with a bias that takes part in
          the choice alone, a first choice among groups of experts, top-k,
          renormalised weights and a factor: ``moe_route_gated``, from router
          logits, or from the token rows through the projection.
``lora``  y = base + scale (x A^T) B^T with the low-rank adapter of each row's
          own request beside a projection that all rows share: ``moe_lora``.

Rows are N(0, 1), weights N(0, 0.02) as the repository draws them elsewhere.  A
token whose choice hangs on a difference of less than 1e-5 (of the largest
score) is drawn again: it is decided by the last bits of a 32-bit sum.
"""
import math

import torch

own = False

DEV = "cuda"
GAP = 1e-5
EPS = 1e-6
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def _norm(name, T, D, dt="bf16", add=True, y=True, q=-1):
    """q: values to a scale (0: the row's, -1: no 8-bit output)."""
    return {"name": name, "op": "norm", "T": T, "D": D, "dt": dt, "add": add, "y": y, "q": q}


def _gate(name, T, E, k, score="sigmoid", groups=1, kept=1, top2=True, bias=True, renorm=True, scale=1.0, D=0):
    """D: width of the token rows (0: the router logits are the input)."""
    return {"name": name, "op": "gate", "T": T, "E": E, "k": k, "score": score, "groups": groups, "kept": kept,
            "top2": top2, "bias": bias, "renorm": renorm, "scale": scale, "D": D}


def _lora(name, T, K, N, r, n, dt="bf16", mixed=False, none=0.0):
    """n adapters; mixed: rows in any order, else a request's rows together;
    none: the share of rows (or requests) without an adapter."""
    return {"name": name, "op": "lora", "T": T, "K": K, "N": N, "r": r, "n": n, "dt": dt, "mixed": mixed, "none": none}


def listed():
    return [
        # one user's next token: nothing but latency
        _norm("norm_T1_2048", 1, 2048),
        # a decode batch of odd size, rows that end inside a vector group, scales for groups
        _norm("norm_T77_2816_g128", 77, 2816, q=128),
        # a prompt in 32 bits, the first norm (nothing to add)
        _norm("norm_T4096_2048_f32", 4096, 2048, dt="f32", add=False),
        # the largest prompt, rows for 8-bit expert products
        _norm("norm_T16384_8192_row", 16384, 8192, q=0),
        # one user's next token, groups of experts
        _gate("gate_T1_E256_g8", 1, 256, 8, groups=8, kept=4, scale=2.5),
        # a decode batch over many experts, softmax scores with a bias
        _gate("gate_T509_E512", 509, 512, 10, score="softmax"),
        # a prompt's rows through the projection
        _gate("gate_T4096_E128_rows", 4096, 128, 8, D=2048),
        # the largest prompt, groups of experts
        _gate("gate_T16384_E256_g8", 16384, 256, 8, groups=8, kept=4, scale=2.5),
        # one user's next token through its own adapter
        _lora("lora_T1_2048_r16", 1, 2048, 2048, 16, 8),
        # a decode batch of many users, rows in any order, some without an adapter
        _lora("lora_T61_4096_r64", 61, 4096, 4096, 64, 40, mixed=True, none=0.1),
        # four users' prompts, a wide projection kept in 32 bits
        _lora("lora_T2000_2048x4224_r24_f32", 2000, 2048, 4224, 24, 4, dt="f32"),
        # the largest batch of prompts
        _lora("lora_T8192_8192_r64", 8192, 8192, 8192, 64, 12),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(v, m):
    return max(m, v // m * m)


_CEIL = {"norm": 1.2e9, "gate": 1.9e7, "lora": 4.2e8}  # bytes: under the largest listed case of each


def draw(rng):
    while True:
        op = rng.choice(["norm", "gate", "lora"])
        if op == "norm":
            q = rng.choice([-1, 0, 0, 32, 64, 128])
            c = _norm("", _logint(rng, 1, 16384), _mult(_logint(rng, 256, 16384), max(q, 8)), rng.choice(["bf16", "bf16", "f32"]),
                      rng.random() < 0.7, q < 0 or rng.random() < 0.6, q)
        elif op == "gate":
            D = rng.choice([0, 0, 1]) * _mult(_logint(rng, 256, 8192), 8)
            groups = rng.choice([1, 1, 2, 4, 8, 16])
            size = _mult(_logint(rng, 2, 512 // groups), 8 if D and groups == 1 else 1)
            if D and groups * size % 8:
                continue
            kept = rng.randint(1, groups)
            c = _gate("", _logint(rng, 1, 16384), groups * size, rng.randint(1, min(10, kept * size)),
                      rng.choice(["softmax", "sigmoid"]), groups, kept, rng.random() < 0.6, rng.random() < 0.7,
                      rng.random() < 0.8, rng.choice([1.0, 2.5]), D)
        else:
            c = _lora("", _logint(rng, 1, 8192), _mult(_logint(rng, 256, 8192), 8), _mult(_logint(rng, 256, 8192), 8),
                      rng.choice([8, 16, 24, 32, 64, 96, 128]), _logint(rng, 1, 48), rng.choice(["bf16", "bf16", "f32"]),
                      rng.random() < 0.4, rng.choice([0.0, 0.2]))
            if 2.0 * c["T"] * c["n"] * c["r"] * (c["K"] + c["N"]) > 3e11:
                continue
        if work(c)["bytes"] <= _CEIL[op]:
            del c["name"]
            return c


def work(case):
    """Every input once, every output once; of the adapters, those that some row
    has (their expected number)."""
    T = case["T"]
    if case["op"] == "norm":
        D, b = case["D"], 4 if case["dt"] == "f32" else 2
        scales = 4 * T * (D // case["q"] if case["q"] > 0 else 1)
        out = b * (case["add"] + case["y"]) * T * D + (T * D + scales if case["q"] >= 0 else 0)
        return {"bytes": b * (1 + case["add"]) * T * D + b * D + out, "flops": 6.0 * T * D}
    if case["op"] == "gate":
        E, D = case["E"], case["D"]
        rows = 2 * T * D + 2 * D * E if D else 0
        return {"bytes": rows + 4 * T * E + 8 * T * case["k"] + 4 * E, "flops": 2.0 * T * D * E + 8.0 * T * E}
    K, N, r, n = (case[m] for m in ("K", "N", "r", "n"))
    rows = T * (1.0 - case["none"])
    used = n * (1.0 - (1.0 - 1.0 / n) ** rows) if case["mixed"] else min(n * (1.0 - case["none"]), rows)
    b = 4 if case["dt"] == "f32" else 2
    return {"bytes": 2 * rows * K + 2 * b * T * N + 2 * used * r * (K + N) + 8 * T, "flops": 2.0 * rows * r * (K + N)}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _normal(shape, std, g, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=g)


def _near(logits, bias, c):
    """Rows whose choice, of groups or of experts, or whose order is decided by
    less than GAP of the largest value compared."""
    p = logits.double()
    p = torch.sigmoid(p) if c["score"] == "sigmoid" else torch.softmax(p, dim=1)
    v = p if bias is None else p + bias.double()
    T, E = v.shape
    near = torch.zeros(T, dtype=torch.bool, device=v.device)
    if c["kept"] < c["groups"]:
        m = v.view(T, c["groups"], -1)
        s = m.topk(min(2 if c["top2"] else 1, m.shape[2]), dim=2).values.sum(2)
        o = s.sort(dim=1, descending=True).values
        near |= o[:, c["kept"] - 1] - o[:, c["kept"]] < GAP * o.abs().amax(1)
        cut = o[:, c["kept"] - 1:c["kept"]]
        v = torch.where((s >= cut).repeat_interleave(m.shape[2], dim=1), v, torch.full_like(v, -1e30))
    o = v.topk(min(E, c["k"] + 1), dim=1).values
    gaps = o[:, :-1] - o[:, 1:]
    return near | (gaps < GAP * o[:, :1].abs()).any(1) if gaps.shape[1] else near


def prepare(case, seed):
    g, T = _gen(seed), case["T"]
    st = {"case": case}
    if case["op"] == "norm":
        D, dt = case["D"], TYPES[case["dt"]]
        st["x"] = _normal((T, D), 1.0, g, dt)
        st["res"] = _normal((T, D), 2.0, g, dt) if case["add"] else None
        st["w"] = (1.0 + _normal((D,), 0.2, g, torch.float32)).to(dt)
        st["sum"] = torch.empty_like(st["x"]) if case["add"] else None
        st["y"] = torch.empty_like(st["x"]) if case["y"] else None
        st["q"] = st["s"] = None
        if case["q"] >= 0:
            st["q"] = torch.empty((T, D), dtype=torch.float8_e4m3fn, device=DEV)
            st["s"] = torch.empty((T, D // (case["q"] or D)), dtype=torch.float32, device=DEV)
        return st
    if case["op"] == "gate":
        E, D, k = case["E"], case["D"], case["k"]
        st["Wg"] = _normal((D, E), 0.02, g) if D else None
        st["bias"] = _normal((E,), 0.1 if case["score"] == "sigmoid" else 0.2 / E, g, torch.float32) if case["bias"] else None
        fresh = lambda: _normal((T, D), 1.0, g) if D else _normal((T, E), 1.3, g, torch.float32)  # noqa: E731
        x = fresh()
        for _ in range(40):
            near = _near(x.float() @ st["Wg"].float() if D else x, st["bias"], case)
            if not bool(near.any()):
                break
            x = torch.where(near[:, None], fresh(), x)
        st["x"] = x if D else None
        st["logits"] = torch.empty((T, E), dtype=torch.float32, device=DEV) if D else x
        st["ids"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
        st["w"] = torch.empty((T, k), dtype=torch.float32, device=DEV)
        return st
    K, N, r, n = (case[m] for m in ("K", "N", "r", "n"))
    st["x"] = _normal((T, K), 1.0, g)
    st["A"] = _normal((n, r, K), 0.02, g)
    st["B"] = _normal((n, N, r), 0.05, g)
    st["scales"] = torch.empty(n, dtype=torch.float32, device=DEV).uniform_(0.5, 2.0, generator=g)
    st["base"] = _normal((T, N), 1.0, g, TYPES[case["dt"]])
    st["y"] = torch.empty_like(st["base"])
    if case["mixed"]:
        ids = torch.randint(0, n, (T,), device=DEV, generator=g)
        off = torch.rand(T, device=DEV, generator=g) < case["none"]
    else:  # n requests of about as many rows each, adapters in an order of their own
        cuts = (torch.rand(n - 1, device=DEV, generator=g) * T).long().sort().values
        req = torch.searchsorted(cuts, torch.arange(T, device=DEV), right=True)
        ids = torch.randperm(n, device=DEV, generator=g)[req]
        off = (torch.rand(n, device=DEV, generator=g) < case["none"])[req]
    st["ids"] = torch.where(off, torch.full_like(ids, -1), ids).to(torch.int32)
    return st


# --------------------------------------------------------------- plain form
def _plain_norm(st):
    c = st["case"]
    h = st["x"].float()
    if c["add"]:
        h = h + st["res"].float()
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * st["w"].float()
    out = {}
    if c["add"]:
        out["sum"] = h.to(st["x"].dtype)
    if c["y"]:
        out["y"] = y.to(st["x"].dtype)
    if c["q"] >= 0:
        m = y.view(c["T"], -1, c["q"] or c["D"])
        s = m.abs().amax(dim=2) / E4M3_MAX
        s = torch.where(s > 0, s, torch.ones_like(s))
        out["q"] = (m / s[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view_as(y).to(torch.float8_e4m3fn)
        out["s"] = s
    return out


def _plain_gate(st):
    c = st["case"]
    k, E = c["k"], c["E"]
    logits = torch.matmul(st["x"].float(), st["Wg"].float()) if c["D"] else st["logits"]
    L = logits.double()
    if c["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-L))
    else:
        p = torch.exp(L - L.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    v = p if st["bias"] is None else p + st["bias"].double()
    if c["kept"] < c["groups"]:
        m = v.view(c["T"], c["groups"], -1)
        best = torch.sort(m, dim=2, descending=True).values[:, :, :2 if c["top2"] else 1].sum(2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        keep = torch.zeros_like(best).scatter_(1, order, 1.0).repeat_interleave(E // c["groups"], dim=1)
        v = torch.where(keep > 0, v, torch.full_like(v, -math.inf))
    ids = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(p, 1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    out = {"ids": ids.to(torch.int32), "w": (w * c["scale"]).float()}
    if c["D"]:
        out["logits"] = logits
    return out


def _plain_lora(st):
    c = st["case"]
    T, K, N, r, n = (c[m] for m in ("T", "K", "N", "r", "n"))
    mine = st["ids"].long()[:, None] == torch.arange(n, device=DEV)  # [T, n]
    v = torch.matmul(st["x"].float(), st["A"].float().view(n * r, K).t()).view(T, n, r)
    v = v * (mine.float() * st["scales"])[:, :, None]
    delta = torch.matmul(v.view(T, n * r), st["B"].float().transpose(1, 2).reshape(n * r, N))
    return (st["base"].float() + delta).to(st["base"].dtype)


# ------------------------------------------------------- the framework's calls
_plans = {}


def _plan(case, make):
    """What a program sets up once for a shape and uses for all its inputs:
    the configuration and the workspace."""
    key = tuple(sorted(case.items()))
    if key not in _plans:
        _plans.clear()
        _plans[key] = make()
    return _plans[key]


def _own_norm(st):
    import mixture_experts_layer_gating_gb300 as moe

    c = st["case"]
    moe.moe_add_rms_norm(c["T"], c["D"], st["x"], st["res"], st["w"], EPS, st["sum"], st["y"], st["q"], st["s"], max(c["q"], 0))
    out = {"sum": st["sum"], "y": st["y"], "q": st["q"], "s": st["s"]}
    return {m: t for m, t in out.items() if t is not None}


def _own_gate(st):
    import mixture_experts_layer_gating_gb300 as moe

    c = st["case"]

    def make():
        cfg = moe.make_config(c["T"], c["D"] or 8, c["E"], c["k"], 8, renormalize=c["renorm"])
        gate = moe.make_gate(c["score"], c["groups"], c["kept"], "top2_sum" if c["top2"] else "max", c["scale"])
        return cfg, gate, moe.alloc_workspace(cfg, DEV)

    cfg, gate, ws = _plan(c, make)
    moe.moe_route_gated(cfg, gate, st["x"], st["Wg"], None, st["bias"], st["logits"], st["ids"], st["w"], ws)
    out = {"ids": st["ids"], "w": st["w"]}
    if c["D"]:
        out["logits"] = st["logits"]
    return out


def _own_lora(st):
    import mixture_experts_layer_gating_gb300 as moe

    c = st["case"]
    T, K, N, r, n = (c[m] for m in ("T", "K", "N", "r", "n"))
    ws = _plan(c, lambda: torch.zeros(moe.moe_lora_workspace_size(T, K, N, r, n), dtype=torch.uint8, device=DEV))
    moe.moe_lora(T, K, N, r, n, st["x"], st["ids"], st["A"], st["B"], st["scales"], st["base"], st["y"], ws)
    return st["y"]


def run(state):
    op = state["case"]["op"]
    if own:
        return _own_norm(state) if op == "norm" else _own_gate(state) if op == "gate" else _own_lora(state)
    return _plain_norm(state) if op == "norm" else _plain_gate(state) if op == "gate" else _plain_lora(state)


# --------------------------------------------------------------- in 64 bits
def _exact_norm(st):
    c = st["case"]
    parts = []
    for a in range(0, c["T"], 2048):
        x = st["x"][a:a + 2048].double()
        if c["add"]:
            x = x + st["res"][a:a + 2048].double()
        one = {"sum": x} if c["add"] else {}
        y = x / torch.sqrt(x.pow(2).sum(1, keepdim=True) / c["D"] + EPS) * st["w"].double()
        if c["y"]:
            one["y"] = y
        if c["q"] >= 0:
            per = c["q"] or c["D"]
            s = torch.stack([b.abs().amax(1) for b in y.split(per, dim=1)], dim=1) / E4M3_MAX
            one["q"] = y / s.repeat_interleave(per, dim=1)
            one["s"] = s
        parts.append(one)
    return {m: torch.cat([p[m] for p in parts]) for m in parts[0]}


def _exact_gate(st):
    c = st["case"]
    L = st["x"].double() @ st["Wg"].double() if c["D"] else st["logits"].double()
    p = torch.sigmoid(L) if c["score"] == "sigmoid" else torch.softmax(L, dim=1)
    v = p + st["bias"].double() if c["bias"] else p.clone()
    size = c["E"] // c["groups"]
    alive = torch.ones_like(v, dtype=torch.bool)
    if c["kept"] < c["groups"]:
        best = torch.stack([m.topk(min(size, 2 if c["top2"] else 1), dim=1).values.sum(1) for m in v.split(size, dim=1)], dim=1)
        alive[:] = False
        for _ in range(c["kept"]):  # the first of the largest, one after another
            at = best.argmax(1, keepdim=True)
            alive.scatter_(1, at * size + torch.arange(size, device=DEV), True)
            best.scatter_(1, at, -math.inf)
    v[~alive] = -math.inf
    ids = []
    for _ in range(c["k"]):
        ids.append(v.argmax(1, keepdim=True))
        v.scatter_(1, ids[-1], -math.inf)
    ids = torch.cat(ids, dim=1)
    w = p.gather(1, ids)
    out = {"ids": ids.to(torch.int32), "w": (w / w.sum(1, keepdim=True) if c["renorm"] else w) * c["scale"]}
    if c["D"]:
        out["logits"] = L
    return out


def _exact_lora(st):
    y = st["base"].double()
    for a in st["ids"].unique().tolist():
        if a < 0:
            continue
        rows = (st["ids"] == a).nonzero()[:, 0]
        low = st["x"][rows].double() @ st["A"][a].double().t()
        y[rows] += float(st["scales"][a]) * (low @ st["B"][a].double().t())
    return y


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_norm(st) if case["op"] == "norm" else _exact_gate(st) if case["op"] == "gate" else _exact_lora(st)
