"""What is measured of the operators for a few tokens.

Two operators, both bound by the bytes of the weights that they stream:

``layer``   the whole MoE layer for 1 to 32 tokens (router projection, top-k
            softmax, the chosen experts' gate/up and down projections, the
            shared expert and the weighted combine) as one kernel launch:
            ``moe_layer_few``, for bf16, per-column-scaled e4m3 (both layouts)
            and group-scaled 4-bit expert weights.
``linear``  y = x W^T for 1 to 32 rows of x with 4-bit weights and group
            scales: ``moe_linear_w4``.

4-bit weights: row n of a matrix with K inputs is K/2 bytes; byte j holds the
codes of inputs 2j (low nibble) and 2j + 1 (high nibble); the weight is
(code - zero) * scale with one bf16 scale (and one zero point, 8 when none are
given) per row and group of 32, 64 or 128 inputs.

Inputs are the repository's synthetic recipe: x ~ N(0, 1), weights ~ N(0,
0.02), Zipf-skewed routing as a per-expert logit bias -a ln(rank).  A token
whose k-th and (k+1)-th logits are closer than 1e-4 is drawn again: which of
the two experts it takes is a matter of the last bits of a 32-bit sum.
"""
import math

import torch

own = False

DEV = "cuda"
GAP = 1e-4


# ------------------------------------------------------------------- cases
def _layer(name, T, D, E, k, I, Is=0, act="swiglu", w="bf16", zipf=0.0, renorm=True):
    return {"name": name, "op": "layer", "T": T, "D": D, "E": E, "k": k, "I": I, "Is": Is,
            "act": act, "w": w, "zipf": zipf, "renorm": renorm}


def _linear(name, M, K, N, g, zeros, out):
    return {"name": name, "op": "linear", "M": M, "K": K, "N": N, "g": g, "zeros": zeros, "out": out}


def listed():
    return [
        # one user's next token in the smallest layer: nothing but latency
        _layer("layer_toy_T1_bf16", 1, 256, 8, 2, 128),
        # one user's next token, Qwen3-MoE layer
        _layer("layer_qwen3_T1_bf16", 1, 2048, 128, 8, 768),
        # eight users (the repository's Gemma-4 decode batch), GEGLU and a dense MLP of another width
        _layer("layer_gemma4_T8_bf16", 8, 2816, 128, 8, 704, 2112, "geglu_tanh"),
        # a draft of five tokens to be verified, 512 experts with skewed routing
        _layer("layer_qwen35_T5_bf16", 5, 4096, 512, 10, 1024, 1024, zipf=1.1),
        # one user's next token, e4m3 weights with the reduction dimension contiguous
        _layer("layer_ling_T1_fp8nk", 1, 8192, 256, 8, 2048, 2048, w="fp8_e4m3_nk"),
        # sixteen users, e4m3 weights as the checkpoint lays them out: the largest
        _layer("layer_ling_T16_fp8", 16, 8192, 256, 8, 2048, 2048, w="fp8_e4m3"),
        # 4-bit experts: one user, and a batch of odd size over a width that ends inside a tile
        _layer("layer_qwen3_T1_w4", 1, 2048, 128, 8, 768, w="w4_g128"),
        _layer("layer_gemma4_T19_w4", 19, 2816, 128, 8, 704, 2112, "geglu_tanh", w="w4_g64"),
        # a small projection for one token: latency
        _linear("linear_T1_2048x2048", 1, 2048, 2048, 128, False, "bf16"),
        # a square projection at one token, zero points
        _linear("linear_T1_8192x8192", 1, 8192, 8192, 128, True, "bf16"),
        # a ragged batch, small groups, a width that ends inside a tile
        _linear("linear_T13_2816x4224", 13, 2816, 4224, 32, False, "bf16"),
        # the logits of a batch of 32: the largest product, fp32 out
        _linear("linear_T32_4096x131072", 32, 4096, 131072, 64, True, "f32"),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(v, m):
    return max(m, v // m * m)


_CEIL = {"layer": 3.0e9, "linear": 3.3e8}  # bytes: under the largest listed case of the operator


def draw(rng):
    while True:
        if rng.random() < 0.6:
            w = rng.choice(["bf16", "fp8_e4m3", "fp8_e4m3_nk", "w4_g32", "w4_g64", "w4_g128"])
            unit = {"bf16": 8, "fp8_e4m3": 16, "fp8_e4m3_nk": 16}.get(w) or int(w[4:])
            E = _logint(rng, 4, 512)
            c = _layer("", _logint(rng, 1, 32), _mult(_logint(rng, 256, 8192), unit), E,
                       rng.randint(1, min(10, E)), _mult(_logint(rng, 128, 2048), unit),
                       rng.choice([0, 1]) * _mult(_logint(rng, 128, 2304), unit),
                       rng.choice(["swiglu", "geglu_tanh"]), w, rng.choice([0.0, 0.0, 1.1]),
                       rng.random() < 0.8)
            # the weights in hand, and what a plain form holds of them in 32 bits
            if 3 * c["E"] * c["D"] * c["I"] * _wbytes(w) > 1.3e10 or 12 * c["T"] * c["k"] * c["D"] * c["I"] > 3e10:
                continue
        else:
            g = rng.choice([32, 64, 128])
            c = _linear("", _logint(rng, 1, 32), _mult(_logint(rng, 256, 16384), g), _logint(rng, 64, 160000),
                        g, rng.random() < 0.5, rng.choice(["bf16", "f32"]))
        if work(c)["bytes"] <= _CEIL[c["op"]]:
            del c["name"]
            return c


def _wbytes(w):
    return 2.0 if w == "bf16" else 1.0 if w.startswith("fp8") else 0.5 + 2.0 / int(w[4:])


def work(case):
    """Each chosen expert's weights once (their expected number under uniform
    routing), the shared expert's and the router's, x in, y out."""
    if case["op"] == "linear":
        M, K, N, g = case["M"], case["K"], case["N"], case["g"]
        per = 0.5 + (3.0 if case["zeros"] else 2.0) / g
        return {"bytes": per * N * K + 2 * M * K + (4 if case["out"] == "f32" else 2) * M * N,
                "flops": 2.0 * M * N * K}
    T, D, E, k, I, Is = (case[n] for n in ("T", "D", "E", "k", "I", "Is"))
    active = E * (1.0 - (1.0 - k / E) ** T)
    cols = 4 * ((2 * I + D) * active + (2 * Is + D if Is else 0)) if case["w"].startswith("fp8") else 0
    return {"bytes": 3 * D * (I * active + Is) * _wbytes(case["w"]) + cols + 2 * D * E + 4 * T * D,
            "flops": 2.0 * T * D * (3 * (k * I + Is) + E)}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(shape, std, g):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(0.0, std, generator=g)


def _w4(rows, K, group, g):
    """Codes and scales of N(0, 0.02) weights: the scale of a group sets its
    code 7 near the largest of `group` such draws, 2.2 to 2.8 deviations."""
    width = 2.2 + 0.3 * math.log2(group / 32)
    q = torch.empty((*rows, K // 2), dtype=torch.uint8, device=DEV)
    flat = q.view(-1)
    step = 1 << 28
    for a in range(0, flat.numel(), step):
        m = min(step, flat.numel() - a)
        c = _normal((2, m), 7.0 / width, g).round_().clamp_(-8, 7).add_(8).to(torch.uint8)
        flat[a:a + m] = c[0] | (c[1] << 4)
    s = torch.empty((*rows, K // group), dtype=torch.float32, device=DEV).uniform_(0.8, 1.2, generator=g)
    return q, (s * (0.02 * width / 7.0)).to(torch.bfloat16)


def _fp8(shape, col_dims, g):
    """e4m3 codes and per-column scales of N(0, 0.02) weights, a column's
    largest value near 448 (four deviations)."""
    q = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    flat = q.view(-1)
    step = 1 << 28
    for a in range(0, flat.numel(), step):
        m = min(step, flat.numel() - a)
        flat[a:a + m] = _normal((m,), 112.0, g).clamp_(-448, 448).to(torch.float8_e4m3fn)
    s = torch.empty(col_dims, dtype=torch.float32, device=DEV).uniform_(0.8, 1.2, generator=g)
    return q, s * (0.02 / 112.0)


def _expert_weights(w, lead, K, N, g):
    """One projection's weights and scales in the layout of kind `w`, for
    `lead` experts (an empty tuple: one matrix)."""
    if w == "bf16":
        return _normal((*lead, K, N), 0.02, g), None
    if w == "fp8_e4m3":
        return _fp8((*lead, K, N), (*lead, N), g)
    if w == "fp8_e4m3_nk":
        return _fp8((*lead, N, K), (*lead, N), g)
    return _w4((*lead, N), K, int(w[4:]), g)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "linear":
        M, K, N, grp = case["M"], case["K"], case["N"], case["g"]
        q, s = _w4((N,), K, grp, g)
        z = None
        if case["zeros"]:
            z = torch.randint(5, 11, (N, K // grp), dtype=torch.uint8, device=DEV, generator=g)
        out = torch.empty((M, N), dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16, device=DEV)
        return {"case": case, "x": _normal((M, K), 1.0, g), "q": q, "s": s, "z": z, "out": out}
    T, D, E, k, I, Is, w = (case[n] for n in ("T", "D", "E", "k", "I", "Is", "w"))
    st = {"case": case}
    st["Wg"] = _normal((D, E), 0.02, g)
    st["bias"] = None
    if case["zipf"]:
        rank = torch.randperm(E, device=DEV, generator=g).double() + 1.0
        st["bias"] = (-case["zipf"] * rank.log()).float()
    st["W13"], st["s13"] = _expert_weights(w, (E,), D, 2 * I, g)
    st["W2"], st["s2"] = _expert_weights(w, (E,), I, D, g)
    st.update(W13s=None, s13s=None, W2s=None, s2s=None)
    if Is:
        st["W13s"], st["s13s"] = _expert_weights(w, (), D, 2 * Is, g)
        st["W2s"], st["s2s"] = _expert_weights(w, (), Is, D, g)
    x = _normal((T, D), 1.0, g)
    for _ in range(50):
        v = torch.sort(x.double() @ st["Wg"].double() + (0.0 if st["bias"] is None else st["bias"].double()),
                       dim=1, descending=True).values
        near = (v[:, k - 1] - v[:, k] < GAP) if k < E else torch.zeros(T, dtype=torch.bool, device=DEV)
        if not bool(near.any()):
            break
        x = torch.where(near[:, None], _normal((T, D), 1.0, g), x)
    st["x"] = x
    st["out"] = torch.empty((T, D), dtype=torch.bfloat16, device=DEV)
    return st


# --------------------------------------------------------------- plain form
def _plain_w(w, s, kind):
    """Weights [..., K, N] in 32 bits, without the per-column e4m3 scales."""
    if kind == "bf16" or kind == "fp8_e4m3":
        return w.float()
    if kind == "fp8_e4m3_nk":
        return w.float().transpose(-1, -2)
    return _plain_w4(w, s, None).transpose(-1, -2)


def _plain_w4(q, s, z):
    codes = torch.stack((q & 15, q >> 4), dim=-1).float()
    codes = codes.view(*s.shape, -1)  # [..., N, groups, inputs of a group]
    codes = codes - (8.0 if z is None else z.float()[..., None])
    return (codes * s.float()[..., None]).flatten(-2)


def _plain_act(g, u, act):
    if act == "swiglu":
        return g * torch.sigmoid(g) * u
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g))) * u


def _plain_ffn(x, W13, s13, W2, s2, kind, act):
    """x [..., rows, D] through one gated FFN per leading index."""
    fp8 = kind.startswith("fp8")
    gu = torch.matmul(x, _plain_w(W13, s13, kind))
    gu = gu * s13[..., None, :] if fp8 else gu
    I = gu.shape[-1] // 2
    h = _plain_act(gu[..., :I], gu[..., I:], act)
    y = torch.matmul(h, _plain_w(W2, s2, kind))
    return y * s2[..., None, :] if fp8 else y


def _plain_layer(st):
    c = st["case"]
    kind, k, scaled = c["w"], c["k"], c["w"] != "bf16"
    logits = st["x"].double() @ st["Wg"].double()
    if st["bias"] is not None:
        logits = logits + st["bias"].double()
    v, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    v, ids = v[:, :k], ids[:, :k].reshape(-1)
    p = torch.exp(v - v[:, :1])
    p = p / (p.sum(1, keepdim=True) if c["renorm"] else torch.exp(logits - v[:, :1]).sum(1, keepdim=True))
    x = st["x"].float()
    rows = x.repeat_interleave(k, dim=0)[:, None, :]
    as_bytes = lambda t: t.view(torch.uint8)[ids].view(t.dtype) if t.dtype == torch.float8_e4m3fn else t[ids]  # noqa: E731
    y = _plain_ffn(rows, as_bytes(st["W13"]), st["s13"][ids] if scaled else None, as_bytes(st["W2"]),
                   st["s2"][ids] if scaled else None, kind, c["act"])
    out = (y[:, 0, :].view(c["T"], k, -1) * p.float()[:, :, None]).sum(1)
    if c["Is"]:
        out = out + _plain_ffn(x, st["W13s"], st["s13s"], st["W2s"], st["s2s"], kind, c["act"])
    return out.to(torch.bfloat16)


def _plain_linear(st):
    return torch.matmul(st["x"].float(), _plain_w4(st["q"], st["s"], st["z"]).t()).to(st["out"].dtype)


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


def _own_layer(st):
    import mixture_experts_layer_gating_gb300 as moe

    c = st["case"]

    def make():
        cfg = moe.make_config(c["T"], c["D"], c["E"], c["k"], c["I"], c["Is"], c["act"], w_dtype=c["w"],
                              renormalize=c["renorm"])
        return cfg, moe.alloc_workspace(cfg, DEV)

    cfg, ws = _plan(c, make)
    moe.moe_layer_few(cfg, st["x"], st["Wg"], st["bias"], st["W13"], st["s13"], st["W2"], st["s2"],
                      st["W13s"], st["s13s"], st["W2s"], st["s2s"], st["out"], ws)
    return st["out"]


def _own_linear(st):
    import mixture_experts_layer_gating_gb300 as moe

    c = st["case"]
    ws = _plan(c, lambda: torch.zeros(moe.moe_linear_w4_workspace_size(c["M"], c["K"], c["N"]),
                                      dtype=torch.uint8, device=DEV))
    moe.moe_linear_w4(c["M"], c["K"], c["N"], c["g"], st["x"], st["q"], st["s"], st["z"], st["out"], ws)
    return st["out"]


def run(state):
    if own:
        return _own_layer(state) if state["case"]["op"] == "layer" else _own_linear(state)
    return _plain_layer(state) if state["case"]["op"] == "layer" else _plain_linear(state)


# --------------------------------------------------------------- in 64 bits
def _exact_matrix(w, s, kind):
    """One expert's [N, K] matrix in 64 bits, scales included."""
    if kind == "bf16":
        return w.double().t()
    if kind == "fp8_e4m3":
        return w.double().t() * s.double()[:, None]
    if kind == "fp8_e4m3_nk":
        return w.double() * s.double()[:, None]
    return _exact_w4(w, s, None, int(kind[4:]))


def _exact_w4(q, s, z, group):
    N, half = q.shape
    W = torch.empty((N, 2 * half), dtype=torch.float64, device=q.device)
    W[:, 0::2] = (q % 16).double()
    W[:, 1::2] = (q // 16).double()
    per = torch.arange(2 * half, device=q.device) // group
    W -= 8.0 if z is None else z.double()[:, per]
    W *= s.double()[:, per]
    return W


def _exact_expert(x, W13, s13, W2, s2, kind, act):
    up = x @ _exact_matrix(W13, s13, kind).t()
    g, u = up.chunk(2, dim=1)
    if act == "swiglu":
        h = g / (1.0 + torch.exp(-g)) * u
    else:
        h = g * u / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))
    return h @ _exact_matrix(W2, s2, kind).t()


def exact(case, seed):
    st = prepare(case, seed)
    x = st["x"].double()
    if case["op"] == "linear":
        rows = max(1, (1 << 27) // case["K"])
        parts = []
        for a in range(0, case["N"], rows):
            z = st["z"][a:a + rows] if case["zeros"] else None
            parts.append(x @ _exact_w4(st["q"][a:a + rows], st["s"][a:a + rows], z, case["g"]).t())
        return torch.cat(parts, dim=1)
    k, kind, act = case["k"], case["w"], case["act"]
    logits = x @ st["Wg"].double()
    if st["bias"] is not None:
        logits = logits + st["bias"].double()
    probs = torch.softmax(logits, dim=1)
    table = logits.cpu().tolist()
    out = torch.zeros((case["T"], case["D"]), dtype=torch.float64, device=DEV)
    chosen = [sorted(range(case["E"]), key=lambda e, row=row: (-row[e], e))[:k] for row in table]
    users = {}
    for t, row in enumerate(chosen):
        for e in row:
            users.setdefault(e, []).append(t)
    total = torch.stack([probs[t, row].sum() for t, row in enumerate(chosen)])
    for e, ts in users.items():
        one = lambda n: None if st[n] is None else st[n][e]  # noqa: E731
        y = _exact_expert(x[ts], st["W13"][e], one("s13"), st["W2"][e], one("s2"), kind, act)
        p = probs[ts, e] / (total[ts] if case["renorm"] else 1.0)
        out[ts] += p[:, None] * y
    if case["Is"]:
        out += _exact_expert(x, st["W13s"], st["s13s"], st["W2s"], st["s2s"], kind, act)
    return out
