"""Timed cases of the 4-bit weight operators and the mixture-of-experts layer.

Three operators, each in a plain form (elementary torch operations in 32 bits)
and as the library's calls:

  round_trip  quantise BF16 weights W[N, K] to 4-bit codes with a BF16 scale
              per group of G columns, and read them back as BF16;
  gemv        y[B, N] (fp32) = x[B, K] . W^T for such a weight;
  moe         one mixture-of-experts layer for T tokens: router, top-k choice,
              SwiGLU experts (BF16 or 4-bit) and their weighted sum, in BF16.

A held 4-bit value is a code c in 0..15 that stands for (c - 8) * scale.
"""
import math

import numpy as np
import torch

own = False

SIGMA = 0.02  # standard deviation of the weights


# ---------------------------------------------------------------------------
# The cases.
# ---------------------------------------------------------------------------
def listed():
    return [
        # one expert's projection, quantised when it is loaded
        {"name": "round_trip 2048x6144 g128", "op": "round_trip", "N": 2048, "K": 6144, "G": 128},
        # the largest weight of the checkpoint workload, quantised when it is loaded
        {"name": "round_trip 16384x53248 g32", "op": "round_trip", "N": 16384, "K": 53248, "G": 32},
        # the smallest projection of a decode step: a launch of a few microseconds
        {"name": "gemv 2048x6144 b1 g128", "op": "gemv", "N": 2048, "K": 6144, "B": 1, "G": 128},
        # an odd shape at an odd batch, a partial last group and a partial last row tile
        {"name": "gemv 5001x7003 b5 g32", "op": "gemv", "N": 5001, "K": 7003, "B": 5, "G": 32},
        # a layer's down projection, a few sequences at once
        {"name": "gemv 6144x16384 b4 g64", "op": "gemv", "N": 6144, "K": 16384, "B": 4, "G": 64},
        # the largest weight, one sequence
        {"name": "gemv 16384x53248 b1 g128", "op": "gemv", "N": 16384, "K": 53248, "B": 1, "G": 128},
        # the largest weight, the largest batch
        {"name": "gemv 16384x53248 b16 g128", "op": "gemv", "N": 16384, "K": 53248, "B": 16, "G": 128},
        # a small layer with odd widths, a few tokens
        {"name": "moe bf16 t5 e12k3 1001x333", "op": "moe", "W": "bf16", "T": 5, "E": 12, "k": 3, "H": 1001,
         "F": 333, "score": "softmax"},
        # one token through a layer of 128 experts, 8 chosen: a decode step of one sequence
        {"name": "moe bf16 t1 e128k8 6144x2048", "op": "moe", "W": "bf16", "T": 1, "E": 128, "k": 8, "H": 6144,
         "F": 2048, "score": "softmax"},
        # the same step with 4-bit experts
        {"name": "moe q4 t1 e128k8 6144x2048", "op": "moe", "W": "q4", "G": 128, "T": 1, "E": 128, "k": 8, "H": 6144,
         "F": 2048, "score": "sigmoid"},
        # sixteen sequences, few wide experts, each with several tokens
        {"name": "moe bf16 t16 e8k2 4096x11008", "op": "moe", "W": "bf16", "T": 16, "E": 8, "k": 2, "H": 4096,
         "F": 11008, "score": "softmax"},
        # sixteen sequences over most of the 128 4-bit experts
        {"name": "moe q4 t16 e128k8 6144x2048", "op": "moe", "W": "q4", "G": 32, "T": 16, "E": 128, "k": 8, "H": 6144,
         "F": 2048, "score": "sigmoid"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["round_trip", "gemv", "moe"])
    # half of the cases have widths that are multiples of 128, as models have;
    # the others any width
    step = rng.choice([128, 1])

    def width(lo, hi):
        return max(step, _log(rng, lo, hi) // step * step)

    G = rng.choice([32, 64, 128])
    if op == "moe":
        E = _log(rng, 4, 128)
        c = {"op": op, "W": rng.choice(["bf16", "q4"]), "T": rng.randint(1, 16), "E": E,
             "k": rng.randint(1, min(8, E)), "H": width(256, 6144), "F": width(128, 2048),
             "score": rng.choice(["softmax", "sigmoid"])}
        if c["W"] == "q4":
            c["G"] = G
        return c
    c = {"op": op, "N": width(128, 16384), "K": width(128, 53248), "G": G}
    if op == "gemv":
        c["B"] = rng.randint(1, 16)
    return c


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _normal(shape, sigma, g):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, sigma, generator=g)


def _held(shape, G, g):
    """4-bit codes (two to a byte, the even column low) and group scales of normal weights."""
    M, N, K = shape
    codes = torch.empty((M, N, (K + 1) // 2), dtype=torch.uint8, device="cuda")
    for m in range(M):
        # a group's largest magnitude is about 2.3 to 3 sigma and stands at code 8 +- 7
        c = _normal((N, K + K % 2), 2.6, g).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
        if K % 2:
            c[:, K] = 8
        codes[m] = c[:, 0::2] | (c[:, 1::2] << 4)
    u = torch.rand((M, N, -(-K // G)), device="cuda", generator=g)
    return codes, ((0.8 + 0.4 * u) * (SIGMA / 2.6)).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    if own:
        from decode_gemv_sign_gb300 import wcomp

        s["lib"] = wcomp

    def held(name, shape):
        codes, scales = _held(shape, case["G"], g)
        if own:
            s[name] = s["lib"].q4_pack(codes, scales, shape[2], case["G"])
        else:
            s[name] = (codes, scales)

    if case["op"] == "round_trip":
        N, K = case["N"], case["K"]
        w = _normal((N, K), SIGMA, g)
        # a thousandth of the weights are outliers of five sigma
        flat = w.view(-1)
        at = torch.randint(0, N * K, (max(1, N * K // 1000),), device="cuda", generator=g)
        flat[at] = flat[at] * 5
        s["w"] = w
    elif case["op"] == "gemv":
        held("w", (1, case["N"], case["K"]))
        s["x"] = _normal((case["B"], case["K"]), 1.0, g)
    else:
        E, H, F = case["E"], case["H"], case["F"]
        s["x"] = _normal((case["T"], H), 1.0, g)
        s["router"] = _normal((E, H), SIGMA, g)
        s["bias"] = 0.1 * torch.randn((E,), device="cuda", generator=g) if case["score"] == "sigmoid" else None
        for name, shape in (("gate", (E, F, H)), ("up", (E, F, H)), ("down", (E, H, F))):
            if case["W"] == "bf16":
                s[name] = _normal(shape, SIGMA, g)
            else:
                held(name, shape)
    return s


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def _quantise(w, G):
    """W[N, K] as float codes c - 8 and BF16 scales, groups along the columns."""
    N, K = w.shape
    pad = -K % G
    v = torch.nn.functional.pad(w.float(), (0, pad)).view(N, -1, G)
    scale = (v.abs().amax(-1) / 7).to(torch.bfloat16)
    s = scale.float().unsqueeze(-1)
    q = torch.where(s > 0, (v / s).round().clamp(-7, 7), torch.zeros_like(v))
    return q, scale


def _values(held, K, G):
    """The fp32 values that held codes and scales stand for, [..., N, K]."""
    codes, scales = held
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)[..., :K].float() - 8
    group = torch.arange(K, device=codes.device) // G
    return c * scales.float()[..., group]


def _route(s, case):
    """Chosen experts [T, k] and their weights."""
    logits = s["x"].float() @ s["router"].float().T
    score = torch.softmax(logits, -1) if case["score"] == "softmax" else torch.sigmoid(logits)
    by = score if s["bias"] is None else score + s["bias"]
    ids = torch.sort(by, dim=-1, descending=True, stable=True).indices[:, :case["k"]]
    p = torch.gather(score, 1, ids)
    return ids, p / p.sum(-1, keepdim=True).clamp_min(1e-20)


def _expert_weight(s, name, case, experts):
    """fp32 weights of the given experts (all of them: None)."""
    w = s[name]
    if case["W"] == "bf16":
        return (w if experts is None else w[experts]).float()
    w = w if experts is None else (w[0][experts], w[1][experts])
    return _values(w, case["F"] if name == "down" else case["H"], case["G"])


def _moe(s, case):
    T, E, k = case["T"], case["E"], case["k"]
    ids, p = _route(s, case)
    x = s["x"].float()
    if T * k < E:  # the chosen experts' weights, one copy for each choice
        at = ids.reshape(-1)
        xs = x.repeat_interleave(k, 0).unsqueeze(-1)
        g = _expert_weight(s, "gate", case, at) @ xs
        u = _expert_weight(s, "up", case, at) @ xs
        z = (_expert_weight(s, "down", case, at) @ (g * torch.sigmoid(g) * u)).view(T, k, -1)
        y = (z * p.unsqueeze(-1)).sum(1)
    else:  # every token through every expert, weighted by zero where it was not chosen
        xs = x.T.expand(E, -1, -1)
        g = _expert_weight(s, "gate", case, None) @ xs
        u = _expert_weight(s, "up", case, None) @ xs
        z = _expert_weight(s, "down", case, None) @ (g * torch.sigmoid(g) * u)
        full = torch.zeros((T, E), device=x.device).scatter_(1, ids, p)
        y = (z * full.T.unsqueeze(1)).sum(0).T
    return y.to(torch.bfloat16).contiguous()


def run(state):
    case = state["case"]
    if case["op"] == "round_trip":
        if own:
            c = state["lib"].q4_encode(state["w"], case["G"])
            out = state["lib"].q4_decode(c).view(torch.bfloat16)
            c.free()
            return out
        q, scale = _quantise(state["w"], case["G"])
        return (q * scale.float().unsqueeze(-1)).flatten(1)[:, :case["K"]].to(torch.bfloat16)
    if case["op"] == "gemv":
        if own:
            return state["lib"].q4_gemv(state["w"], state["x"])
        return state["x"].float() @ _values(state["w"], case["K"], case["G"])[0].T
    if own:
        return state["lib"].moe(state["x"], state["router"], state["gate"], state["up"], state["down"], case["k"],
                                scoring=case["score"], bias=state["bias"])
    return _moe(state, case)


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------
def _held_bytes(N, K, G):
    return N * K / 2 + 2 * N * -(-K // G)


def work(case):
    if case["op"] == "round_trip":
        N, K = case["N"], case["K"]
        # read W, write the held form; read it, write the values
        return {"bytes": 4 * N * K + 2 * _held_bytes(N, K, case["G"]), "flops": 4 * N * K}
    if case["op"] == "gemv":
        N, K, B = case["N"], case["K"], case["B"]
        return {"bytes": _held_bytes(N, K, case["G"]) + 2 * B * K + 4 * B * N, "flops": 2 * B * N * K}
    T, E, k, H, F = (case[n] for n in ("T", "E", "k", "H", "F"))
    if case["W"] == "bf16":
        expert = 6 * H * F
    else:
        expert = 2 * _held_bytes(F, H, case["G"]) + _held_bytes(H, F, case["G"])
    # experts that at least one of T tokens chooses, on average
    used = E * (1 - (1 - k / E) ** T)
    return {"bytes": used * expert + 2 * E * H + 4 * T * H, "flops": 2 * T * E * H + 6 * T * k * H * F}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------
def _plain_inputs(case, seed):
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def _held64(held, K, G, m):
    """Matrix m of a held weight in 64 bits."""
    codes, scales = held[0][m], held[1][m].double()
    N = codes.shape[0]
    v = torch.empty((N, 2 * codes.shape[1]), dtype=torch.float64, device=codes.device)
    v[:, 0::2] = (codes % 16).double()
    v[:, 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
    v = v[:, :K] - 8.0
    for j in range(scales.shape[1]):
        v[:, j * G:(j + 1) * G] *= scales[:, j:j + 1]
    return v


def exact(case, seed):
    s = _plain_inputs(case, seed)
    if case["op"] == "round_trip":
        w, G = s["w"], case["G"]
        N, K = w.shape
        out = torch.empty((N, K), dtype=torch.float64, device=w.device)
        rows = max(1, (1 << 26) // K)  # some rows at a time
        for r in range(0, N, rows):
            v = w[r:r + rows].double()
            v = torch.cat((v, v.new_zeros((v.shape[0], -K % G))), 1).unflatten(1, (-1, G))
            step = (torch.amax(torch.abs(v), 2, keepdim=True) / 7.0).to(torch.bfloat16).double()
            q = torch.clamp(torch.round(v / torch.where(step > 0, step, torch.ones_like(step))), -7.0, 7.0)
            out[r:r + rows] = (q * step).reshape(v.shape[0], -1)[:, :K]
        return out
    if case["op"] == "gemv":
        K, G = case["K"], case["G"]
        return s["x"].double() @ _held64(s["w"], K, G, 0).T
    T, k, H, F = case["T"], case["k"], case["H"], case["F"]

    def weight(name, e):
        if case["W"] == "bf16":
            return s[name][e].double()
        return _held64(s[name], F if name == "down" else H, case["G"], e)

    x = s["x"].double()
    logits = torch.einsum("th,eh->te", x, s["router"].double())
    if case["score"] == "softmax":
        e = torch.exp(logits - logits.max(1, keepdim=True).values)
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-logits))
    pick = (score if s["bias"] is None else score + s["bias"].double()).cpu().numpy()
    score = score.cpu().numpy()
    y = torch.zeros((T, H), dtype=torch.float64, device=x.device)
    chosen = np.argsort(-pick, axis=1, kind="stable")[:, :k]
    for e in sorted(set(chosen.reshape(-1).tolist())):
        ts = np.nonzero((chosen == e).any(1))[0]
        p = torch.from_numpy(score[ts, e] / score[ts[:, None], chosen[ts]].sum(1)).to(x.device)
        xe = x[torch.from_numpy(ts).to(x.device)]
        g, u = xe @ weight("gate", e).T, xe @ weight("up", e).T
        z = (g / (1.0 + torch.exp(-g)) * u) @ weight("down", e).T
        y[torch.from_numpy(ts).to(x.device)] += p[:, None] * z
    return y
