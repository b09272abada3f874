"""Plain numpy definitions, in 64 bits, of the 4-bit weights and the mixture-of-experts layer.

Test infrastructure only; shares no code with the library.  BF16 data comes
and goes as uint16 bit patterns.
"""
from __future__ import annotations

import numpy as np

EPS = 2.0 ** -23  # one step of an fp32 sum (the tensor cores may truncate)


def f64(bits: np.ndarray) -> np.ndarray:
    """Values of BF16 bit patterns."""
    return (np.ascontiguousarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def bf16(v: np.ndarray) -> np.ndarray:
    """Bits of the nearest BF16 (ties to even) of 64-bit values, rounded once; NaN becomes 0x7FC0."""
    v = np.asarray(v, np.float64)
    with np.errstate(all="ignore"):
        a = np.abs(v)
        e = np.floor(np.log2(np.where((a > 0) & np.isfinite(a), a, 1.0)))
        ulp = 2.0 ** (np.maximum(e, -126) - 7)
        r = np.where(np.isfinite(v), np.rint(v / ulp) * ulp, v)  # rint is half to even
        r = np.where(np.abs(r) >= 2.0 ** 128, np.copysign(np.inf, r), r)
        out = (r.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    return np.where(np.isnan(v), np.uint16(0x7FC0), out)


def q4_encode(w: np.ndarray, group: int):
    """codes uint8 [..., N, K] (one per weight) and scale bits [..., N, ceil(K / group)] of BF16 bits w."""
    v = f64(w)
    K = v.shape[-1]
    groups = -(-K // group)
    codes = np.full(v.shape, 8, np.uint8)
    scales = np.zeros((*v.shape[:-1], groups), np.uint16)
    for j in range(groups):
        g = v[..., j * group:(j + 1) * group]
        bad = ~np.isfinite(g).all(-1)
        m = np.where(bad, 0.0, np.abs(np.where(np.isfinite(g), g, 0.0)).max(-1))
        s = bf16(m / 7.0)
        sv = f64(s)
        ok = (sv > 0) & ~bad
        q = np.rint(np.where(ok[..., None], np.where(np.isfinite(g), g, 0.0) / np.where(ok, sv, 1.0)[..., None], 0.0))
        codes[..., j * group:(j + 1) * group] = (np.clip(q, -7, 7) + 8).astype(np.uint8)
        scales[..., j] = np.where(bad, np.uint16(0x7FC0), s)
    return codes, scales


def q4_values(codes: np.ndarray, scales: np.ndarray, group: int) -> np.ndarray:
    K = codes.shape[-1]
    return (codes.astype(np.float64) - 8.0) * f64(scales)[..., np.arange(K) // group]


def pack_codes(codes: np.ndarray) -> np.ndarray:
    """Two codes a byte, the even column low; an odd row ends with code 8."""
    if codes.shape[-1] % 2:
        codes = np.concatenate([codes, np.full((*codes.shape[:-1], 1), 8, np.uint8)], -1)
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def gemv(w: np.ndarray, x: np.ndarray, group: int):
    """y [B, N] of weight values w [N, K], and how far an fp32 sum may be from it.

    Products of 4-bit integers and BF16 are exact in fp32.  A result is at most
    K / group scaled sums, each of at most eight 16-term tensor-core steps, and
    a few dozen additions over warps and blocks: every addition errs by at most
    EPS of the sum of magnitudes.
    """
    xv = f64(x)
    steps = -(-w.shape[1] // group) + 64
    return xv @ w.T, steps * EPS * (np.abs(xv) @ np.abs(w).T) + 1e-40


def silu(g):
    return g / (1.0 + np.exp(-g))


def scores(x, router, scoring):
    """Scores [T, E] and how far fp32 logits may move each of them (relative for softmax, absolute for sigmoid)."""
    xv, rv = f64(x), f64(router)
    logits = xv @ rv.T
    dl = (x.shape[1] / 16 + 64) * EPS * (np.abs(xv) @ np.abs(rv).T).max(1, keepdims=True)
    if scoring == "softmax":
        e = np.exp(logits - logits.max(1, keepdims=True))
        s = e / e.sum(1, keepdims=True)
        return s, s * (2.0 * dl + 64 * EPS)
    s = 1.0 / (1.0 + np.exp(-logits))
    return s, s * (dl + 8 * EPS)


TWO_BF16 = 2.0 ** -16  # what holding a hidden value as two BF16 parts may lose of it: 2^-8 of 2^-8
FP16 = 2.0 ** -11  # in fp16 under a power of two: 11 significant bits


def moe(x, gate, up, down, ids, weights, held=TWO_BF16):
    """y [T, H] for a given choice and its weights, in 64 bits, and the fp32 kernel's error bound.

    gate, up [E, F, H] and down [E, H, F] are values; ids, weights [T, k].
    The hidden values lose at most `held` of themselves between the products
    (TWO_BF16 for BF16 experts, FP16 for 4-bit ones, where a value below 2^-31
    of the largest of its 32 neighbours also errs by 2^-39 of that); sums are in
    fp32; y is rounded once to BF16, whose 8 significant bits err by at most
    2^-8 of a value (1 + 2^-8 rounds to 1).
    """
    xv = f64(x)
    T, H = xv.shape
    F = gate.shape[1]
    eh, ef = (H / 16 + 64) * EPS, (F * ids.shape[1] / 16 + 64) * EPS
    y, dy = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for e, v in zip(ids[t], weights[t]):
            g, u = gate[e] @ xv[t], up[e] @ xv[t]
            dg, du = eh * (np.abs(gate[e]) @ np.abs(xv[t])), eh * (np.abs(up[e]) @ np.abs(xv[t]))
            h = silu(g) * u
            # |silu'| <= 1.1
            dh = 1.1 * dg * (np.abs(u) + du) + (np.abs(silu(g)) + 1.1 * dg) * du + (held + 16 * EPS) * np.abs(h) + 2.0 ** -39 * np.abs(h).max()
            y[t] += v * (down[e] @ h)
            dy[t] += abs(v) * (np.abs(down[e]) @ (dh + ef * np.abs(h)))
    return y, dy + 2.0 ** -8 * (np.abs(y) + dy) + 1e-38
