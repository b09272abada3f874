"""Plain numpy definitions, in 64 bits, of the 4-bit key/value cache's calls and of log probabilities.

Test infrastructure only; shares no code with the library.  BF16 data comes
and goes as uint16 bit patterns; a sequence's keys and values are [n, H, D].
"""
from __future__ import annotations

import numpy as np

from oracle.q4_moe_oracle import EPS, f64, q4_encode, q4_values

GROUP = 32
PAGE = 64


def held(w: np.ndarray) -> np.ndarray:
    """The values that BF16 rows [..., D] have in 4 bits."""
    codes, scales = q4_encode(w, GROUP)
    return q4_values(codes, scales, GROUP)


def seen(n: int, rows: int, i: int, window: int) -> tuple:
    """First and one past the last position that row i of `rows` sees in a sequence of n tokens."""
    last = n - rows + i
    return (max(0, last - window + 1) if window else 0), max(last + 1, 0)


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, window: int = 0):
    """Rows q [T, Hq, D] (values) of one sequence over its keys and values [n, H, D] (values).

    Returns out, lse, mass [H, n], and how far results of the library may be from
    them.  Products of a code and an activation are exact; a score is summed in fp32
    over D / 32 scaled groups of at most two steps each and scaled (D / 4 + 8 steps of
    at most EPS of the sum of magnitudes, an exponential's 2^-21 besides); sums over n tokens are fp32
    (n EPS); the weights that multiply v are rounded to fp16 (2^-11), out to BF16 (2^-8).

    Those weights are x = p * s under a power of two 2^k that brings the largest scale of the
    sequence's values, s_max in [2^E, 2^(E + 1)), to [2^14, 2^15): k = 14 - E.  Below
    2^-14 fp16 has steps of 2^-24, so x errs by up to 2^-25, which is 2^(-25 - k) = 2^(E - 39) <= 2^-39
    s_max before the power of two.  Times a code of at most 7 that is 2^-39 of the largest value
    of the head, 7 s_max; the scale's own rounding to BF16 adds 2^-8 of that.  Each of the n terms
    may err by as much, and the sum is divided by one of at least 1.
    """
    T, Hq, D = q.shape
    n, H, _ = k.shape
    share = Hq // H
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    out_tol, lse_tol = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    mass, mass_tol = np.zeros((H, n)), np.zeros((H, n))
    with np.errstate(all="ignore"):
        for i in range(T):
            lo, hi = seen(n, T, i, window)
            if lo >= hi:
                continue
            for hq in range(Hq):
                h = hq // share
                z = scale * (k[lo:hi, h] @ q[i, hq])
                mag = abs(scale) * (np.abs(k[lo:hi, h]) @ np.abs(q[i, hq]))
                m = z.max()
                e = np.exp(z - m)
                p = e / e.sum()
                dz = EPS * ((D / 4 + 8) * mag + 4 * np.abs(z - m)) + 2.0 ** -21
                off = (p * dz).sum() + (hi - lo) * EPS  # of the sum of exponentials
                out[i, hq] = p @ v[lo:hi, h]
                lse[i, hq] = m + np.log(e.sum())
                out_tol[i, hq] = 2.0 ** -8 * np.abs(out[i, hq]) + (p * (dz + 2 * off + 2.0 ** -11)) @ np.abs(v[lo:hi, h])
                out_tol[i, hq] += (hi - lo) * 2.0 ** -39 * (1 + 2.0 ** -8) * np.nanmax(np.abs(v[:, h]))
                lse_tol[i, hq] = 2 * off + dz.max() + 4 * EPS * (abs(m) + abs(lse[i, hq]))
                mass[h, lo:hi] += p
                mass_tol[h, lo:hi] += p * (dz + lse_tol[i, hq] + T * share * EPS)
    return out, lse, mass, out_tol + 1e-37, lse_tol, mass_tol + 1e-37


def evict(mass: np.ndarray, n: int, keep: int, recent: int) -> np.ndarray:
    """Positions that one head of a sequence of n tokens keeps, ascending."""
    if n <= keep:
        return np.arange(n)
    m = np.asarray(mass[:n - recent], np.float64)
    rank = np.where(np.isnan(m), -np.inf, m)
    # a NaN ranks below minus infinity too
    order = sorted(range(n - recent), key=lambda j: (np.isnan(m[j]), -rank[j], j))
    return np.array(sorted(order[:keep - recent]) + list(range(n - recent, n)), np.int64)


def logprobs(z: np.ndarray, ids, top_k: int, scale: float = 1.0):
    """(logprob, entropy, lse, top_logprobs, top_ids) of rows z [T, V] (values), and a bound of the errors of logprobs.

    A term exp(scale (z - m)) is off by 2^-21 and twice the rounding of its exponent; sums over V
    terms run in parallel parts of at most V / 128 + 64 steps.
    """
    T, V = z.shape
    lp, ent, lse = np.zeros(T), np.zeros(T), np.zeros(T)
    top, top_ids = np.zeros((T, top_k)), np.zeros((T, top_k), np.int32)
    tol = np.zeros(T)
    with np.errstate(all="ignore"):
        for t in range(T):
            x = z[t].astype(np.float64)
            order = sorted(range(V), key=lambda j: (np.isnan(x[j]), -x[j] if not np.isnan(x[j]) else 0.0, j))
            top_ids[t] = order[:top_k]
            x = x * scale
            m = np.nan if np.isnan(x).any() else x.max()
            d = x - m
            e = np.exp(d)
            m_ok = np.isfinite(m)
            # everything from the distances to the largest, which leaves 1 out of the sum: 64 bits lose it too
            e[np.argmax(x) if m_ok else 0] = 0.0
            log_sum = np.log1p(e.sum()) if m_ok else np.nan
            lse[t] = m + log_sum
            logp = d - log_sum
            p = np.exp(logp)
            ent[t] = -np.where(p > 0, p * np.where(p > 0, logp, 0.0), 0.0).sum() if m_ok else np.nan
            top[t] = logp[top_ids[t]]
            if ids is not None:
                i = int(ids[t])
                lp[t] = 0.0 if i < 0 else np.nan if i >= V else logp[i]
            d = np.where(p > 0, -d, 0.0)
            # the error of the terms, but for the largest, which is exact
            tol[t] = ((p * (2.0 ** -21 + 3 * EPS * d)).sum() + (1 - p.max()) * (V / 128 + 64) * EPS) if m_ok else 0.0
    return lp, ent, lse, top, top_ids, tol
