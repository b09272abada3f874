"""Timed cases of the operators that a decode step needs around its weights.

Four operators, each in a plain form (elementary torch operations in 32 bits)
and as the library's calls:

  append    quantise new rows of keys and values k, v [T, H, D] into a paged
            4-bit cache, and read them back as BF16;
  attend    attention of query rows q [T, Hq, D] over such a cache, Hq / H query
            heads to a cached head, with its log-sum-exp and, if asked for, the
            attention weight that every cached token has got so far ("mass");
  evict     for every sequence and cached head keep the last tokens and those of
            the largest mass, in their order, in other pages;
  logprobs  log probability of a given token under each row of logits [T, V],
            the row's entropy and its largest logits with their tokens.

A page holds 64 tokens of one sequence; row b of a table names the pages of
sequence b.  A cached value is a code c in 0..15 that stands for (c - 8) * s,
with a BF16 scale s for each 32 columns of a row.
"""
import math
import random

import torch

own = False

PAGE = 64
GROUP = 32


# ---------------------------------------------------------------------------
# The cases.
# ---------------------------------------------------------------------------
def listed():
    return [
        # a decode step of sixteen sequences: one new token each
        {"name": "append b16 1 token 8x128", "op": "append", "B": 16, "L": 4096, "rows": 1, "H": 8, "D": 128,
         "ragged": True},
        # eight prompts of different lengths enter the cache
        {"name": "append 8 prompts to 8192 8x128", "op": "append", "B": 8, "L": 8192, "rows": 8192, "H": 8, "D": 128,
         "ragged": True},
        # one sequence's decode step, a few thousand tokens: latency counts
        {"name": "attend b1 32/8x128 L4097", "op": "attend", "B": 1, "L": 4097, "rows": 1, "Hq": 32, "H": 8, "D": 128,
         "ragged": False, "window": 0, "mass": False},
        # an odd set: seven query heads to a cached one, several new tokens a sequence, an empty sequence and one of
        # one token, weights gathered for eviction
        {"name": "attend b7 35/5x64 L1001 mass", "op": "attend", "B": 7, "L": 1001, "rows": 4, "Hq": 35, "H": 5,
         "D": 64, "ragged": True, "window": 0, "mass": True},
        # sixteen sequences of all lengths that gather weights for eviction
        {"name": "attend b16 32/8x128 L16384 mass", "op": "attend", "B": 16, "L": 16384, "rows": 1, "Hq": 32, "H": 8,
         "D": 128, "ragged": True, "window": 0, "mass": True},
        # one long document
        {"name": "attend b1 64/8x128 L262143", "op": "attend", "B": 1, "L": 262143, "rows": 1, "Hq": 64, "H": 8,
         "D": 128, "ragged": False, "window": 0, "mass": False},
        # a full batch: the largest
        {"name": "attend b64 64/8x128 L8192", "op": "attend", "B": 64, "L": 8192, "rows": 1, "Hq": 64, "H": 8,
         "D": 128, "ragged": False, "window": 0, "mass": False},
        # one sequence is halved
        {"name": "evict b1 8x128 4096 to 2048", "op": "evict", "B": 1, "L": 4096, "keep": 2048, "recent": 256, "H": 8,
         "D": 128, "ragged": False},
        # a batch of different lengths is brought down to one size
        {"name": "evict b32 8x128 16384 to 2000", "op": "evict", "B": 32, "L": 16384, "keep": 2000, "recent": 100,
         "H": 8, "D": 128, "ragged": True},
        # the tokens that a decode step of four sequences chose, from the head's fp32 logits
        {"name": "logprobs t4 v16384 fp32 top 8", "op": "logprobs", "T": 4, "V": 16384, "k": 8, "dtype": "fp32"},
        # an odd vocabulary, without alternatives
        {"name": "logprobs t33 v50001 bf16", "op": "logprobs", "T": 33, "V": 50001, "k": 0, "dtype": "bf16"},
        # a prompt is scored under the checkpoint workload's vocabulary
        {"name": "logprobs t1024 v151552 fp32 top 20", "op": "logprobs", "T": 1024, "V": 151552, "k": 20,
         "dtype": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "evict", "logprobs"])
    if op == "logprobs":
        T = _log(rng, 1, 1024)
        return {"op": op, "T": T, "V": _log(rng, 1000, 151552), "k": rng.choice([0, rng.randint(1, 32)]),
                "dtype": rng.choice(["fp32", "bf16"])}
    c = {"op": op, "B": _log(rng, 1, 64), "H": rng.choice([1, 2, 4, 5, 8, 16]), "D": rng.choice([64, 128, 128, 256]),
         "ragged": rng.choice([True, True, False])}
    # values of the cache's keys: up to 2^29 for reads of the cache, 2^26 for new rows and moved ones
    most = max(1, (1 << (29 if op == "attend" else 26)) // (c["B"] * c["H"] * c["D"]))
    if op == "append":
        c["L"] = _log(rng, 1, min(most, 16384))
        c["rows"] = rng.choice([1, c["L"]])
    elif op == "evict":
        c["L"] = _log(rng, 2, min(most, 65536))
        c["keep"] = rng.randint(1, c["L"])
        c["recent"] = rng.randint(0, c["keep"])
    else:
        c["L"] = _log(rng, 1, min(most // 4, 131072))
        c["rows"] = rng.choice([1, 1, rng.randint(2, 4)])
        c["Hq"] = c["H"] * rng.choice([1, 2, 3, 4, 7, 8, 16])
        c["window"] = rng.choice([0, 0, _log(rng, 1, c["L"] + 1)])
        c["mass"] = rng.choice([True, False])
    return c


def _lengths(case):
    """Tokens that each sequence holds, the new ones among them: all L, or spread over 0 .. L (their logarithm)."""
    B, L = case["B"], case["L"]
    if not case["ragged"]:
        return [L] * B
    rng = random.Random(B * 1000003 + L)
    lengths = [L] + [_log(rng, 1, L + 1) - 1 for _ in range(B - 1)]
    if B > 4:  # a place of the batch without a sequence, and a sequence that has just begun
        lengths[1:3] = [0, 1]
    return lengths


def _rows(case):
    """New tokens of each sequence: one, or up to as many as `rows` and the sequence's length."""
    lengths = _lengths(case)
    if case.get("rows", 1) == 1:
        return [1] * case["B"]
    rng = random.Random(case["L"])
    if case["op"] == "append":
        return lengths
    return [min(lengths[0], case["rows"])] + [rng.randint(0, min(n, case["rows"])) for n in lengths[1:]]


def _width(case):
    return -(-max(case["L"], 1) // PAGE)


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _normal(shape, g, sigma=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, sigma, generator=g)


def _keys_values(T, case, g):
    """Rows of keys and values; some channels of the keys are large, as keys' are."""
    H, D = case["H"], case["D"]
    k, v = _normal((T, H, D), g), _normal((T, H, D), g)
    channel = torch.where(torch.rand((H, D), device="cuda", generator=g) < 0.03, 5.0, 1.0)
    return k.mul_(channel.to(torch.bfloat16)), v


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(rows):
    at = [0]
    for n in rows:
        at.append(at[-1] + n)
    return _ints(at)


def _cache(s, case, pages, fill, g):
    """The cache, filled from `fill`: (table, lengths) or None.

    Plain: codes as whole numbers in 8 bits and scales, by page, head and place.
    """
    H, D = case["H"], case["D"]
    k = v = None
    if fill is not None:
        table, lengths = fill
        starts = _starts(lengths)
        k, v = _keys_values(sum(lengths), case, g)
    if own:
        from decode_gemv_sign_gb300 import wcomp

        s["lib"] = wcomp
        s["cache"] = wcomp.kv4_create(pages, H, D)
        if fill is not None and len(k):
            wcomp.kv4_append(s["cache"], k, v, table, _ints(lengths), starts)
        return
    s["codes"] = torch.full((2, pages, H, PAGE, D), 8, dtype=torch.uint8, device="cuda")
    s["scales"] = torch.zeros((2, pages, H, PAGE, D // GROUP), dtype=torch.bfloat16, device="cuda")
    if fill is not None and len(k):
        _write(s, k, v, *_places(table, _ints(lengths), starts, len(k)))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "logprobs":
        if own:
            from decode_gemv_sign_gb300 import wcomp

            s["lib"] = wcomp
        T, V = case["T"], case["V"]
        dtype = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        s["logits"] = torch.empty((T, V), dtype=dtype, device="cuda").normal_(0.0, 3.0, generator=g)
        # most given tokens are likely ones: the largest of a few drawn
        some = torch.randint(0, V, (T, 64), device="cuda", generator=g)
        s["ids"] = some.gather(1, s["logits"].gather(1, some).float().argmax(1, keepdim=True)).squeeze(1)
        return s
    B, W = case["B"], _width(case)
    lengths, rows = _lengths(case), _rows(case)
    pages = B * W
    table = torch.randperm(pages, device="cuda", generator=g).to(torch.int32).view(B, W)
    s["table"], s["lengths"] = table, _ints(lengths)
    # one row a sequence needs no starts
    s["starts"] = None if case.get("rows", 1) == 1 else _starts(rows)
    T = sum(rows)
    s["T"] = T
    if case["op"] == "append":
        _cache(s, case, pages, None, g)
        # views of one tensor of projections, as a layer's k and v are
        s["k"], s["v"] = torch.cat(_keys_values(T, case, g), 1).chunk(2, 1)
    elif case["op"] == "attend":
        _cache(s, case, pages, (table, lengths), g)
        s["q"] = _normal((T, case["Hq"], case["D"]), g, 1.5)
        if case["mass"]:
            s["mass"] = torch.rand((B, case["H"], W * PAGE), device="cuda", generator=g)
    else:
        keep = case["keep"]
        other = -(-keep // PAGE)
        _cache(s, case, pages + B * other, (table, lengths), g)
        s["table_out"] = (pages + torch.randperm(B * other, device="cuda", generator=g)).to(torch.int32).view(B, other)
        # few tokens get most of the weight; many have got next to nothing
        s["mass"] = torch.rand((B, case["H"], W * PAGE), device="cuda", generator=g).pow_(8).mul_(20.0)
        s["all"], s["all_starts"] = _ints([keep] * B), _starts([keep] * B)
    return s


# ---------------------------------------------------------------------------
# The plain forms.
# ---------------------------------------------------------------------------
def _places(table, lengths, starts, T):
    """Sequence, position, page and place in it of the T rows."""
    i = torch.arange(T, device=table.device)
    if starts is None:
        seq, back = i, torch.ones_like(i)
    else:
        ends = starts[1:].long()
        seq = torch.searchsorted(ends, i, right=True)
        back = ends[seq] - i
    pos = lengths.long()[seq] - back
    at = pos.clamp_min(0)
    return seq, pos, table.long()[seq, at // PAGE], at % PAGE


def _quantise(w):
    """Codes and BF16 scales of rows [..., D]."""
    v = w.float().unflatten(-1, (-1, GROUP))
    scale = (v.abs().amax(-1) / 7).to(torch.bfloat16)
    s = scale.float().unsqueeze(-1)
    c = torch.where(s > 0, (v / s).round().clamp(-7, 7), torch.zeros_like(v)) + 8
    return c.flatten(-2).to(torch.uint8), scale


def _write(s, k, v, seq, pos, page, place):
    there = pos >= 0
    page, place = page[there], place[there]
    for i, w in enumerate((k, v)):
        codes, scales = _quantise(w[there])
        s["codes"][i, page, :, place] = codes
        s["scales"][i, page, :, place] = scales


def _values(codes, scales):
    return (codes.float() - 8) * scales.float().repeat_interleave(GROUP, -1)


def _append(s):
    at = _places(s["table"], s["lengths"], s["starts"], s["T"])
    _write(s, s["k"], s["v"], *at)
    _, pos, page, place = at
    out = _values(s["codes"][:, page, :, place], s["scales"][:, page, :, place]).transpose(0, 1)
    out = torch.where((pos >= 0)[None, :, None, None], out, torch.zeros_like(out)).to(torch.bfloat16)
    return {"k": out[0], "v": out[1]}


def _attend(s, case):
    T, Hq, H, D = s["T"], case["Hq"], case["H"], case["D"]
    seq, pos, _, _ = _places(s["table"], s["lengths"], s["starts"], T)
    pages = s["table"].long()[seq]  # [T, W]

    def cached(i):  # [T, H, W * PAGE, D]
        return _values(s["codes"][i, pages], s["scales"][i, pages]).transpose(1, 2).flatten(2, 3)

    q = s["q"].float().view(T, H, Hq // H, D)
    score = q @ cached(0).transpose(-1, -2) * D ** -0.5
    j = torch.arange(score.shape[-1], device=q.device)
    seen = j[None] <= pos[:, None]
    if case["window"]:
        seen &= j[None] > pos[:, None] - case["window"]
    score = torch.where(seen[:, None, None], score, torch.full_like(score, -math.inf))
    m = score.amax(-1, keepdim=True).clamp_min(-3e38)
    e = torch.exp(score - m)
    total = e.sum(-1, keepdim=True)
    p = e / total.clamp_min(1e-38)
    v = torch.where(seen[:, None, :, None], cached(1), torch.zeros((), device=q.device))
    out = {"out": (p @ v).view(T, Hq, D).to(torch.bfloat16), "lse": (m + torch.log(total)).view(T, Hq)}
    if case["mass"]:
        out["mass"] = s["mass"].index_add(0, seq, p.sum(2))
    return out


def _evict(s, case):
    keep, recent = case["keep"], case["recent"]
    B, H, M = s["mass"].shape
    n = s["lengths"].long().view(B, 1, 1)
    j = torch.arange(M, device=n.device)
    # the last ones first, then by mass (none is below 0), then what does not exist
    key = torch.where(j >= n - recent, torch.full_like(s["mass"], math.inf), s["mass"])
    key = torch.where(j < n, key, torch.full_like(key, -1.0))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.sort(torch.where(order < n, order, torch.full_like(order, M)), -1).values
    kept = torch.nn.functional.pad(kept, (0, keep - kept.shape[-1]), value=M)
    there = kept < M
    kept = kept.clamp_max(M - 1)
    b, h = torch.arange(B, device=n.device).view(B, 1, 1), torch.arange(H, device=n.device).view(1, H, 1)
    page, place = s["table"].long()[b, kept // PAGE], kept % PAGE
    i = torch.arange(keep, device=n.device)
    page_out, place_out = s["table_out"].long()[:, i // PAGE].view(B, 1, keep).expand(B, H, keep)[there], i.expand(
        B, H, keep)[there] % PAGE
    h_out = h.expand(B, H, keep)[there]
    for w in (s["codes"], s["scales"]):
        w[:, page_out, h_out, place_out] = w[:, page, h, place][:, there]
    mass = s["mass"].new_zeros(B, H, s["table_out"].shape[1] * PAGE)
    mass[..., :keep] = torch.where(there, s["mass"].gather(2, kept), mass[..., :keep])
    # what the new pages hold
    page, place = s["table_out"].long()[:, i // PAGE].view(B, 1, keep), (i % PAGE).view(1, 1, keep)
    out = _values(s["codes"][:, page, h, place], s["scales"][:, page, h, place])
    out = torch.where(there[None, ..., None], out, torch.zeros_like(out)).to(torch.bfloat16).transpose(2, 3)
    return {"kept": torch.where(there, kept, torch.full_like(kept, -1)).int(), "mass": mass,
            "lengths": s["lengths"].clamp_max(keep), "k": out[0], "v": out[1]}


def _logprobs(s, case):
    z = s["logits"].float()
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    logp = z - m - torch.log(total)
    out = {"logprob": logp.gather(1, s["ids"].view(-1, 1)).squeeze(1), "entropy": -(e / total * logp).sum(1)}
    if case["k"]:
        ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :case["k"]]
        out["top_logprobs"], out["top_ids"] = logp.gather(1, ids), ids.int()
    return out


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    if case["op"] == "append":
        return _append(state)
    if case["op"] == "attend":
        return _attend(state, case)
    return _evict(state, case) if case["op"] == "evict" else _logprobs(state, case)


def _own(s, case):
    lib = s["lib"]
    if case["op"] == "logprobs":
        logprob, entropy, top_logprobs, top_ids = lib.logprobs(s["logits"], s["ids"], case["k"])
        out = {"logprob": logprob, "entropy": entropy}
        return {**out, "top_logprobs": top_logprobs, "top_ids": top_ids} if case["k"] else out
    where = (s["table"], s["lengths"], s["starts"])
    if case["op"] == "append":
        lib.kv4_append(s["cache"], s["k"], s["v"], *where)
        k, v = lib.kv4_read(s["cache"], *where, rows=s["T"])
        return {"k": k, "v": v}
    if case["op"] == "attend":
        lse = torch.empty((s["T"], case["Hq"]), dtype=torch.float32, device="cuda")
        mass = s["mass"].clone() if case["mass"] else None
        out = lib.kv4_attend(s["cache"], s["q"], *where, window=case["window"], lse=lse, mass=mass)
        return {"out": out, "lse": lse, "mass": mass} if case["mass"] else {"out": out, "lse": lse}
    B, H, keep, D = case["B"], case["H"], case["keep"], case["D"]
    kept = torch.empty((B, H, keep), dtype=torch.int32, device="cuda")
    lengths, mass = lib.kv4_evict(s["cache"], s["table"], s["lengths"], s["mass"], keep, case["recent"],
                                  s["table_out"], kept=kept)
    # what the new pages hold: `keep` rows of each sequence, zeros where it has fewer
    k, v = lib.kv4_read(s["cache"], s["table_out"], s["all"], s["all_starts"], rows=B * keep)
    return {"kept": kept, "mass": mass, "lengths": lengths, "k": k.view(B, keep, H, D), "v": v.view(B, keep, H, D)}


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "logprobs":
        T, V, k = case["T"], case["V"], case["k"]
        return {"bytes": T * V * (4 if case["dtype"] == "fp32" else 2) + T * (8 + 8 + 8 * k), "flops": 6 * T * V}
    H, D, lengths, rows = case["H"], case["D"], _lengths(case), _rows(case)
    held = H * (D + 2 * 2 * D // GROUP)  # bytes of a token's codes and scales, keys and values
    if case["op"] == "append":
        T = sum(min(r, n) for r, n in zip(rows, lengths))
        return {"bytes": T * (8 * D * H + 2 * held), "flops": 8 * T * H * D}
    if case["op"] == "attend":
        Hq, w = case["Hq"], case["window"]
        tokens = pairs = 0
        for r, n in zip(rows, lengths):
            first = max(0, n - max(r, 1) + 1 - w) if w else 0
            tokens += (n - first) if r else 0
            pairs += sum(min(n - i, w) if w else n - i for i in range(min(r, n)))
        return {"bytes": tokens * (held + (8 * H if case["mass"] else 0)) + 4 * sum(rows) * Hq * (D + 1),
                "flops": 4 * pairs * Hq * D}
    tokens, kept = sum(lengths), sum(min(n, case["keep"]) for n in lengths)
    # read the mass and what is kept; write it, its mass and its places; read it, write its values
    return {"bytes": 4 * H * tokens + kept * (3 * held + 8 * H + 4 * H * D), "flops": H * tokens}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------
def _held64(w):
    """The values that rows [..., D] have in 4 bits."""
    groups = w.double().reshape(*w.shape[:-1], w.shape[-1] // 32, 32)
    step = (torch.amax(torch.abs(groups), -1, keepdim=True) / 7.0).to(torch.bfloat16).double()
    steps = torch.where(step > 0, step, torch.ones_like(step))
    return (torch.clamp(torch.round(groups / steps), -7.0, 7.0) * step).reshape(w.shape)


def exact(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = "cuda"
    if case["op"] == "logprobs":
        T, V, k = case["T"], case["V"], case["k"]
        dtype = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        logits = torch.empty((T, V), dtype=dtype, device=dev).normal_(0.0, 3.0, generator=g)
        some = torch.randint(0, V, (T, 64), device=dev, generator=g)
        ids = some.gather(1, logits.gather(1, some).float().argmax(1, keepdim=True)).squeeze(1)
        parts = []
        for t in range(0, T, 64):  # some rows at a time
            z = logits[t:t + 64].double()
            logp = z - torch.logsumexp(z, 1, keepdim=True)
            part = [logp[torch.arange(len(z), device=dev), ids[t:t + 64]], -(torch.exp(logp) * logp).sum(1)]
            if k:
                order = torch.argsort(-z, dim=1, stable=True)[:, :k]
                part += [torch.take_along_dim(logp, order, 1), order.int()]
            parts.append(part)
        out = [torch.cat(p) for p in zip(*parts)]
        return dict(zip(("logprob", "entropy", "top_logprobs", "top_ids"), out))
    B, H, D, W = case["B"], case["H"], case["D"], -(-max(case["L"], 1) // 64)
    lengths, rows = _lengths(case), _rows(case)
    torch.randperm(B * W, device=dev, generator=g)  # the pages' order, which no result depends on
    if case["op"] == "append":
        k, v = _keys_values(sum(rows), case, g)
        out = {"k": _held64(k), "v": _held64(v)}
        at = 0
        for n, r in zip(lengths, rows):  # rows that would stand before the first position
            out["k"][at:at + max(0, r - n)] = 0
            out["v"][at:at + max(0, r - n)] = 0
            at += r
        return out
    k, v = _keys_values(sum(lengths), case, g)
    if case["op"] == "attend":
        Hq, w = case["Hq"], case["window"]
        q = _normal((sum(rows), Hq, D), g, 1.5).double()
        out = torch.zeros((sum(rows), Hq, D), dtype=torch.float64, device=dev)
        lse = torch.full((sum(rows), Hq), -math.inf, dtype=torch.float64, device=dev)
        mass = torch.rand((B, H, W * 64), device=dev, generator=g).double() if case["mass"] else None
        row = first = 0
        for b in range(B):
            n = lengths[b]
            kb, vb = _held64(k[first:first + n]), _held64(v[first:first + n])
            first += n
            for r in range(rows[b]):
                last = n - rows[b] + r  # this row's position
                lo = max(0, last - w + 1) if w else 0
                if last >= lo:
                    x = q[row].reshape(H, Hq // H, D)
                    z = torch.einsum("hgd,nhd->hgn", x, kb[lo:last + 1]) / math.sqrt(D)
                    lse[row] = torch.logsumexp(z, -1).flatten()
                    p = torch.softmax(z, -1)
                    out[row] = torch.einsum("hgn,nhd->hgd", p, vb[lo:last + 1]).reshape(Hq, D)
                    if mass is not None:
                        mass[b, :, lo:last + 1] += p.sum(1)
                row += 1
        return {"out": out, "lse": lse, "mass": mass} if case["mass"] else {"out": out, "lse": lse}
    keep, recent = case["keep"], case["recent"]
    torch.randperm(B * -(-keep // 64), device=dev, generator=g)
    mass = torch.rand((B, H, W * 64), device=dev, generator=g).pow_(8).mul_(20.0)
    kept = torch.full((B, H, keep), -1, dtype=torch.int32, device=dev)
    left = torch.zeros((B, H, -(-keep // 64) * 64), dtype=torch.float64, device=dev)
    ks, vs = (torch.zeros((B, keep, H, D), dtype=torch.float64, device=dev) for _ in range(2))
    first = 0
    for b in range(B):
        n = lengths[b]
        m, tail = min(n, keep), min(n, recent)
        kb, vb = k[first:first + n], v[first:first + n]
        first += n
        for h in range(H):
            best = torch.argsort(-mass[b, h, :n - tail], stable=True)[:m - tail]
            at = torch.cat((torch.sort(best).values, torch.arange(n - tail, n, device=dev)))
            kept[b, h, :m] = at.int()
            left[b, h, :m] = mass[b, h, at].double()
            ks[b, :m, h], vs[b, :m, h] = _held64(kb[at, h]), _held64(vb[at, h])
    return {"kept": kept, "mass": left, "lengths": torch.tensor([min(n, keep) for n in lengths], dtype=torch.int32,
                                                                device=dev), "k": ks, "v": vs}
