"""Greedy decoding through one quantised expert block, as a serving loop would run it.

    python -m decode_gemv_sign_gb300.expert_block --tokens 4 --steps 16
    python -m decode_gemv_sign_gb300.expert_block --tokens 4 --steps 300 --context 512 --keep 128

A step takes the last token of each of 1 to 16 sequences through
  * with --context, attention over a cache of keys and values in 4 bits (kv4_append,
    kv4_attend) and a residual addition,
  * a projection in 4 bits (q4_gemv) and a residual addition,
  * a mixture-of-experts layer, its experts in 4 bits (moe), and a second one,
  * a lossless head (encode, gemv), whose largest logit is the next token (with
    --context by logprobs, which gives its log probability and the entropy too).
The weights are random.  They are quantised and laid out once; a step is
captured in a CUDA graph and replayed, the tokens staying on the device.  With
--keep the cache is brought down to that many tokens (kv4_evict) whenever it has
reached --context.
Prints one JSON line: the bytes the weights take and the time of a step.
"""
from __future__ import annotations

import argparse
import json

import torch

from decode_gemv_sign_gb300 import wcomp


class CachedAttention:
    """Attention of `sequences` sequences over a 4-bit cache of up to `most` tokens each, its projections in 4 bits.

    qkv [(heads + 2 kv_heads) dim, H] gives a token's queries, keys and values (without positions), out [H, heads
    dim] takes the heads together.  The weight that every cached token gets is gathered, and `evict` keeps the
    tokens of largest weight: for that each sequence has a second set of pages.
    """

    def __init__(self, qkv, out, heads: int, kv_heads: int, dim: int, sequences: int, most: int, group: int = 64):
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.qkv, self.out = wcomp.q4_encode(qkv, group), wcomp.q4_encode(out, group)
        width = -(-most // 64)
        self.most = width * 64
        self.cache = wcomp.kv4_create(2 * sequences * width, kv_heads, dim)
        pages = torch.arange(2 * sequences * width, dtype=torch.int32, device=qkv.device)
        self.table, self.spare = pages.view(2, sequences, width).unbind(0)
        self.lengths = torch.zeros(sequences, dtype=torch.int32, device=qkv.device)
        self.mass = torch.zeros(sequences, kv_heads, width * 64, device=qkv.device)

    def __call__(self, x):
        """x [T, H] of one new token a sequence: adds it to the cache and returns what it attends to, fp32 [T, H]."""
        self.lengths += 1
        y = wcomp.q4_gemv(self.qkv, x).bfloat16().view(len(x), -1, self.dim)
        q, k, v = y.split((self.heads, self.kv_heads, self.kv_heads), 1)
        wcomp.kv4_append(self.cache, k, v, self.table, self.lengths)
        o = wcomp.kv4_attend(self.cache, q, self.table, self.lengths, mass=self.mass)
        return wcomp.q4_gemv(self.out, o.view(len(x), -1))

    def evict(self, keep: int, recent: int):
        """Keep the last `recent` tokens and those of largest weight.  Tables and lengths stay where they are."""
        lengths, _ = wcomp.kv4_evict(self.cache, self.table, self.lengths, self.mass.clone(), keep, recent, self.spare,
                                     mass_out=self.mass)
        self.lengths.copy_(lengths)
        was = self.table.clone()
        self.table.copy_(self.spare)
        self.spare.copy_(was)

    def weights(self):
        return self.qkv, self.out

    def free(self):
        for c in (self.qkv, self.out, self.cache):
            c.free()


class ExpertBlock:
    """embed [V, H], proj [H, H], router [E, H], gate and up [E, F, H], down [E, H, F], head [V, H]: BF16 on one GPU.

    Keeps the embedding and the router as they are, the head losslessly coded
    and everything else in 4 bits with one scale per `group` columns.  `attention`
    (a CachedAttention) comes first if it is given.
    """

    def __init__(self, embed, proj, router, gate, up, down, head, top_k: int, group: int = 64, scoring="softmax",
                 attention=None):
        self.embed, self.router = embed, router
        self.proj = wcomp.q4_encode(proj, group)
        self.experts = [wcomp.q4_encode(w, group) for w in (gate, up, down)]
        self.head = wcomp.encode(head, "bytesplit")
        self.top_k, self.scoring, self.attention = top_k, scoring, attention

    @classmethod
    def random(cls, V, H, F, E, top_k, group=64, seed=0, device="cuda", attention=None):
        """Random weights.  attention: (heads, kv_heads, dim, sequences, most tokens) or None."""
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def draw(*shape):
            w = torch.empty(*shape, dtype=torch.bfloat16, device=device)
            return w.normal_(0.0, shape[-1] ** -0.5, generator=g)

        embed = torch.empty(V, H, dtype=torch.bfloat16, device=device).normal_(0.0, 1.0, generator=g)
        weights = draw(H, H), draw(E, H), draw(E, F, H), draw(E, F, H), draw(E, H, F), draw(V, H)
        if attention is not None:
            heads, kv_heads, dim, sequences, most = attention
            attention = CachedAttention(draw((heads + 2 * kv_heads) * dim, H), draw(H, heads * dim), heads, kv_heads,
                                        dim, sequences, most, group)
        return cls(embed, *weights, top_k, group, attention=attention)

    def _held(self):
        return (self.proj, *self.experts, *(self.attention.weights() if self.attention else ()))

    def bytes(self) -> int:
        """What the coded weights take on the device."""
        return sum(c.info()["bytes"] for c in self._held()) + self.head.info()["serialized_bytes"]

    def hidden(self, x):
        """x [T, H] through the attention, if there is one, the projection and the experts."""
        if self.attention is not None:
            x = (x.float() + self.attention(x)).bfloat16()
        r = (x.float() + wcomp.q4_gemv(self.proj, x)).bfloat16()
        return r + wcomp.moe(r, self.router, *self.experts, self.top_k, scoring=self.scoring)

    def step(self, tokens):
        """The next token of each sequence, int64 [T]."""
        return wcomp.gemv(self.head, self.hidden(self.embed[tokens])).argmax(1)

    def scored_step(self, tokens):
        """The next token of each sequence, int64 [T], its log probability and the entropy it was chosen from."""
        logits = wcomp.gemv(self.head, self.hidden(self.embed[tokens]))
        _, entropy, top, ids = wcomp.logprobs(logits, top_k=1)
        return ids[:, 0].long(), top[:, 0], entropy

    def graph(self, tokens, logprob=None, entropy=None):
        """A CUDA graph whose replay replaces `tokens` by the next ones (and the others, if given, by what they had)."""

        def step():
            if logprob is None:
                tokens.copy_(self.step(tokens))
            else:
                for to, value in zip((tokens, logprob, entropy), self.scored_step(tokens)):
                    to.copy_(value)

        keep, cached = tokens.clone(), self.attention
        if cached is not None:
            if (cached.lengths >= cached.most).any():
                raise ValueError("the cache has no place for a token: evict first")
            weights = cached.mass.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()  # first calls set the library's buffers up
            tokens.copy_(keep)
            if cached is not None:  # as if it had not been
                cached.lengths -= 1
                cached.mass.copy_(weights)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        return graph

    def free(self):
        for c in (self.proj, *self.experts, self.head, *([self.attention] if self.attention else [])):
            c.free()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=4, help="sequences, 1 to 16")
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--vocabulary", type=int, default=16384)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--ffn", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--top-k", type=int, default=4)
    ap.add_argument("--group", type=int, default=64, choices=[32, 64, 128])
    ap.add_argument("--context", type=int, default=0, help="tokens of the cache; 0: no attention")
    ap.add_argument("--keep", type=int, default=0, help="tokens left when the cache is full; 0: none is evicted")
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--kv-heads", type=int, default=4)
    ap.add_argument("--dim", type=int, default=128, choices=[64, 128, 256])
    a = ap.parse_args()
    if a.context:
        return attended(a)
    block = ExpertBlock.random(a.vocabulary, a.hidden, a.ffn, a.experts, a.top_k, a.group)
    tokens = torch.arange(a.tokens, device="cuda")
    graph = block.graph(tokens)
    out = torch.empty(a.steps, a.tokens, dtype=torch.int64, device="cuda")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for i in range(a.steps):
        graph.replay()
        out[i].copy_(tokens)
    end.record()
    end.synchronize()
    wcomp.device_check()
    print(json.dumps({"weight_bytes": block.bytes(), "us_per_step": round(1e3 * start.elapsed_time(end) / a.steps, 1),
                      "tokens": out.t().tolist()}))


def attended(a):
    if a.steps > a.context and not 0 < a.keep < a.context:
        raise SystemExit("more steps than --context tokens want a --keep below it")
    block = ExpertBlock.random(a.vocabulary, a.hidden, a.ffn, a.experts, a.top_k, a.group,
                               attention=(a.heads, a.kv_heads, a.dim, a.tokens, a.context))
    tokens = torch.arange(a.tokens, device="cuda")
    logprob, entropy = (torch.empty(a.tokens, device="cuda") for _ in range(2))
    graph = block.graph(tokens, logprob, entropy)
    out = torch.empty(a.steps, a.tokens, dtype=torch.int64, device="cuda")
    scores = torch.empty(2, a.steps, a.tokens, device="cuda")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    held = evictions = 0
    for i in range(a.steps):
        if held == a.context:
            block.attention.evict(a.keep, a.keep // 4)
            held, evictions = a.keep, evictions + 1
        graph.replay()
        held += 1
        out[i].copy_(tokens)
        scores[0, i].copy_(logprob)
        scores[1, i].copy_(entropy)
    end.record()
    end.synchronize()
    wcomp.device_check()
    print(json.dumps({"weight_bytes": block.bytes(), "cache_bytes": block.attention.cache.info()["bytes"],
                      "us_per_step": round(1e3 * start.elapsed_time(end) / a.steps, 1), "evictions": evictions,
                      "mean_logprob": round(float(scores[0].mean()), 4), "mean_entropy": round(float(scores[1].mean()), 4),
                      "tokens": out.t().tolist()}))


if __name__ == "__main__":
    main()
