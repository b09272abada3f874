"""Greedy decoding through one quantised expert block, as a serving loop would run it.

    python -m decode_gemv_sign_gb300.expert_block --tokens 4 --steps 16

A step takes the last token of each of 1 to 16 sequences through
  * a projection in 4 bits (q4_gemv) and a residual addition,
  * a mixture-of-experts layer, its experts in 4 bits (moe), and a second one,
  * a lossless head (encode, gemv), whose largest logit is the next token.
The weights are random.  They are quantised and laid out once; a step is
captured in a CUDA graph and replayed, the tokens staying on the device.
Prints one JSON line: the bytes the weights take and the time of a step.
"""
from __future__ import annotations

import argparse
import json

import torch

from decode_gemv_sign_gb300 import wcomp


class ExpertBlock:
    """embed [V, H], proj [H, H], router [E, H], gate and up [E, F, H], down [E, H, F], head [V, H]: BF16 on one GPU.

    Keeps the embedding and the router as they are, the head losslessly coded
    and everything else in 4 bits with one scale per `group` columns.
    """

    def __init__(self, embed, proj, router, gate, up, down, head, top_k: int, group: int = 64, scoring="softmax"):
        self.embed, self.router = embed, router
        self.proj = wcomp.q4_encode(proj, group)
        self.experts = [wcomp.q4_encode(w, group) for w in (gate, up, down)]
        self.head = wcomp.encode(head, "bytesplit")
        self.top_k, self.scoring = top_k, scoring

    @classmethod
    def random(cls, V, H, F, E, top_k, group=64, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def draw(*shape):
            w = torch.empty(*shape, dtype=torch.bfloat16, device=device)
            return w.normal_(0.0, shape[-1] ** -0.5, generator=g)

        embed = torch.empty(V, H, dtype=torch.bfloat16, device=device).normal_(0.0, 1.0, generator=g)
        return cls(embed, draw(H, H), draw(E, H), draw(E, F, H), draw(E, F, H), draw(E, H, F), draw(V, H), top_k, group)

    def bytes(self) -> int:
        """What the coded weights take on the device."""
        return sum(c.info()["bytes"] for c in (self.proj, *self.experts)) + self.head.info()["serialized_bytes"]

    def hidden(self, x):
        """x [T, H] through the projection and the experts."""
        r = (x.float() + wcomp.q4_gemv(self.proj, x)).bfloat16()
        return r + wcomp.moe(r, self.router, *self.experts, self.top_k, scoring=self.scoring)

    def step(self, tokens):
        """The next token of each sequence, int64 [T]."""
        return wcomp.gemv(self.head, self.hidden(self.embed[tokens])).argmax(1)

    def graph(self, tokens):
        """A CUDA graph whose replay replaces `tokens` by the next ones."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step(tokens)  # first calls set the library's buffers up
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            tokens.copy_(self.step(tokens))
        return graph

    def free(self):
        for c in (self.proj, *self.experts, self.head):
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
    a = ap.parse_args()
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


if __name__ == "__main__":
    main()
