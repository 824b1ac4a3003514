"""Serve a small decoder with random Q8_0 weights from a paged key-value cache: ragged prompts in chunks, then greedy
decoding replayed from a CUDA graph.

Every layer of a step is: q, k, v (gemv_parts) -> norms, rotation and append (rope_append) -> attention (attn_prefill or
attn_decode) -> output projection, residual and norm (gemv_residual_norm) -> gated pair (gemv_glu) -> down projection,
residual and the next norm; kv_slots gives the step its pages, positions and slots, gemv_argmax ends it.

    python examples/serve.py --requests 8 --prompt 300 --tokens 64 --cache q8 --window 256
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import q8_block_quantized_gemv_gb300 as q8  # noqa: E402

EPS = 1e-6
CHUNK = 512  # rows of a step: the most the projections take


class Weight:
    """A random Q8_0 weight [K, N] with entries of variance 1 / K, row-major (for reference) and tiled (as used)."""

    def __init__(self, K, N, generator):
        Np = q8.padded_n(N)
        self.K, self.N = K, N
        self.q = torch.randint(-127, 128, (K, Np), dtype=torch.int8, device="cuda", generator=generator)
        self.q[:, N:] = 0
        self.s = torch.full((K // 32, Np), (3.0 / K) ** 0.5 / 127.0, device="cuda")
        self.s[:, N:] = 0
        self.tiled = q8.tile_device(self.q, self.s, N)

    def dense(self):
        return (self.q.double() * self.s.double().repeat_interleave(32, 0))[:, :self.N]


class Model:
    def __init__(self, layers=4, width=2048, heads=16, kv_heads=4, dim=128, ffn=5632, vocab=32000, positions=16384,
                 rotary=None, scaling=None, seed=1):
        g = torch.Generator("cuda").manual_seed(seed)
        self.width, self.heads, self.kv_heads, self.dim, self.ffn, self.vocab = width, heads, kv_heads, dim, ffn, vocab

        def gamma(n):
            return 0.5 + torch.rand(n, device="cuda", generator=g)

        self.embedding = torch.randn(vocab, width, device="cuda", generator=g)
        self.rope = q8.rope_table(positions, rotary or dim, scaling=scaling)
        self.first_norm = gamma(width)
        self.layers = [{"q": Weight(width, heads * dim, g), "k": Weight(width, kv_heads * dim, g),
                        "v": Weight(width, kv_heads * dim, g), "o": Weight(heads * dim, width, g),
                        "gate": Weight(width, ffn, g), "up": Weight(width, ffn, g), "down": Weight(ffn, width, g),
                        "q_norm": gamma(dim), "k_norm": gamma(dim), "mid_norm": gamma(width),
                        "next_norm": gamma(width)} for _ in range(layers)]
        self.head = Weight(width, vocab, g)


class Server:
    """The cache, block table and workspaces of ``requests`` conversations over one model."""

    def __init__(self, model, requests, pages, page_size=64, cache="bf16", window=0, sinks=0):
        if not 1 <= requests <= CHUNK:
            raise ValueError(f"1 to {CHUNK} requests: every step has a row of each")
        self.lengths = [0] * requests  # as self.cached, on the host
        self.model, self.R, self.page_size, self.window, self.sinks = model, requests, page_size, window, sinks
        self.caches = [q8.KVCache.empty(pages, model.kv_heads, page_size, model.dim, cache) for _ in model.layers]
        self.table = torch.full((requests, pages), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, device="cuda").to(torch.int32)  # the pages in any order
        self.head = torch.zeros(1, dtype=torch.int32, device="cuda")      # the next free page
        self.cached = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.tokens = torch.zeros(requests, dtype=torch.int64, device="cuda")
        self.logits = torch.empty((requests, q8.padded_n(model.vocab)), device="cuda")
        self.workspace = q8.attn_workspace()
        self.graph = None

    def make_room(self, counts):
        """Count counts[r] more tokens for request r; refused where pages or the rotation table's positions run out (what
        the kernels then do, tokens without a place and NaN, is for steps that cannot ask)."""
        lengths = [n + more for n, more in zip(self.lengths, counts)]
        if sum(-(-n // self.page_size) for n in lengths) > self.free.numel():
            raise ValueError("not enough pages for that many tokens")
        if max(lengths) > self.model.rope.shape[0]:
            raise ValueError("more tokens than the rotation table has positions")
        self.lengths = lengths

    def step(self, tokens, fresh, decode):
        """One step over tokens [rows], fresh[r] of them request r's next; leaves each request's next token in
        self.tokens and its logits in self.logits.  Nothing waits for the device, so that a step can be captured."""
        m = self.model
        at = q8.kv_slots(self.cached, fresh, self.table, self.free, self.page_size, tokens.numel(), head=self.head)
        h = m.embedding[tokens]
        x = (h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * m.first_norm).bfloat16()
        for layer, cache in zip(m.layers, self.caches):
            q, k, v = q8.gemv_parts(x, [(*layer[n].tiled, layer[n].N) for n in "qkv"], tiled=True)
            q = q8.rope_append(q, k, v, cache, at["positions"], at["slots"], table=m.rope, q_heads=m.heads,
                               q_gamma=layer["q_norm"], k_gamma=layer["k_norm"], eps=EPS)
            options = {"window": self.window, "sinks": self.sinks, "workspace": self.workspace}
            if decode:
                a = q8.attn_decode(q, cache, at["table"], at["lens"], **options)
            else:
                a = q8.attn_prefill(q, cache, at["table"], at["lens"], at["row_start"], **options)
            h, x = q8.gemv_residual_norm(a, *layer["o"].tiled, m.width, h, layer["mid_norm"], EPS)
            _, g = q8.gemv_glu(x, layer["gate"].tiled, layer["up"].tiled, m.ffn, want=("bf16",))
            h, x = q8.gemv_residual_norm(g, *layer["down"].tiled, m.width, h, layer["next_norm"], EPS)
        if not decode:  # the requests' last rows
            x = x[(at["row_start"][1:] - 1).clamp(min=0).long()]
        q8.gemv_argmax(x, *m.head.tiled, m.vocab, idx=self.tokens, logits=self.logits, tiled=True)
        self.cached.copy_(at["lens"])
        self.head.copy_(at["head"])

    def prefill(self, prompts):
        """The prompts (lists of token ids), as many rows a step as fit; every request's last chunk comes in the last
        step, so that self.tokens and self.logits are those of all requests.  Returns the first new tokens."""
        left = [list(p) for p in prompts]
        if len(left) != self.R or not all(left):
            raise ValueError("a prompt of one token or more for each request")
        self.make_room([len(p) for p in left])
        while any(left):
            room, take = CHUNK, []
            for i, p in enumerate(left):
                later = len(left) - 1 - i  # each of the others may need a row
                take.append(min(len(p), max(room - later, 0)))
                room -= take[-1]
            if take != [len(p) for p in left]:  # not the last step: everybody keeps a token for it
                take = [min(n, max(len(p) - 1, 0)) for n, p in zip(take, left)]
            rows = [t for n, p in zip(take, left) for t in p[:n]]
            left = [p[n:] for n, p in zip(take, left)]
            self.step(torch.tensor(rows, device="cuda"), torch.tensor(take, dtype=torch.int32, device="cuda"), False)
        return self.tokens.clone()

    def decode(self, count):
        """``count`` more greedy tokens of every request, [count, requests]; the step is captured once and replayed."""
        self.make_room([count] * self.R)
        out = torch.empty((count, self.R), dtype=torch.int64, device="cuda")
        start = 0
        if self.graph is None and count:
            ones = torch.ones(self.R, dtype=torch.int32, device="cuda")
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):  # a first step outside: what initializes on first use has then done so
                self.step(self.tokens, ones, True)
                out[0], start = self.tokens, 1
                side.synchronize()
                self.graph, self.ones = torch.cuda.CUDAGraph(), ones
                with torch.cuda.graph(self.graph, stream=side):
                    self.step(self.tokens, ones, True)
            torch.cuda.current_stream().wait_stream(side)
        for i in range(start, count):
            self.graph.replay()
            out[i] = self.tokens
        return out


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("requests", 8), ("prompt", 300), ("tokens", 64), ("layers", 4), ("page", 64), ("window", 0),
                        ("sinks", 0)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--cache", choices=("bf16", "q8"), default="bf16")
    a = ap.parse_args()
    model = Model(layers=a.layers, positions=a.prompt + a.tokens + 1)
    pages = a.requests * -(-(a.prompt + a.tokens) // a.page)
    server = Server(model, a.requests, pages, a.page, a.cache, a.window, a.sinks)
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randint(model.vocab, (max(a.prompt - 7 * r, 1),), generator=g).tolist() for r in range(a.requests)]

    def timed(what):
        t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        t[0].record()
        result = what()
        t[1].record()
        torch.cuda.synchronize()
        return result, t[0].elapsed_time(t[1])

    Server(model, 1, 1, a.page, a.cache).prefill([[0]])  # what initializes on first use
    first, ms = timed(lambda: server.prefill(prompts))
    print(f"prefill: {sum(map(len, prompts))} tokens of {a.requests} prompts in {ms:.2f} ms")
    few = min(2, a.tokens)
    head = server.decode(few)  # with the capture
    rest, ms = timed(lambda: server.decode(a.tokens - few))
    if a.tokens > few:
        print(f"decode: {a.tokens - few} steps of {a.requests} requests, {ms / (a.tokens - few) * 1e3:.1f} us a step")
    for r in range(min(a.requests, 4)):
        print(f"request {r}:", [first[r].item()] + torch.cat([head, rest])[:8, r].tolist())
    if q8.device_fault():
        raise SystemExit("a kernel's bounded wait ran out")


if __name__ == "__main__":
    main()
