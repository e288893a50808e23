"""A server's steps: prompts come in by chunks next to rows that decode, pages come and go.

    PYTHONPATH=. python examples/prompts.py [--rows 8] [--requests 24] [--chunk 128]

The target is a small random transformer, as in speculate.py; what matters is how the
calls fit together.  Per step

    assign        pages for every row's tokens, given back where a request has ended, and
                  the packed tokens' rows and positions, all on the device
    attend_chunk  the packed tokens over their rows' earlier ones in the 8-bit cache and
                  over one another: chunks of prompts and single tokens in one call
    write         their keys and values enter the cache

The host decides only what it knows anyway: which request a row serves, and how many of
its tokens a step takes.

One call for all rows is the simplest, not the fastest, where most of many rows decode: with
254 rows of one token and 2 of 512 over 1024 to 4096 it takes 1.16 ms.  Such a server keeps the
rows that decode in front, and after the write gives them to `attend` and the others alone to
`attend_chunk` (slices of the table, the lengths and the starts, these from 0 again): 0.31 ms.
"""
from __future__ import annotations

import argparse
import time

import torch

from model_free_suffix_gb300 import KVCache


class Server:
    """A random decoder of `layers` blocks that serves `rows` requests at a time."""

    def __init__(self, rows=8, room=1024, chunk=128, vocab=512, width=256, layers=2, kv_heads=2, group=4, head_dim=64,
                 page=64, pages=None, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.kv_heads, self.q_heads, self.dim, self.chunk, self.room = kv_heads, kv_heads * group, head_dim, chunk, room

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g) * cols ** -0.5).to(torch.bfloat16).cuda()

        self.embed = (torch.randn(vocab, width, generator=g) * 0.5).to(torch.bfloat16).cuda()
        self.qkv = [weight((self.q_heads + 2 * kv_heads) * head_dim, width) * 2 for _ in range(layers)]
        self.proj = [weight(width, self.q_heads * head_dim) for _ in range(layers)]
        width_pages = -(-room // page)
        self.cache = KVCache(pages or rows * width_pages, page, kv_heads, head_dim, rows, width_pages, q_heads=self.q_heads,
                             num_layers=layers)
        self.pages = self.cache.new_pages()
        self.tokens = torch.zeros(rows, room, dtype=torch.int32, device="cuda")
        self.requests = [None] * rows          # [tokens in the cache, prompt's length, tokens wanted]

    def step(self, waiting):
        """One step; `waiting`: (prompt, tokens wanted) of requests to come, the next one last.  The finished ones' tokens."""
        B = len(self.requests)
        keep, new = [0] * B, [0] * B
        for b in range(B):
            if self.requests[b] is None and waiting:
                prompt, more = waiting.pop()
                self.tokens[b, :len(prompt)] = torch.tensor(prompt, dtype=torch.int32)
                self.requests[b] = [0, len(prompt), more]
            if self.requests[b] is not None:
                done, prompt, _ = self.requests[b]
                keep[b], new[b] = done, min(self.chunk, prompt - done) if done < prompt else 1
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        plan = self.cache.assign(self.pages, i32(keep), i32(new), total=sum(new))
        x = self.embed[self.tokens[plan.rows.long(), plan.positions.long()].long()]
        for i, (w_in, w_out) in enumerate(zip(self.qkv, self.proj)):
            h = torch.nn.functional.layer_norm(x, x.shape[1:])
            qkv = (h @ w_in.T).view(len(x), -1, self.dim)
            q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
            o = self.cache.attend_chunk(q, k, v, self.pages.block_table, plan.seq_lens, plan.q_start, layer=i)
            self.cache.write(k, v, self.pages.block_table, plan.seq_lens, plan.q_start, layer=i)
            x = x + o.view(len(x), -1) @ w_out.T
        last = plan.q_start[1:].long() - 1     # (rows without tokens: another's, which is not used)
        best = (torch.nn.functional.layer_norm(x[last], x.shape[1:]) @ self.embed.T).argmax(-1).int()
        finished = []
        for b, r in enumerate(self.requests):
            if r is None:
                continue
            r[0] += new[b]
            if r[0] >= r[1]:
                self.tokens[b, r[0]] = best[b]
                if r[0] + 1 - r[1] == r[2]:
                    finished.append(self.tokens[b, r[1]:r[0] + 1].tolist())
                    self.requests[b] = None    # (its pages go back with the next step's assign)
        return finished

    def serve(self, requests):
        waiting, out, steps = list(requests)[::-1], [], 0
        while waiting or any(r is not None for r in self.requests):
            out += self.step(waiting)
            steps += 1
        zero = torch.zeros(len(self.requests), dtype=torch.int32, device="cuda")
        self.cache.assign(self.pages, zero, zero, total=0)
        assert self.cache.get_error() == 0
        return out, steps


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--rows", type=int, default=8)
    p.add_argument("--requests", type=int, default=24)
    p.add_argument("--chunk", type=int, default=128)
    a = p.parse_args()
    g = torch.Generator().manual_seed(0)
    requests = [(torch.randint(0, 512, (int(n),), generator=g).tolist(), 16)
                for n in torch.randint(1, 700, (a.requests,), generator=g)]
    server = Server(a.rows, chunk=a.chunk)
    began = time.perf_counter()
    out, steps = server.serve(requests)
    print("%d requests, %d prompt tokens, %d new ones in %d steps, %.2f ms a step"
          % (len(out), sum(len(r[0]) for r in requests), sum(map(len, out)), steps,
             (time.perf_counter() - began) / steps * 1e3))


if __name__ == "__main__":
    main()
