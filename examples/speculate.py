"""A whole speculative decoding loop: drafts, verification pass, next step.

    PYTHONPATH=. python examples/speculate.py [--batch 8] [--steps 60] [--temperature 0]

The target is a small random transformer (plain torch products around the cache
and its attention); what matters is how the calls fit together.  Per step

    drafts   the row's last token and its drafts are packed, 1 + num_valid each
    write    their keys and values enter the paged 8-bit cache
    attend   they attend over their rows' cache
    verify   accepts a prefix of the drafts and draws one more token
    propose_with_update   appends them and drafts the next ones

without the host waiting for the device: the packed tensors have room for k
drafts in every row, and q_start says on the device where each row's tokens are.
A rejected draft needs no call of its own, since the row's length does not count
it and the next write takes its place.
"""
from __future__ import annotations

import argparse
import time

import torch

from model_free_suffix_gb300 import KVCache, SuffixDrafter


class Target:
    """A random decoder: `layers` blocks of attention, tied embeddings."""

    def __init__(self, vocab=512, width=256, layers=2, kv_heads=2, group=4, head_dim=64, batch=8, capacity=1024,
                 page=64, window=0, sinks=0, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.kv_heads, self.q_heads, self.dim = kv_heads, kv_heads * group, head_dim
        self.window, self.sinks = window, sinks
        heads = self.q_heads + 2 * kv_heads

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g) * cols ** -0.5).to(torch.bfloat16).cuda()

        self.embed = (torch.randn(vocab, width, generator=g) * 0.5).to(torch.bfloat16).cuda()
        self.qkv = [weight(heads * head_dim, width) * 2 for _ in range(layers)]
        self.proj = [weight(width, self.q_heads * head_dim) for _ in range(layers)]
        pages = -(-capacity // page)
        self.cache = KVCache(batch * pages, page, kv_heads, head_dim, batch, pages, q_heads=self.q_heads,
                             num_layers=layers)
        # any assignment of pages to rows will do
        order = torch.randperm(batch * pages, generator=g, dtype=torch.int32)
        self.table = order.view(batch, pages).cuda()

    def __call__(self, ids, seq_lens, q_start, max_q):
        """Logits of the packed new tokens, which enter the cache."""
        x = self.embed[ids.long()]
        for i, (w_in, w_out) in enumerate(zip(self.qkv, self.proj)):
            h = torch.nn.functional.layer_norm(x, x.shape[1:])
            qkv = (h @ w_in.T).view(len(ids), -1, self.dim)
            q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
            self.cache.write(k, v, self.table, seq_lens, q_start, layer=i)
            # (zeros: tokens that no row claims are not touched)
            o = self.cache.attend(q, self.table, seq_lens, q_start, max_q, window=self.window, sinks=self.sinks,
                                  out=torch.zeros(q.shape, dtype=q.dtype, device=q.device), layer=i)
            x = x + o.view(len(ids), -1) @ w_out.T
        return torch.nn.functional.layer_norm(x, x.shape[1:]) @ self.embed.T


def pack(tok, n, drafts, num_valid):
    """The rows' last tokens and drafts, packed: ids, lengths with them, starts."""
    B, k = drafts.shape
    q_start = torch.zeros(B + 1, dtype=torch.int32, device=tok.device)
    q_start[1:] = torch.cumsum(num_valid + 1, 0)
    at = torch.arange(B * (k + 1), device=tok.device, dtype=torch.int32)
    row = torch.searchsorted(q_start[1:], at, right=True).clamp(max=B - 1)
    last = tok.gather(1, (n - 1).long()[:, None])
    new = torch.cat([last, drafts.clamp(min=0)], 1)
    ids = new[row, (at - q_start[row]).clamp(max=k).long()]
    return ids, n + num_valid, q_start


def generate(target, prompts, steps, k=7, temperature=0.0, seed=1):
    """Tokens of each row after `steps` steps, and the mean number a step gave."""
    B, V = len(prompts), target.embed.shape[0]
    S = target.table.shape[1] * target.cache.page_size
    dr = SuffixDrafter(max_batch=B, seq_capacity=S, vocab_size=V, k=k, corpus_capacity=1 << 12)
    g = torch.Generator("cuda").manual_seed(seed)
    tok = torch.zeros(B, S, dtype=torch.int32, device="cuda")
    n = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
    for b, p in enumerate(prompts):
        tok[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    # the prompts but for their last tokens
    lens = n - 1
    starts = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    starts[1:] = torch.cumsum(lens, 0)
    target(torch.tensor([t for p in prompts for t in p[:-1]], dtype=torch.int32, device="cuda"), lens, starts,
           max(len(p) for p in prompts) - 1)
    t = torch.full((B,), temperature, device="cuda")
    out, verdict = dr.propose(tok, n), dr.new_verdict(B)
    began = n.clone()
    for _ in range(steps):
        ids, seq_lens, q_start = pack(tok, n, out.drafts, out.num_valid)
        logits = target(ids, seq_lens, q_start, k + 1)
        dr.verify(logits, out.drafts, out.num_valid, torch.rand(B, k, device="cuda", generator=g),
                  torch.empty(B, V, device="cuda").exponential_(generator=g), row_start=q_start[:B],
                  temperature=t, out=verdict)
        dr.propose_with_update(tok, n, verdict.sampled, out=out)
    new = (n - began).float().mean().item()
    assert dr.get_error() == 0 and target.cache.get_error() == 0
    dr.close()
    return [tok[b, :m].tolist() for b, m in enumerate(n.tolist())], new / steps


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--k", type=int, default=7)
    p.add_argument("--temperature", type=float, default=0.0)
    a = p.parse_args()
    rng = torch.Generator().manual_seed(0)
    prompts = [torch.randint(0, 512, (20 + 9 * b,), generator=rng).tolist() for b in range(a.batch)]
    target = Target(batch=a.batch, capacity=20 + 9 * a.batch + a.steps * (a.k + 1) + 16)
    began = time.perf_counter()
    _, rate = generate(target, prompts, a.steps, a.k, a.temperature)
    print("%d rows, %d steps: %.2f tokens a step and row, %.2f ms a step"
          % (a.batch, a.steps, rate, (time.perf_counter() - began) / a.steps * 1e3))


if __name__ == "__main__":
    main()
