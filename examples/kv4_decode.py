"""A decode machine's side of one attention layer: receive the prompts' KV, keep it in 4 bits, decode, evict.

    python examples/kv4_decode.py [--requests 8] [--prompt 4096] [--budget 1024] [--steps 64]

Synthetic prompts' K and V (bf16) arrive as lossless streams (``Codec``), are decoded and appended to a
``KV4Cache``; the prompts' last queries are weighed and every sequence is cut to the budget; then each step
appends a token a request, attends, and adds up the weights, and sequences that have outgrown the budget by a
page are cut again.  No step copies anything back from the GPU.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lossless_bf16_kv_amd as sz  # noqa: E402
from lossless_bf16_kv_amd import kv4  # noqa: E402


class Pages:
    """Free pages, and each request's."""

    def __init__(self, count: int, requests: int, width: int):
        self.free = list(range(count))
        self.rows = torch.full((requests, width), -1, dtype=torch.int32)

    def cover(self, request: int, pages: int) -> None:
        """Gives a request pages 0 .. pages - 1."""
        row = self.rows[request]
        for i in range(pages):
            if row[i] < 0:
                row[i] = self.free.pop()

    def take_back(self, row) -> None:
        self.free += [int(p) for p in row if p >= 0]


def run(requests=8, prompt=4096, budget=1024, steps=64, heads=32, kv_heads=8, d=128, page=64, seed=0):
    """Returns the largest rounding error of the first attention over the cache's values (of sum p |v| + |o|), its
    relative distance from attention over the bf16 KV, the last lengths and the streams' ratios."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = torch.linspace(prompt // 2, prompt, requests).int()
    total = int(lens.sum())
    cu = torch.cat([torch.zeros(1, dtype=torch.int32), lens.cumsum(0, dtype=torch.int32)])
    spread = torch.exp(0.75 * torch.randn(kv_heads, d, generator=g, device="cuda"))
    k = (torch.randn(total, kv_heads, d, generator=g, device="cuda") * spread).bfloat16()
    v = torch.randn(total, kv_heads, d, generator=g, device="cuda").bfloat16()

    # what arrives: lossless streams, decoded bit for bit
    codec = sz.Codec("cuda", chunk_size=1024)
    codec.calibrate(torch.cat([k.flatten()[:1 << 20], v.flatten()[:1 << 20]]))
    streams = codec.encode_batch([k, v])
    k, v = codec.decode_batch(streams)

    # pages for the prompts, and for the cut sequences with the tokens to come before the next cut
    slack, sinks, recent = page, 4, budget // 4
    wide = -(-(max(prompt, budget) + slack) // page)
    cut = -(-budget // page)
    pages = Pages(requests * (wide + cut + 1), requests, wide)
    cache = kv4.KV4Cache(len(pages.free), page, kv_heads, d)
    for r in range(requests):
        pages.cover(r, -(-int(lens[r]) // page))
    table, dev_lens = pages.rows.cuda(), lens.cuda()
    cache.append(k, v, table, dev_lens, cu.cuda())

    # the last queries of the prompts say which tokens matter
    seen = min(32, prompt // 2)
    qcu = torch.arange(requests + 1, dtype=torch.int32) * seen
    scale = d ** -0.5
    q = (torch.randn(requests * seen, heads, d, generator=g, device="cuda") /
         spread.repeat_interleave(heads // kv_heads, 0)).bfloat16()
    kw = {"max_q": seen, "max_len": prompt}
    out, lse = cache.attend(q, table, dev_lens, qcu.cuda(), **kw)
    cache.weigh(q, lse, table, dev_lens, qcu.cuda(), **kw)

    # the last query of request 0 against plain attention over the KV as the cache holds it, and as it came
    n, group = int(lens[0]), heads // kv_heads

    def plain(k, v):
        k, v = (x[:n].float().repeat_interleave(group, 1) for x in (k, v))
        p = torch.softmax((q[seen - 1].float()[None] * k).sum(-1) * scale, 0)[..., None]       # [tokens, heads, 1]
        return (p * v).sum(0), (p * v.abs()).sum(0)
    got = out[seen - 1].float()
    held, size = plain(*cache.read(table, dev_lens, cu.cuda(), total=total))
    rounding = float(((got - held).abs() / (size + held.abs())).max())
    came, _ = plain(k, v)
    error = float((got - came).norm() / came.norm())

    def evict():
        nonlocal table, dev_lens
        old = pages.rows.clone()
        pages.rows.fill_(-1)
        for r in range(requests):
            pages.cover(r, -(-min(int(lens[r]), budget) // page))
        new = pages.rows.cuda()
        dev_lens, _ = cache.evict(table, dev_lens, new[:, :cut].contiguous(), budget, sinks=sinks, recent=recent,
                                  max_len=int(lens.max()))
        lens.clamp_(max=budget)
        table = new
        for r in range(requests):
            pages.take_back(old[r])

    evict()
    for _ in range(steps):
        if int(lens.max()) >= budget + slack:
            evict()
        lens.add_(1)
        for r in range(requests):
            pages.cover(r, -(-int(lens[r]) // page))
        table, dev_lens = pages.rows.cuda(), dev_lens + 1
        q, k, v = (torch.randn(requests, h, d, generator=g, device="cuda").bfloat16() for h in (heads, kv_heads, kv_heads))
        cache.append(k, v, table, dev_lens)
        out, lse = cache.attend(q, table, dev_lens, max_len=int(lens.max()))
        cache.weigh(q, lse, table, dev_lens, max_len=int(lens.max()))
    cache.check()                        # the one wait: no page, length or offset was out of range
    assert torch.equal(dev_lens.cpu(), lens) and bool(out.isfinite().all())
    ratio = [s.ratio for s in streams]
    return rounding, error, lens.tolist(), ratio


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("requests", 8), ("prompt", 4096), ("budget", 1024), ("steps", 64)):
        p.add_argument("--" + name, type=int, default=default)
    rounding, error, lens, ratio = run(**vars(p.parse_args()))
    print(f"received at {min(ratio):.2f}x lossless; attention rounds by {rounding:.1e}; 4 bits take it {100 * error:.1f} % "
          f"from the bf16 KV's; lengths at the end {min(lens)} .. {max(lens)}")


if __name__ == "__main__":
    main()
