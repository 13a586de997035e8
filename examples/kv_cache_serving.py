"""One attention layer served from a paged 4-bit key/value cache.

A batch of prompts of different lengths is taken in by chunks (their keys and
values quantized into the cache, their queries attending over what is there),
then every sequence decodes one token at a time: the step is captured once as a
HIP graph, and slots, lengths and page tables change in place between replays,
pages being handed out as sequences grow.  At the end the first sequence's
cache is read back, as a layer that wants dense keys and values would.

Prints how far the layer's outputs are from attention over the keys and values
before they were quantized, and the time of a step.  Keys and values are random
numbers with a few large channels, the ones that the rotation is for.

    python examples/kv_cache_serving.py [--format mxfp4] [--steps 64] ...
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp4_block_scaled_row_amd as fq


class PageTable:
    """Which pages each sequence has: a free list on the host, the table on the GPU."""

    def __init__(self, pages, page_size, seqs, longest):
        self.page_size = page_size
        self.free = list(range(pages))[::-1]
        self.rows = [[] for _ in range(seqs)]
        self.table = torch.full((seqs, -(-longest // page_size)), -1, dtype=torch.int32, device="cuda")

    def grow(self, seq, length):
        """Pages for `length` tokens."""
        row = self.rows[seq]
        while len(row) * self.page_size < length:
            self.table[seq, len(row)] = self.free[-1]
            row.append(self.free.pop())

    def slots(self, seq, first, last):
        """Slots of tokens [first, last)."""
        return [self.rows[seq][t // self.page_size] * self.page_size + t % self.page_size for t in range(first, last)]


def ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def serve(prompts, steps, *, chunk=256, q_heads=32, kv_heads=8, head_dim=128, page_size=16, format="nvfp4", seed=0,
          verbose=True):
    """Relative root mean square errors of the keys and values read back, and of the attention outputs."""
    torch.manual_seed(seed)
    seqs, total = len(prompts), [n + steps for n in prompts]
    rotation = "fwht128" if head_dim % 128 == 0 else None
    # what the projections of this layer would give for every token of every sequence
    spread = 1.0 + 7.0 * (torch.rand(kv_heads, head_dim, device="cuda") > 0.97).float()
    keys = [(torch.randn(n, kv_heads, head_dim, device="cuda") * spread).bfloat16() for n in total]
    values = [torch.randn(n, kv_heads, head_dim, device="cuda").bfloat16() for n in total]
    queries = [torch.randn(n, q_heads, head_dim, device="cuda").bfloat16() for n in total]

    # tensor scales from a calibration sample, fixed before the first token is written
    scales = {}
    if format == "nvfp4":
        sample = torch.cat([k[:64] for k in keys]).reshape(-1, head_dim)
        if rotation:
            sample = fq.fwht(sample, transform_size=128)
        scales = dict(k_global=fq.quantize_nvfp4(sample).global_scale,
                      v_global=fq.quantize_nvfp4(torch.cat([v[:64] for v in values]).reshape(-1, head_dim)).global_scale)
    pages = sum(-(-n // page_size) for n in total)
    cache = fq.kv_cache(pages, page_size, kv_heads, head_dim, format=format, **scales)
    paging = PageTable(pages, page_size, seqs, max(total))
    outputs = [torch.zeros(n, q_heads, head_dim, dtype=torch.bfloat16, device="cuda") for n in total]

    # prompts: a chunk of each sequence at a time
    done = [0] * seqs
    while done != list(prompts):
        upto = [min(n, d + chunk) for n, d in zip(prompts, done)]
        new = [u - d for u, d in zip(upto, done)]
        for b in range(seqs):
            paging.grow(b, upto[b])
        take = lambda x: torch.cat([x[b][done[b]:upto[b]] for b in range(seqs)])
        slots = ints([s for b in range(seqs) for s in paging.slots(b, done[b], upto[b])], torch.int64)
        fq.kv_cache_write(cache, take(keys), take(values), slots, rotation=rotation)
        cu = [sum(new[:b]) for b in range(seqs + 1)]
        out = fq.kv_cache_attention(take(queries), cache, paging.table, ints(upto), cu_q=ints(cu), max_q=max(new),
                                    rotation=rotation)
        for b in range(seqs):
            outputs[b][done[b]:upto[b]] = out[cu[b]:cu[b + 1]]
        done = upto

    # decoding: one step captured, its inputs changed in place
    q, out = (torch.zeros(seqs, q_heads, head_dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.zeros(seqs, kv_heads, head_dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots, lengths = ints([-1] * seqs, torch.int64), ints([0] * seqs)

    def step():
        fq.kv_cache_write(cache, k, v, slots, rotation=rotation)
        fq.kv_cache_attention(q, cache, paging.table, lengths, rotation=rotation, out=out)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()          # once outside the capture, for the stream's workspace (slots of -1: nothing is written)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    spent = []
    for i in range(steps):
        at = [n + i for n in prompts]
        for b in range(seqs):
            paging.grow(b, at[b] + 1)
        for buffer, source in ((q, queries), (k, keys), (v, values)):
            buffer.copy_(torch.stack([source[b][at[b]] for b in range(seqs)]))
        slots.copy_(ints([paging.slots(b, at[b], at[b] + 1)[0] for b in range(seqs)], torch.int64))
        lengths.copy_(ints([t + 1 for t in at]))
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        graph.replay()
        end.record()
        for b in range(seqs):
            outputs[b][at[b]] = out[b]
        spent.append((begin, end))
    torch.cuda.synchronize()
    us = sorted(a.elapsed_time(b) * 1e3 for a, b in spent)[len(spent) // 2] if spent else 0.0

    # the first sequence's keys and values, dense, in their own basis
    dense_k, dense_v = fq.kv_cache_read(cache, paging.table[:1], ints([0, total[0]]), total=total[0], rotation=rotation)
    k_error = float((dense_k.float() - keys[0].float()).norm() / keys[0].float().norm())
    v_error = float((dense_v.float() - values[0].float()).norm() / values[0].float().norm())

    # against attention over what was there before quantization
    wrong = size = 0.0
    for b in range(seqs):
        share = q_heads // kv_heads
        kk, vv = (x[b].float().repeat_interleave(share, 1).transpose(0, 1).contiguous() for x in (keys, values))
        s = torch.matmul(queries[b].float().transpose(0, 1).contiguous(), kk.transpose(1, 2).contiguous()) * head_dim ** -0.5
        s.masked_fill_(torch.ones(total[b], total[b], dtype=torch.bool, device="cuda").triu(1), float("-inf"))
        want = torch.matmul(s.softmax(-1), vv).transpose(0, 1)
        wrong += float((outputs[b].float() - want).square().sum())
        size += float(want.square().sum())
    error = (wrong / size) ** 0.5
    if verbose:
        print("%s, %d sequences of %d to %d tokens, %d query heads on %d: cache of %.1f MB (bf16 %.1f MB)" %
              (format, seqs, min(total), max(total), q_heads, kv_heads,
               sum(p.numel() for p in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)) / 1e6,
               4e-6 * pages * page_size * kv_heads * head_dim))
        print("keys read back: relative error %.4f, values %.4f; attention outputs %.4f" % (k_error, v_error, error))
        print("decode step (write and attention): %.1f us" % us)
    return k_error, v_error, error


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--format", choices=("nvfp4", "mxfp4"), default="nvfp4")
    p.add_argument("--prompts", type=int, nargs="+", default=[1500, 37, 640, 2000])
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--head-dim", type=int, default=128)
    a = p.parse_args()
    serve(a.prompts, a.steps, format=a.format, head_dim=a.head_dim)


if __name__ == "__main__":
    main()
