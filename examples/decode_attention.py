"""The attention part of a decode layer, end to end: input projection, planner, rotary
positions with the cache write, paged attention, output projection with the residual.

    python examples/decode_attention.py [--steps 64] [--seqs 8] [--e4m3]

Prompts of different lengths go in as chunks of rows, then every sequence gets one token a
step through a captured graph: lengths, block tables and slots are worked out on the GPU, so
the same graph serves every step. Random weights; prints the time of a step.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import split_switched_decode_gb300 as ssd
from split_switched_decode_gb300 import inputs


class AttentionLayer:
    """Weights, a paged cache with its free list, and the buffers of one layer."""

    def __init__(self, hidden=1024, heads=16, kv_heads=2, dim=64, seqs=8, max_len=1024, page=16,
                 e4m3=False, max_rows=512, seed=0, device="cuda"):
        self.heads, self.kv_heads, self.dim, self.page = heads, kv_heads, dim, page
        width = (heads + 2 * kv_heads) * dim
        self.w_in = inputs.weight(width, hidden, device, seed, "w_in")
        self.w_out = inputs.weight(hidden, heads * dim, device, seed, "w_out")
        table_width = -(-max_len // page)
        pages = seqs * table_width
        dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        cache = torch.zeros((2, pages, kv_heads, page, dim), device=device).to(dtype)
        self.k_cache, self.v_cache = cache[0], cache[1]
        # one step of the 8-bit grid per head: keys and values of unit size use its middle
        self.scale = torch.full((kv_heads,), 0.05, device=device) if e4m3 else None
        self.inv_freq, self.magnitude = ssd.rope_frequencies(dim, device=device)

        def ints(*shape, fill=0):
            return torch.full(shape, fill, dtype=torch.int32, device=device)
        self.length, self.table = ints(seqs), ints(seqs, table_width, fill=-1)
        self.free = torch.randperm(pages, device=device).to(torch.int32)
        self.summary, self.q_start = ints(4), ints(seqs + 1)
        self.positions, self.slots = ints(max_rows), ints(max_rows)
        self.rows = torch.empty((max_rows, width), dtype=torch.bfloat16, device=device)
        self.mixed = torch.empty((max_rows, heads * dim), dtype=torch.bfloat16, device=device)
        self.ws = {}

    def _workspaces(self, T):
        """Zero-filled once per number of rows; every call leaves them ready."""
        if T not in self.ws:
            S, hidden = self.length.numel(), self.w_in.shape[1]
            self.ws[T] = (
                ssd.workspace(ssd.dec_linear_workspace_bytes(T, self.w_in.shape[0], hidden)),
                ssd.workspace(ssd.attn_decode_workspace_bytes(S, T, self.heads, self.kv_heads,
                                                              self.dim)),
                ssd.workspace(ssd.dec_linear_workspace_bytes(T, hidden, self.w_out.shape[1])))
        return self.ws[T]

    def step(self, x, out, new_len=None):
        """x, out [T, hidden]: row t belongs to the sequence that new_len [S] (None: one row
        each) puts it in; out = x + attention. Everything runs on the current stream."""
        T, H, G, D = x.shape[0], self.heads, self.kv_heads, self.dim
        ws_in, ws_attn, ws_out = self._workspaces(T)
        rows, mixed = self.rows[:T], self.mixed[:T]
        ssd.dec_linear(x, self.w_in, None, rows, ws_in)
        ssd.kv_plan(self.length, new_len, self.table, self.free, self.summary[1:2], self.page,
                    self.length, self.q_start, self.positions[:T], self.slots[:T], self.summary)
        q = rows[:, :H * D].view(T, H, D)
        k = rows[:, H * D:(H + G) * D].view(T, G, D)
        v = rows[:, (H + G) * D:].view(T, G, D)
        ssd.rope_append(q, k, v, self.positions[:T], self.slots[:T], self.inv_freq, q,
                        self.k_cache, self.v_cache, magnitude=self.magnitude,
                        k_scale=self.scale, v_scale=self.scale)
        ssd.attn_decode(q, self.k_cache, self.v_cache, self.table, self.length,
                        mixed.view(T, H, D), ws_attn, q_start=self.q_start, k_scale=self.scale,
                        v_scale=self.scale)
        ssd.dec_linear(mixed, self.w_out, x, out, ws_out)

    def capture(self, x, out):
        """A graph of one decode step (one row a sequence) on x and out."""
        self._workspaces(x.shape[0])
        saved = [t.clone() for t in (self.length, self.table, self.summary)]
        self.step(x, out)  # launch once outside: attributes, lazy loading
        for t, s in zip((self.length, self.table, self.summary), saved):
            t.copy_(s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            self.step(x, out)
        return graph


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--seqs", type=int, default=8, choices=range(1, 65), metavar="1..64")
    ap.add_argument("--e4m3", action="store_true")
    a = ap.parse_args(argv)
    layer = AttentionLayer(seqs=a.seqs, e4m3=a.e4m3)
    hidden = layer.w_in.shape[1]
    prompts = torch.arange(a.seqs, dtype=torch.int32, device="cuda") % 8 + 1  # <= 512 rows
    x = inputs.activations(int(prompts.sum()), hidden, "cuda", 1, "prompt")
    layer.step(x, torch.empty_like(x), prompts)
    x = inputs.activations(a.seqs, hidden, "cuda", 1, "token")
    out = torch.empty_like(x)
    graph = layer.capture(x, out)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
        x.copy_(out)
    torch.cuda.synchronize()
    us = (time.perf_counter() - t) / a.steps * 1e6
    print(f"{a.seqs} sequences, lengths {layer.length.tolist()}: {us:.1f} us a step, "
          f"{int(layer.summary[1])} pages used")
    return layer, out


if __name__ == "__main__":
    main()
