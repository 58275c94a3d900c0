#!/usr/bin/env python3
"""One decoder layer's token step on the library's calls, captured into a CUDA graph.

    h += x;  a = norm(h) in E4M3  ->  q, k, v = a Wqkv (FP8)  ->  k, v into the 4-bit cache
    ->  attention over the cache  ->  o = attn Wo  ->  h += o;  y = norm(h)
    ->  logits = y Wr  ->  out = experts(y, logits)

`out` is the next layer's x, the residual stream h is FP32 and updated in place.  Weights are
random.  Queries and keys get no position: the library has no call that rotates them, and a model
that does so would between the projection and the cache.  The eight calls of a step enqueue eleven kernels at most and allocate nothing once the
first step has run.

    python examples/decoder_layer.py [--batch 16] [--context 4000] [--steps 8]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_sm_gb300 as dg  # noqa: E402

EPS = 1e-5


class DecoderLayer:
    def __init__(self, batch, width=4096, heads_q=32, heads_kv=8, d=128, experts=16, inter=1536, top=4,
                 page_size=64, max_tokens=8192, seed=0):
        self.batch, self.width, self.heads_q, self.heads_kv, self.d = batch, width, heads_q, heads_kv, d
        self.experts, self.inter, self.top, self.page_size = experts, inter, top, page_size
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(*shape, fan_in):
            return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(1 / math.sqrt(fan_in))

        self.gain1, self.gain2 = (torch.ones(width, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        # The fused projection's weights by output column, quantised once.
        n = (heads_q + 2 * heads_kv) * d
        w = weight(n, width, fan_in=width)
        self.wqkv = torch.empty((n, width), dtype=torch.uint8, device="cuda")
        self.wqkv_scale = torch.empty(n, device="cuda")
        dg.quantize_rows_e4m3(n, width, w, width, self.wqkv, width, self.wqkv_scale)
        self.wo = weight(heads_q * d, width, fan_in=heads_q * d)
        self.wr = weight(width, experts, fan_in=width)
        self.wg, self.wu = (weight(experts, width, inter, fan_in=width) for _ in range(2))
        self.wd = weight(experts, inter, width, fan_in=inter)
        # The cache: every sequence may grow to max_tokens; pages are handed out as it does.
        self.table_width = -(-max_tokens // page_size)
        pages = batch * self.table_width
        self.pool = torch.zeros((pages, heads_kv, dg.dg_kv4_block_bytes(page_size, d)), dtype=torch.uint8, device="cuda")
        self.cache = dg.dg_kv4_cache(self.pool, pages, page_size, heads_kv, d)
        self.table = torch.full((batch, self.table_width), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32).tolist()
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.slots = torch.zeros(batch, dtype=torch.int64, device="cuda")

        def buf(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device="cuda")

        self.x, self.h = torch.zeros((batch, width), dtype=torch.bfloat16, device="cuda"), torch.zeros((batch, width), device="cuda")
        self.a, self.a_scale = buf(batch, width, dtype=torch.uint8), buf(batch, dtype=torch.float32)
        self.qkv, self.attn, self.o = buf(batch, n), buf(batch, heads_q * d), buf(batch, width)
        self.y, self.logits, self.out = buf(batch, width), buf(batch, experts, dtype=torch.float32), buf(batch, width)
        # Workspaces are zeroed once and reused by every step.
        self.attn_ws = torch.zeros(dg.dg_attention_kv4_workspace_bytes(batch, 1, heads_q, heads_kv, d), dtype=torch.uint8, device="cuda")
        self.moe_ws = torch.zeros(dg.dg_moe_workspace_bytes(batch, width, inter, experts, top), dtype=torch.uint8, device="cuda")

    def grow(self, tokens):
        """Room for `tokens` more tokens of every sequence (host side): pages for them."""
        for b, n in enumerate(self.lens.tolist()):
            have, need = -(-n // self.page_size), -(-(n + tokens) // self.page_size)
            for i in range(have, need):
                self.table[b, i] = self.free.pop()

    def advance(self):
        """The next token of every sequence: its slot, and the length that includes it."""
        page = torch.gather(self.table, 1, (self.lens // self.page_size).long()[:, None])[:, 0]
        self.slots.copy_(page.long() * self.page_size + self.lens % self.page_size)
        self.lens.add_(1)

    def prompt(self, k, v):
        """Writes a prompt's keys and values, [batch, tokens, heads_kv * d] BF16, to the cache."""
        b, t, w = k.shape
        self.grow(t)
        at = torch.arange(t, device="cuda")[None] + self.lens.long()[:, None]
        page = torch.gather(self.table.long(), 1, at // self.page_size)
        slots = (page * self.page_size + at % self.page_size).flatten()
        dg.kv4_append(self.cache, b * t, k, w, v, w, slots)
        self.lens.add_(t)

    def step(self):
        """One token of every sequence: x and h in, out and h out.  advance() comes before."""
        b, w, hq, hkv, d = self.batch, self.width, self.heads_q, self.heads_kv, self.d
        n = (hq + 2 * hkv) * d
        dg.rmsnorm_residual_e4m3(b, w, self.x, w, dg.DG_OUT_BF16, self.h, w, dg.DG_OUT_F32, self.h, w, self.gain1, EPS,
                                 self.a, w, self.a_scale)
        dg.gemm_fp8_e4m3(b, n, w, self.a, w, self.a_scale, self.wqkv, w, self.wqkv_scale, self.qkv, n)
        dg.kv4_append(self.cache, b, self.qkv[:, hq * d:], n, self.qkv[:, (hq + hkv) * d:], n, self.slots)
        dg.attention_kv4(self.cache, b, 1, hq, 1 / math.sqrt(d), self.qkv, n, n, self.table, self.table_width, self.lens,
                         self.attn, hq * d, hq * d, self.attn_ws, self.attn_ws.numel())
        dg.gemm_bf16(b, w, hq * d, 1.0, self.attn, hq * d, self.wo, w, 0.0, self.o, w)
        dg.rmsnorm_residual_bf16(b, w, self.o, w, dg.DG_OUT_BF16, self.h, w, dg.DG_OUT_F32, self.h, w, self.gain2, EPS,
                                 self.y, w)
        dg.gemm_bf16(b, self.experts, w, 1.0, self.y, w, self.wr, self.experts, 0.0, self.logits, self.experts, dg.DG_OUT_F32)
        dg.moe_bf16(b, w, self.inter, self.experts, self.top, True, self.y, w, self.logits, self.experts,
                    self.wg, self.inter, w * self.inter, self.wu, self.inter, w * self.inter, self.wd, w, w * self.inter,
                    self.out, w, self.moe_ws, self.moe_ws.numel())

    def capture(self):
        """A graph of step(), for replay().  Runs one step: gemm_bf16 keeps a workspace per stream,
        which has to exist on the capturing stream before the capture."""
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            self.step()
        torch.cuda.current_stream().wait_stream(stream)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            self.step()
        return graph


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--context", type=int, default=4000)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    layer = DecoderLayer(a.batch, max_tokens=a.context + a.steps + 8)
    kv = (a.batch, a.context, layer.heads_kv * layer.d)
    layer.prompt(torch.randn(kv, device="cuda", dtype=torch.bfloat16), torch.randn(kv, device="cuda", dtype=torch.bfloat16))
    layer.grow(a.steps + 1)
    layer.x.copy_(torch.randn_like(layer.x))
    layer.advance()
    graph = layer.capture()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    times = []
    for _ in range(a.steps):
        layer.advance()
        start.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end) * 1e3)
    status = dg.dg_device_status()
    assert status == dg.DG_OK, dg.status_string(status)
    assert bool(layer.out.isfinite().all())
    print(f"batch {a.batch}, context {a.context}: {min(times):.1f} us a layer step (of {a.steps}), "
          f"cache {layer.pool.numel() / 2**20:.0f} MiB")


if __name__ == "__main__":
    main()
