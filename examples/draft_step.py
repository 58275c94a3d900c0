#!/usr/bin/env python3
"""One step of speculative decoding in 4 bits on the library's calls, captured into a CUDA graph: a tree
of drafted tokens goes through an attention layer and the vocabulary, and what the model agrees with is kept.

    q, k, v = x Wqkv (4-bit weights)  ->  k, v into the 4-bit cache behind the context
    ->  attention of the tree over the cache  ->  logits = (attn Wo) Wh
    ->  accept(): the longest path of drafted tokens that the logits predict; its rows move to the front

Node 0 of a tree is the last token that is certain, the others are guesses for what follows their parent.
Weights and drafts are random here (every node's token is made a likely one, so that paths are
found).  fork() gives a sequence's cache to another one: full pages are shared through the page
tables, the page that both would write next is copied.  The host counts each page's users, so that
no sequence writes into a page that another one reads.

    python examples/draft_step.py [--batch 8] [--nodes 16] [--context 4000] [--steps 4]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_sm_gb300 as dg  # noqa: E402


class Weight4:
    """A weight [n, k] by output column in 4 bits with group scales."""

    def __init__(self, w, group):
        self.n, self.k, self.group = w.shape[0], w.shape[1], group
        self.ldq, self.ldp = -(-self.k // 32) * 16, -(-self.n // 4) * 4
        self.q = torch.zeros((self.n, self.ldq), dtype=torch.uint8, device="cuda")
        self.params = torch.zeros((-(-self.k // group), self.ldp), dtype=torch.int32, device="cuda")
        dg.quantize_groups_w4(self.n, self.k, group, w, w.stride(0), self.q, self.ldq, self.params, self.ldp)

    def times(self, m, x, ldx, out, ws):
        dg.gemm_w4_bf16(m, self.n, self.k, self.group, x, ldx, self.q, self.ldq, self.params, self.ldp, out, self.n,
                        dg.DG_OUT_F32 if out.dtype == torch.float32 else dg.DG_OUT_BF16, ws, ws.numel())


class DraftStep:
    def __init__(self, batch, nodes, width=2048, heads_q=16, heads_kv=4, d=128, vocab=32000, group=128, page_size=64,
                 max_tokens=8192, seed=0):
        self.batch, self.nodes, self.width, self.heads_q, self.heads_kv, self.d = batch, nodes, width, heads_q, heads_kv, d
        self.vocab, self.page_size = vocab, page_size
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(n, k):
            return Weight4(torch.randn((n, k), generator=g, device="cuda", dtype=torch.bfloat16).mul_(1 / math.sqrt(k)), group)

        self.n = (heads_q + 2 * heads_kv) * d
        self.wqkv, self.wo, self.wh = weight(self.n, width), weight(width, heads_q * d), weight(vocab, width)
        self.table_width = -(-max_tokens // page_size)
        pages = batch * self.table_width
        self.pool = torch.zeros((pages, heads_kv, dg.dg_kv4_block_bytes(page_size, d)), dtype=torch.uint8, device="cuda")
        self.cache = dg.dg_kv4_cache(self.pool, pages, page_size, heads_kv, d)
        # Every sequence has pages for max_tokens (a program would hand them out as sequences grow).
        self.table = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32).view(batch, -1)
        self.users, self.free = [1] * pages, []                   # sequences whose tables name a page; pages that none names
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")

        def buf(*shape, dtype=torch.bfloat16):
            return torch.zeros(shape, dtype=dtype, device="cuda")

        m = batch * nodes
        self.x = buf(m, width)
        self.mask = buf(batch, nodes, dtype=torch.int64)          # bit t: node t is seen
        self.parent, self.token = buf(batch, nodes, dtype=torch.int64), buf(batch, nodes, dtype=torch.int64)
        self.qkv, self.attn, self.o = buf(m, self.n), buf(m, heads_q * d), buf(m, width)
        self.logits = buf(m, vocab, dtype=torch.float32)
        self.path, self.counts = buf(batch, nodes, dtype=torch.int32), buf(batch, dtype=torch.int32)
        # Workspaces are zeroed once and reused by every step.
        self.attn_ws = buf(dg.dg_attention_kv4_workspace_bytes(batch, nodes, heads_q, heads_kv, d), dtype=torch.uint8)
        self.gemm_ws = buf(max(dg.dg_gemm_w4_workspace_bytes(m, w.n, w.k) for w in (self.wqkv, self.wo, self.wh)), dtype=torch.uint8)

    def slots(self, tokens):
        """Slots of the next `tokens` tokens of every sequence; past its pages -1, which kv4_append passes over (and
        attention_kv4_tree reports the length)."""
        at = torch.arange(tokens, device="cuda")[None] + self.lens.long()[:, None]
        nth = at // self.page_size
        page = torch.gather(self.table.long(), 1, nth.clamp(max=self.table_width - 1))
        return torch.where(nth < self.table_width, page * self.page_size + at % self.page_size, -1).flatten()

    def prompt(self, k, v):
        """Writes a prompt's keys and values, [batch, tokens, heads_kv * d] BF16, to the cache."""
        b, t, w = k.shape
        dg.kv4_append(self.cache, b * t, k, w, v, w, self.slots(t))
        self.lens.add_(t)

    def draft(self, parent, token):
        """The trees: parents [batch, nodes] (of node 0: itself) and tokens."""
        self.parent.copy_(parent)
        self.token.copy_(token)
        bit = torch.ones(self.nodes, dtype=torch.int64, device="cuda") << torch.arange(self.nodes, device="cuda")
        self.mask.copy_(bit[None].expand(self.batch, -1))
        for i in range(1, self.nodes):
            self.mask[:, i] |= self.mask.gather(1, self.parent[:, i:i + 1])[:, 0]

    def verify(self):
        """x [batch * nodes, width] -> logits; the trees' keys and values are in the cache then, lens include them."""
        b, t, hq, hkv, d, n = self.batch, self.nodes, self.heads_q, self.heads_kv, self.d, self.n
        self.wqkv.times(b * t, self.x, self.width, self.qkv, self.gemm_ws)
        dg.kv4_append(self.cache, b * t, self.qkv[:, hq * d:], n, self.qkv[:, (hq + hkv) * d:], n, self.slots(t))
        self.lens.add_(t)
        dg.attention_kv4_tree(self.cache, b, t, hq, 1 / math.sqrt(d), self.qkv, n, t * n, self.table, self.table_width, self.lens,
                              None, self.mask, self.attn, hq * d, t * hq * d, self.attn_ws, self.attn_ws.numel())
        self.wo.times(b * t, self.attn, hq * d, self.o, self.gemm_ws)
        self.wh.times(b * t, self.o, self.width, self.logits, self.gemm_ws)

    def accept(self):
        """Keeps each tree's longest path of tokens that its logits predict (node 0 always)."""
        b, t = self.batch, self.nodes
        best = self.logits.view(b, t, -1).argmax(-1)
        depth = torch.zeros((b, t), dtype=torch.int64, device="cuda")  # of accepted nodes; 0: not accepted
        depth[:, 0] = 1
        for i in range(1, t):
            up = self.parent[:, i:i + 1]
            agrees = best.gather(1, up)[:, 0] == self.token[:, i]
            depth[:, i] = torch.where(agrees & (depth.gather(1, up)[:, 0] > 0), depth.gather(1, up)[:, 0] + 1, 0)
        count, end = depth.max(1)
        self.counts.copy_(count)
        # The path's nodes in ascending order: the bits of its end's mask.
        on = (self.mask.gather(1, end[:, None]) >> torch.arange(t, device="cuda")[None]) & 1 == 1
        self.path.copy_(torch.where(on, torch.arange(t, device="cuda")[None], t).sort(1)[0])
        dg.kv4_accept(self.cache, b, t, self.table, self.table_width, self.lens, None, self.path, t, self.counts, self.lens)

    def fork(self, src, dst):
        """Sequence dst goes on from what src has (lists of sequences, one pair after the other; what dst had is gone)."""
        for a, b in zip(src, dst):
            if a == b:
                continue
            n = int(self.lens[a])
            full = n // self.page_size
            if n > self.table_width * self.page_size:
                raise ValueError(f"sequence {a} has outgrown its pages")
            old, source = self.table[b].tolist(), self.table[a].tolist()
            for page in old:
                self.users[page] -= 1
                if self.users[page] == 0:
                    self.free.append(page)
            # Full pages are shared; the others are dst's own.  (The other tables name at most all pages but a
            # table's width of them, so there are enough.)
            new = source[:full] + [self.free.pop() for _ in range(full, self.table_width)]
            for page in new:
                self.users[page] += 1
            self.table[b].copy_(torch.tensor(new, dtype=torch.int32))
            if n % self.page_size:
                dg.kv4_copy_pages(self.cache, 1, self.table[a, full:full + 1].contiguous(), self.table[b, full:full + 1].contiguous())
            self.lens[b] = n

    def capture(self):
        """A graph of verify() and accept(), for replay().  Runs one step."""
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            self.verify()
            self.accept()
        torch.cuda.current_stream().wait_stream(stream)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            self.verify()
            self.accept()
        return graph


def random_trees(batch, nodes, vocab, generator=None):
    """(parents, tokens) of random trees: every node's parent is an earlier one."""
    parent = (torch.rand((batch, nodes), generator=generator, device="cuda") * torch.arange(nodes, device="cuda")).long()
    return parent, torch.randint(0, vocab, (batch, nodes), generator=generator, device="cuda")


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--nodes", type=int, default=16)
    ap.add_argument("--context", type=int, default=4000)
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args()
    step = DraftStep(a.batch, a.nodes, max_tokens=a.context + (a.steps + 2) * a.nodes)
    kv = (a.batch, a.context, step.heads_kv * step.d)
    step.prompt(torch.randn(kv, device="cuda", dtype=torch.bfloat16), torch.randn(kv, device="cuda", dtype=torch.bfloat16))
    step.x.copy_(torch.randn_like(step.x))
    parent, token = random_trees(a.batch, a.nodes, step.vocab)
    step.draft(parent, token)
    before = step.lens.clone()
    step.verify()
    # The tokens that the model would choose at each parent, for half of the nodes.
    best = step.logits.view(a.batch, a.nodes, -1).argmax(-1)
    step.draft(parent, torch.where(torch.rand_like(parent, dtype=torch.float32) < 0.5, best.gather(1, parent), token))
    step.lens.copy_(before)
    graph = step.capture()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    times = []
    for _ in range(a.steps):
        start.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end) * 1e3)
    status = dg.dg_device_status()
    assert status == dg.DG_OK, dg.status_string(status)
    assert bool(step.logits.isfinite().all())
    print(f"batch {a.batch}, trees of {a.nodes}, context {a.context}: {min(times):.1f} us a step (of {a.steps}), "
          f"{float(step.counts.float().mean()):.1f} tokens kept")


if __name__ == "__main__":
    main()
