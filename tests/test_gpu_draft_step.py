"""examples/draft_step.py: the calls of a speculative decoding step one after the other, each against the
oracle on its own inputs, eagerly and from a graph; forks; and the example's command."""
import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest

import dense_gemm_sm_gb300 as dg
from oracle import serving as ref

from .helpers import torch_mod

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("draft_step", os.path.join(ROOT, "examples", "draft_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f32(t):
    return t.detach().float().cpu().numpy()


def unpack(w):
    """(codes, scale, zero) of a Weight4."""
    q = w.q.cpu().numpy().view(np.uint32)
    k = np.arange(w.k)
    codes = ((q[:, k // 8] >> (4 * (k % 8 // 2) + 16 * (k % 2)).astype(np.uint32)) & 15).astype(np.uint8)
    p = w.params.cpu().numpy().view(np.uint32)[:, :w.n].T
    return codes, ref.widen(p & 0xFFFF), ref.widen(p >> 16)


def close(got, want, bound):
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.nanmax(np.abs(got - want) / (bound + 1e-30)):.3g}"


@pytest.mark.parametrize("batch,nodes,hq,d,graphed", [(3, 7, 8, 64, False), (3, 7, 4, 128, True), (2, 40, 8, 128, True)])
def test_steps(example, batch, nodes, hq, d, graphed):
    torch = torch_mod()
    width, hkv, vocab, page, ctx = 192, 2, 300, 16, 37
    s = example.DraftStep(batch, nodes, width, hq, hkv, d, vocab, 64, page, max_tokens=ctx + 5 * nodes)
    g = torch.Generator(device="cuda").manual_seed(nodes)
    pool = ref.Kv4Pool(s.pool.shape[0], page, hkv, d)
    table = s.table.cpu().numpy()

    def slots(b, pos):
        return table[b, np.asarray(pos) // page] * page + np.asarray(pos) % page

    k, v = (torch.randn((batch, ctx, hkv * d), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    s.prompt(k, v)
    for b in range(batch):
        pool.append(f32(k[b]).reshape(ctx, hkv, d), f32(v[b]).reshape(ctx, hkv, d), slots(b, np.arange(ctx)))
    weights = [unpack(w) for w in (s.wqkv, s.wo, s.wh)]
    parent, token = example.random_trees(batch, nodes, vocab, g)
    graph = None
    if graphed:  # a step to warm up and the capture, on a cache that is put back
        s.draft(parent, token)
        kept = s.pool.clone(), s.lens.clone()
        graph = s.capture()
        s.pool.copy_(kept[0])
        s.lens.copy_(kept[1])
    lens = np.full(batch, ctx)
    moved = 0
    for turn in range(3):
        parent, token = example.random_trees(batch, nodes, vocab, g)
        s.x.copy_(torch.randn(s.x.shape, generator=g, device="cuda"))
        if turn:  # drafts that the model agrees with: what it chose at their parents (a step ahead, put back)
            s.draft(parent, token)
            kept = s.pool.clone(), s.lens.clone()
            s.verify()
            best = s.logits.view(batch, nodes, -1).argmax(-1)
            token = torch.where(torch.rand(token.shape, generator=g, device="cuda") < 0.7, best.gather(1, parent), token)
            s.pool.copy_(kept[0])
            s.lens.copy_(kept[1])
        s.draft(parent, token)
        if graphed:
            graph.replay()
        else:
            s.verify()
            s.accept()
        torch.cuda.synchronize()
        assert dg.dg_device_status() == dg.DG_OK
        close(f32(s.qkv), *ref.w4_gemm(f32(s.x), *weights[0], 64, ref.BF16))
        qkv = f32(s.qkv).reshape(batch, nodes, -1)
        new = qkv[..., hq * d:].reshape(batch, nodes, 2, hkv, d)
        for b in range(batch):
            pool.append(new[b, :, 0], new[b, :, 1], slots(b, lens[b] + np.arange(nodes)))
        lens = lens + nodes
        mask = s.mask.cpu().numpy().view(np.uint64)
        q = qkv[..., :hq * d].reshape(batch, nodes, hq, d).astype(np.float64)
        want, bound = ref.kv4_attention(pool, q, table, lens, float(np.float32(1 / np.sqrt(d))),
                                        ref.tree_sees(lens, [nodes] * batch, mask), middle=8)
        close(f32(s.attn).reshape(want.shape), want, bound)
        close(f32(s.o), *ref.w4_gemm(f32(s.attn), *weights[1], 64, ref.BF16))
        close(f32(s.logits), *ref.w4_gemm(f32(s.o), *weights[2], 64, ref.F32))
        # The accepted path, from the logits that were computed.
        best = s.logits.view(batch, nodes, -1).argmax(-1).cpu().numpy()
        par, tok = parent.cpu().numpy(), token.cpu().numpy()
        for b in range(batch):
            paths = {0: [0]}
            for i in range(1, nodes):
                if par[b, i] in paths and best[b, par[b, i]] == tok[b, i]:
                    paths[i] = paths[par[b, i]] + [i]
            path = max(paths.values(), key=len)
            assert int(s.counts[b]) == len(path)
            got = s.path[b, :len(path)].tolist()
            assert got in list(paths.values())
            base = lens[b] - nodes
            pool.move(slots(b, base + np.array(got)), slots(b, base + np.arange(len(got))))
            moved += sum(i != j for i, j in enumerate(got))
            lens[b] = base + len(got)
        assert s.lens.tolist() == lens.tolist()
        for b in range(batch):                               # what the sequences keep, bit for bit
            at = slots(b, np.arange(lens[b]))
            K, V = (torch.empty((lens[b], hkv * d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
            dg.kv4_gather(s.cache, int(lens[b]), torch.from_numpy(at).cuda(), K, hkv * d, V, hkv * d)
            for w, x in enumerate((K, V)):
                assert np.array_equal(f32(x), ref.bf16(pool.rows(w, at).astype(np.float32)).reshape(lens[b], -1))
    assert moved > 0


def test_a_fork_goes_on_by_itself(example):
    torch = torch_mod()
    s = example.DraftStep(3, 5, 128, 4, 2, 64, 200, 32, 16, max_tokens=96)
    k, v = (torch.randn((3, 41, 128), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    s.prompt(k, v)
    s.fork([0], [2])
    assert s.lens.tolist() == [41, 41, 41] and s.table[2, :2].tolist() == s.table[0, :2].tolist() and int(s.table[2, 2]) != int(s.table[0, 2])
    parent, token = example.random_trees(3, 5, 200)
    s.draft(parent[:1].expand(3, -1), token[:1].expand(3, -1))
    s.x.copy_(torch.randn((5, 128), device="cuda").repeat(3, 1))
    s.verify()
    torch.cuda.synchronize()
    assert dg.dg_device_status() == dg.DG_OK
    # The fork computes what its source does, and sequence 1, of another context, does not.
    out = s.logits.view(3, 5, -1)
    assert torch.equal(out[0], out[2]) and not torch.equal(out[0], out[1])
    # Different tokens behind the same context: the source's own page is not the fork's.
    a, b = s.slots(1)[0], s.slots(1)[2]
    assert int(a) != int(b)


def kept(s, b):
    """Sequence b's rows of K and V as they stand in the cache."""
    torch = torch_mod()
    n, w = int(s.lens[b]), s.heads_kv * s.d
    at = torch.arange(n, device="cuda")
    slots = s.table[b].long()[at // s.page_size] * s.page_size + at % s.page_size
    k, v = (torch.empty((n, w), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dg.kv4_gather(s.cache, n, slots, k, w, v, w)
    return k, v


@pytest.mark.parametrize("forks", [
    [(0, 2), (1, 2)],                                         # into a former copy, from a shorter sequence
    [(0, 2), (1, 0)],                                         # into a former source
    [(0, 2), (0, 1), (3, 0), (2, 3)],
    [(0, 2), (2, 0), (1, 1)],                                 # back again; to itself
])
def test_forks_of_forks_write_into_no_shared_page(example, forks):
    torch = torch_mod()
    s = example.DraftStep(4, 5, 128, 4, 2, 64, 200, 32, 16, max_tokens=96)
    k, v = (torch.randn((4, 41, 128), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    s.prompt(k, v)
    s.lens.copy_(torch.tensor([41, 20, 33, 16]))              # contexts of different lengths, one that ends with its page
    rows = {b: kept(s, b) for b in range(4)}
    for a, b in forks:
        s.fork([a], [b])
        rows[b] = rows[a]
    for step in range(2):
        before = s.lens.tolist()
        table = s.table.tolist()
        for b in range(4):                                    # where b writes nobody else reads
            others = [p for c in range(4) if c != b for p in table[c]]
            assert len(set(table[b])) == len(table[b]) and not set(table[b][before[b] // 16:]) & set(others)
        parent, token = example.random_trees(4, 5, 200)
        s.draft(parent, token)
        s.x.copy_(torch.randn_like(s.x))
        s.verify()
        s.accept()
        torch.cuda.synchronize()
        assert dg.dg_device_status() == dg.DG_OK
        for b in range(4):
            for x, y in zip(kept(s, b), rows[b]):
                assert torch.equal(x[:len(y)], y)


def test_a_sequence_that_outgrows_its_pages_is_reported(example):
    torch = torch_mod()
    s = example.DraftStep(2, 5, 128, 4, 2, 64, 200, 32, 16, max_tokens=48)
    k, v = (torch.randn((2, 44, 128), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    s.prompt(k, v)
    s.lens[1] = 20
    first = kept(s, 0)
    assert s.slots(5)[4] == -1 and (s.slots(5)[:4] >= 0).all() and (s.slots(5)[5:] >= 0).all()
    s.draft(*example.random_trees(2, 5, 200))
    s.verify()                                                # 49 tokens in 48 places
    torch.cuda.synchronize()
    assert dg.dg_device_status() == dg.DG_ERR_BAD_INDEX
    with pytest.raises(ValueError):
        s.fork([0], [1])
    s.lens.copy_(torch.tensor([44, 20]))
    for x, y in zip(kept(s, 0), first):
        assert torch.equal(x, y)


def test_the_command_runs(example):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "draft_step.py"), "--batch", "2", "--nodes", "6", "--context", "100",
                        "--steps", "2"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "us a step" in r.stdout, r.stdout + r.stderr
