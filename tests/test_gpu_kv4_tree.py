"""Trees of drafted tokens over the 4-bit cache: attention_kv4_tree against the float64 oracle within
its bound, kv4_accept and kv4_copy_pages bit for bit."""
import numpy as np
import pytest

import dense_gemm_sm_gb300 as dg
from oracle import serving as ref

from .helpers import torch_mod
from .test_gpu_kv4 import build, dev, host, rows, sync

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    dg.load()
    return t


def trees(rng, batch, lq):
    """Masks [batch, lq] (uint64) of random trees: ancestors and the node itself."""
    mask = np.zeros((batch, lq), np.uint64)
    for b in range(batch):
        for i in range(lq):
            up = rng.integers(-1, i) if i else -1
            mask[b, i] = np.uint64(1 << i) | (mask[b, up] if up >= 0 else np.uint64(0))
    return mask


def oracle(pool, q, table, lens, scale, sees=None):
    return ref.kv4_attention(pool, q, table, lens, scale, sees, middle=8)


def attend(torch, pool, data, table, lens, nodes, mask, q, scale, pad=0, batch_pad=0, ws=None):
    batch, lq, hq, d = q.shape
    ld = hq * d + pad
    stride = lq * ld + batch_pad
    Q = torch.full((batch * stride,), float("nan"), dtype=torch.bfloat16, device="cuda")
    O = torch.full((batch * stride,), -3.0, dtype=torch.bfloat16, device="cuda")
    Q.as_strided((batch, lq, hq * d), (stride, ld, 1)).copy_(dev(torch, q.astype(np.float32).reshape(batch, lq, -1)))
    cache = dg.dg_kv4_cache(data, pool.pages, pool.page_size, pool.heads, d)
    if ws is None:
        ws = torch.zeros(dg.dg_attention_kv4_workspace_bytes(batch, lq, hq, pool.heads, d), dtype=torch.uint8, device="cuda")
    T = torch.from_numpy(table.astype(np.int32)).cuda()
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    n = None if nodes is None else torch.tensor(nodes, dtype=torch.int32, device="cuda")
    M = torch.from_numpy(np.ascontiguousarray(mask).view(np.int64)).cuda()
    dg.attention_kv4_tree(cache, batch, lq, hq, scale, Q, ld, stride, T, table.shape[1], L, n, M, O, ld, stride, ws, ws.numel())
    ov = O.as_strided((batch, lq, hq * d), (stride, ld, 1))
    got = ov.float().cpu().numpy().reshape(batch, lq, hq, d).astype(np.float64)
    ov.fill_(-3.0)
    assert bool((O == -3.0).all())                            # nothing between the rows is written
    return got


def check(torch, lens, nodes, lq, hq, heads, d, page_size, seed=0, mask=None, **more):
    rng = np.random.default_rng(seed + sum(lens) + d + hq + lq)
    pool, data, table = build(torch, rng, lens, page_size, heads, d, spare_cols=seed % 3)
    q = ref.bf16(rng.standard_normal((len(lens), lq, hq, d)) * more.pop("std", 1.0)).astype(np.float64)
    mask = trees(rng, len(lens), lq) if mask is None else mask
    scale = float(np.float32(1 / np.sqrt(d)))
    got = attend(torch, pool, data, table, lens, nodes, mask, q, scale, **more)
    sync(torch)
    n = [lq] * len(lens) if nodes is None else nodes
    want, bound = oracle(pool, q, table, lens, scale, ref.tree_sees(lens, n, mask))
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, first {np.argwhere(bad)[0]}, worst {np.nanmax(np.abs(got - want) / (bound + 1e-30)):.3g}"
    for b, m in enumerate(n):
        assert not got[b, m:].any()
    return got


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 300, 1000])
def test_tree_contexts(torch, ctx, d):
    check(torch, [ctx + 10], None, 10, 8, 2, d, 16, seed=ctx)
    check(torch, [ctx + 40], None, 40, 4, 1, d, 32, seed=ctx)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lq", [1, 2, 7, 8, 9, 31, 32, 33, 63, 64])
def test_tree_sizes(torch, lq, d):
    check(torch, [200 + lq, lq, 65 + lq], None, lq, 4, 2, d, 48, seed=lq)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,heads,lq", [(1, 1, 5), (7, 1, 9), (14, 2, 13), (8, 1, 16), (16, 1, 25), (33, 1, 4), (12, 3, 21), (8, 1, 64), (28, 4, 25)])
def test_tree_heads(torch, hq, heads, lq, d):
    check(torch, [230, 70, 512 + lq], None, lq, hq, heads, d, 64, seed=lq)


@pytest.mark.parametrize("page_size", [16, 32, 48, 64, 80, 128, 256])
def test_tree_pages(torch, page_size):
    check(torch, [300, 40, 77], None, 30, 8, 2, 128, page_size, seed=page_size)
    check(torch, [300, 40, 77], None, 30, 8, 2, 64, page_size, seed=page_size)


@pytest.mark.parametrize("lq,hq", [(12, 8), (40, 8), (64, 16)])
def test_trees_of_different_sizes(torch, lq, hq):
    # Fewer nodes than queries, none, and a sequence without a token.
    nodes = [lq, 1, 0, lq // 2, 0, lq - 1]
    lens = [400, 90, 33, lq // 2, 0, 2000]
    check(torch, lens, nodes, lq, hq, 2, 128, 32, seed=3)
    check(torch, lens, nodes, lq, hq, 2, 64, 32, seed=4)


@pytest.mark.parametrize("lq,hq", [(2, 4), (4, 8), (8, 4), (6, 16)])
@pytest.mark.parametrize("nodes,lens", [([0, 2, 0, 1], [3000, 40, 500, 2]), ([1, 0], [33, 1500]), ([0, 0, 0], [100, 0, 700]),
                                        ([2] + [0, 1, 0, 2, 0] * 30, [50] + [700, 90, 33, 64, 1] * 30)])
def test_sequences_without_a_draft(torch, lq, hq, nodes, lens):
    # Contexts without a query among others: zeros, and the others as ever.
    check(torch, lens, nodes, lq, hq, 2, 128 if len(lens) < 5 else 64, 32, seed=lq)


@pytest.mark.parametrize("lq", [2, 40])
def test_context_without_a_draft_is_not_read(torch, lq):
    # Not a page of it, which a page outside the cache would tell.
    rng = np.random.default_rng(lq)
    lens, nodes = [300, 600, 70], [lq, 0, lq]
    pool, data, table = build(torch, rng, lens, 16, 2, 64)
    table[1] = pool.pages
    q = ref.bf16(rng.standard_normal((3, lq, 4, 64))).astype(np.float64)
    mask = trees(rng, 3, lq)
    got = attend(torch, pool, data, table, lens, nodes, mask, q, 0.125)
    sync(torch)
    want, bound = oracle(pool, q, table, lens, 0.125, ref.tree_sees(lens, nodes, mask))
    assert np.all(np.abs(got - want) <= bound) and not got[1].any()


@pytest.mark.parametrize("hq", [2, 16])
def test_tree_longer_than_its_sequence(torch, hq):
    # The first nodes would lie before position 0: there are no such keys.
    check(torch, [3, 9, 1], None, 12, hq, 2, 128, 16)


def test_masks_that_leave_nothing(torch):
    rng = np.random.default_rng(1)
    for lq in (8, 40):
        mask = trees(rng, 3, lq)
        mask[0, ::2] = 0                                     # no context in the first sequence: rows without a key
        mask[1, 1] = 0                                       # the context alone
        mask[2] = ~np.uint64(0)                              # every node, itself and later ones too
        got = check(torch, [lq, 100, lq + 5], None, lq, 16, 2, 128, 16, mask=mask)
        assert not got[0, ::2].any() and got[0, 1].any()


@pytest.mark.parametrize("d", [64, 128])
def test_bits_past_the_tree_name_nothing(torch, d):
    rng = np.random.default_rng(2)
    mask = trees(rng, 2, 20) | np.uint64(0xFFFFFFFFFFF00000)
    check(torch, [150, 60], [20, 11], 20, 8, 2, d, 16, mask=mask)


def test_a_chain_is_attention_of_the_newest_tokens(torch):
    rng = np.random.default_rng(3)
    for lq, hq in ((5, 8), (40, 8)):
        lens = [700, 40, 333]
        pool, data, table = build(torch, rng, lens, 64, 2, 128)
        q = ref.bf16(rng.standard_normal((3, lq, hq, 128))).astype(np.float64)
        mask = np.array([[(1 << (i + 1)) - 1 for i in range(lq)]] * 3, np.uint64)
        got = attend(torch, pool, data, table, lens, None, mask, q, 0.09)
        want, bound = oracle(pool, q, table, lens, float(np.float32(0.09)))
        sync(torch)
        assert np.all(np.abs(got - want) <= bound)


def test_tree_strides_and_peaked_scores(torch):
    check(torch, [130, 60], None, 20, 8, 2, 128, 16, pad=72, batch_pad=16)
    check(torch, [130, 60], [9, 20], 20, 8, 2, 64, 16, pad=8, batch_pad=64, std=30.0)
    check(torch, [700], None, 33, 8, 1, 128, 64, std=30.0)


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("lq,ctx", [(3, 40), (40, 0), (40, 200), (64, 3000)])
def test_tree_scores_far_from_zero(torch, lq, ctx, sign):
    # All scores at about +-900 in units of log2; the context's first unit far below what follows.
    rng = np.random.default_rng(ctx + lq)
    n, heads, d, page_size = ctx + lq, 2, 128, 32
    pool = ref.Kv4Pool(-(-n // page_size), page_size, heads, d)
    k = np.ones((n, heads, d), np.float32) + 0.02 * rng.standard_normal((n, heads, d)).astype(np.float32)
    k[:min(ctx, 128)] *= 1.5
    pool.append(ref.bf16(k), rows(rng, (n, heads, d)), np.arange(n))
    q = ref.bf16(sign * (30 + rng.standard_normal((1, lq, 8, d)))).astype(np.float64)
    table, mask = np.arange(pool.pages)[None], trees(rng, 1, lq)
    scale = float(np.float32(0.17))
    got = attend(torch, pool, torch.from_numpy(pool.pack()).cuda(), table, [n], None, mask, q, scale)
    sync(torch)
    want, bound = oracle(pool, q, table, [n], scale, ref.tree_sees([n], [lq], mask))
    assert np.isfinite(got).all() and np.all(np.abs(got - want) <= bound)


@pytest.mark.parametrize("lens,lq,hq,heads,d", [([6000], 16, 8, 1, 128), ([9000, 0, 4000], 8, 8, 1, 64), ([5000, 300], 64, 8, 2, 128),
                                               ([2000] * 9, 30, 8, 2, 64)])
def test_tree_long_contexts_in_one_workspace(torch, lens, lq, hq, heads, d):
    ws = torch.zeros(dg.dg_attention_kv4_workspace_bytes(len(lens), lq, hq, heads, d), dtype=torch.uint8, device="cuda")
    nodes = [min(n, lq) for n in lens]
    for seed in (1, 2):
        check(torch, lens, nodes, lq, hq, heads, d, 64, seed=seed, ws=ws)


# Items (sequence, cache head, 128 query rows) of one size, which get CTAs of their own where no CTA's
# share grows by more than a unit of 128 keys, and of nearly one size; few items of many parts, which
# threads share, many of few.
@pytest.mark.parametrize("batch,length,other,lq,hq,heads,d", [
    (1, 8208, 8208, 16, 16, 8, 128), (1, 19500, 19500, 40, 1, 1, 64), (1, 19500, 19500, 60, 8, 1, 128), (3, 512, 512, 20, 8, 4, 64),
    (3, 512, 400, 20, 8, 4, 64), (19, 1000, 1000, 18, 2, 2, 128), (40, 300, 300, 20, 4, 4, 64), (75, 130, 257, 33, 2, 2, 64), (150, 129, 1, 17, 1, 1, 128)])
def test_items_of_one_size(torch, batch, length, other, lq, hq, heads, d):
    check(torch, [length] * (batch - 1) + [other], None if other >= lq else [lq] * (batch - 1) + [other], lq, hq, heads, d, 64, std=4.0)


@pytest.mark.parametrize("lq", [3, 40])
def test_trees_and_tokens_in_one_workspace(torch, lq):
    """A workspace that attention_kv4 and attention_kv4_tree use in turn."""
    rng = np.random.default_rng(9)
    lens, hq, heads, d = [1500, 700], 8, 2, 128
    pool, data, table = build(torch, rng, lens, 64, heads, d)
    q = ref.bf16(rng.standard_normal((2, lq, hq, d))).astype(np.float64)
    mask = trees(rng, 2, lq)
    scale = float(np.float32(0.09))
    ws = torch.zeros(dg.dg_attention_kv4_workspace_bytes(2, lq, hq, heads, d), dtype=torch.uint8, device="cuda")
    want, bound = oracle(pool, q, table, lens, scale, ref.tree_sees(lens, [lq] * 2, mask))
    plain, plain_bound = oracle(pool, q, table, lens, scale)
    cache = dg.dg_kv4_cache(data, pool.pages, 64, heads, d)
    Q = dev(torch, q.astype(np.float32).reshape(2, -1))
    T, L = torch.from_numpy(table.astype(np.int32)).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    for _ in range(3):
        got = attend(torch, pool, data, table, lens, None, mask, q, scale, ws=ws)
        assert np.all(np.abs(got - want) <= bound)
        O = torch.zeros_like(Q)
        dg.attention_kv4(cache, 2, lq, hq, scale, Q, hq * d, lq * hq * d, T, table.shape[1], L, O, hq * d, lq * hq * d, ws, ws.numel())
        sync(torch)
        assert np.all(np.abs(O.float().cpu().numpy().reshape(plain.shape) - plain) <= plain_bound)


@pytest.mark.parametrize("lq", [3, 40])
def test_two_streams_of_trees(torch, lq):
    """Calls on two streams at once, each with a workspace of its own, on one cache."""
    rng = np.random.default_rng(10)
    lens, hq, heads, d = [3000, 900, 20], 8, 2, 64
    pool, data, table = build(torch, rng, lens, 48, heads, d)
    cache = dg.dg_kv4_cache(data, pool.pages, 48, heads, d)
    T, L = torch.from_numpy(table.astype(np.int32)).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    calls = []
    for _ in range(2):
        q = ref.bf16(rng.standard_normal((3, lq, hq, d))).astype(np.float64)
        n = [min(lq, k) for k in lens]
        mask = trees(rng, 3, lq)
        Q = dev(torch, q.astype(np.float32).reshape(3, -1))
        calls.append((torch.cuda.Stream(), Q, torch.zeros((8,) + tuple(Q.shape), dtype=Q.dtype, device="cuda"), torch.from_numpy(mask.view(np.int64)).cuda(),
                      torch.tensor(n, dtype=torch.int32, device="cuda"),
                      torch.zeros(dg.dg_attention_kv4_workspace_bytes(3, lq, hq, heads, d), dtype=torch.uint8, device="cuda"),
                      oracle(pool, q, table, lens, float(np.float32(0.125)), ref.tree_sees(lens, n, mask))))
    torch.cuda.synchronize()
    for k in range(8):
        for stream, Q, O, M, N, ws, _ in calls:
            dg.attention_kv4_tree(cache, 3, lq, hq, 0.125, Q, hq * d, lq * hq * d, T, table.shape[1], L, N, M, O[k], hq * d, lq * hq * d, ws, ws.numel(),
                                  stream=stream)
    sync(torch)
    for _, _, O, _, _, _, (want, bound) in calls:
        for k in range(8):
            assert np.all(np.abs(O[k].float().cpu().numpy().reshape(want.shape) - want) <= bound)


@pytest.mark.parametrize("lq", [6, 40])
def test_tree_repeats_bit_for_bit_and_in_a_graph(torch, lq):
    rng = np.random.default_rng(12)
    lens = [1800, 60, 333]
    pool, data, table = build(torch, rng, lens, 64, 2, 128)
    q = ref.bf16(rng.standard_normal((3, lq, 16, 128))).astype(np.float64)
    mask = trees(rng, 3, lq)
    first = attend(torch, pool, data, table, lens, None, mask, q, 0.09)
    for _ in range(3):
        assert np.array_equal(attend(torch, pool, data, table, lens, None, mask, q, 0.09), first)
    cache = dg.dg_kv4_cache(data, pool.pages, 64, 2, 128)
    ws = torch.zeros(dg.dg_attention_kv4_workspace_bytes(3, lq, 16, 2, 128), dtype=torch.uint8, device="cuda")
    Q = dev(torch, q.astype(np.float32).reshape(3, -1))
    O = torch.zeros_like(Q)
    T, L = torch.from_numpy(table.astype(np.int32)).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    N = torch.full((3,), lq, dtype=torch.int32, device="cuda")
    M = torch.from_numpy(mask.view(np.int64)).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.attention_kv4_tree(cache, 3, lq, 16, 0.09, Q, 2048, 2048 * lq, T, table.shape[1], L, N, M, O, 2048, 2048 * lq, ws, ws.numel())
    for _ in range(3):
        graph.replay()
        sync(torch)
        assert np.array_equal(O.float().cpu().numpy().reshape(first.shape), first)
    L.copy_(torch.tensor([1, 50, 0], dtype=torch.int32))      # the graph follows lengths, sizes and masks
    N.copy_(torch.tensor([1, 3, 0], dtype=torch.int32))
    mask = trees(rng, 3, lq)
    M.copy_(torch.from_numpy(mask.view(np.int64)))
    graph.replay()
    sync(torch)
    want, bound = oracle(pool, q, table, [1, 50, 0], float(np.float32(0.09)), ref.tree_sees([1, 50, 0], [1, 3, 0], mask))
    assert np.all(np.abs(O.float().cpu().numpy().reshape(first.shape) - want) <= bound)


@pytest.mark.parametrize("lq", [4, 40])
def test_tree_bad_pages_lengths_and_sizes(torch, lq):
    rng = np.random.default_rng(13)
    lens = [100, 100, 100]
    pool, data, table = build(torch, rng, lens, 16, 1, 64)
    table[0, 2], table[1, 6] = -1, pool.pages                # pages outside the cache are not visible
    q = ref.bf16(rng.standard_normal((3, lq, 4, 64))).astype(np.float64)
    mask = trees(rng, 3, lq)
    got = attend(torch, pool, data, table, lens, None, mask, q, 0.125)
    sync(torch, dg.DG_ERR_BAD_INDEX)
    want, bound = oracle(pool, q, table, lens, 0.125, ref.tree_sees(lens, [lq] * 3, mask))
    assert np.all(np.abs(got - want) <= bound)
    pool, data, table = build(torch, rng, [112, 112, 112], 16, 1, 64)
    got = attend(torch, pool, data, table, [-5, 10 ** 9, 112], [lq, lq, 2], mask, q, 0.125)
    sync(torch, dg.DG_ERR_BAD_INDEX)
    want, bound = oracle(pool, q, table, [0, 112, 112], 0.125, ref.tree_sees([0, 112, 112], [lq, lq, 2], mask))
    assert np.all(np.abs(got - want) <= bound)
    got = attend(torch, pool, data, table, [112, 112, 112], [-1, lq + 1, lq], mask, q, 0.125)
    sync(torch, dg.DG_ERR_BAD_INDEX)
    want, bound = oracle(pool, q, table, [112] * 3, 0.125, ref.tree_sees([112] * 3, [0, lq, lq], mask))
    assert np.all(np.abs(got - want) <= bound)


@pytest.mark.parametrize("lq", [4, 40])
def test_queries_that_are_not_finite_stay_alone(torch, lq):
    rng = np.random.default_rng(14)
    lens = [900, 60]
    pool, data, table = build(torch, rng, lens, 32, 2, 128)
    mask = trees(rng, 2, lq)
    q = ref.bf16(rng.standard_normal((2, lq, 8, 128))).astype(np.float64)
    good = attend(torch, pool, data, table, lens, None, mask, q, 0.09)
    q[0, 1, 3, 7] = np.nan
    q[1, lq - 1, 0, 64] = np.inf
    cache = dg.dg_kv4_cache(data, pool.pages, 32, 2, 128)
    Q = torch.from_numpy(q.astype(np.float32)).to(torch.bfloat16).cuda()
    O = torch.zeros((2, lq, 1024), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(dg.dg_attention_kv4_workspace_bytes(2, lq, 8, 2, 128), dtype=torch.uint8, device="cuda")
    dg.attention_kv4_tree(cache, 2, lq, 8, 0.09, Q, 1024, 1024 * lq, torch.from_numpy(table.astype(np.int32)).cuda(), table.shape[1],
                          torch.tensor(lens, dtype=torch.int32, device="cuda"), None, torch.from_numpy(mask.view(np.int64)).cuda(),
                          O, 1024, 1024 * lq, ws, ws.numel())
    sync(torch)
    got = O.float().cpu().numpy().reshape(2, lq, 8, 128)
    bad = np.zeros((2, lq, 8), bool)
    bad[0, 1, 3] = bad[1, lq - 1, 0] = True
    assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], good[~bad])


@pytest.mark.parametrize("lq,hq,heads,d", [(8, 4, 2, 128), (40, 4, 1, 64), (64, 8, 2, 128)])
def test_every_unit_of_keys_and_every_node_counts(torch, lq, hq, heads, d):
    # Queries of zeros weigh all visible keys alike; values are 1 in one column for each unit of 32 keys, so
    # that a lost, doubled or stale part moves a column by its whole share.
    rng = np.random.default_rng(15)
    ctx, page_size = 1000, 64                                 # a node's share, 0.001, is over the bound
    n = ctx + lq
    need = -(-n // page_size)
    table = rng.permutation(need + 1)[:need][None]
    pool = ref.Kv4Pool(need + 1, page_size, heads, d)
    slots = table[0, np.arange(n) // page_size] * page_size + np.arange(n) % page_size
    v = ref.unit_rows(n, d, 1)
    v[ctx:] = np.eye(d, dtype=np.float32)[np.arange(lq) % d]  # every node a column of its own
    k = rows(rng, (n, heads, d))
    pool.append(k, np.repeat(v[:, None], heads, 1), slots)
    mask = trees(rng, 1, lq)
    got = attend(torch, pool, torch.from_numpy(pool.pack()).cuda(), table, [n], None, mask, np.zeros((1, lq, hq, d)), 0.1)
    sync(torch)
    for i in range(lq):
        see = np.array([j < ctx or (int(mask[0, i]) >> (j - ctx)) & 1 for j in range(n)], bool)
        mean, err = ref.unit_mean(v[see], see.sum())
        assert np.all(np.abs(got[0, i] - mean) <= err)


# ------------------------------------------------------------------ accepted tokens
def accept_pool(rng, lens, page_size, heads, d):
    need = [-(-n // page_size) for n in lens]
    pages = sum(need) + 2
    table = np.full((len(lens), max(need + [1])), -1, np.int64)
    order, at = rng.permutation(pages), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    pool = ref.Kv4Pool(pages, page_size, heads, d)
    everything = np.arange(pages * page_size)
    pool.append(rows(rng, (len(everything), heads, d)), rows(rng, (len(everything), heads, d)), everything)
    return pool, table


def slot(pool, table, b, pos):
    pos = np.asarray(pos, np.int64)
    return table[b, pos // pool.page_size] * pool.page_size + pos % pool.page_size


def accept(torch, pool, data, table, lens, nodes, path, counts, lq, in_place=False):
    cache = dg.dg_kv4_cache(data, pool.pages, pool.page_size, pool.heads, pool.d)
    i32 = dict(dtype=torch.int32, device="cuda")
    L, C = torch.tensor(lens, **i32), torch.tensor(counts, **i32)
    N = None if nodes is None else torch.tensor(nodes, **i32)
    P = torch.tensor(np.asarray(path).reshape(len(lens), -1), **i32)
    new = L if in_place else torch.full_like(L, -9)
    dg.kv4_accept(cache, len(lens), lq, torch.from_numpy(table.astype(np.int32)).cuda(), table.shape[1], L, N, P, P.shape[1], C, new)
    return new


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page_size,heads,lq,lens", [(16, 1, 8, [8]), (16, 3, 64, [64, 100, 500]), (64, 8, 25, [1000, 30, 63, 64, 65, 25]),
                                                     (48, 2, 1, [1, 49, 50]), (16, 11, 40, [47, 48, 49])])
@pytest.mark.parametrize("in_place", [False, True])
def test_accept(torch, page_size, heads, lq, lens, d, in_place):
    rng = np.random.default_rng(d + lq + heads)
    pool, table = accept_pool(rng, lens, page_size, heads, d)
    data = torch.from_numpy(pool.pack()).cuda()
    nodes = [lq - (b % 3 if lq > 3 else 0) for b in range(len(lens))]
    counts = [int(rng.integers(0, n + 1)) for n in nodes]
    counts[0] = nodes[0]
    path = np.full((len(lens), lq + 2), 10 ** 6)             # entries past the count are not read
    for b, (n, c) in enumerate(zip(nodes, counts)):
        path[b, :c] = np.sort(rng.permutation(n)[:c]) if b % 2 else rng.integers(0, n, c)
    new = accept(torch, pool, data, table, lens, nodes, path, counts, lq, in_place)
    sync(torch)
    for b, (n, c) in enumerate(zip(nodes, counts)):
        base = lens[b] - n
        pool.move(slot(pool, table, b, base + path[b, :c]), slot(pool, table, b, base + np.arange(c)))
    assert new.tolist() == [m - n + c for m, n, c in zip(lens, nodes, counts)]
    assert np.array_equal(data.cpu().numpy(), pool.pack())


def test_accept_reports_what_it_leaves(torch):
    rng = np.random.default_rng(3)
    lens = [40] * 8
    pool, table = accept_pool(rng, lens, 16, 2, 64)
    lens = [40, 40, -1, 10 ** 6, 40, 40, 3, 40]
    table[7, 1] = pool.pages                                 # a node's page outside the cache
    data = torch.from_numpy(pool.pack()).cuda()
    nodes, counts = [8, 8, 8, 8, 9, 8, 8, 20], [2, 2, 2, 2, 2, 9, 2, 2]
    path = [[3, 5] + [0] * 6, [7, 8] + [0] * 6] + [[3, 4] + [0] * 6] * 5 + [[19, 0] + [0] * 6]
    new = accept(torch, pool, data, table, lens, nodes, path, counts, 8)
    sync(torch, dg.DG_ERR_BAD_INDEX)
    sync(torch)
    want = [34, 34, -1, 10 ** 6, 40, 40, 3, 40]
    assert new.tolist() == want
    for b, p in ((0, [3, 5]), (1, [7])):
        pool.move(slot(pool, table, b, 32 + np.array(p)), slot(pool, table, b, 32 + np.arange(len(p))))
    assert np.array_equal(data.cpu().numpy(), pool.pack())
    # A page outside the cache: that row stays, the others move.
    new = accept(torch, pool, data, table[7:], [40], [8], [[7, 1]], [2], 8)
    sync(torch)
    pool.move(slot(pool, table, 7, [39, 33]), slot(pool, table, 7, [32, 33]))
    assert np.array_equal(data.cpu().numpy(), pool.pack())
    table[7, 2] = -1
    accept(torch, pool, data, table[7:], [40], [8], [[7, 1]], [2], 8)
    sync(torch, dg.DG_ERR_BAD_INDEX)
    assert np.array_equal(data.cpu().numpy(), pool.pack())


def test_accept_in_a_graph(torch):
    rng = np.random.default_rng(4)
    pool, table = accept_pool(rng, [100, 90], 16, 2, 128)
    data = torch.from_numpy(pool.pack()).cuda()
    cache = dg.dg_kv4_cache(data, pool.pages, 16, 2, 128)
    i32 = dict(dtype=torch.int32, device="cuda")
    L, P, C = torch.tensor([100, 90], **i32), torch.tensor([[1, 2, 9, 9, 9], [0, 2, 4, 9, 9]], **i32), torch.tensor([2, 3], **i32)
    T = torch.from_numpy(table.astype(np.int32)).cuda()
    nodes = torch.tensor([3, 5], **i32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.kv4_accept(cache, 2, 5, T, table.shape[1], L, nodes, P, 5, C, L)
    lens = [100, 90]
    for _ in range(3):                                       # each replay goes on from the lengths of the one before
        graph.replay()
        sync(torch)
        for b, (n, p) in enumerate(((3, [1, 2]), (5, [0, 2, 4]))):
            base = lens[b] - n
            pool.move(slot(pool, table, b, base + np.array(p)), slot(pool, table, b, base + np.arange(len(p))))
            lens[b] = base + len(p)
        assert L.tolist() == lens and np.array_equal(data.cpu().numpy(), pool.pack())


# ------------------------------------------------------------------ pages
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page_size,heads,pages,n", [(16, 1, 3, 1), (48, 3, 40, 19), (64, 8, 64, 32), (16, 5, 700, 300), (256, 8, 9, 4)])
def test_copy_pages(torch, page_size, heads, pages, n, d):
    rng = np.random.default_rng(pages + d)
    block = dg.dg_kv4_block_bytes(page_size, d)
    before = rng.integers(0, 256, (pages, heads, block)).astype(np.uint8)
    order = rng.permutation(pages)
    src, dst = rng.choice(order[:pages - n], n), order[pages - n:]     # a page may go to several places
    data = torch.from_numpy(before).cuda()
    cache = dg.dg_kv4_cache(data, pages, page_size, heads, d)
    for _ in range(2):
        dg.kv4_copy_pages(cache, n, torch.tensor(src, dtype=torch.int32, device="cuda"), torch.tensor(dst, dtype=torch.int32, device="cuda"))
    sync(torch)
    want = before.copy()
    want[dst] = before[src]
    assert np.array_equal(data.cpu().numpy(), want)


def test_copy_pages_that_are_passed_over(torch):
    rng = np.random.default_rng(1)
    before = rng.integers(0, 256, (6, 2, 16 * 72)).astype(np.uint8)
    data = torch.from_numpy(before).cuda()
    cache = dg.dg_kv4_cache(data, 6, 16, 2, 64)

    def copy(src, dst):
        dg.kv4_copy_pages(cache, len(src), torch.tensor(src, dtype=torch.int32, device="cuda"), torch.tensor(dst, dtype=torch.int32, device="cuda"))
    copy([-1, 2, 3, -5], [1, -1, 3, -2 ** 31])
    sync(torch)
    assert np.array_equal(data.cpu().numpy(), before)
    copy([6, 1, 0], [1, 6, 5])
    sync(torch, dg.DG_ERR_BAD_INDEX)
    sync(torch)
    want = before.copy()
    want[5] = before[0]
    assert np.array_equal(data.cpu().numpy(), want)


def test_copy_page_offsets_past_32_bits(torch):
    page_size, heads, d = 256, 8, 128
    block = dg.dg_kv4_block_bytes(page_size, d)
    pages = (1 << 32) // (block * heads) + 4
    data = torch.zeros((pages, heads, block), dtype=torch.uint8, device="cuda")
    cache = dg.dg_kv4_cache(data, pages, page_size, heads, d)
    data[1].random_(1, 256)
    dg.kv4_copy_pages(cache, 1, torch.tensor([1], dtype=torch.int32, device="cuda"), torch.tensor([pages - 1], dtype=torch.int32, device="cuda"))
    dg.kv4_copy_pages(cache, 1, torch.tensor([pages - 1], dtype=torch.int32, device="cuda"), torch.tensor([0], dtype=torch.int32, device="cuda"))
    sync(torch)
    assert torch.equal(data[pages - 1], data[1]) and torch.equal(data[0], data[1]) and not data[pages - 2].any() and not data[2].any()
