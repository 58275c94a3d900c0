"""Attention over the 4-bit cache where drafted keys are not finite: they touch the queries that see them and
no others; and where queries hold an infinity: they give NaN whatever the signs."""
import numpy as np
import pytest

import dense_gemm_sm_gb300 as dg
from oracle import serving as ref

from .helpers import torch_mod
from .test_gpu_kv4 import attend as attend_newest
from .test_gpu_kv4 import build, rows, sync
from .test_gpu_kv4_tree import attend, trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    dg.load()
    return t


NAN, INF, HUGE = 0x7FC0, 0x7F80, 0x7F70  # BF16 bits; 8 * HUGE is past FP32's range
BAD = [(NAN, 0), (0x3F80, NAN), (INF, 0x3F80), (0x3F80, INF), (0x3F80, 0xFF80), (HUGE, 0x3F80), (NAN, NAN)]


def plant(torch, pool, data, slot, which, scale, zero):
    """Sets the parameters of K (0) or V (1) of a slot, in all heads, to BF16 bits."""
    page, t = divmod(int(slot), pool.page_size)
    at = t // 16 * 16 * (pool.d + 8) + 16 * pool.d + 64 * which + t % 16 * 4
    word = torch.tensor([scale & 255, scale >> 8, zero & 255, zero >> 8], dtype=torch.uint8, device="cuda")
    data[page, :, at:at + 4] = word


# Query rows a cache head: 8, 16 (mma.sync), 64, 80, 160 (tcgen05, one block of rows and two); items that
# are whole and items cut over many CTAs.
FORMS = [(4, 4, 2, 128, [34, 20, 4]), (4, 4, 2, 64, [3000, 40, 300]), (8, 4, 2, 64, [38, 200, 8]), (8, 2, 1, 128, [2500, 40, 300]),
         (16, 4, 1, 128, [50, 16, 300]), (16, 16, 4, 128, [2050, 40, 300]), (20, 8, 2, 64, [70, 20, 150]), (40, 8, 2, 128, [2000, 128, 41])]


@pytest.mark.parametrize("seen", [False, True])
@pytest.mark.parametrize("lq,hq,heads,d,lens", FORMS)
def test_nodes_that_are_not_finite(torch, lq, hq, heads, d, lens, seen):
    # `seen`: by those queries whose masks name the node, else by none, as the padding of a tree.
    rng = np.random.default_rng(lq + d + seen)
    pool, data, table = build(torch, rng, lens, 32, heads, d)
    scale = float(np.float32(1 / np.sqrt(d)))
    q = ref.bf16(rng.standard_normal((len(lens), lq, hq, d))).astype(np.float64)
    mask, sees, slots = trees(rng, len(lens), lq), np.zeros((len(lens), lq), bool), []
    for b, (n, node) in enumerate(zip(lens, (1 if seen else lq - 1, 2, lq // 2))):
        if not seen:
            mask[b] &= ~np.uint64(1 << node)
        sees[b] = (mask[b] >> np.uint64(node)) & np.uint64(1)
        at = n - lq + node
        slots.append(table[b, at // 32] * 32 + at % 32)
    assert sees.any() == seen
    # (Of clean keys, which is right for the queries that do not see a planted one.)
    want, bound = ref.kv4_attention(pool, q, table, lens, scale, ref.tree_sees(lens, [lq] * len(lens), mask), middle=8)
    clean = data.clone()
    for s, z in BAD:
        for which in (0, 1):
            data.copy_(clean)
            for slot in slots:
                plant(torch, pool, data, slot, which, s, z)
            got = attend(torch, pool, data, table, lens, None, mask, q, scale)
            sync(torch)
            close = np.abs(got - want) <= bound
            assert close[~sees].all(), f"{which} {s:x} {z:x}: {(~close[~sees]).sum()} of {close[~sees].size}"
            if which == 1 and s != HUGE:
                assert not np.isfinite(got[sees]).any()


@pytest.mark.parametrize("lq,hq,heads,d,lens", [(4, 4, 2, 128, [34, 20, 4]), (7, 1, 1, 64, [5000, 40, 300]), (8, 4, 2, 128, [3000, 200, 8]),
                                                (20, 8, 2, 64, [70, 20, 150]), (40, 8, 2, 128, [3000, 128, 41])])
def test_newest_tokens_that_are_not_finite(torch, lq, hq, heads, d, lens):
    # attention_kv4: token t of the newest is seen by queries t and later.
    rng = np.random.default_rng(lq + d)
    pool, data, table = build(torch, rng, lens, 32, heads, d)
    scale = float(np.float32(1 / np.sqrt(d)))
    q = ref.bf16(rng.standard_normal((len(lens), lq, hq, d))).astype(np.float64)
    want, bound = ref.kv4_attention(pool, q, table, lens, scale, middle=8)
    clean = data.clone()
    for s, z in BAD:
        for which in (0, 1):
            data.copy_(clean)
            sees = np.zeros((len(lens), lq), bool)
            for b, (n, t) in enumerate(zip(lens, (lq - 1, 1, lq // 2))):
                at = n - lq + t
                plant(torch, pool, data, table[b, at // 32] * 32 + at % 32, which, s, z)
                sees[b, t:] = True
            got = attend_newest(torch, pool, data, table, lens, q, scale)
            sync(torch)
            close = np.abs(got - want) <= bound
            assert close[~sees].all(), f"{which} {s:x} {z:x}: {(~close[~sees]).sum()} of {close[~sees].size}"
            if which == 1 and s != HUGE:
                assert not np.isfinite(got[sees]).any()


@pytest.mark.parametrize("lq,hq,heads,d,lens", FORMS)
def test_infinite_queries_over_keys_far_from_zero(torch, lq, hq, heads, d, lens):
    # Keys whose smallest element is far above their range: codes and zeros pull a score the same way, and with
    # -Inf in the query every score is -Inf.
    rng = np.random.default_rng(lq + d)
    pool = ref.Kv4Pool(sum(-(-n // 32) for n in lens), 32, heads, d)
    table, first = np.full((len(lens), max(-(-n // 32) for n in lens)), -1, np.int64), 0
    for b, n in enumerate(lens):
        need = -(-n // 32)
        table[b, :need] = np.arange(first, first + need)
        k = ref.bf16(100 + rng.standard_normal((n, heads, d)).astype(np.float32))
        pool.append(k, rows(rng, (n, heads, d)), first * 32 + np.arange(n))
        first += need
    assert (pool.zero[0][pool.scale[0] > 0] > 128 * pool.scale[0][pool.scale[0] > 0]).all()
    data = torch.from_numpy(pool.pack()).cuda()
    q = ref.bf16(0.1 * rng.standard_normal((len(lens), lq, hq, d))).astype(np.float64)
    mask = trees(rng, len(lens), lq)
    mask[2, 1] = 0                                            # sees the context, where there is one
    bad = np.zeros((len(lens), lq, hq), bool)
    for b, i, h in [(0, 0, 0), (0, lq - 1, hq - 1), (1, 2, 1), (2, 1, 0), (2, 1, 1)]:
        bad[b, i, h] = True
    hit = q.copy()
    hit[..., d // 2 + 3] = np.where(bad, -np.inf, hit[..., d // 2 + 3])
    scale = float(np.float32(1 / np.sqrt(d)))

    def run(queries, tree):
        T, L = torch.from_numpy(table.astype(np.int32)).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
        Q = torch.from_numpy(queries.astype(np.float32)).to(torch.bfloat16).cuda()
        O = torch.full_like(Q, -3.0)
        ws = torch.zeros(dg.dg_attention_kv4_workspace_bytes(len(lens), lq, hq, heads, d), dtype=torch.uint8, device="cuda")
        cache = dg.dg_kv4_cache(data, pool.pages, 32, heads, d)
        if tree:
            dg.attention_kv4_tree(cache, len(lens), lq, hq, scale, Q, hq * d, lq * hq * d, T, table.shape[1], L, None,
                                  torch.from_numpy(mask.view(np.int64)).cuda(), O, hq * d, lq * hq * d, ws, ws.numel())
        else:
            dg.attention_kv4(cache, len(lens), lq, hq, scale, Q, hq * d, lq * hq * d, T, table.shape[1], L, O, hq * d, lq * hq * d, ws, ws.numel())
        sync(torch)
        return O.float().cpu().numpy()
    for tree in (True, False):
        good, got = run(q, tree), run(hit, tree)
        sees = bad.copy()
        if tree and lens[2] == lq:                            # no context and an empty mask: no key
            sees[2, 1] = False
            assert not got[2, 1, :2].any()
        assert np.isnan(got[sees]).all(), tree
        assert np.array_equal(got[~bad], good[~bad])
