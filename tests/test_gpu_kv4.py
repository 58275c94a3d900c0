"""The 4-bit key-value cache (kv4_append, kv4_gather) bit for bit against its definition, and
attention_kv4 against the float64 oracle within the bound derived there."""
import numpy as np
import pytest

import dense_gemm_sm_gb300 as dg
from oracle import serving as ref

from .helpers import torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    dg.load()
    return t


def sync(torch, want=dg.DG_OK):
    torch.cuda.synchronize()
    assert dg.dg_device_status() == want


def rows(rng, shape):
    x = rng.standard_normal(shape).astype(np.float32) * np.exp(rng.normal(0, 1, shape[:-1] + (1,))).astype(np.float32)
    return ref.bf16(x)


def dev(torch, x):
    return torch.from_numpy(np.ascontiguousarray(ref.bf16_bits(x)).view(np.int16)).view(torch.bfloat16).cuda()


def host(t):
    return t.detach().float().cpu().numpy()


# ------------------------------------------------------------------ rows
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page_size,pages,heads,tokens,pad", [(16, 5, 1, 70, 0), (48, 3, 3, 101, 8), (64, 2, 8, 128, 1),
                                                             (128, 2, 2, 1, 0), (16, 40, 5, 333, 4)])
def test_append_and_gather(torch, d, page_size, pages, heads, tokens, pad):
    rng = np.random.default_rng(tokens + d)
    k, v = rows(rng, (tokens, heads, d)), rows(rng, (tokens, heads, d))
    k[0, 0] = 2.5                                             # a constant row
    v[0, 0, :] = 0
    v[0, 0, d - 1] = -1e-38
    k[tokens // 2, heads - 1, 3] = 1e30                       # a step so large that the rest falls on one code
    slots = rng.permutation(pages * page_size)[:tokens]
    ld = heads * d + pad
    K, V = (torch.full((tokens, ld), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    K[:, :heads * d], V[:, :heads * d] = dev(torch, k.reshape(tokens, -1)), dev(torch, v.reshape(tokens, -1))
    pool = ref.Kv4Pool(pages, page_size, heads, d)
    pool.append(k, v, slots)
    data = torch.zeros((pages, heads, dg.dg_kv4_block_bytes(page_size, d)), dtype=torch.uint8, device="cuda")
    cache = dg.dg_kv4_cache(data, pages, page_size, heads, d)
    S = torch.from_numpy(slots).cuda()
    dg.kv4_append(cache, tokens, K, ld, V, ld, S)
    sync(torch)
    assert np.array_equal(data.cpu().numpy(), pool.pack())
    Ko, Vo = (torch.full((tokens, ld), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dg.kv4_gather(cache, tokens, S, Ko, ld, Vo, ld)
    sync(torch)
    for which, out in ((0, Ko), (1, Vo)):
        got = host(out)
        want = ref.bf16(pool.rows(which, slots).astype(np.float32)).reshape(tokens, -1)
        assert np.array_equal(got[:, :heads * d], want) and np.isnan(got[:, heads * d:]).all()


def test_overwriting_a_slot_leaves_its_neighbours(torch):
    rng = np.random.default_rng(9)
    k, v = rows(rng, (32, 2, 128)), rows(rng, (32, 2, 128))
    pool = ref.Kv4Pool(1, 32, 2, 128)
    pool.append(k, v, np.arange(32))
    data = torch.from_numpy(pool.pack()).cuda()
    cache = dg.dg_kv4_cache(data, 1, 32, 2, 128)
    for at in (0, 1, 7, 8, 15, 16, 31):
        x, y = rows(rng, (1, 2, 128)), rows(rng, (1, 2, 128))
        pool.append(x, y, [at])
        dg.kv4_append(cache, 1, dev(torch, x.reshape(1, -1)), 256, dev(torch, y.reshape(1, -1)), 256,
                      torch.tensor([at], device="cuda"))
        sync(torch)
        assert np.array_equal(data.cpu().numpy(), pool.pack()), at


def test_slots_outside_the_cache(torch):
    rng = np.random.default_rng(10)
    k = rows(rng, (4, 1, 64))
    data = torch.zeros((2, 1, 16 * 72), dtype=torch.uint8, device="cuda")
    cache = dg.dg_kv4_cache(data, 2, 16, 1, 64)
    K = dev(torch, k.reshape(4, -1))
    S = torch.tensor([-1, 32, 2 ** 40, -2 ** 62], device="cuda")
    dg.kv4_append(cache, 4, K, 64, K, 64, S)
    sync(torch, dg.DG_ERR_BAD_INDEX)
    sync(torch)                                               # read once, cleared
    assert not data.any()
    dg.kv4_append(cache, 1, K, 64, K, 64, S)                  # a negative slot is no error
    sync(torch)
    out = torch.full((4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    dg.kv4_gather(cache, 4, S, out, 64, out.clone(), 64)
    sync(torch, dg.DG_ERR_BAD_INDEX)
    assert not out.any()


# ------------------------------------------------------------------ attention
def build(torch, rng, lens, page_size, heads, d, extra=2, spare_cols=0):
    """A pool with the sequences' tokens, every unused byte 0xFF (NaN scales), and its table."""
    need = [-(-n // page_size) for n in lens]
    pages = sum(need) + extra
    width = max(need + [1]) + spare_cols
    order = rng.permutation(pages)
    pool = ref.Kv4Pool(pages, page_size, heads, d)
    pool.codes[:] = 15
    pool.scale[:] = pool.zero[:] = np.nan
    table = np.full((len(lens), width), -7, np.int64)
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        if n:
            slots = table[b, np.arange(n) // page_size] * page_size + np.arange(n) % page_size
            pool.append(rows(rng, (n, heads, d)), rows(rng, (n, heads, d)), slots)
    nan = np.isnan(pool.scale)
    pool.scale[nan] = pool.zero[nan] = 0.0
    packed = pool.pack()
    rec = packed.reshape(pages, heads, page_size // 16, -1)
    prm = rec[..., 16 * d:].reshape(pages, heads, page_size // 16, 2, 16, 4)
    stale = nan.reshape(2, pages, page_size // 16, 16, heads)
    for w in range(2):
        prm[:, :, :, w][stale[w].transpose(0, 3, 1, 2)] = 255
    data = torch.from_numpy(packed).cuda()
    return pool, data, table


def attend(torch, pool, data, table, lens, q, scale, pad=0, batch_pad=0, ws=None, heads_kv=None):
    batch, lq, hq, d = q.shape
    ld = hq * d + pad
    stride = lq * ld + batch_pad
    Q = torch.full((batch * stride,), float("nan"), dtype=torch.bfloat16, device="cuda")
    O = torch.full((batch * stride,), -3.0, dtype=torch.bfloat16, device="cuda")
    qv = Q.as_strided((batch, lq, hq * d), (stride, ld, 1))
    qv.copy_(dev(torch, q.astype(np.float32).reshape(batch, lq, -1)))
    cache = dg.dg_kv4_cache(data, pool.pages, pool.page_size, pool.heads, d)
    if ws is None:
        ws = torch.zeros(dg.dg_attention_kv4_workspace_bytes(batch, lq, hq, pool.heads, d), dtype=torch.uint8, device="cuda")
    T = torch.from_numpy(table.astype(np.int32)).cuda()
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    dg.attention_kv4(cache, batch, lq, hq, scale, Q, ld, stride, T, table.shape[1], L, O, ld, stride, ws, ws.numel())
    ov = O.as_strided((batch, lq, hq * d), (stride, ld, 1))
    got = ov.float().cpu().numpy().reshape(batch, lq, hq, d).astype(np.float64)
    ov.fill_(-3.0)
    assert bool((O == -3.0).all())                            # nothing between the rows is written
    return got


def check(torch, lens, lq, hq, heads, d, page_size, pad=0, batch_pad=0, std=1.0, seed=0, ws=None):
    rng = np.random.default_rng(seed + sum(lens) + d + hq)
    pool, data, table = build(torch, rng, lens, page_size, heads, d, spare_cols=seed % 3)
    q = ref.bf16(rng.standard_normal((len(lens), lq, hq, d)) * std).astype(np.float64)
    scale = float(np.float32(1 / np.sqrt(d)))
    got = attend(torch, pool, data, table, lens, q, scale, pad, batch_pad, ws)
    sync(torch)
    want, bound = ref.kv4_attention(pool, q, table, lens, scale)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, first {np.argwhere(bad)[0]}, worst {np.nanmax(np.abs(got - want) / (bound + 1e-30)):.3g}"


LENGTHS = [1, 2, 15, 16, 17, 63, 64, 65, 100, 127, 128, 129, 511, 513, 1025]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", LENGTHS)
def test_attention_lengths(torch, n, d):
    check(torch, [n], 1, 4, 1, d, 16, seed=n)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page_size", [16, 32, 48, 64, 80, 128, 256])
def test_attention_pages(torch, page_size, d):
    check(torch, [300, 0, 77], 1, 8, 2, d, page_size, seed=page_size)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,heads,lq", [(1, 1, 1), (2, 1, 1), (7, 1, 1), (8, 1, 1), (9, 1, 1), (16, 2, 1), (17, 1, 1), (32, 1, 1),
                                         (33, 1, 1), (12, 3, 1), (4, 4, 3), (8, 1, 5), (10, 2, 7), (3, 1, 40)])
def test_attention_heads_and_queries(torch, hq, heads, lq, d):
    check(torch, [200, 3, 65], lq, hq, heads, d, 32, seed=lq)


@pytest.mark.parametrize("lens", [[0], [0, 0, 0], [1] * 20, [0, 5000, 1, 17], list(range(0, 400, 13)), [2500, 2500]])
def test_attention_batches(torch, lens):
    check(torch, lens, 1, 8, 2, 128, 64, seed=len(lens))


@pytest.mark.parametrize("lens,lq,hq,d", [([6000], 1, 16, 128), ([9000, 0, 4000], 2, 16, 64), ([20000], 1, 8, 64),
                                          ([3000, 2600, 2700], 1, 32, 128), ([40, 4100, 4200, 70], 1, 16, 128)])
def test_attention_of_long_sequences_and_one_cache_head(torch, lens, lq, hq, d):
    # So many CTAs share a sequence that their sums are joined in two steps; twice with one workspace.
    ws = torch.zeros(dg.dg_attention_kv4_workspace_bytes(len(lens), lq, hq, 1, d), dtype=torch.uint8, device="cuda")
    for seed in (1, 2):
        check(torch, lens, lq, hq, 1, d, 64, seed=seed, ws=ws)
    assert not ws[:1024].any()


def test_attention_strides(torch):
    check(torch, [130, 40], 2, 4, 2, 128, 16, pad=72, batch_pad=16)


def test_attention_queries_before_the_first_key(torch):
    # Fewer tokens than queries: the first queries see nothing and get zeros.
    check(torch, [2, 0, 5, 1], 4, 4, 2, 128, 16, seed=4)


def test_attention_peaked_scores(torch):
    check(torch, [700], 1, 8, 1, 128, 64, std=30.0, seed=5)


def test_attention_many_sequences_one_workspace(torch):
    # Calls of different sizes share one workspace, zeroed once.
    ws = torch.zeros(dg.dg_attention_kv4_workspace_bytes(64, 4, 16, 2, 128), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(11)
    check(torch, [int(x) for x in rng.integers(0, 300, 64)], 1, 16, 2, 128, 16, seed=7, ws=ws)
    check(torch, [3000], 4, 4, 1, 64, 32, seed=8, ws=ws)
    check(torch, [int(x) for x in rng.integers(0, 900, 9)], 2, 16, 2, 128, 48, seed=9, ws=ws)


def test_attention_repeats_bit_for_bit_and_in_a_graph(torch):
    rng = np.random.default_rng(12)
    lens = [1800, 40, 333]
    pool, data, table = build(torch, rng, lens, 64, 2, 128)
    q = ref.bf16(rng.standard_normal((3, 1, 16, 128))).astype(np.float64)
    first = attend(torch, pool, data, table, lens, q, 0.09)
    for _ in range(3):
        assert np.array_equal(attend(torch, pool, data, table, lens, q, 0.09), first)
    cache = dg.dg_kv4_cache(data, pool.pages, 64, 2, 128)
    ws = torch.zeros(dg.dg_attention_kv4_workspace_bytes(3, 1, 16, 2, 128), dtype=torch.uint8, device="cuda")
    Q = dev(torch, q.astype(np.float32).reshape(3, -1))
    O = torch.zeros_like(Q)
    T, L = torch.from_numpy(table.astype(np.int32)).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.attention_kv4(cache, 3, 1, 16, 0.09, Q, 2048, 2048, T, table.shape[1], L, O, 2048, 2048, ws, ws.numel())
    for _ in range(3):
        graph.replay()
        sync(torch)
        assert np.array_equal(O.float().cpu().numpy().reshape(first.shape), first)
    L.copy_(torch.tensor([1, 40, 0], dtype=torch.int32))      # the graph follows the lengths
    graph.replay()
    sync(torch)
    want, bound = ref.kv4_attention(pool, q, table, [1, 40, 0], float(np.float32(0.09)))
    assert np.all(np.abs(O.float().cpu().numpy().reshape(first.shape) - want) <= bound)


def test_attention_bad_pages_and_lengths(torch):
    rng = np.random.default_rng(13)
    lens = [100, 100, 100]
    pool, data, table = build(torch, rng, lens, 16, 1, 64)
    table[0, 2], table[1, 3] = -1, pool.pages                 # pages outside the cache are not visible
    q = ref.bf16(rng.standard_normal((3, 1, 4, 64))).astype(np.float64)
    got = attend(torch, pool, data, table, lens, q, 0.125)
    sync(torch, dg.DG_ERR_BAD_INDEX)
    want, bound = ref.kv4_attention(pool, q, table, lens, 0.125)
    assert np.all(np.abs(got - want) <= bound)
    # Lengths outside the table are taken as its bounds.
    pool, data, table = build(torch, rng, [112, 112, 112], 16, 1, 64)
    got = attend(torch, pool, data, table, [-5, 10 ** 9, 112], q, 0.125)
    sync(torch, dg.DG_ERR_BAD_INDEX)
    want, bound = ref.kv4_attention(pool, q, table, [0, 112, 112], 0.125)
    assert np.all(np.abs(got - want) <= bound)
    got = attend(torch, pool, data, table[:, :0], [0, 0, 5], q, 0.125)
    sync(torch, dg.DG_ERR_BAD_INDEX)
    assert not got.any()


def test_attention_page_offsets_past_32_bits(torch):
    # A pool of over 4 GiB; the sequence lies at its end.
    page_size, heads, d, n = 256, 8, 128, 300
    block = dg.dg_kv4_block_bytes(page_size, d)
    pages = (1 << 32) // (block * heads) + 4
    rng = np.random.default_rng(14)
    data = torch.zeros((pages, heads, block), dtype=torch.uint8, device="cuda")
    cache = dg.dg_kv4_cache(data, pages, page_size, heads, d)
    k, v = rows(rng, (n, heads, d)), rows(rng, (n, heads, d))
    at = np.concatenate([np.arange(256) + (pages - 1) * page_size, np.arange(n - 256) + (pages - 3) * page_size])
    S = torch.from_numpy(at).cuda()
    dg.kv4_append(cache, n, dev(torch, k.reshape(n, -1)), heads * d, dev(torch, v.reshape(n, -1)), heads * d, S)
    small = ref.Kv4Pool(2, page_size, heads, d)
    small.append(k, v, np.arange(n))
    q = ref.bf16(rng.standard_normal((1, 1, 16, d))).astype(np.float64)
    small_table = np.array([[0, 1]])
    big = ref.Kv4Pool(2, page_size, heads, d)
    big.pages = pages
    got = attend(torch, big, data, np.array([[pages - 1, pages - 3]]), [n], q, 0.09)
    sync(torch)
    want, bound = ref.kv4_attention(small, q, small_table, [n], float(np.float32(0.09)))
    assert np.all(np.abs(got - want) <= bound)
    Ko, Vo = (torch.empty((n, heads * d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dg.kv4_gather(cache, n, S, Ko, heads * d, Vo, heads * d)
    sync(torch)
    assert np.array_equal(host(Vo), ref.bf16(small.rows(1, np.arange(n)).astype(np.float32)).reshape(n, -1))
