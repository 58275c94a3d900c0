"""attention_kv4 and the cache where a call takes another way than small ordinary ones do."""
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


def random_cache(torch, lens, page, heads, d, seed):
    """A cache of random codes and parameters, and the sequences' pages in random order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 1
    data = torch.randint(0, 256, (pages, heads, dg.dg_kv4_block_bytes(page, d)), generator=g, device="cuda", dtype=torch.uint8)
    params = data.view(pages, heads, page // 16, -1)[..., 16 * d:].view(torch.bfloat16)
    params.copy_(torch.randn(params.shape, generator=g, device="cuda"))
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return data, table, g


def attend(torch, data, table, lens, q, heads, page, scale):
    batch, lq, hq, d = q.shape
    cache = dg.dg_kv4_cache(data, data.shape[0], page, heads, d)
    ws = torch.zeros(dg.dg_attention_kv4_workspace_bytes(batch, lq, hq, heads, d), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, -3.0)
    dg.attention_kv4(cache, batch, lq, hq, scale, q, hq * d, lq * hq * d, table, table.shape[1],
                     torch.tensor(lens, dtype=torch.int32, device="cuda"), out, hq * d, lq * hq * d, ws, ws.numel())
    torch.cuda.synchronize()
    assert dg.dg_device_status() == dg.DG_OK
    return out


# Items that are whole in a warp, cut between warps, cut between CTAs, joined in two steps.
@pytest.mark.parametrize("lens,lq,hq,heads,d", [
    ([20, 33, 5], 1, 8, 2, 128), ([300, 700], 1, 16, 2, 64), ([3000], 1, 8, 1, 128), ([8192], 1, 32, 8, 128), ([20000], 1, 16, 1, 64),
    ([6000, 40], 3, 8, 1, 128), ([1500, 9, 0, 2500], 5, 12, 2, 64)])
def test_a_query_that_is_not_finite_gives_nan_and_only_there(torch, lens, lq, hq, heads, d):
    data, table, g = random_cache(torch, lens, 64, heads, d, sum(lens))
    q = torch.randn((len(lens), lq, hq, d), generator=g, device="cuda").to(torch.bfloat16)
    plain = attend(torch, data, table, lens, q, heads, 64, 0.1)
    assert bool(plain.isfinite().all())
    bad = q.clone()
    where = torch.zeros((len(lens), lq, hq), dtype=torch.bool, device="cuda")
    for b in range(len(lens)):
        for i in range(lq):
            for h, value in ((b % hq, float("nan")), ((b + 3 * i + 5) % hq, float("inf"))):
                bad[b, i, h, (7 * i + h) % d] = value
                where[b, i, h] = lens[b] - lq + i >= 0            # a row without a key stays 0
    out = attend(torch, data, table, lens, bad, heads, 64, 0.1)
    assert bool(out[where].isnan().all())
    assert torch.equal(out[~where], plain[~where])


# Every unit of keys is visible in these outputs (tests/test_kv4_units.py): a part that a join loses,
# doubles or takes from an earlier call changes them.  Items of one warp, of one CTA, of neighbouring
# CTAs, and those joined in two steps; one workspace for calls whose units are dealt differently.
@pytest.mark.parametrize("lens,lq,hq,heads,d", [
    ([6000], 1, 16, 1, 128), ([9000, 0, 4000], 2, 16, 1, 64), ([20000], 1, 8, 1, 64), ([20000], 1, 8, 1, 128), ([33000], 1, 32, 1, 128),
    ([3000, 2600, 2700], 1, 32, 1, 128), ([40, 4100, 4200, 70], 1, 16, 1, 128), ([16768, 16768], 4, 8, 1, 64), ([8192], 1, 32, 8, 128),
    ([0, 5000, 1, 17], 1, 8, 2, 128), ([1024] * 20, 1, 32, 8, 128), ([1024] * 5, 1, 128, 8, 64), ([700, 33, 1500, 64, 3100] * 3, 1, 16, 4, 64),
    ([2000] * 40, 1, 8, 8, 128), ([512] * 16, 3, 32, 4, 64)])
def test_every_unit_of_keys_counts_once(torch, lens, lq, hq, heads, d):
    batch, page = len(lens), 48
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 1
    g = torch.Generator(device="cuda").manual_seed(sum(lens) + hq)
    data = torch.full((pages, heads, dg.dg_kv4_block_bytes(page, d)), 255, dtype=torch.uint8, device="cuda")
    cache = dg.dg_kv4_cache(data, pages, page, heads, d)
    order = torch.randperm(pages, generator=g, device="cuda")
    table = torch.full((batch, max(need)), -1, dtype=torch.int32, device="cuda")
    q = torch.zeros((batch, lq, hq * d), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    ws = torch.zeros(dg.dg_attention_kv4_workspace_bytes(batch, lq, hq, heads, d), dtype=torch.uint8, device="cuda")
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    units = sum(-(-n // 32) for n in lens) * heads * -(-(lq * hq // heads) // 8)
    for call in range(3):
        want, bound = np.zeros((batch, lq, hq, d)), np.zeros((batch, lq, hq, d))
        at = 0
        for b, n in enumerate(lens):
            mine = order[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = mine.to(torch.int32)
            if n == 0:
                continue
            rows = [ref.unit_rows(n, d, 1 + (3 * b + h + 5 * call) % 11) for h in range(heads)]
            v = torch.from_numpy(np.stack(rows, 1)).cuda().to(torch.bfloat16)
            k = torch.randn((n, heads, d), generator=g, device="cuda").to(torch.bfloat16)
            token = torch.arange(n, device="cuda")
            dg.kv4_append(cache, n, k, heads * d, v, heads * d, mine[token // page] * page + token % page)
            for h in range(heads):
                for i in range(lq):
                    heads_of = slice(h * (hq // heads), (h + 1) * (hq // heads))
                    want[b, i, heads_of], bound[b, i, heads_of] = ref.unit_mean(rows[h], max(n - lq + i + 1, 0), units)
        out.fill_(-3.0)
        dg.attention_kv4(cache, batch, lq, hq, 0.5, q, hq * d, lq * hq * d, table, table.shape[1], L, out, hq * d, lq * hq * d, ws,
                         ws.numel())
        torch.cuda.synchronize()
        assert dg.dg_device_status() == dg.DG_OK
        got = out.float().cpu().numpy().astype(np.float64).reshape(want.shape)
        off = np.abs(got - want) > bound
        assert not off.any(), f"call {call}: {off.sum()} of {off.size}, first {np.argwhere(off)[0]}"


# A prompt's rows: 4 and 8 heads in flight, runs of heads cut over warps, more tokens than the grid
# has warps; 16-byte, 8-byte and single accesses.
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens,heads,page,pad,offset", [
    (5000, 8, 64, 0, 0), (3500, 8, 16, 8, 0), (9800, 4, 48, 4, 0), (5003, 12, 32, 1, 0), (5003, 16, 64, 0, 1), (5003, 5, 16, 3, 0),
    (20011, 8, 128, 0, 4), (3300, 8, 16, 0, 2), (2432, 16, 64, 8, 0)])
def test_a_prompt_written_and_read_back(torch, tokens, heads, page, pad, offset, d):
    rng = np.random.default_rng(tokens + d)
    width, pages = heads * d, -(-tokens // page) + 3
    ld = width + pad
    slots = rng.permutation(pages * page)[:tokens]
    skipped = rng.choice(tokens, 40, replace=False)
    pool = ref.Kv4Pool(pages, page, heads, d)
    rows, given = [], slots.copy()
    given[skipped] = -1 - skipped                             # negative: passed over, read as zeros
    kept = given >= 0
    for which in range(2):
        x = rng.standard_normal((tokens, heads, d)).astype(np.float32) * np.exp(rng.normal(0, 1, (tokens, heads, 1))).astype(np.float32)
        x[rng.integers(0, tokens, 9), rng.integers(0, heads, 9)] = 1.5
        x = ref.bf16(x)
        buf = torch.full((tokens * ld + offset,), float("nan"), dtype=torch.bfloat16, device="cuda")
        buf[offset:].view(tokens, ld)[:, :width] = torch.from_numpy(x.reshape(tokens, width)).cuda()
        rows.append(buf[offset:].view(tokens, ld))
        pool.codes[which, slots[kept]], pool.scale[which, slots[kept]], pool.zero[which, slots[kept]] = \
            (a[kept] for a in ref.kv4_quantise(x))
    data = torch.zeros((pages, heads, dg.dg_kv4_block_bytes(page, d)), dtype=torch.uint8, device="cuda")
    cache = dg.dg_kv4_cache(data, pages, page, heads, d)
    S = torch.from_numpy(given).cuda()
    dg.kv4_append(cache, tokens, rows[0], ld, rows[1], ld, S)
    torch.cuda.synchronize()
    assert dg.dg_device_status() == dg.DG_OK
    assert np.array_equal(data.cpu().numpy(), pool.pack_all())
    bufs = [torch.full((tokens * ld + offset,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    outs = [b[offset:].view(tokens, ld) for b in bufs]
    dg.kv4_gather(cache, tokens, S, outs[0], ld, outs[1], ld)
    torch.cuda.synchronize()
    assert dg.dg_device_status() == dg.DG_OK
    for which, out in enumerate(outs):
        want = ref.bf16(pool.rows(which, slots).astype(np.float32)).reshape(tokens, width)
        want[~kept] = 0
        assert np.array_equal(out[:, :width].float().cpu().numpy(), want)
        assert bool((out[:, width:] == 7.0).all()) and bool((bufs[which][:offset] == 7.0).all())


# More sequences than the first four of every lane: their places are searched for.
@pytest.mark.parametrize("batch,lq,hq,heads,d,lone", [(129, 1, 4, 2, 64, 0), (161, 2, 12, 1, 64, 700), (300, 1, 8, 2, 128, 0), (700, 1, 2, 2, 64, 1500),
                                                      (1000, 1, 1, 1, 64, 0)])
def test_batches_of_many_sequences(torch, batch, lq, hq, heads, d, lone):
    rng = np.random.default_rng(batch)
    lens = [int(n) for n in rng.integers(0, 90, batch) * (rng.random(batch) < 0.8)]
    if lone:
        lens[batch * 2 // 3] = lone                           # one far longer, past every lane's first four
    lens[-1], page = 40, 16
    need = [-(-n // page) for n in lens]
    order = rng.permutation(sum(need) + 2)
    pool = ref.Kv4Pool(len(order), page, heads, d)
    table = np.full((batch, max(need)), -9, np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    slots = np.concatenate([table[b, np.arange(n) // page] * page + np.arange(n) % page for b, n in enumerate(lens)])
    for which in range(2):
        x = ref.bf16(rng.standard_normal((len(slots), heads, d)).astype(np.float32))
        pool.codes[which, slots], pool.scale[which, slots], pool.zero[which, slots] = ref.kv4_quantise(x)
    q = ref.bf16(rng.standard_normal((batch, lq, hq, d))).astype(np.float64)
    scale = float(np.float32(1 / np.sqrt(d)))
    out = attend(torch, torch.from_numpy(pool.pack_all()).cuda(), torch.from_numpy(table.astype(np.int32)).cuda(), lens,
                 torch.from_numpy(q).cuda().to(torch.bfloat16), heads, page, scale)
    want, bound = ref.kv4_attention(pool, q, table, lens, scale)
    off = ~(np.abs(out.float().cpu().numpy() - want) <= bound)
    assert not off.any(), f"{off.sum()} of {off.size}, first {np.argwhere(off)[0]}"


# A piece of a prompt: many blocks of query rows, each with its own last key, some before the first.
@pytest.mark.parametrize("lens,lq,hq,heads,d", [([500, 150, 0], 200, 8, 2, 64), ([1300], 257, 4, 1, 128), ([90, 64], 90, 6, 3, 128)])
def test_queries_of_a_prompt(torch, lens, lq, hq, heads, d):
    rng = np.random.default_rng(lq)
    page = 32
    need = [-(-n // page) for n in lens]
    order = rng.permutation(sum(need) + 1)
    pool = ref.Kv4Pool(len(order), page, heads, d)
    table = np.full((len(lens), max(need)), -1, np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    slots = np.concatenate([table[b, np.arange(n) // page] * page + np.arange(n) % page for b, n in enumerate(lens)])
    for which in range(2):
        x = ref.bf16(rng.standard_normal((len(slots), heads, d)).astype(np.float32))
        pool.codes[which, slots], pool.scale[which, slots], pool.zero[which, slots] = ref.kv4_quantise(x)
    q = ref.bf16(rng.standard_normal((len(lens), lq, hq, d))).astype(np.float64)
    scale = float(np.float32(1 / np.sqrt(d)))
    out = attend(torch, torch.from_numpy(pool.pack_all()).cuda(), torch.from_numpy(table.astype(np.int32)).cuda(), lens,
                 torch.from_numpy(q).cuda().to(torch.bfloat16), heads, page, scale)
    want, bound = ref.kv4_attention(pool, q, table, lens, scale)
    off = ~(np.abs(out.float().cpu().numpy() - want) <= bound)
    assert not off.any(), f"{off.sum()} of {off.size}, first {np.argwhere(off)[0]}"
