"""Bounded waits of gemm_w4_bf16 and attention_kv4_tree (tests/test_gpu_serving_faults.py says how they are
made to run out): the call reports DG_ERR_TIMEOUT and ends, and on a workspace zeroed again gives what
it gave before."""
import pytest

import dense_gemm_sm_gb300 as dg

from .helpers import torch_mod
from .test_gpu_serving_faults import expire

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    dg.load()
    return t


# More units (128 columns, 256 k) for each CTA than its ring has stages.
@pytest.mark.parametrize("m,group", [(3, 128), (20, 64), (64, 32), (100, 128)])
def test_products_that_give_up(torch, m, group):
    n, k = 40000, 2048
    g = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn((m, k), generator=g, device="cuda", dtype=torch.bfloat16)
    q = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    p = torch.randn((k // group, n, 2), generator=g, device="cuda", dtype=torch.bfloat16)
    out = torch.empty((m, n), device="cuda")
    ws = torch.zeros(dg.dg_gemm_w4_workspace_bytes(m, n, k), dtype=torch.uint8, device="cuda")

    def call():
        dg.gemm_w4_bf16(m, n, k, group, x, k, q, k // 2, p, n, out, n, dg.DG_OUT_F32, ws, ws.numel())
    expire(torch, call, out, ws)


# More units (128 keys of a cache head and block of rows) for each CTA, or (32 keys, few rows) for each
# warp, than its ring has stages.
@pytest.mark.parametrize("d,lq,hq", [(128, 16, 32), (128, 64, 32), (64, 40, 16), (128, 2, 32), (64, 3, 16)])
def test_trees_that_give_up(torch, d, lq, hq):
    batch, n, heads, page = 4, 16384, 8, 64
    g = torch.Generator(device="cuda").manual_seed(d + lq)
    pages = batch * n // page
    data = torch.randint(0, 256, (pages, heads, dg.dg_kv4_block_bytes(page, d)), generator=g, device="cuda", dtype=torch.uint8)
    params = data.view(pages, heads, page // 16, -1)[..., 16 * d:].view(torch.bfloat16)
    params.copy_(torch.randn(params.shape, generator=g, device="cuda"))
    cache = dg.dg_kv4_cache(data, pages, page, heads, d)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(batch, -1)
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    mask = torch.randint(-2 ** 62, 2 ** 62, (batch, lq), generator=g, device="cuda")
    q = torch.randn((batch, lq, hq * d), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    ws = torch.zeros(dg.dg_attention_kv4_workspace_bytes(batch, lq, hq, heads, d), dtype=torch.uint8, device="cuda")

    def call():
        dg.attention_kv4_tree(cache, batch, lq, hq, 0.02, q, hq * d, lq * hq * d, table, table.shape[1], lens, None, mask, out, hq * d,
                              lq * hq * d, ws, ws.numel())
    expire(torch, call, out, ws)
