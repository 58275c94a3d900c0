"""Bounded waits of the serving operators: with dg_set_fault_injection(1) the stages of their rings
are not released, so the waits for a free stage, and then those for a full one, run out.  Every
CTA that gives up waits for its own copies, returns, and the call reports DG_ERR_TIMEOUT; on a
workspace zeroed again the same call then gives what it gave before.
"""
import pytest

import dense_gemm_sm_gb300 as dg

from .helpers import torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    dg.load()
    return t


def expire(torch, call, out, ws):
    """`call` with waits that run out between two calls without; they agree bit for bit."""
    call()
    torch.cuda.synchronize()
    assert dg.dg_device_status() == dg.DG_OK
    first = out.clone()
    dg.dg_set_fault_injection(1)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        dg.dg_set_fault_injection(0)
    assert dg.dg_device_status() == dg.DG_ERR_TIMEOUT
    assert dg.dg_device_status() == dg.DG_OK  # read and cleared
    ws.zero_()
    out.fill_(-3.0)
    call()
    torch.cuda.synchronize()
    assert dg.dg_device_status() == dg.DG_OK
    assert torch.equal(out, first) and bool(first.isfinite().all())


# More units (32 keys of a cache head) for each warp than its ring has stages.
@pytest.mark.parametrize("d,hq", [(128, 32), (128, 128), (128, 256), (64, 32), (64, 128), (64, 256)])
def test_attention_that_gives_up(torch, d, hq):
    batch, n, heads, page = 4, 16384, 8, 64
    g = torch.Generator(device="cuda").manual_seed(d + hq)
    pages = batch * n // page
    block = dg.dg_kv4_block_bytes(page, d)
    data = torch.randint(0, 256, (pages, heads, block), generator=g, device="cuda", dtype=torch.uint8)
    params = data.view(pages, heads, page // 16, -1)[..., 16 * d:].view(torch.bfloat16)
    params.copy_(torch.randn(params.shape, generator=g, device="cuda"))
    cache = dg.dg_kv4_cache(data, pages, page, heads, d)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(batch, -1)
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    q = torch.randn((batch, hq * d), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    ws = torch.zeros(dg.dg_attention_kv4_workspace_bytes(batch, 1, hq, heads, d), dtype=torch.uint8, device="cuda")

    def call():
        dg.attention_kv4(cache, batch, 1, hq, 0.02, q, hq * d, hq * d, table, table.shape[1], lens, out, hq * d, hq * d, ws,
                         ws.numel())
    expire(torch, call, out, ws)


# More units (64 rows of a 128-column tile) for each CTA than its rings have stages, in both kernels.
@pytest.mark.parametrize("T", [1, 20, 64])
def test_experts_that_give_up(torch, T):
    K, I, E, top = 2048, 4096, 4, 2
    g = torch.Generator(device="cuda").manual_seed(T)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(std)
    x, logits = normal(T, K), torch.randn((T, E), generator=g, device="cuda")
    wg, wu, wd = normal(E, K, I, std=K ** -0.5), normal(E, K, I, std=K ** -0.5), normal(E, I, K, std=I ** -0.5)
    out = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(dg.dg_moe_workspace_bytes(T, K, I, E, top), dtype=torch.uint8, device="cuda")

    def call():
        dg.moe_bf16(T, K, I, E, top, True, x, K, logits, E, wg, I, K * I, wu, I, K * I, wd, K, I * K, out, K, ws, ws.numel())
    expire(torch, call, out, ws)
