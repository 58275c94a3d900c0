"""The serving operators on streams of their own: results on a side stream and from a graph against
the oracle, and calls of two streams at once, each with its workspace, bit for bit as alone."""
import numpy as np
import pytest

import dense_gemm_sm_gb300 as dg
from oracle import serving as ref

from .helpers import torch_mod

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def torch():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    dg.load()
    return t


def sync(torch):
    torch.cuda.synchronize()
    assert dg.dg_device_status() == dg.DG_OK


def test_norm_on_a_side_stream_and_from_a_graph(torch):
    rows, cols = 64, 4096
    rng = np.random.default_rng(1)
    first, second = (ref.bf16(rng.standard_normal((rows, cols))) for _ in range(2))
    gain = ref.bf16(1 + 0.1 * rng.standard_normal(cols))
    X = torch.from_numpy(first).cuda().to(torch.bfloat16)
    next_x = torch.from_numpy(second).cuda().to(torch.bfloat16)
    G = torch.from_numpy(gain).cuda().to(torch.bfloat16)
    Y, Z = (torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def norm(out, stream=None):
        dg.rmsnorm_residual_bf16(rows, cols, X, cols, dg.DG_OUT_BF16, None, 0, dg.DG_OUT_BF16, None, 0, G, EPS, out, cols,
                                 stream=stream)

    def right(out, x):
        _, y = ref.rmsnorm(x, None, gain, EPS)
        rel = (cols / 32 + 40) * 2.0 ** -25 + 6 * ref.F32
        return np.all(np.abs(out.float().cpu().numpy() - y) <= np.abs(y) * (ref.BF16 + 2 * rel) + 1e-38)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm(Y, side)                                             # a stream named in the call
    with torch.cuda.stream(side):
        norm(Z)                                               # the current one
    torch.cuda.current_stream().wait_stream(side)
    X.copy_(next_x)
    sync(torch)
    assert right(Y, first) and right(Z, first) and not right(Y, second)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm(Z)
    for x in (first, second):
        X.copy_(torch.from_numpy(x))
        Z.zero_()
        graph.replay()
        sync(torch)
        assert right(Z, x)


class Attention:
    def __init__(self, torch, seed, lens, hq, heads, d, page=32):
        g = torch.Generator(device="cuda").manual_seed(seed)
        need = [-(-n // page) for n in lens]
        pages, batch = sum(need), len(lens)
        self.data = torch.randint(0, 256, (pages, heads, dg.dg_kv4_block_bytes(page, d)), generator=g, device="cuda", dtype=torch.uint8)
        params = self.data.view(pages, heads, page // 16, -1)[..., 16 * d:].view(torch.bfloat16)
        params.copy_(torch.randn(params.shape, generator=g, device="cuda"))
        self.cache = dg.dg_kv4_cache(self.data, pages, page, heads, d)
        self.table = torch.full((batch, max(need)), -1, dtype=torch.int32, device="cuda")
        order, at = torch.randperm(pages, generator=g, device="cuda").to(torch.int32), 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.q = torch.randn((batch, hq * d), generator=g, device="cuda").to(torch.bfloat16)
        self.out = torch.empty_like(self.q)
        self.ws = torch.zeros(dg.dg_attention_kv4_workspace_bytes(batch, 1, hq, heads, d), dtype=torch.uint8, device="cuda")
        self.hq, self.w = hq, hq * d

    def __call__(self):
        dg.attention_kv4(self.cache, len(self.lens), 1, self.hq, 0.05, self.q, self.w, self.w, self.table, self.table.shape[1],
                         self.lens, self.out, self.w, self.w, self.ws, self.ws.numel())


class Experts:
    def __init__(self, torch, seed, T, K, I, E, top):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std=1.0):
            return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(std)
        self.sizes = T, K, I, E, top
        self.x, self.logits = normal(T, K), torch.randn((T, E), generator=g, device="cuda")
        self.wg, self.wu, self.wd = normal(E, K, I, std=K ** -0.5), normal(E, K, I, std=K ** -0.5), normal(E, I, K, std=I ** -0.5)
        self.out = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
        self.ws = torch.zeros(dg.dg_moe_workspace_bytes(T, K, I, E, top), dtype=torch.uint8, device="cuda")

    def __call__(self):
        T, K, I, E, top = self.sizes
        dg.moe_bf16(T, K, I, E, top, True, self.x, K, self.logits, E, self.wg, I, K * I, self.wu, I, K * I, self.wd, K, I * K,
                    self.out, K, self.ws, self.ws.numel())


@pytest.mark.parametrize("pair", ["attention and experts", "two attentions", "two experts"])
def test_calls_on_two_streams_at_once(torch, pair):
    make = {"attention and experts": lambda: [Attention(torch, 1, [6000, 40, 900], 32, 8, 128), Experts(torch, 2, 20, 1024, 520, 16, 4)],
            "two attentions": lambda: [Attention(torch, 3, [20000], 8, 1, 64), Attention(torch, 4, [700] * 30, 16, 2, 128)],
            "two experts": lambda: [Experts(torch, 5, 1, 2048, 1024, 8, 2), Experts(torch, 6, 48, 512, 264, 32, 8)]}[pair]
    calls = make()
    alone = []
    for c in calls:
        c()
        sync(torch)
        alone.append(c.out.clone())
        c.out.fill_(-3.0)
    streams = [torch.cuda.Stream() for _ in calls]
    kept = [[] for _ in calls]
    torch.cuda.synchronize()
    for _ in range(25):
        for c, s, k in zip(calls, streams, kept):
            with torch.cuda.stream(s):
                c()
                k.append(c.out.clone())
                c.out.fill_(-3.0)
    sync(torch)
    for a, k in zip(alone, kept):
        assert bool(a.isfinite().all())
        for i, out in enumerate(k):
            assert torch.equal(out, a), i
