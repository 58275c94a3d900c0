"""moe_bf16 against the float64 oracle, within the bound derived there."""
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


def dev(torch, x):
    return torch.from_numpy(np.ascontiguousarray(ref.bf16_bits(x)).view(np.int16)).view(torch.bfloat16).cuda()


def padded(torch, x, ld, gap=0):
    """[.., rows, cols] in a buffer with row stride ld and `gap` elements between matrices, NaN between."""
    x = x if x.ndim == 3 else x[None]
    e, r, c = x.shape
    stride = r * ld + gap
    buf = torch.full((e * stride,), float("nan"), dtype=torch.bfloat16, device="cuda")
    buf.as_strided((e, r, c), (stride, ld, 1)).copy_(dev(torch, x))
    return buf, stride


def make(rng, T, K, I, E):
    x = ref.bf16(rng.standard_normal((T, K)))
    wg, wu = (ref.bf16(rng.standard_normal((E, K, I)) / np.sqrt(K)) for _ in range(2))
    wd = ref.bf16(rng.standard_normal((E, I, K)) / np.sqrt(I))
    return x, wg, wu, wd


def up8(n):
    return (n + 7) // 8 * 8


def call(torch, x, logits, wg, wu, wd, top, renorm, pad=0, gap=0, ws=None):
    T, K = x.shape
    E, _, I = wg.shape
    ldx, ldi, ldk = up8(K) + pad, up8(I) + pad, up8(K) + pad
    X, _ = padded(torch, x, ldx)
    Wg, sg = padded(torch, wg, ldi, gap)
    Wu, su = padded(torch, wu, ldi + pad, gap)
    Wd, sd = padded(torch, wd, ldk, gap)
    ldl, ldy = E + pad // 8, K + pad // 8
    L = torch.full((T, ldl), float("inf"), device="cuda")
    L[:, :E] = torch.from_numpy(np.asarray(logits, dtype=np.float32))
    Y = torch.full((T, ldy), -3.0, dtype=torch.bfloat16, device="cuda")
    if ws is None:
        ws = torch.zeros(dg.dg_moe_workspace_bytes(T, K, I, E, top), dtype=torch.uint8, device="cuda")
    dg.moe_bf16(T, K, I, E, top, renorm, X, ldx, L, ldl, Wg, ldi, sg, Wu, ldi + pad, su, Wd, ldk, sd, Y, ldy, ws, ws.numel())
    sync(torch)
    assert bool((Y[:, K:] == -3.0).all())
    return Y[:, :K].float().cpu().numpy().astype(np.float64)


def check(torch, T, K, I, E, top, renorm=True, seed=0, logits=None, **kw):
    rng = np.random.default_rng(seed + T + K + I + E)
    x, wg, wu, wd = make(rng, T, K, I, E)
    if logits is None:
        logits = rng.standard_normal((T, E)).astype(np.float32) * 1.5
    got = call(torch, x, logits, wg, wu, wd, top, renorm, **kw)
    want, bound = ref.moe(x, logits, wg, wu, wd, top, renorm)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, first {np.argwhere(bad)[0]}, worst {np.nanmax(np.abs(got - want) / (bound + 1e-30)):.3g}"


@pytest.mark.parametrize("T", [1, 2, 7, 8, 15, 16, 17, 31, 33, 48, 63, 64])
def test_tokens(torch, T):
    check(torch, T, 256, 128, 8, 2)


@pytest.mark.parametrize("K,I", [(64, 64), (8, 8), (1, 1), (63, 65), (64, 1), (1, 64), (130, 72), (200, 1000), (1000, 200),
                                 (777, 333), (2048, 128), (128, 2048)])
@pytest.mark.parametrize("T", [1, 19])
def test_sizes(torch, K, I, T):
    check(torch, T, K, I, 5, 3)


# Rows off 128-byte lines: CTAs in groups on neighbouring column tiles, the last group's tiles fewer.
@pytest.mark.parametrize("K,I", [(1288, 1160), (1160, 2056), (2600, 520), (520, 2600), (264, 1032)])
@pytest.mark.parametrize("T", [1, 24, 64])
def test_rows_off_lines(torch, K, I, T):
    check(torch, T, K, I, 6, 2)


@pytest.mark.parametrize("E,top", [(1, 1), (2, 1), (2, 2), (8, 8), (16, 16), (33, 4), (64, 8), (128, 1), (512, 3)])
@pytest.mark.parametrize("renorm", [False, True])
def test_experts(torch, E, top, renorm):
    check(torch, 5, 72, 40, E, top, renorm)


@pytest.mark.parametrize("T", [3, 40])
def test_strides(torch, T):
    check(torch, T, 264, 136, 6, 2, pad=16, gap=64)


def test_one_expert_takes_every_token(torch):
    logits = np.zeros((64, 8), np.float32)
    logits[:, 5] = 9.0
    check(torch, 64, 320, 192, 8, 1, logits=logits)


def test_ties_go_to_the_lowest_expert(torch):
    logits = np.zeros((9, 12), np.float32)
    logits[3, 7] = logits[3, 9] = 1.0
    check(torch, 9, 64, 64, 12, 3, logits=logits)


def test_experts_switched_off(torch):
    # Experts at -inf and NaN are never read (their weights are NaN), one row has no expert at all.
    rng = np.random.default_rng(5)
    x, wg, wu, wd = make(rng, 4, 96, 80, 6)
    logits = rng.standard_normal((4, 6)).astype(np.float32)
    logits[:, 1], logits[:, 4] = -np.inf, np.nan
    logits[2] = -np.inf
    logits[3, [0, 2, 5]] = -np.inf                            # one expert left for two places
    want, bound = ref.moe(x, logits, wg, wu, wd, 2, True)
    for e in (1, 4):
        wg[e] = wu[e] = np.nan
    got = call(torch, x, logits, wg, wu, wd, 2, True)
    assert np.all(np.abs(got - want) <= bound)
    assert not got[2].any()
    none = call(torch, x, np.full((4, 6), -np.inf, np.float32), wg, wu, wd, 2, False)
    assert not none.any()


def test_far_logits(torch):
    logits = np.random.default_rng(6).standard_normal((6, 10)).astype(np.float32) * 60
    check(torch, 6, 64, 48, 10, 4, renorm=False, logits=logits)


def test_calls_share_a_workspace_and_repeat_bit_for_bit(torch):
    ws = torch.zeros(dg.dg_moe_workspace_bytes(64, 1000, 1000, 32, 8), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(7)
    x, wg, wu, wd = make(rng, 20, 520, 264, 16)
    logits = rng.standard_normal((20, 16)).astype(np.float32)
    first = call(torch, x, logits, wg, wu, wd, 4, True, ws=ws)
    check(torch, 64, 128, 1000, 32, 8, seed=1, ws=ws)
    check(torch, 1, 1000, 64, 4, 1, seed=2, ws=ws)
    for _ in range(3):
        assert np.array_equal(call(torch, x, logits, wg, wu, wd, 4, True, ws=ws), first)


def test_graph_follows_the_router(torch):
    rng = np.random.default_rng(8)
    T, K, I, E, top = 3, 512, 256, 8, 2
    x, wg, wu, wd = make(rng, T, K, I, E)
    X, Wg, Wu, Wd = (dev(torch, a) for a in (x, wg, wu, wd))
    L = torch.zeros((T, E), device="cuda")
    Y = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(dg.dg_moe_workspace_bytes(T, K, I, E, top), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.moe_bf16(T, K, I, E, top, True, X, K, L, E, Wg, I, K * I, Wu, I, K * I, Wd, K, K * I, Y, K, ws, ws.numel())
    for seed in range(3):
        logits = np.random.default_rng(seed).standard_normal((T, E)).astype(np.float32)
        L.copy_(torch.from_numpy(logits))
        graph.replay()
        sync(torch)
        want, bound = ref.moe(x, logits, wg, wu, wd, top, True)
        assert np.all(np.abs(Y.float().cpu().numpy() - want) <= bound)


def test_expert_offsets_past_32_bits(torch):
    # The last expert's matrices start past 2^32 bytes.
    T, K, I, E = 2, 1024, 1024, 512
    stride = (1 << 32) // 2 // (E - 1) // 8 * 8 + 8 * 1024
    rng = np.random.default_rng(15)
    x, wg, wu, wd = make(rng, T, K, I, 1)
    logits = np.zeros((T, E), np.float32)
    logits[:, E - 1] = 5.0
    buf = []
    for w in (wg, wu, wd):
        b = torch.full((stride * (E - 1) + K * I,), float("nan"), dtype=torch.bfloat16, device="cuda")
        b[stride * (E - 1):].copy_(dev(torch, w[0]).flatten())
        buf.append(b)
    L = torch.from_numpy(logits).cuda()
    Y = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(dg.dg_moe_workspace_bytes(T, K, I, E, 1), dtype=torch.uint8, device="cuda")
    dg.moe_bf16(T, K, I, E, 1, True, dev(torch, x), K, L, E, buf[0], I, stride, buf[1], I, stride, buf[2], K, stride, Y, K, ws, ws.numel())
    sync(torch)
    want, bound = ref.moe(x, np.zeros((T, 1)), wg, wu, wd, 1, True)
    assert np.all(np.abs(Y.float().cpu().numpy() - want) <= bound)
