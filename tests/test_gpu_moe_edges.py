"""moe_bf16 where a call takes another way than small ordinary ones do."""
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


def dev(torch, x):
    return torch.from_numpy(np.ascontiguousarray(ref.bf16_bits(x)).view(np.int16)).view(torch.bfloat16).cuda()


def call(torch, x, logits, wg, wu, wd, top, renorm):
    T, K = x.shape
    E, _, I = wg.shape
    Y = torch.full((T, K), -3.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(dg.dg_moe_workspace_bytes(T, K, I, E, top), dtype=torch.uint8, device="cuda")
    L = torch.from_numpy(np.asarray(logits, dtype=np.float32)).cuda()
    dg.moe_bf16(T, K, I, E, top, renorm, dev(torch, x), K, L, E, dev(torch, wg), I, K * I, dev(torch, wu), I, K * I,
                dev(torch, wd), K, I * K, Y, K, ws, ws.numel())
    torch.cuda.synchronize()
    assert dg.dg_device_status() == dg.DG_OK
    return Y.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("T", [1, 20])
@pytest.mark.parametrize("K", [64, 1024])                     # whole tiles, and tiles joined from parts
@pytest.mark.parametrize("least", [False, True])
def test_an_activation_past_the_range_is_infinite(torch, T, K, least):
    I = 64
    x, wg, wu, wd = np.zeros((T, K), np.float32), *(np.zeros((1, K, I), np.float32) for _ in range(2)), np.zeros((1, I, K), np.float32)
    x[:, 0] = x[:, K - 1] = 2.0 ** 40
    wg[0, 0, 5] = 2.0 ** 24
    if least:                                                 # 2^128 (1 - 2^-10): FP32 has it, BF16 rounds it up to Inf
        wu[0, 0, 5], wu[0, K - 1, 5] = 2.0 ** 24 * (1 - 2.0 ** -8), 0.75 * 2.0 ** 16
    else:
        wu[0, 0, 5] = 2.0 ** 30
    wd[0, 5, ::2], wd[0, 5, 1::2] = 1.0, -2.0
    y = call(torch, x, np.zeros((T, 1)), wg, wu, wd, 1, True)
    assert np.all(y[:, ::2] == np.inf) and np.all(y[:, 1::2] == -np.inf)


def check(torch, T, E, top, renorm, logits, K=72, I=40):
    rng = np.random.default_rng(T + E + top)
    x = ref.bf16(rng.standard_normal((T, K)))
    wg, wu = (ref.bf16(rng.standard_normal((E, K, I)) / np.sqrt(K)) for _ in range(2))
    wd = ref.bf16(rng.standard_normal((E, I, K)) / np.sqrt(I))
    got = call(torch, x, logits, wg, wu, wd, top, renorm)
    want, bound = ref.moe(x, logits, wg, wu, wd, top, renorm)
    off = ~(np.abs(got - want) <= bound)
    assert not off.any(), f"{off.sum()} of {off.size}, first {np.argwhere(off)[0]}"


# More than 16 tokens have a routing launch of their own, whose lanes hold 2, 4 or 16 logits each.
@pytest.mark.parametrize("E", [40, 64, 65, 100, 128, 129, 300, 512])
@pytest.mark.parametrize("T,top,renorm", [(17, 1, False), (33, 8, True), (64, 16, False), (48, 11, True)])
def test_routing_of_many_experts(torch, T, E, top, renorm):
    rng = np.random.default_rng(E + T)
    check(torch, T, E, top, renorm, rng.standard_normal((T, E)).astype(np.float32) * 1.5)


@pytest.mark.parametrize("T", [5, 16, 21, 64])
@pytest.mark.parametrize("E,top", [(17, 16), (33, 9), (40, 16), (65, 12), (128, 16), (129, 10), (512, 16)])
def test_routing_of_ties_and_of_experts_switched_off(torch, T, E, top):
    # Logits in steps of a half tie at the last place of nearly every row; whole experts and single
    # logits are off; one row has a single expert left, one none, one equal logits throughout.
    rng = np.random.default_rng(E * T)
    logits = np.round(rng.standard_normal((T, E)) * 2).astype(np.float32) / 2
    logits[:, rng.choice(E, E // 8, replace=False)] = -np.inf
    logits[rng.random((T, E)) < 0.05] = np.nan
    logits[0], logits[1], logits[2] = -np.inf, -np.inf, -0.0
    logits[0, E - 1] = -3.0
    logits[2, ::2] = 0.0
    check(torch, T, E, top, T % 2 == 0, logits)
