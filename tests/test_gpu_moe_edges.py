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
