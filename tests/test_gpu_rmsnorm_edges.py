"""rmsnorm_residual_bf16 and _e4m3 at the ends of their range, in every form of the kernel."""
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


def to_codes(torch, x, r, gain, eps, ld):
    """x [rows, cols] float32 on the host -> (code values, scales) of BF16 rows with stride ld."""
    rows, cols = x.shape
    X = torch.full((rows, ld), float("nan"), dtype=torch.bfloat16, device="cuda")
    X[:, :cols] = torch.from_numpy(x).cuda()
    R = None
    if r is not None:
        R = torch.full((rows, ld), float("nan"), device="cuda")
        R[:, :cols] = torch.from_numpy(r).cuda()
    Q = torch.full((rows, ld), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((rows,), -1.0, device="cuda")
    dg.rmsnorm_residual_e4m3(rows, cols, X, ld, dg.DG_OUT_BF16, R, ld, dg.DG_OUT_F32, None if R is None else torch.empty_like(R), ld,
                             torch.from_numpy(gain).to(torch.bfloat16).cuda(), eps, Q, ld, s)
    torch.cuda.synchronize()
    assert dg.dg_device_status() == dg.DG_OK
    return Q[:, :cols].contiguous().view(torch.float8_e4m3fn).float().cpu().numpy(), s.cpu().numpy()


# A few lanes a row, a warp, CTAs with one to four chunks a thread, rows that begin anywhere, two passes.
FORMS = [(64, 64), (40, 41), (500, 504), (777, 777), (4096, 4096), (4096, 4099), (12288, 12288), (16384, 16384), (40000, 40000)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("cols,ld", FORMS)
def test_rows_of_zeros_without_eps(torch, cols, ld, residual):
    rng = np.random.default_rng(cols)
    x = ref.bf16(rng.standard_normal((6, cols)))
    gain = ref.bf16(1 + 0.1 * rng.standard_normal(cols))
    x[1] = x[4] = 0
    r = None
    if residual:
        r = rng.standard_normal((6, cols)).astype(np.float32)
        r[1], r[4] = 0, 0
        r[3] = -x[3]                                          # what cancels is a row of zeros too
    codes, s = to_codes(torch, x, r, gain, 0.0, ld)
    zero = [1, 3, 4] if residual else [1, 4]
    rest = [i for i in range(6) if i not in zero]
    assert not codes[zero].any() and not s[zero].any()
    assert np.all(np.abs(codes[rest]).max(1) == 448) and np.all(s[rest] > 0)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("cols,ld", FORMS)
def test_rows_whose_reciprocal_passes_fp32(torch, cols, ld, residual):
    # Largest outputs from 2^-116 down to 2^-140, zeros among the elements: by small rows, by a small
    # gain, by both, and by a small gain on a row so large that its norm is small.
    rng = np.random.default_rng(cols + 1)
    for x_exp, gain_exp, eps in ((-126, 0, 1.0), (-120, -10, 1.0), (0, -124, 1e-5), (50, -121, 1e-5), (-130, 0, 1e-5), (0, -122, 1e-9)):
        x = ref.bf16(rng.uniform(0.25, 1, (4, cols)) * rng.choice([-1, 1], (4, cols)) * 2.0 ** x_exp)
        gain = ref.bf16(rng.uniform(0.5, 1, cols) * 2.0 ** gain_exp)
        x[:, 1::3] = 0
        x[2] = 0
        r = (rng.uniform(-0.25, 0.25, (4, cols)) * 2.0 ** x_exp).astype(np.float32) if residual else None
        if residual:
            r[:, 1::3] = 0
            r[2] = 0
        codes, s = to_codes(torch, x, r, gain, eps, ld)
        _, y = ref.rmsnorm(x, r, gain, eps)
        want, scales = ref.rmsnorm_codes(y)
        # FP32 subnormals: h, h * gain and the largest output are off by up to 2^-150 each.
        top = np.abs((x if r is None else x.astype(np.float64) + r) * gain.astype(np.float64)).max(1, keepdims=True)
        tiny = 2.0 ** -149 / np.where(top > 0, top, 1) * 2
        rel = (cols / 32 + 40) * 2.0 ** -25 + 8 * ref.F32
        assert np.all(np.abs(codes - want) <= np.abs(want) * (ref.E4M3 + 4 * rel + tiny) + 448 * tiny + 2.0 ** -10)
        assert np.all(np.abs(s - scales) <= scales * (4 * rel + tiny[:, 0]) + 2.0 ** -148)
        assert not codes[2].any() and s[2] == 0 and not codes[:, 1::3].any()
