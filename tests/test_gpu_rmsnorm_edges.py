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
