"""rmsnorm_residual_bf16 and _e4m3 against the float64 oracle.

Every output may be off by half a step of its type (BF16 2^-8, E4M3 2^-4 and half a subnormal
step, FP32 2^-24) and by the FP32 arithmetic before it: the mean of n squares has at most
n / 32 + 40 roundings of 2^-24 in a row (a thread's terms, then two shuffle trees), half of
that in its root, and five more operations follow.
"""
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


def sync(torch, want=dg.DG_OK):
    torch.cuda.synchronize()
    assert dg.dg_device_status() == want


def make(torch, shape, ld, dtype, seed, std=1.0, offset=0):
    """A [rows, cols] view with row stride ld, `offset` elements into its buffer; NaN around it."""
    g = torch.Generator().manual_seed(seed)
    rows, cols = shape
    buf = torch.full((rows * ld + offset + 64,), float("nan"), dtype=dtype)
    v = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    x = torch.randn((rows, cols), generator=g) * std * torch.exp(torch.randn((rows, 1), generator=g))
    v.copy_(x.to(dtype))
    buf = buf.cuda()
    return buf, buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]


def host(t):
    return t.detach().float().cpu().numpy()


def code_values(torch, q):
    return q.view(torch.float8_e4m3fn).float().cpu().numpy()


def check(torch, h, y, H, Y, r_type, cols):
    rel = (cols / 32 + 40) * 2.0 ** -25 + 6 * ref.F32
    if H is not None:
        step = ref.F32 if r_type == torch.float32 else ref.BF16
        assert np.all(np.abs(host(H) - h) <= np.abs(h) * (step + 2 * ref.F32))
    assert np.all(np.abs(host(Y) - y) <= np.abs(y) * (ref.BF16 + 2 * rel) + 1e-38)


def check_codes(torch, y, Q, s, cols):
    rel = (cols / 32 + 40) * 2.0 ** -25 + 6 * ref.F32
    v, scales = ref.rmsnorm_codes(y)
    assert np.all(np.abs(s.cpu().numpy() - scales) <= scales * (rel + 4 * ref.F32))
    got = code_values(torch, Q)
    assert np.all(np.abs(got - v) <= np.abs(v) * (ref.E4M3 + 4 * rel) + 2.0 ** -10)


def run(torch, rows, cols, xt, rt, ld, off, e4m3, inplace=False, ldy=None):
    X0, X = make(torch, (rows, cols), ld, xt, 1, offset=off)
    R0, R = make(torch, (rows, cols), ld, rt, 2, 2.0, offset=off) if rt is not None else (None, None)
    _, gain = make(torch, (1, cols), cols, torch.bfloat16, 3)
    h, y = ref.rmsnorm(host(X), None if R is None else host(R), host(gain)[0], EPS)
    H0, H = (R0, R) if inplace else ((None, None) if R is None else make(torch, (rows, cols), ld, rt, 4, offset=off))
    keep = None if H0 is None else H0.clone()
    ldy = ldy or cols
    T = {torch.float32: dg.DG_OUT_F32, torch.bfloat16: dg.DG_OUT_BF16, None: dg.DG_OUT_BF16}
    args = (rows, cols, X, ld, T[xt], R, ld if R is not None else 0, T[rt], H, ld if R is not None else 0, gain, EPS)
    if e4m3:
        Y = torch.full((rows, ldy), 0xA5, dtype=torch.uint8, device="cuda")
        s = torch.full((rows + 1,), -1.0, device="cuda")
        dg.rmsnorm_residual_e4m3(*args, Y, ldy, s)
        sync(torch)
        check_codes(torch, y, Y[:, :cols].contiguous(), s[:rows], cols)
        assert s[rows].item() == -1.0 and bool((Y[:, cols:] == 0xA5).all())
        if H is not None:
            check(torch, h, np.zeros_like(y), H, torch.zeros_like(X), rt, cols)
    else:
        Y = torch.full((rows, ldy), float("nan"), dtype=torch.bfloat16, device="cuda")
        dg.rmsnorm_residual_bf16(*args, Y, ldy)
        sync(torch)
        check(torch, h, y, H, Y[:, :cols], rt, cols)
        assert bool(Y[:, cols:].isnan().all())
    if H0 is not None:  # nothing around the rows of H is written
        mask = torch.ones_like(H0, dtype=torch.bool)
        mask[off:off + rows * ld].view(rows, ld)[:, :cols] = False
        a, b = H0[mask], keep[mask]
        assert bool(((a == b) | (a.isnan() & b.isnan())).all())


WIDTHS = [1, 7, 8, 31, 64, 256, 257, 264, 777, 1024, 4096, 8192, 8200, 12345, 16384, 32768, 32776, 40001]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("cols", WIDTHS)
def test_widths(torch, cols, e4m3):
    run(torch, 5, cols, torch.bfloat16, torch.bfloat16, (cols + 7) // 8 * 8, 0, e4m3)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rt", ["none", "bf16", "f32"])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("ld_off", [(1000, 0), (1001, 0), (1008, 3), (1008, 8)])
def test_types_strides_and_alignment(torch, xt, rt, e4m3, ld_off):
    t = {"bf16": torch.bfloat16, "f32": torch.float32, "none": None}
    run(torch, 37, 1000, t[xt], t[rt], ld_off[0], ld_off[1], e4m3, ldy=1005 if ld_off[1] == 3 else 1000)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("xt,rt", [("bf16", "none"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "none"), ("f32", "f32")])
@pytest.mark.parametrize("cols,ld", [(128, 133), (143, 143), (600, 605), (1031, 1033), (4096, 4101), (8179, 8179), (9001, 9010), (16500, 16501)])
def test_rows_that_begin_anywhere(torch, cols, ld, xt, rt, e4m3):
    # Each operand a different distance from an aligned address, H and Y the same.
    t = {"bf16": torch.bfloat16, "f32": torch.float32, "none": None}
    xt, rt = t[xt], t[rt]
    rows = 5
    for k in range(8):
        _, X = make(torch, (rows, cols), ld + 2 * k, xt, k, offset=k)
        _, R = make(torch, (rows, cols), ld + k, rt, 20 + k, offset=(5 * k + 3) % 8) if rt is not None else (None, None)
        _, gain = make(torch, (1, cols), cols, torch.bfloat16, 40 + k, offset=(3 * k + 1) % 8)
        H0, H = make(torch, (rows, cols), ld, rt, 60 + k, offset=7 - k) if rt is not None else (None, None)
        keep = None if H0 is None else H0.clone()
        Y0 = torch.full((rows * ld + 16,), 0xA5 if e4m3 else 7.0, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda")
        Y = Y0[7 - k:7 - k + rows * ld].view(rows, ld)[:, :cols]
        s = torch.full((rows,), -1.0, device="cuda")
        T = {torch.float32: dg.DG_OUT_F32, torch.bfloat16: dg.DG_OUT_BF16, None: dg.DG_OUT_BF16}
        args = (rows, cols, X, ld + 2 * k, T[xt], R, ld + k if R is not None else 0, T[rt], H, ld if R is not None else 0, gain, EPS)
        if e4m3:
            dg.rmsnorm_residual_e4m3(*args, Y, ld, s)
        else:
            dg.rmsnorm_residual_bf16(*args, Y, ld)
        sync(torch)
        h, y = ref.rmsnorm(host(X), None if R is None else host(R), host(gain)[0], EPS)
        if e4m3:
            check_codes(torch, y, Y.contiguous(), s, cols)
            if H is not None:
                check(torch, h, np.zeros_like(y), H, torch.zeros_like(X), rt, cols)
        else:
            check(torch, h, y, H, Y, rt, cols)
        for buf, old, off in ((Y0, None, 7 - k), (H0, keep, 7 - k)):  # nothing around the rows is written
            if buf is None:
                continue
            mask = torch.ones_like(buf, dtype=torch.bool)
            mask[off:off + rows * ld].view(rows, ld)[:, :cols] = False
            got = buf[mask]
            same = (got == (0xA5 if e4m3 else 7.0)) if old is None else (got == old[mask]) | (got.isnan() & old[mask].isnan())
            assert bool(same.all())


@pytest.mark.parametrize("cols,ld", [(777, 777), (4099, 4100)])
@pytest.mark.parametrize("rt", ["bf16", "f32"])
def test_in_place_residual_of_rows_that_begin_anywhere(torch, cols, ld, rt):
    run(torch, 6, cols, torch.bfloat16, torch.bfloat16 if rt == "bf16" else torch.float32, ld, 0, False, inplace=True, ldy=ld)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows", [1, 3, 4, 15, 17, 31, 33, 70])
@pytest.mark.parametrize("cols,ld", [(1, 1), (5, 9), (40, 40), (64, 64), (65, 65), (120, 128), (127, 127), (128, 136)])
def test_short_rows(torch, rows, cols, ld, e4m3):
    run(torch, rows, cols, torch.bfloat16, torch.float32, ld, 0, e4m3)
    run(torch, rows, cols, torch.float32, torch.bfloat16, ld, 0, e4m3, inplace=True, ldy=ld)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("cols", [8208, 10240, 12288, 12296, 20000, 24576, 24584])
def test_long_rows(torch, cols, e4m3):
    run(torch, 3, cols, torch.bfloat16, torch.bfloat16, cols, 0, e4m3)
    run(torch, 2, cols, torch.float32, None, cols + 8, 0, e4m3)


@pytest.mark.parametrize("rows", [1, 2, 8, 9, 4097])
@pytest.mark.parametrize("cols", [96, 520])
def test_rows(torch, rows, cols):
    run(torch, rows, cols, torch.bfloat16, torch.float32, cols, 0, True)


@pytest.mark.parametrize("cols", [200, 4096, 40000])
@pytest.mark.parametrize("rt", ["bf16", "f32"])
def test_in_place_residual(torch, cols, rt):
    run(torch, 6, cols, torch.bfloat16, torch.bfloat16 if rt == "bf16" else torch.float32, cols, 0, False, inplace=True)


def test_zero_rows_and_non_finite_rows(torch):
    X = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    X[1, 3], X[2, 5] = float("inf"), float("nan")
    X[3] = 1.0
    gain = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    Q = torch.full((4, 256), 9, dtype=torch.uint8, device="cuda")
    s = torch.full((4,), -1.0, device="cuda")
    dg.rmsnorm_residual_e4m3(4, 256, X, 256, dg.DG_OUT_BF16, None, 0, dg.DG_OUT_BF16, None, 0, gain, 0.0, Q, 256, s)
    Y = torch.empty((4, 256), dtype=torch.bfloat16, device="cuda")
    dg.rmsnorm_residual_bf16(4, 256, X, 256, dg.DG_OUT_BF16, None, 0, dg.DG_OUT_BF16, None, 0, gain, EPS, Y, 256)
    sync(torch)
    # eps = 0 and a row of zeros: 0 / 0; with eps the norm of zeros is zeros.
    assert not Y[0].any() and Y[2].isnan().all() and bool((Y[3] - 1).abs().max() < 2 ** -7)
    assert bool((code_values(torch, Q[3:]) == 448).all()) and abs(s[3].item() * 448 - 1) < 1e-6
    dg.rmsnorm_residual_e4m3(1, 256, X, 256, dg.DG_OUT_BF16, None, 0, dg.DG_OUT_BF16, None, 0, gain, EPS, Q, 256, s)
    sync(torch)
    assert not Q[0].any() and s[0].item() == 0.0


def test_feeds_the_fp8_gemm(torch):
    # The codes and scales go straight into gemm_fp8_e4m3; against the float64 product of what they stand for.
    M, K, N = 64, 512, 128
    _, X = make(torch, (M, K), K, torch.bfloat16, 5)
    gain = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    Q, s = torch.empty((M, K), dtype=torch.uint8, device="cuda"), torch.empty(M, device="cuda")
    dg.rmsnorm_residual_e4m3(M, K, X, K, dg.DG_OUT_BF16, None, 0, dg.DG_OUT_BF16, None, 0, gain, EPS, Q, K, s)
    W = torch.randn((N, K), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    qw, sw = torch.empty((N, K), dtype=torch.uint8, device="cuda"), torch.empty(N, device="cuda")
    dg.quantize_rows_e4m3(N, K, W, K, qw, K, sw)
    C = torch.empty((M, N), device="cuda")
    dg.gemm_fp8_e4m3(M, N, K, Q, K, s, qw, K, sw, C, N, dg.DG_OUT_F32)
    sync(torch)
    a = code_values(torch, Q).astype(np.float64) * s.cpu().numpy()[:, None].astype(np.float64)
    b = code_values(torch, qw).astype(np.float64) * sw.cpu().numpy()[:, None].astype(np.float64)
    assert np.all(np.abs(C.cpu().numpy() - a @ b.T) <= 1e-5 * (np.abs(a) @ np.abs(b).T))


def test_graph_and_side_stream(torch):
    _, X = make(torch, (64, 4096), 4096, torch.bfloat16, 7)
    gain = torch.ones(4096, dtype=torch.bfloat16, device="cuda")
    Y, Z = (torch.zeros((64, 4096), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def call(out):
        dg.rmsnorm_residual_bf16(64, 4096, X, 4096, dg.DG_OUT_BF16, None, 0, dg.DG_OUT_BF16, None, 0, gain, EPS, out, 4096)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(Y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(Z)
    X.mul_(2)
    graph.replay()
    sync(torch)
    Y2 = torch.empty_like(Y)
    call(Y2)
    sync(torch)
    assert torch.equal(Z, Y2) and not torch.equal(Y, torch.zeros_like(Y))
