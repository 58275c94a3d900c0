"""4-bit weights: quantize_groups_w4 and dequantize_groups_w4 bit for bit against their definition,
gemm_w4_bf16 against the float64 oracle within the bound derived there, and exactly where all sums
are."""
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


def words(torch, x):
    return torch.from_numpy(np.ascontiguousarray(x).view(np.int32)).cuda()


def weights(rng, n, k):
    return ref.bf16((rng.standard_normal((n, k)) * np.exp(rng.normal(0, 1, (n, 1)))).astype(np.float32))


# ------------------------------------------------------------------ rows
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,k,pad", [(1, 1, 0), (3, 7, 1), (5, 31, 0), (4, 32, 0), (7, 33, 7), (17, 129, 3), (8, 256, 0), (33, 1000, 0),
                                     (2, 4096, 8), (130, 777, 2), (300, 264, 5)])
def test_rows(torch, n, k, pad, group):
    rng = np.random.default_rng(n + k + group)
    w = weights(rng, n, k)
    w[0, :min(k, group)] = -2.5                       # a constant group
    w[n // 2, k // 2] = 1e30                          # a step so large that the rest falls on one code
    w[n - 1, k - 1] = -1e-38
    codes, scale, zero = ref.w4_quantise(w, group)
    groups = scale.shape[1]
    ldw, ldq, ldp = k + pad, -(-k // 32) * 16 + 16, -(-n // 4) * 4 + 4
    W = torch.full((n, ldw), float("nan"), dtype=torch.bfloat16, device="cuda")
    W[:, :k] = dev(torch, w)
    Q = torch.full((n, ldq), 0xAB, dtype=torch.uint8, device="cuda")
    P = torch.full((groups, ldp), -7, dtype=torch.int32, device="cuda")
    dg.quantize_groups_w4(n, k, group, W, ldw, Q, ldq, P, ldp)
    sync(torch)
    want, used = ref.w4_pack(codes, ldq), -(-k // 8) * 4
    got = Q.cpu().numpy()
    assert np.array_equal(got[:, :used], want[:, :used]) and (got[:, used:] == 0xAB).all()
    got = P.cpu().numpy()
    assert np.array_equal(got[:, :n].view(np.uint32), ref.w4_params(scale, zero, ldp)[:, :n]) and (got[:, n:] == -7).all()
    back = torch.full((n, ldw), 3.0, dtype=torch.bfloat16, device="cuda")
    dg.dequantize_groups_w4(n, k, group, Q, ldq, P, ldp, back, ldw)
    sync(torch)
    got = back.float().cpu().numpy()
    assert np.array_equal(got[:, :k], ref.bf16(ref.w4_value(codes, scale, zero, group).astype(np.float32))) and (got[:, k:] == 3.0).all()


def test_rows_from_odd_addresses(torch):
    n, k, group = 6, 200, 64
    w = weights(np.random.default_rng(2), n, k)
    flat = torch.zeros(n * 203 + 1, dtype=torch.bfloat16, device="cuda")
    W = flat[1:].as_strided((n, k), (203, 1))
    W.copy_(dev(torch, w))
    Q, P = torch.zeros((n, 112), dtype=torch.uint8, device="cuda"), torch.zeros((4, 8), dtype=torch.int32, device="cuda")
    dg.quantize_groups_w4(n, k, group, W, 203, Q, 112, P, 8)
    sync(torch)
    codes, scale, zero = ref.w4_quantise(w, group)
    assert np.array_equal(Q.cpu().numpy(), ref.w4_pack(codes, 112))
    W.zero_()
    dg.dequantize_groups_w4(n, k, group, Q, 112, P, 8, W, 203)
    sync(torch)
    assert np.array_equal(W.float().cpu().numpy(), ref.bf16(ref.w4_value(codes, scale, zero, group).astype(np.float32)))
    assert flat[0] == 0 and not flat[1:].as_strided((n - 1, 3), (203, 1), 1 + k).any()


# ------------------------------------------------------------------ product
class Weights:
    def __init__(self, torch, rng, n, k, group, exact=False, spare=0):
        groups = -(-k // group)
        self.n, self.k, self.group = n, k, group
        self.codes = rng.integers(0, 16, (n, k)).astype(np.uint8)
        if exact:
            self.scale = ref.bf16(2.0 ** rng.integers(-1, 2, (n, groups)))
            self.zero = ref.bf16(rng.integers(-8, 3, (n, groups)) * 0.5)
        else:
            self.scale = ref.bf16(np.exp(rng.normal(0, 0.5, (n, groups))) * 0.3)
            self.zero = ref.bf16(-7.5 * self.scale + rng.normal(0, 0.3, (n, groups)))
        self.ldq, self.ldp = -(-k // 32) * 16 + 16 * spare, -(-n // 4) * 4 + 4 * spare
        q = ref.w4_pack(self.codes, self.ldq)
        at = np.arange(self.ldq * 2)                    # codes past K may be anything
        bit = 4 * (at % 8 // 2) + 16 * (at % 2)
        for j in at[k:]:
            q[:, j // 8 * 4 + bit[j] // 8] |= np.uint8(15 << (bit[j] % 8))
        p = ref.w4_params(self.scale, self.zero, self.ldp)
        p[:, n:] = 0xFFFFFFFF                           # and parameters past N
        self.Q, self.P = torch.from_numpy(q).cuda(), words(torch, p)

    def times(self, torch, x, f32, pad=0, padc=0, ws=None, stream=None):
        m = x.shape[0]
        ldx, ldc = -(-self.k // 8) * 8 + pad, self.n + padc
        X = torch.full((m, ldx), float("nan"), dtype=torch.bfloat16, device="cuda")
        X[:, :self.k] = x if torch.is_tensor(x) else dev(torch, x)
        C = torch.full((m, ldc), -3.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        if ws is None:
            ws = torch.zeros(dg.dg_gemm_w4_workspace_bytes(m, self.n, self.k), dtype=torch.uint8, device="cuda")
        dg.gemm_w4_bf16(m, self.n, self.k, self.group, X, ldx, self.Q, self.ldq, self.P, self.ldp, C, ldc,
                        dg.DG_OUT_F32 if f32 else dg.DG_OUT_BF16, ws, ws.numel())
        sync(torch)
        assert bool((C[:, self.n:] == -3.0).all())
        return C[:, :self.n].float().cpu().numpy()


def check(torch, m, n, k, group, f32, seed=0, pad=0, padc=0, ws=None, spare=0):
    rng = np.random.default_rng(seed + m + n + k)
    w = Weights(torch, rng, n, k, group, spare=spare)
    x = ref.bf16((rng.standard_normal((m, k)) * np.exp(rng.normal(0, 1, (m, 1)))).astype(np.float32))
    got = w.times(torch, x, f32, pad, padc, ws)
    want, bound = ref.w4_gemm(x, w.codes, w.scale, w.zero, group, ref.F32 if f32 else ref.BF16)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, first {np.argwhere(bad)[0]}, worst {np.nanmax(np.abs(got - want) / (bound + 1e-30)):.3g}"


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 129, 200])
def test_product_rows(torch, m, f32):
    check(torch, m, 300, 520, 128, f32)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("k", [1, 7, 8, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 4096, 5000])
def test_product_depths(torch, k, group):
    check(torch, 3, 130, k, group, True, spare=k % 2)
    check(torch, 20, 70, k, group, False)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 127, 128, 129, 1000, 5001, 20000])
def test_product_columns(torch, n):
    check(torch, 5, n, 384, 64, True, padc=n % 3)
    check(torch, 40, n, 200, 32, False, padc=5)


@pytest.mark.parametrize("pad,padc", [(0, 1), (8, 0), (64, 7)])
def test_product_strides(torch, pad, padc):
    check(torch, 18, 260, 300, 128, False, pad=pad, padc=padc)
    check(torch, 18, 260, 300, 128, True, pad=pad, padc=padc)


@pytest.mark.parametrize("m,n,k,group", [(1, 4096, 4096, 128), (16, 1000, 2048, 64), (64, 515, 1500, 32), (61, 3000, 4096, 128), (150, 129, 900, 32)])
def test_product_is_exact_where_all_sums_are(torch, m, n, k, group):
    # Small whole numbers and halves: no sum passes 2^24 of its last place, so every order gives the same.
    rng = np.random.default_rng(k + m)
    w = Weights(torch, rng, n, k, group, exact=True)
    x = rng.integers(-2, 3, (m, k)).astype(np.float32)
    got = w.times(torch, x, True)
    assert np.array_equal(got, x.astype(np.float64) @ ref.w4_value(w.codes, w.scale, w.zero, group).T)


def test_product_of_single_elements(torch):
    # Row m of X has one 1: every weight of its k comes out by itself.
    rng = np.random.default_rng(5)
    n, k, group = 140, 300, 64
    w = Weights(torch, rng, n, k, group, exact=True)
    got = w.times(torch, np.eye(k, dtype=np.float32), True)
    assert np.array_equal(got, ref.w4_value(w.codes, w.scale, w.zero, group).T)


def test_rows_that_are_not_finite_stay_alone(torch):
    rng = np.random.default_rng(6)
    w = Weights(torch, rng, 200, 640, 128)
    x = ref.bf16(rng.standard_normal((20, 640)).astype(np.float32))
    good = w.times(torch, x, True)
    X = dev(torch, x)
    X[3, 100], X[7, 5], X[11, 600] = float("nan"), float("inf"), -float("inf")
    got = w.times(torch, X, True)
    bad = [3, 7, 11]
    assert not np.isfinite(got[bad]).any()
    keep = [i for i in range(20) if i not in bad]
    assert np.array_equal(got[keep], good[keep])


def test_columns_whose_parameters_are_not_finite_stay_alone(torch):
    rng = np.random.default_rng(7)
    w = Weights(torch, rng, 150, 256, 128)
    x = ref.bf16(rng.standard_normal((5, 256)).astype(np.float32))
    good = w.times(torch, x, True)
    w.P[1, 70] = 0x7FC07FC0
    got = w.times(torch, x, True)
    assert not np.isfinite(got[:, 70]).any()
    keep = np.arange(150) != 70
    assert np.array_equal(got[:, keep], good[:, keep])


def test_calls_of_different_sizes_share_a_workspace(torch):
    sizes = [(1, 4096, 4096, 128), (64, 300, 5000, 32), (3, 20000, 130, 64), (17, 128, 9000, 128), (100, 700, 700, 64)]
    ws = torch.zeros(max(dg.dg_gemm_w4_workspace_bytes(m, n, k) for m, n, k, _ in sizes), dtype=torch.uint8, device="cuda")
    for seed in range(2):
        for m, n, k, group in sizes:
            check(torch, m, n, k, group, seed % 2 == 0, seed=seed, ws=ws)


@pytest.mark.parametrize("m", [1, 16, 33, 64, 70])
def test_product_repeats_bit_for_bit_and_in_a_graph(torch, m):
    rng = np.random.default_rng(8)
    n, k = 1500, 4096
    w = Weights(torch, rng, n, k, 128)
    X = dev(torch, ref.bf16(rng.standard_normal((m, k)).astype(np.float32)))
    first = w.times(torch, X, True)
    for _ in range(3):
        assert np.array_equal(w.times(torch, X, True), first)
    C = torch.zeros((m, n), device="cuda")
    ws = torch.zeros(dg.dg_gemm_w4_workspace_bytes(m, n, k), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            dg.gemm_w4_bf16(m, n, k, 128, X, k, w.Q, w.ldq, w.P, w.ldp, C, n, dg.DG_OUT_F32, ws, ws.numel())
    for _ in range(3):
        C.zero_()
        graph.replay()
        sync(torch)
        assert np.array_equal(C.cpu().numpy(), first)
    X.mul_(2)                                                # the graph follows its inputs
    graph.replay()
    sync(torch)
    assert np.array_equal(C.cpu().numpy(), 2 * first)


@pytest.mark.parametrize("m,n,k,group", [(1, 1000, 2048, 128), (16, 3000, 1024, 32), (30, 1000, 2048, 64), (61, 3000, 1024, 128)])
def test_stages_are_used_after_they_have_come(torch, m, n, k, group):
    # Lanes of a warp wait for different barriers of a stage and use what the others waited for.  All sums are
    # exact, and two inputs take turns in rings and tensor memory: what is used too early is another call's.
    rng = np.random.default_rng(m)
    ws = torch.zeros(dg.dg_gemm_w4_workspace_bytes(m, n, k), dtype=torch.uint8, device="cuda")
    turns = []
    for _ in range(2):
        w = Weights(torch, rng, n, k, group, exact=True)
        x = rng.integers(-2, 3, (m, k)).astype(np.float32)
        turns.append((w, dev(torch, x), torch.from_numpy((x.astype(np.float64) @ ref.w4_value(w.codes, w.scale, w.zero, group).T)).cuda(),
                      torch.zeros((50, m, n), device="cuda")))
    for i in range(50):
        for w, x, _, c in turns:
            dg.gemm_w4_bf16(m, n, k, group, x, k, w.Q, w.ldq, w.P, w.ldp, c[i], n, dg.DG_OUT_F32, ws, ws.numel())
    sync(torch)
    for _, _, want, c in turns:
        assert bool((c.double() == want).all())


def test_two_streams_with_their_own_workspaces(torch):
    rng = np.random.default_rng(9)
    w = [Weights(torch, rng, 3000, 4096, 128), Weights(torch, rng, 5000, 1024, 32)]
    X = [dev(torch, ref.bf16(rng.standard_normal((m, v.k)).astype(np.float32))) for m, v in zip((16, 40), w)]
    alone = [v.times(torch, x, True) for v, x in zip(w, X)]
    ws = [torch.zeros(dg.dg_gemm_w4_workspace_bytes(x.shape[0], v.n, v.k), dtype=torch.uint8, device="cuda") for v, x in zip(w, X)]
    C = [torch.zeros((x.shape[0], v.n), device="cuda") for v, x in zip(w, X)]
    streams = [torch.cuda.Stream() for _ in w]
    torch.cuda.synchronize()
    for _ in range(10):
        for v, x, c, u, s in zip(w, X, C, ws, streams):
            dg.gemm_w4_bf16(x.shape[0], v.n, v.k, v.group, x, v.k, v.Q, v.ldq, v.P, v.ldp, c, v.n, dg.DG_OUT_F32, u, u.numel(), stream=s)
    sync(torch)
    for c, a in zip(C, alone):
        assert np.array_equal(c.cpu().numpy(), a)


def test_no_depth_and_no_rows(torch):
    C = torch.full((4, 10), 5.0, dtype=torch.bfloat16, device="cuda")
    dg.gemm_w4_bf16(4, 8, 0, 32, None, 0, None, 0, None, 0, C, 10, dg.DG_OUT_BF16, None, 0)
    sync(torch)
    assert not C[:, :8].any() and bool((C[:, 8:] == 5.0).all())
    dg.gemm_w4_bf16(0, 8, 64, 32, None, 0, None, 0, None, 0, None, 0, dg.DG_OUT_BF16, None, 0)
    sync(torch)


def test_offsets_past_32_bits(torch):
    # 8.6 GB of codes; columns from all over are checked.
    n, k, group, m = (1 << 21) + 5, 8192, 128, 2
    rng = np.random.default_rng(10)
    g = torch.Generator(device="cuda").manual_seed(1)
    Q = torch.randint(-2 ** 62, 2 ** 62, (n, k // 16), generator=g, device="cuda", dtype=torch.int64)
    ldp = -(-n // 4) * 4
    P = torch.empty((k // group, ldp, 2), dtype=torch.bfloat16, device="cuda")
    P[..., 0].fill_(0.25)
    P[..., 1] = torch.randn((k // group, ldp), generator=g, device="cuda")
    x = ref.bf16(rng.standard_normal((m, k)).astype(np.float32))
    C = torch.zeros((m, n), device="cuda")
    ws = torch.zeros(dg.dg_gemm_w4_workspace_bytes(m, n, k), dtype=torch.uint8, device="cuda")
    dg.gemm_w4_bf16(m, n, k, group, dev(torch, x), k, Q, k // 2, P, ldp, C, n, dg.DG_OUT_F32, ws, ws.numel())
    sync(torch)
    at = np.unique(np.concatenate([[0, 1, 127, 128, n // 2, n - 2, n - 1], rng.integers(0, n, 60)]))
    q = Q[torch.from_numpy(at).cuda()].cpu().numpy().view(np.uint32)
    j = np.arange(k)
    codes = ((q[:, j // 8] >> (4 * (j % 8 // 2) + 16 * (j % 2)).astype(np.uint32)) & 15).astype(np.uint8)
    zero = P[:, torch.from_numpy(at).cuda(), 1].float().cpu().numpy().T
    want, bound = ref.w4_gemm(x, codes, np.full_like(zero, 0.25), zero, group, ref.F32)
    assert np.all(np.abs(C.cpu().numpy()[:, at] - want) <= bound)
    back = torch.empty((5, k), dtype=torch.bfloat16, device="cuda")
    dg.dequantize_groups_w4(5, k, group, Q[n - 5:], k // 2, P.view(torch.int32)[:, n - 5:].squeeze(-1).contiguous().new_zeros((k // group, 8)).copy_(
        torch.nn.functional.pad(P.view(torch.int32)[:, n - 5:n].squeeze(-1), (0, 3))), 8, back, k)
    sync(torch)
    last = at >= n - 5
    rows = torch.from_numpy(at[last] - (n - 5)).cuda()
    assert np.array_equal(back[rows].float().cpu().numpy(), ref.bf16(ref.w4_value(codes[last], np.full_like(zero[last], 0.25), zero[last], group).astype(np.float32)))


# ------------------------------------------------------------------ the ends of the range
@pytest.mark.parametrize("group", [32, 64, 128])
def test_rows_of_tiny_weights(torch, group):
    # Ranges from one subnormal BF16 step (2^-133) to 2^-96, across 1e-30, where quotients are taken another way.
    # Where the scale rounds to 0 codes are 0.
    rng = np.random.default_rng(group)
    n, k = 160, 2 * group + 9
    w = np.ldexp(rng.standard_normal((n, k)).astype(np.float32), -rng.integers(96, 134, (n, 1)))
    w[0] = 0
    w[0, 3] = 2.0 ** -133
    w[1] = np.ldexp(rng.integers(0, 20, k).astype(np.float32), -133)
    w[2] = 2.0 ** -126 + np.ldexp(rng.integers(0, 2, k).astype(np.float32), -133)
    w[3:40] += ref.bf16(np.float32(1e-30) * (1 + rng.standard_normal((37, k)).astype(np.float32) * 0.3))
    w = ref.bf16(w)
    codes, scale, zero = ref.w4_quantise(w, group)
    assert (scale == 0).any() and ((scale > 0) & (scale < 2.0 ** -126)).any()
    ldq, ldp = -(-k // 32) * 16, n
    Q, P = torch.zeros((n, ldq), dtype=torch.uint8, device="cuda"), torch.zeros((scale.shape[1], ldp), dtype=torch.int32, device="cuda")
    dg.quantize_groups_w4(n, k, group, dev(torch, w), k, Q, ldq, P, ldp)
    sync(torch)
    assert np.array_equal(P.cpu().numpy().view(np.uint32), ref.w4_params(scale, zero, ldp))
    assert np.array_equal(Q.cpu().numpy(), ref.w4_pack(codes, ldq))
    back = torch.full((n, k), 3.0, dtype=torch.bfloat16, device="cuda")
    dg.dequantize_groups_w4(n, k, group, Q, ldq, P, ldp, back, k)
    sync(torch)
    assert np.array_equal(back.float().cpu().numpy(), ref.bf16(ref.w4_value(codes, scale, zero, group).astype(np.float32)))


@pytest.mark.parametrize("m,group", [(3, 128), (30, 64), (40, 128), (64, 32)])
def test_product_with_weights_near_the_end_of_the_range(torch, m, group):
    # 16 times the largest scale is past FP32's range, as is 16 scale - zero.
    rng = np.random.default_rng(m)
    n, k = 150, 600
    w = Weights(torch, rng, n, k, group)
    w.scale[:, ::2] = ref.bf16(np.float32(2.25e37))
    w.zero[:, ::2] = ref.bf16(np.float32(-1.68e38))
    w.P = words(torch, ref.w4_params(w.scale, w.zero, w.ldp))
    x = ref.bf16((1e-6 * rng.standard_normal((m, k))).astype(np.float32))
    got = w.times(torch, x, True)
    want, bound = ref.w4_gemm(x, w.codes, w.scale, w.zero, group, ref.F32)
    assert np.all(np.abs(got - want) <= bound)
