"""The serving operators without a GPU: refused arguments, and the oracle's own pins."""
import numpy as np
import pytest

import dense_gemm_sm_gb300 as dg
from oracle import serving as ref

P = 0x10000  # an aligned address that no refused call reaches
INV, MIS, UNS = dg.DG_ERR_INVALID_ARG, dg.DG_ERR_MISALIGNED, dg.DG_ERR_UNSUPPORTED


# ------------------------------------------------------------------ refusals
NORM = dict(rows=4, cols=64, X=P, ldx=64, x_type=dg.DG_OUT_BF16, R=P, ldr=64, r_type=dg.DG_OUT_F32, H=P, ldh=64,
            gain=P, eps=1e-5, Y=P, ldy=64)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INV), (dict(cols=-1), INV), (dict(x_type=7), INV), (dict(r_type=-1), INV), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV), (dict(ldx=63), INV), (dict(ldr=63), INV),
    (dict(ldh=63), INV), (dict(ldy=63), INV), (dict(X=None), INV), (dict(gain=None), INV), (dict(Y=None), INV),
    (dict(R=None), INV), (dict(H=None), INV), (dict(X=P + 1), MIS), (dict(R=P + 2), MIS), (dict(H=P + 2), MIS),
    (dict(gain=P + 1), MIS), (dict(rows=2 ** 31), UNS), (dict(cols=2 ** 31, ldx=2 ** 31, ldr=2 ** 31, ldh=2 ** 31, ldy=2 ** 31), UNS),
    (dict(rows=0), dg.DG_OK), (dict(cols=0), dg.DG_OK)])
def test_norm_refuses(change, status):
    a = {**NORM, **change}
    assert dg.rmsnorm_residual_bf16(*a.values(), stream=0, check=False) == status
    assert dg.rmsnorm_residual_e4m3(*a.values(), P, stream=0, check=False) == status


def test_norm_refuses_its_own_outputs():
    assert dg.rmsnorm_residual_e4m3(*NORM.values(), None, stream=0, check=False) == INV
    assert dg.rmsnorm_residual_e4m3(*NORM.values(), P + 2, stream=0, check=False) == MIS
    assert dg.rmsnorm_residual_bf16(*{**NORM, "Y": P + 1}.values(), stream=0, check=False) == MIS


def cache(data=P, pages=8, page_size=32, heads=2, d=128):
    return dg.dg_kv4_cache(data, pages, page_size, heads, d)


@pytest.mark.parametrize("c,status", [
    (dict(pages=-1), INV), (dict(page_size=0), INV), (dict(page_size=24), INV), (dict(heads=0), INV), (dict(d=0), INV),
    (dict(data=None), INV), (dict(d=96), UNS), (dict(page_size=4112), UNS), (dict(heads=4097), UNS), (dict(pages=2 ** 31), UNS), (dict(data=P + 8), MIS)])
def test_cache_refuses(c, status):
    c = cache(**c)
    assert dg.kv4_append(c, 4, P, 256, P, 256, P, stream=0, check=False) == status
    assert dg.kv4_gather(c, 4, P, P, 256, P, 256, stream=0, check=False) == status
    assert dg.attention_kv4(c, 1, 1, 2, 1.0, P, 256, 256, P, 1, P, P, 256, 256, P, 1 << 40, stream=0, check=False) == status


@pytest.mark.parametrize("a,status", [
    ((-1, P, 256, P, 256, P), INV), ((4, None, 256, P, 256, P), INV), ((4, P, 255, P, 256, P), INV),
    ((4, P, 256, None, 256, P), INV), ((4, P, 256, P, 255, P), INV), ((4, P, 256, P, 256, None), INV),
    ((4, P + 1, 256, P, 256, P), MIS), ((4, P, 256, P, 256, P + 4), MIS), ((2 ** 31, P, 256, P, 256, P), UNS),
    ((0, None, 0, None, 0, None), dg.DG_OK)])
def test_rows_refuse(a, status):
    tokens, k, ldk, v, ldv, slots = a
    assert dg.kv4_append(cache(), tokens, k, ldk, v, ldv, slots, stream=0, check=False) == status
    assert dg.kv4_gather(cache(), tokens, slots, k, ldk, v, ldv, stream=0, check=False) == status


ATTN = dict(batch=3, Lq=2, heads_q=8, scale=0.1, Q=P, ldq=1024, strideQ=2048, page_table=P, ldt=4, lens=P, O=P, ldo=1024,
            strideO=2048, workspace=P, workspace_bytes=1 << 40)


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), INV), (dict(Lq=-1), INV), (dict(heads_q=-8), INV), (dict(heads_q=7), INV), (dict(ldt=-1), INV),
    (dict(scale=0.0), INV), (dict(scale=float("inf")), INV), (dict(scale=float("nan")), INV), (dict(Q=None), INV),
    (dict(O=None), INV), (dict(lens=None), INV), (dict(page_table=None), INV), (dict(ldq=1016), INV), (dict(ldo=1016), INV),
    (dict(strideQ=2040), INV), (dict(strideO=2040), INV), (dict(workspace=None), INV), (dict(workspace_bytes=0), INV),
    (dict(Q=P + 8), MIS), (dict(O=P + 8), MIS), (dict(ldq=1028, strideQ=4096), MIS), (dict(strideO=2052), MIS), (dict(lens=P + 2), MIS),
    (dict(page_table=P + 2), MIS), (dict(workspace=P + 16), MIS), (dict(ldt=2 ** 27), UNS),
    (dict(batch=65537), UNS), (dict(batch=65536, Lq=65536, strideQ=65536 * 1024, strideO=65536 * 1024), UNS),
    (dict(batch=0), dg.DG_OK), (dict(Lq=0), dg.DG_OK), (dict(heads_q=0), dg.DG_OK)])
def test_attention_refuses(change, status):
    assert dg.attention_kv4(cache(), *{**ATTN, **change}.values(), stream=0, check=False) == status


def test_attention_workspace():
    need = dg.dg_attention_kv4_workspace_bytes(3, 2, 8, 2, 128)
    assert need > 0
    assert dg.attention_kv4(cache(), *{**ATTN, "workspace_bytes": need - 1}.values(), stream=0, check=False) == INV
    for bad in [(0, 2, 8, 2, 128), (3, 0, 8, 2, 128), (3, 2, 0, 2, 128), (3, 2, 8, 0, 128), (3, 2, 8, 3, 128), (3, 2, 8, 2, 80)]:
        assert dg.dg_attention_kv4_workspace_bytes(*bad) == 0
    assert dg.dg_kv4_block_bytes(32, 128) == 32 * 136 and dg.dg_kv4_block_bytes(48, 64) == 48 * 72
    for bad in [(0, 128), (24, 128), (-16, 128), (32, 96)]:
        assert dg.dg_kv4_block_bytes(*bad) == 0


MOE = dict(T=4, K=64, I=32, E=8, top=2, renorm=True, X=P, ldx=64, logits=P, ldl=8, Wg=P, ldwg=32, strideWg=2048, Wu=P, ldwu=32,
           strideWu=2048, Wd=P, ldwd=64, strideWd=2048, Y=P, ldy=64, workspace=P, workspace_bytes=1 << 40)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INV), (dict(K=-1), INV), (dict(I=-1), INV), (dict(E=0), INV), (dict(top=0), INV), (dict(top=9), INV), (dict(I=0), INV),
    (dict(X=None), INV), (dict(logits=None), INV), (dict(Wg=None), INV), (dict(Wu=None), INV), (dict(Wd=None), INV),
    (dict(Y=None), INV), (dict(ldx=56), INV), (dict(ldl=7), INV), (dict(ldwg=24), INV), (dict(ldwu=24), INV), (dict(ldwd=56), INV),
    (dict(ldy=63), INV), (dict(strideWg=2040), INV), (dict(strideWu=2040), INV), (dict(strideWd=2040), INV),
    (dict(workspace=None), INV), (dict(workspace_bytes=0), INV), (dict(T=65), UNS), (dict(top=17, E=32, ldl=32), UNS),
    (dict(E=513, ldl=513), UNS), (dict(X=P + 8), MIS), (dict(Wg=P + 8), MIS), (dict(Wu=P + 2), MIS), (dict(Wd=P + 4), MIS),
    (dict(ldx=65), MIS), (dict(ldwg=36, strideWg=4096), MIS), (dict(strideWd=2052), MIS), (dict(Y=P + 1), MIS),
    (dict(workspace=P + 128), MIS), (dict(logits=P + 2), MIS), (dict(T=0), dg.DG_OK), (dict(K=0), dg.DG_OK)])
def test_moe_refuses(change, status):
    assert dg.moe_bf16(*{**MOE, **change}.values(), stream=0, check=False) == status


def test_moe_workspace():
    need = dg.dg_moe_workspace_bytes(4, 64, 32, 8, 2)
    assert need > 0
    assert dg.moe_bf16(*{**MOE, "workspace_bytes": need - 1}.values(), stream=0, check=False) == INV
    for bad in [(0, 64, 32, 8, 2), (4, 0, 32, 8, 2), (4, 64, 0, 8, 2), (4, 64, 32, 0, 2), (4, 64, 32, 8, 0), (4, 64, 32, 8, 9)]:
        assert dg.dg_moe_workspace_bytes(*bad) == 0


# ------------------------------------------------------------------ the oracle's pins
def test_norm_closed_forms():
    x = np.full((2, 4), 3.0, np.float32)
    h, y = ref.rmsnorm(x, None, np.array([1, 2, 3, 4], np.float32), 0.0)
    assert np.array_equal(h, x) and np.allclose(y, [[1, 2, 3, 4]] * 2, rtol=1e-15)
    h, y = ref.rmsnorm(x, -x, np.ones(4, np.float32), 1e-5)
    assert not h.any() and not y.any()
    v, s = ref.rmsnorm_codes(np.array([[1.0, -10.0, 0.0], [0.0, 0.0, 0.0]]))
    assert np.allclose(v, [[44.8, -448, 0], [0, 0, 0]]) and np.allclose(s, [10 / 448, 0])
    # A row of one size and its negative halves: mean of squares 2.5.
    assert np.allclose(ref.rmsnorm(np.array([[1.0, 2.0]], np.float32), None, np.ones(2, np.float32), 0.0)[1],
                       np.array([[1, 2]]) / np.sqrt(2.5))


def test_kv4_row_by_hand():
    # 0..15: scale 1, the codes are the values; a row of -2 and 5.5: scale 0.5, codes 0 and 15.
    c, s, z = ref.kv4_quantise(np.arange(16, dtype=np.float32)[None])
    assert c.tolist() == [list(range(16))] and s[0] == 1 and z[0] == 0
    c, s, z = ref.kv4_quantise(np.array([[-2.0, 5.5, 0.25, 0.0]], np.float32))
    assert c.tolist() == [[0, 15, 4, 4]] and s[0] == 0.5 and z[0] == -2.0  # 4.5 goes to the even 4
    c, s, z = ref.kv4_quantise(np.full((1, 8), -7.0, np.float32))
    assert not c.any() and s[0] == 0 and z[0] == -7 and np.all(ref.kv4_value(c, s, z) == -7)


def test_kv4_step_bounds_the_error():
    x = ref.bf16(np.random.default_rng(1).standard_normal((200, 128)))
    c, s, z = ref.kv4_quantise(x)
    # Half a step, and the scale's own rounding over 15 steps.
    assert np.all(np.abs(ref.kv4_value(c, s, z) - x) <= s[:, None] * (0.5 + 16 * ref.BF16))


def test_kv4_layout_by_hand():
    p = ref.Kv4Pool(2, 32, 2, 64)
    p.codes[1, 32 + 16 + 11, 1, 13] = 9     # page 1, record 1, token 11 of the record, column 13
    b = p.pack()
    # Group 1 (columns 8-15), token 11: half 1, pair 1, odd; column 13 is the second of piece 1.
    at = 16 * 72 + 8 * 64 + (((1 * 8 + 1) * 4 + 1) * 2 + 1) * 4 + 2 + 0
    assert b[1, 1, at] == 9 << 4 and np.count_nonzero(b) == 1
    p = ref.Kv4Pool(1, 16, 1, 128)
    p.scale[0, 3], p.zero[1, 3] = 1.0, -2.0
    b = p.pack()[0, 0]
    assert b[16 * 128 + 12:16 * 128 + 16].tolist() == [0x80, 0x3F, 0, 0]
    assert b[16 * 128 + 76:16 * 128 + 80].tolist() == [0, 0, 0, 0xC0] and b.size == 16 * 136


def test_attention_closed_forms():
    rng = np.random.default_rng(2)
    p = ref.Kv4Pool(4, 16, 1, 64)
    k, v = ref.bf16(rng.standard_normal((40, 1, 64))), ref.bf16(rng.standard_normal((40, 1, 64)))
    p.append(k, v, np.arange(40))
    table, lens = np.array([[0, 1, 2, -1]]), np.array([40])
    q = np.zeros((1, 3, 2, 64))
    o, _ = ref.kv4_attention(p, q, table, lens, 1.0)
    rows = p.rows(1, np.arange(40))[:, 0]
    for i in range(3):  # query 0: the mean over the keys that each query sees
        assert np.allclose(o[0, i, 0], rows[:38 + i].mean(0), rtol=1e-12)
    q[0, 2, 1] = 100 * p.rows(0, np.array([7]))[0, 0]
    o, _ = ref.kv4_attention(p, q, table, lens, 1.0)
    best = np.argmax(p.rows(0, np.arange(40))[:, 0] @ q[0, 2, 1])
    assert np.allclose(o[0, 2, 1], rows[best])
    o, _ = ref.kv4_attention(p, q[:, :], table, np.array([2]), 1.0)  # the first query sees nothing
    assert not o[0, 0].any() and np.allclose(o[0, 1, 0], rows[0])


def test_attention_bound_rejects_a_planted_mistake():
    rng = np.random.default_rng(3)
    p = ref.Kv4Pool(4, 16, 1, 64)
    p.append(ref.bf16(rng.standard_normal((50, 1, 64))), ref.bf16(rng.standard_normal((50, 1, 64))), np.arange(50))
    q = ref.bf16(rng.standard_normal((1, 1, 4, 64))).astype(np.float64)
    table = np.array([[0, 1, 2, 3]])
    o, bound = ref.kv4_attention(p, q, table, np.array([50]), 0.125)
    for wrong in (ref.kv4_attention(p, q, table, np.array([49]), 0.125)[0],       # the last key lost
                  ref.kv4_attention(p, q, table[:, [0, 2, 1, 3]], np.array([50]), 0.125)[0] * 1.03,
                  ref.kv4_attention(p, q, table, np.array([50]), 0.12)[0]):       # another scale
        assert np.any(np.abs(wrong - o) > bound)


def test_moe_closed_forms():
    assert ref.moe_route([[1.0, 3.0, 3.0, 0.0]], 2, True) == [[(1, 0.5), (2, 0.5)]]      # a tie: the lowest first
    assert [e for e, _ in ref.moe_route([[2.0, 2.0, 2.0]], 2, False)[0]] == [0, 1]
    assert np.allclose([w for _, w in ref.moe_route([[2.0, 2.0, 2.0]], 2, False)[0]], 1 / 3)
    assert ref.moe_route([[-np.inf, np.nan]], 1, True) == [[]]
    assert ref.moe_route([[-np.inf, 5.0]], 2, True) == [[(1, 1.0)]]
    x = np.array([[1.0, 2.0]], np.float32)
    wg, wu, wd = (np.zeros((2, 2, 2), np.float32) for _ in range(3))
    wg[1], wu[1], wd[1] = np.eye(2), np.eye(2), np.eye(2)
    y, _ = ref.moe(x, [[0.0, 9.0]], wg, wu, wd, 1, True)
    assert np.allclose(y, x * x / (1 + np.exp(-x)))
    y, _ = ref.moe(x, [[9.0, 0.0]], wg, wu, wd, 1, True)
    assert not y.any()


def test_moe_bound_rejects_a_planted_mistake():
    rng = np.random.default_rng(4)
    x = ref.bf16(rng.standard_normal((3, 64)))
    wg, wu = (ref.bf16(rng.standard_normal((4, 64, 40)) / 8) for _ in range(2))
    wd = ref.bf16(rng.standard_normal((4, 40, 64)) / 6)
    logits = rng.standard_normal((3, 4))
    y, bound = ref.moe(x, logits, wg, wu, wd, 2, True)
    for wrong in (ref.moe(x, logits, wg, wu, wd, 2, False)[0], ref.moe(x, logits, wu, wg, wd, 2, True)[0],
                  ref.moe(x, logits, wg[:, :, :39], wu[:, :, :39], wd[:, :39], 2, True)[0]):
        assert np.any(np.abs(wrong - y) > bound)
