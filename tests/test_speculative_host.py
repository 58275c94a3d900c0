"""The operators of a speculative decoding step without a GPU: refused arguments, sizes without a
workspace, and the oracle's own pins."""
import numpy as np
import pytest

import dense_gemm_sm_gb300 as dg
from oracle import serving as ref

P = 0x10000  # an aligned address that no refused call reaches
BIG = 1 << 40
INV, MIS, UNS, OK = dg.DG_ERR_INVALID_ARG, dg.DG_ERR_MISALIGNED, dg.DG_ERR_UNSUPPORTED, dg.DG_OK


def cache(data=P, pages=8, page_size=32, heads=2, d=128):
    return dg.dg_kv4_cache(data, pages, page_size, heads, d)


BAD_CACHES = [(dict(pages=-1), INV), (dict(page_size=24), INV), (dict(heads=0), INV), (dict(data=None), INV), (dict(d=96), UNS),
              (dict(page_size=4112), UNS), (dict(heads=4097), UNS), (dict(pages=2 ** 31), UNS), (dict(data=P + 8), MIS)]

TREE = dict(batch=3, Lq=2, heads_q=8, scale=0.1, Q=P, ldq=1024, strideQ=2048, page_table=P, ldt=4, lens=P, nodes=P, mask=P, O=P, ldo=1024,
            strideO=2048, workspace=P, workspace_bytes=BIG)


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), INV), (dict(Lq=-1), INV), (dict(heads_q=-8), INV), (dict(heads_q=7), INV), (dict(ldt=-1), INV),
    (dict(scale=0.0), INV), (dict(scale=float("inf")), INV), (dict(scale=float("nan")), INV), (dict(Q=None), INV),
    (dict(O=None), INV), (dict(lens=None), INV), (dict(mask=None), INV), (dict(page_table=None), INV), (dict(ldq=1016), INV), (dict(ldo=1016), INV),
    (dict(strideQ=2040), INV), (dict(strideO=2040), INV), (dict(workspace=None), INV), (dict(workspace_bytes=0), INV),
    (dict(Q=P + 8), MIS), (dict(O=P + 8), MIS), (dict(ldq=1028, strideQ=4096), MIS), (dict(strideO=2052), MIS), (dict(lens=P + 2), MIS),
    (dict(nodes=P + 2), MIS), (dict(mask=P + 4), MIS), (dict(page_table=P + 2), MIS), (dict(workspace=P + 16), MIS), (dict(ldt=2 ** 27), UNS),
    (dict(batch=65537), UNS), (dict(Lq=65, strideQ=65 * 1024, strideO=65 * 1024), UNS), (dict(heads_q=131072, ldq=BIG, ldo=BIG, strideQ=4 * BIG, strideO=4 * BIG), UNS),
    (dict(batch=0), OK), (dict(Lq=0), OK), (dict(heads_q=0), OK), (dict(batch=0, mask=None), OK)])
def test_tree_refuses(change, status):
    assert dg.attention_kv4_tree(cache(), *{**TREE, **change}.values(), stream=0, check=False) == status


def test_tree_workspace_is_the_attention_s():
    need = dg.dg_attention_kv4_workspace_bytes(3, 2, 8, 2, 128)
    assert dg.attention_kv4_tree(cache(), *{**TREE, "workspace_bytes": need - 1}.values(), stream=0, check=False) == INV


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lq,hq,heads", [(17, 1, 1), (5, 8, 2), (64, 32, 8), (1, 68, 4)])
def test_workspace_has_room_for_every_tree(lq, hq, heads, d):
    # More than 16 query rows a cache head: two parts of 128 rows (outputs, reference and sum in FP32) and a
    # record of 32 bytes for each of 160 CTAs, behind 1024 bytes of counters.
    assert dg.dg_attention_kv4_workspace_bytes(3, lq, hq, heads, d) >= 1024 + 160 * (2 * 128 * (d + 2) * 4 + 32)


ACCEPT = dict(batch=3, Lq=4, page_table=P, ldt=4, lens=P, nodes=P, path=P, ldp=4, counts=P, new_lens=P)


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), INV), (dict(Lq=-1), INV), (dict(ldt=-1), INV), (dict(page_table=None), INV), (dict(lens=None), INV), (dict(path=None), INV),
    (dict(ldp=3), INV), (dict(counts=None), INV), (dict(new_lens=None), INV), (dict(page_table=P + 2), MIS), (dict(lens=P + 1), MIS),
    (dict(nodes=P + 2), MIS), (dict(path=P + 2), MIS), (dict(counts=P + 2), MIS), (dict(new_lens=P + 2), MIS), (dict(Lq=65, ldp=65), UNS),
    (dict(batch=65537), UNS), (dict(ldt=2 ** 27), UNS), (dict(batch=0), OK)])
def test_accept_refuses(change, status):
    assert dg.kv4_accept(cache(), *{**ACCEPT, **change}.values(), stream=0, check=False) == status


@pytest.mark.parametrize("n,src,dst,status", [(-1, P, P, INV), (2, None, P, INV), (2, P, None, INV), (2, P + 2, P, MIS), (2, P, P + 1, MIS),
                                              (2 ** 31, P, P, UNS), (0, None, None, OK)])
def test_copy_refuses(n, src, dst, status):
    assert dg.kv4_copy_pages(cache(), n, src, dst, stream=0, check=False) == status


@pytest.mark.parametrize("c,status", BAD_CACHES)
def test_caches_are_refused(c, status):
    c = cache(**c)
    assert dg.attention_kv4_tree(c, *TREE.values(), stream=0, check=False) == status
    assert dg.kv4_accept(c, *ACCEPT.values(), stream=0, check=False) == status
    assert dg.kv4_copy_pages(c, 2, P, P, stream=0, check=False) == status


ROWS = dict(N=10, K=100, group=64, W=P, ldw=104, Q=P, ldq=64, params=P, ldp=12)


@pytest.mark.parametrize("change,status", [
    (dict(N=-1), INV), (dict(K=-1), INV), (dict(group=0), INV), (dict(group=-32), INV), (dict(group=48), UNS), (dict(group=256), UNS), (dict(W=None), INV),
    (dict(ldw=99), INV), (dict(Q=None), INV), (dict(ldq=48), INV), (dict(ldq=-16), INV), (dict(params=None), INV), (dict(ldp=8), INV), (dict(W=P + 1), MIS),
    (dict(Q=P + 8), MIS), (dict(ldq=68), MIS), (dict(params=P + 4), MIS), (dict(ldp=13), MIS), (dict(N=(1 << 30) + 1, ldp=BIG), UNS),
    (dict(K=(1 << 30) + 1, ldw=BIG, ldq=BIG), UNS), (dict(N=0), OK), (dict(K=0), OK)])
def test_weight_rows_refuse(change, status):
    a = {**ROWS, **change}
    assert dg.quantize_groups_w4(*a.values(), stream=0, check=False) == status
    n, k, group, w, ldw, q, ldq, params, ldp = a.values()
    assert dg.dequantize_groups_w4(n, k, group, q, ldq, params, ldp, w, ldw, stream=0, check=False) == status


GEMM = dict(M=4, N=10, K=100, group=64, X=P, ldx=104, Q=P, ldq=64, params=P, ldp=12, C=P, ldc=10, c_type=dg.DG_OUT_F32, workspace=P, workspace_bytes=BIG)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), INV), (dict(N=-1), INV), (dict(K=-1), INV), (dict(group=0), INV), (dict(group=16), UNS), (dict(X=None), INV), (dict(ldx=96), INV),
    (dict(Q=None), INV), (dict(ldq=48), INV), (dict(params=None), INV), (dict(ldp=8), INV), (dict(C=None), INV), (dict(ldc=9), INV), (dict(c_type=5), INV),
    (dict(workspace=None), INV), (dict(workspace_bytes=0), INV), (dict(X=P + 8), MIS), (dict(ldx=101), MIS), (dict(Q=P + 8), MIS), (dict(ldq=72), MIS),
    (dict(params=P + 8), MIS), (dict(ldp=10), MIS), (dict(C=P + 2), MIS), (dict(workspace=P + 128), MIS), (dict(M=(1 << 30) + 1), UNS),
    (dict(N=(1 << 30) + 1, ldp=BIG, ldc=BIG), UNS), (dict(K=(1 << 30) + 1, ldx=BIG, ldq=BIG), UNS), (dict(M=0), OK), (dict(N=0), OK)])
def test_product_refuses(change, status):
    assert dg.gemm_w4_bf16(*{**GEMM, **change}.values(), stream=0, check=False) == status


def test_product_workspace():
    need = dg.dg_gemm_w4_workspace_bytes(4, 10, 100)
    assert need > 0
    assert dg.gemm_w4_bf16(*{**GEMM, "workspace_bytes": need - 1}.values(), stream=0, check=False) == INV
    # Units of 128 columns, 256 k and 64 rows are counted in 31 bits.
    assert dg.dg_gemm_w4_workspace_bytes(1, 1 << 30, 1 << 15) > 0
    for bad in [(1, 1 << 30, 1 << 17), (1 << 30, 1 << 30, 1 << 30), (0, 10, 100), (4, 0, 100), (4, 10, 0), (-1, 10, 100), (4, (1 << 30) + 1, 100), (1 << 62, 10, 100), (4, 10, 1 << 62)]:
        assert dg.dg_gemm_w4_workspace_bytes(*bad) == 0


# ------------------------------------------------------------------ the oracle's pins
def test_weights_by_hand():
    w = np.array([[0, 15, 7, 7.5, 7.25, 1, 2, 3, -1, -1]], np.float32)      # groups of 8: a full one, a constant one
    codes = np.concatenate([ref.kv4_quantise(w[:, :8])[0], ref.kv4_quantise(w[:, 8:])[0]], 1)
    assert codes.tolist() == [[0, 15, 7, 8, 7, 1, 2, 3, 0, 0]]              # halves to even
    packed = ref.w4_pack(codes, 16)
    # Word 0: even k (0, 7, 7, 2) in the low half, odd k (15, 8, 1, 3) in the high half, low bits first.
    assert packed[0, :4].tolist() == [0x70, 0x27, 0x8F, 0x31] and packed[0, 4:].tolist() == [0] * 12
    scale, zero = np.array([[1.0, 0.0]], np.float32), np.array([[0.0, -1.0]], np.float32)
    assert ref.w4_params(scale, zero, 4).tolist() == [[0x00003F80, 0, 0, 0], [0xBF800000, 0, 0, 0]]


def test_weights_are_their_values_times_rows():
    rng = np.random.default_rng(1)
    w = ref.bf16(rng.standard_normal((5, 100)).astype(np.float32))
    codes, scale, zero = ref.w4_quantise(w, 32)
    assert scale.shape == (5, 4)
    back = ref.w4_value(codes, scale, zero, 32)
    assert np.all(np.abs(back - w) <= 0.52 * scale[:, np.arange(100) // 32])
    c, bound = ref.w4_gemm(np.eye(100, dtype=np.float32), codes, scale, zero, 32, ref.F32)
    assert np.array_equal(c, back.T) and np.all(bound > 0)


def test_a_shifted_group_fails_the_product_s_bound():
    # The planted mistake: the parameters of the neighbouring group for one group of 32.
    rng = np.random.default_rng(2)
    w = ref.bf16(rng.standard_normal((20, 4096)).astype(np.float32))
    x = ref.bf16(rng.standard_normal((3, 4096)).astype(np.float32))
    codes, scale, zero = ref.w4_quantise(w, 32)
    c, bound = ref.w4_gemm(x, codes, scale, zero, 32, ref.BF16)
    scale[:, 50], zero[:, 50] = scale[:, 51], zero[:, 51]
    wrong, _ = ref.w4_gemm(x, codes, scale, zero, 32, ref.BF16)
    assert (np.abs(wrong - c) > bound).mean() > 0.5


def test_trees_by_hand():
    # 0 - 1 - 3, 0 - 2: lens 7, 4 nodes, 3 tokens of context.
    sees = ref.tree_sees([7], [4], [[0b1, 0b11, 0b101, 0b1011, 0]])
    assert [sees(0, i, 7).astype(int).tolist() for i in range(5)] == [
        [1, 1, 1, 1, 0, 0, 0], [1, 1, 1, 1, 1, 0, 0], [1, 1, 1, 1, 0, 1, 0], [1, 1, 1, 1, 1, 0, 1], [0] * 7]


def test_a_chain_sees_what_the_newest_tokens_see():
    rng = np.random.default_rng(3)
    pool = ref.Kv4Pool(3, 16, 1, 64)
    pool.append(ref.bf16(rng.standard_normal((48, 1, 64))), ref.bf16(rng.standard_normal((48, 1, 64))), np.arange(48))
    q = rng.standard_normal((1, 4, 2, 64))
    chain = ref.tree_sees([40], [4], [[1, 3, 7, 15]])
    a, _ = ref.kv4_attention(pool, q, [[0, 1, 2]], [40], 0.1)
    b, _ = ref.kv4_attention(pool, q, [[0, 1, 2]], [40], 0.1, chain)
    assert np.array_equal(a, b)
    # A node that its mask leaves out is past the bound somewhere, which is what fails a comparison.
    c, bound = ref.kv4_attention(pool, q, [[0, 1, 2]], [40], 0.1, ref.tree_sees([40], [4], [[1, 3, 7, 13]]))
    assert (np.abs(c - a)[0, 3] > bound[0, 3]).any() and np.array_equal(c[0, :3], a[0, :3])


def test_rows_move_as_if_at_once():
    pool = ref.Kv4Pool(1, 16, 1, 64)
    pool.codes[0, :, 0, 0] = np.arange(16)
    pool.move([1, 0, 5], [0, 1, 2])
    assert pool.codes[0, :, 0, 0].tolist() == [1, 0, 5] + list(range(3, 16))
