"""The serving operators' limits without a GPU: sizes that are refused have no workspace, and no
check multiplies sizes or strides that overflow."""
import pytest

import dense_gemm_sm_gb300 as dg

P = 0x10000  # an aligned address that no refused call reaches
BIG = 1 << 40
INV, UNS = dg.DG_ERR_INVALID_ARG, dg.DG_ERR_UNSUPPORTED


@pytest.mark.parametrize("sizes", [
    (65537, 1, 8, 8, 128), (1, 65537, 8, 8, 128), (1, 1, 131072, 1, 128), (65536, 65536, 8, 8, 128), (1, 1, 8192, 8192, 64),
    (1 << 40, 1 << 40, 8, 8, 64), (1, 1 << 62, 8, 1, 64), (1, 1, 1 << 62, 1, 64)])
def test_attention_sizes_that_have_no_workspace(sizes):
    batch, lq, hq, hkv, d = sizes
    assert dg.dg_attention_kv4_workspace_bytes(*sizes) == 0
    if hkv <= 4096:
        cache = dg.dg_kv4_cache(P, 8, 16, hkv, d)
        assert dg.attention_kv4(cache, batch, lq, hq, 1.0, P, BIG, BIG, P, 1, P, P, BIG, BIG, P, BIG, stream=0, check=False) == UNS


def test_a_page_size_that_the_cache_does_not_have_has_no_block():
    assert dg.dg_kv4_block_bytes(4096, 128) == 4096 * 136
    assert dg.dg_kv4_block_bytes(4112, 128) == 0 and dg.dg_kv4_block_bytes(2 ** 31 - 16, 64) == 0


@pytest.mark.parametrize("sizes", [
    (1, 64, 64, 513, 2), (1, 2 ** 31, 64, 2, 1), (1, 64, 2 ** 31, 2, 1), (1, 2 ** 31 - 1, 2 ** 31 - 1, 2, 1), (65, 64, 64, 8, 2),
    (1, 64, 64, 32, 17), (1, 1 << 62, 1 << 62, 8, 2), (1 << 62, 64, 64, 8, 2), (1, 64, 64, 1 << 62, 2)])
def test_expert_sizes_that_have_no_workspace(sizes):
    T, K, I, E, top = sizes
    assert dg.dg_moe_workspace_bytes(*sizes) == 0
    w = (1 << 62) + (1 << 40)
    assert dg.moe_bf16(T, K, I, E, top, True, P, w, P, w, P, w, w, P, w, w, P, w, w, P, w, P, BIG, stream=0, check=False) == UNS


# (Lq - 1) ld = 2^63, K ld = 2^64 and the like: as products they come out negative or 0.
@pytest.mark.parametrize("name", ["Q", "O"])
def test_attention_strides_that_overflow(name):
    ld, span = {"Q": 1024, "O": 1024}, {"Q": 1 << 30, "O": 1 << 30}
    ld[name] = 1 << 50
    cache = dg.dg_kv4_cache(P, 8, 16, 8, 128)
    assert dg.attention_kv4(cache, 2, 8193, 8, 1.0, P, ld["Q"], span["Q"], P, 1, P, P, ld["O"], span["O"], P, BIG, stream=0,
                            check=False) == INV


@pytest.mark.parametrize("which", [0, 1, 2])
def test_expert_strides_that_overflow(which):
    K = I = 64
    ld = [64, 64, 64]
    ld[which] = 1 << 58
    args = []
    for n in ld:
        args += [P, n, 1 << 30]
    assert dg.moe_bf16(1, K, I, 8, 2, True, P, K, P, 8, *args, P, K, P, BIG, stream=0, check=False) == INV
