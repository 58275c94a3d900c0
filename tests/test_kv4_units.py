"""What the tests of the 4-bit cache stand on (no GPU): the rows that make each unit of keys visible,
so that a lost, doubled or stale unit is seen, and the packing of whole pools."""
import numpy as np
import pytest

from oracle import serving as ref


@pytest.mark.parametrize("n,d", [(6000, 128), (9000, 64), (20000, 64), (20000, 128), (33000, 128), (700, 64)])
@pytest.mark.parametrize("turn", [1, 5])
def test_every_unit_counts(n, d, turn):
    rows = ref.unit_rows(n, d, turn)
    assert np.all(rows.sum(1) == 1)
    want, bound = ref.unit_mean(rows, n)
    other = ref.unit_rows(n, d, 6 - turn)
    assert np.all((rows * other).sum(1) == 0)                 # every unit is dealt to another column
    s = float(ref.bf16(np.float32(1) / np.float32(15))[0])
    for at in range(0, n, 32):
        one = rows[at:at + 32].astype(np.float64).sum(0) * 15 * s / n
        if n - at < 32:
            continue                                          # the last may be a few keys
        stale = other[at:at + 32].astype(np.float64).sum(0) * 15 * s / n
        for wrong in (want - one, want + one, want - one + stale, (want - one) * n / (n - 32)):
            assert np.any(np.abs(wrong - want) > 2 * bound), at
    # A share of one CTA, and of one warp, in a sequence cut over all of them.
    for keys in (n // 152 // 32 * 32 + 32, 64):
        for at in range(0, n - keys, keys):
            lost = rows[at:at + keys].astype(np.float64).sum(0) * 15 * s / n
            assert np.any(lost > 2 * bound)
            assert np.any(np.abs((want - lost) * n / (n - keys) - want) > 2 * bound)


def test_the_oracle_agrees():
    pool = ref.Kv4Pool(20, 16, 1, 64)
    rows = ref.unit_rows(300, 64, 1)
    pool.append(np.random.default_rng(0).standard_normal((300, 1, 64)).astype(np.float32), rows[:, None], np.arange(300))
    o, _ = ref.kv4_attention(pool, np.zeros((1, 3, 1, 64)), np.arange(20)[None], [300], 1.0)
    for i in range(3):
        assert np.allclose(o[0, i, 0], ref.unit_mean(rows, 298 + i)[0], rtol=1e-12)


@pytest.mark.parametrize("pages,page_size,heads,d", [(3, 16, 1, 64), (2, 48, 3, 128), (1, 64, 2, 64)])
def test_pools_packed_at_once(pages, page_size, heads, d):
    rng = np.random.default_rng(pages)
    pool = ref.Kv4Pool(pages, page_size, heads, d)
    pool.codes[:] = rng.integers(0, 16, pool.codes.shape)
    pool.scale[:], pool.zero[:] = (ref.bf16(rng.standard_normal(pool.scale.shape)) for _ in range(2))
    assert np.array_equal(pool.pack_all(), pool.pack())
