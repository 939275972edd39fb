"""Pins of the oracle's serving operators (no GPU): the latent attention against
the numpy definition and closed forms, the merge against one softmax over the
whole, the block copies against numpy indexing."""
import numpy as np
import pytest

import refattn as R


def run(orc, pg, q, cu, kv, causal=True, scale=R.SCALE):
    return orc.latent_attention(q, pg.cache, pg.fmt, pg.num_blocks, pg.block, pg.block_stride,
                                pg.entry_stride, pg.table, np.asarray(cu, np.int32),
                                np.asarray(kv, np.int32), scale,
                                1.0 if pg.k_scale is None else float(np.float32(pg.k_scale)), causal)


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_matches_the_numpy_definition(orc, fmt, causal):
    kv, cu = [37, 5, 0, 3], [0, 4, 5, 6, 11]  # the last has more new tokens than rows
    pg = R.paged(kv, fmt, 16, pad_entry=16, pad_block=32)
    q = R.queries(12, 3)
    out, lse, err = run(orc, pg, q, cu, kv, causal)
    r = R.attention(pg, q, cu, kv, causal=causal)
    ro, rl = r.out, r.lse
    assert err == 0
    np.testing.assert_allclose(out[:11], ro[:11], rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(lse[:11], rl[:11], rtol=1e-12)
    assert np.isnan(out[11]).all() and np.isnan(lse[11]).all()
    assert (out[5] == 0).all() and np.isneginf(lse[5]).all()
    if causal:
        assert (out[6:8] == 0).all() and np.isneginf(lse[6:8]).all()


def test_attention_closed_forms(orc):
    pg = R.paged([40], 0, 16)
    rows, _ = R.rows_of(pg, 0, 40)
    q = np.zeros((1, 2, R.ENTRY), np.uint16)  # zero query: the plain mean, lse = ln n
    out, lse, _ = run(orc, pg, q, [0, 1], [40])
    np.testing.assert_allclose(out[0, 1], rows[:, :R.RANK].mean(0), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(lse, np.log(40.0))
    q = R.queries(1, 1)  # one row: itself, lse = its score
    out, lse, _ = run(orc, pg, q, [0, 1], [1])
    np.testing.assert_array_equal(out[0, 0], rows[0, :R.RANK])
    np.testing.assert_allclose(lse[0, 0], R.SCALE * (orc.bf16_bits_to_f64(q[0, 0]) @ rows[0]))


def test_attention_leaves_out_rows_without_a_block(orc):
    pg = R.paged([40], 1, 16)
    pg.table[0, 1] = pg.num_blocks
    q = R.queries(1, 2)
    out, lse, err = run(orc, pg, q, [0, 1], [40])
    r = R.attention(pg, q, [0, 1], [40])
    ro, rl = r.out, r.lse
    assert err == 2
    np.testing.assert_allclose(out, ro, rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(lse, rl, rtol=1e-12)


def test_merge_of_parts_is_the_whole(orc):
    rng = np.random.default_rng(3)
    x, v = rng.standard_normal((2, 3, 60)) * 4, rng.standard_normal((60, 8))
    cuts = [0, 1, 17, 60]
    parts, lses = [], []
    for a, b in zip(cuts, cuts[1:]):
        w = np.exp(x[..., a:b])
        parts.append(w @ v[a:b] / w.sum(-1, keepdims=True))
        lses.append(np.log(w.sum(-1)))
    parts.append(np.full_like(parts[0], np.nan))  # an empty part does not count
    lses.append(np.full_like(lses[0], -np.inf))
    out, lse = orc.merge_attn_states(np.stack(parts), np.stack(lses))
    w = np.exp(x)
    np.testing.assert_allclose(out, w @ v / w.sum(-1, keepdims=True), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(lse, np.log(w.sum(-1)), rtol=1e-13)
    out, lse = orc.merge_attn_states(np.stack(parts)[3:], np.stack(lses)[3:])
    assert (out == 0).all() and np.isneginf(lse).all()


@pytest.mark.parametrize("esz", [1, 2])
def test_copy_blocks_against_numpy(orc, esz):
    nb, bs, es, ed = 9, 4, 40, 32
    bst = bs * es + 16
    rng = np.random.default_rng(5)
    caches = [rng.integers(0, 255, nb * bst).astype(np.uint8 if esz == 1 else np.uint16)
              for _ in range(2)]
    ref = [c.copy().reshape(nb, bst) for c in caches]
    src = np.array([3, 3, -1, 1, 2, 99, 0], np.int32)
    dst = np.array([5, 6, 7, -1, 4, 8, 8], np.int32)
    cnt = np.array([4, 2, 3, 4, 0, 1, 5], np.int32)
    err = orc.copy_blocks(caches, esz, nb, bs, bst, es, ed, src, dst, cnt)
    assert err == 2
    for r in ref:
        e = r[:, :bs * es].reshape(nb, bs, es)
        e[5, :4, :ed] = e[3, :4, :ed]
        e[6, :2, :ed] = e[3, :2, :ed]
        e[7, :3, :ed] = 0
    for c, r in zip(caches, ref):
        np.testing.assert_array_equal(c.reshape(nb, bst), r)


def test_copy_blocks_of_no_rows_are_padding(orc):
    """A count of 0 is padding whatever the ids are; equal ids out of range are reported."""
    i = lambda *v: np.array(v, np.int32)
    cache = np.arange(4 * 2 * 32, dtype=np.uint8)
    ref = cache.copy()
    args = (1, 4, 2, 64, 32, 32)
    assert orc.copy_blocks([cache], *args, i(99, 0, -9), i(1, 99, -9), i(0, 0, 0)) == 0
    assert orc.copy_blocks([cache], *args, i(99), i(99), i(1)) == 2
    assert orc.copy_blocks([cache], *args, i(1), i(1), i(2)) == 0
    np.testing.assert_array_equal(cache, ref)
