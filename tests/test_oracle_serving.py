"""The serving oracle against closed forms and hand-made examples (no GPU)."""

import math

import numpy as np

from oracle.serving import attention_bound, attention_ref, lse_bound, paged_plan_ref


def test_plan_by_hand():
    # pages of 4; request 0 has 3 tokens in page 7 and brings 2 (one starts a page), request 1 is new and
    # brings 5 (two pages, of which the free list has one left), request 2 brings nothing
    cu, lens, pos, slots, table, taken, missing = paged_plan_ref([3, 0, 8], [2, 5, 0], [[7, 9], [9, 9], [5, 6]], [11, 12, 13], 1, 9, 4)
    assert cu.tolist() == [0, 2, 7, 7] and lens.tolist() == [5, 5, 8]
    assert pos.tolist() == [3, 4, 0, 1, 2, 3, 4, -1, -1]
    assert slots.tolist() == [31, 48, 52, 53, 54, 55, -1, -1, -1]
    assert table.tolist() == [[7, 12], [13, -1], [5, 6]] and (taken, missing) == (3, 1)


def test_attention_of_one_key_is_its_value():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((1, 4, 8)), rng.standard_normal((1, 2, 8)), rng.standard_normal((1, 2, 8))
    out, lse, spread, size = attention_ref(q, k, v, 0, 0.3)
    assert np.allclose(out[0], v[0][[0, 0, 1, 1]]) and np.allclose(spread, np.abs(out))
    assert np.allclose(lse[0], [0.3 * q[0, h] @ k[0, h // 2] for h in range(4)])


def test_attention_of_equal_scores_is_the_mean_of_what_is_seen():
    v = np.arange(12, dtype=float).reshape(6, 1, 2)
    out, lse, _, _ = attention_ref(np.zeros((3, 1, 2)), np.ones((6, 1, 2)), v, 3, 1.0)
    for i in range(3):
        assert np.allclose(out[i, 0], v[:4 + i, 0].mean(0)) and math.isclose(lse[i, 0], math.log(4 + i))
    out, lse, _, _ = attention_ref(np.zeros((3, 1, 2)), np.ones((6, 1, 2)), v, 3, 1.0, window=2)
    for i in range(3):
        assert np.allclose(out[i, 0], v[2 + i:4 + i, 0].mean(0)) and math.isclose(lse[i, 0], math.log(2))


def test_attention_against_a_dense_softmax():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((5, 3, 16)), rng.standard_normal((9, 3, 16)), rng.standard_normal((9, 3, 16))
    out, lse, _, _ = attention_ref(q, k, v, 4, 0.25)
    x = np.einsum("ihd,jhd->hij", q, k) * 0.25
    x = np.where(np.arange(9) <= 4 + np.arange(5)[:, None], x, -np.inf)
    p = np.exp(x)
    assert np.allclose(out, np.einsum("hij,jhd->ihd", p / p.sum(-1, keepdims=True), v))
    assert np.allclose(lse, np.log(p.sum(-1)).T)


def test_rows_without_keys():
    out, lse, spread, size = attention_ref(np.ones((3, 1, 2)), np.ones((1, 1, 2)), np.ones((1, 1, 2)), -2, 1.0)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and (out[2] == 1).all()


def test_masked_values_never_enter():
    k, v = np.ones((4, 1, 2)), np.ones((4, 1, 2))
    k[3], v[2:] = np.nan, np.inf
    out, lse, _, _ = attention_ref(np.ones((2, 1, 2)), k, v, 0, 1.0)
    assert (out == 1).all() and np.isfinite(lse).all()


def test_bounds_cover_the_roundings_they_name():
    """Weights and result rounded to 16 bits in a float32 computation stay inside; a key left out does not."""
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal(s).astype(np.float16) for s in ((4, 2, 64), (300, 2, 64), (300, 2, 64)))
    ref = attention_ref(q.astype(float), k.astype(float), v.astype(float), 296, 0.125)
    bound = attention_bound(ref[0], ref[2], ref[3], 300, 64, "f16", float(np.abs(v).max()))
    for drop in (0, 1):
        for i in range(4):
            for h in range(2):
                n = 297 + i - drop * 40
                s = (k[:n, h].astype(np.float32) @ q[i, h].astype(np.float32)) * np.float32(0.125)
                p = np.exp(s - s.max())
                o = (p.astype(np.float16).astype(np.float32) @ v[:n, h].astype(np.float32) / p.sum()).astype(np.float16)
                inside = (np.abs(o - ref[0][i, h]) <= bound[i, h]).all()
                assert inside == (drop == 0)
                if not drop:
                    assert abs(s.max() + np.log(p.sum()) - ref[1][i, h]) <= lse_bound(ref[1], ref[3], 300, 64)[i, h]
