"""Pins of the attention oracle: small cases by hand, and its parts against each other."""
import numpy as np
import pytest

from oracle import attention as OA


def cache(seed, n_pages, page, hkv, d):
    rng = np.random.default_rng(seed)
    return rng.standard_normal((n_pages, page, hkv, d)), rng.standard_normal((n_pages, page, hkv, d)), rng


def test_turn_by_a_quarter():
    cos_sin = np.array([[1.0, 1.0, 0.0, 0.0], [0.0, 0.0, 1.0, 1.0]])  # rot 4: angles 0 and pi / 2
    x = np.array([1.0, 2.0, 3.0, 4.0, 5.0])
    assert np.array_equal(OA.turn(x, cos_sin, 0), x)
    assert np.array_equal(OA.turn(x, cos_sin, 1), [-3.0, -4.0, 1.0, 2.0, 5.0])
    assert np.array_equal(OA.turn(x, cos_sin, 1, interleaved=True), [-2.0, 1.0, -4.0, 3.0, 5.0])


def test_turned_scores_depend_on_the_distance_alone():
    rng = np.random.default_rng(1)
    angle = np.arange(40)[:, None] * 100.0 ** (-np.arange(4) / 4)
    cos_sin = np.concatenate([np.cos(angle), np.sin(angle)], axis=1)
    q, k = rng.standard_normal(8), rng.standard_normal(8)
    for inter in (False, True):
        a = OA.turn(q, cos_sin, 9, inter) @ OA.turn(k, cos_sin, 4, inter)
        b = OA.turn(q, cos_sin, 35, inter) @ OA.turn(k, cos_sin, 30, inter)
        assert a == pytest.approx(b, abs=1e-12)


def test_one_visible_slot_returns_its_value():
    k, v, rng = cache(2, 3, 4, 1, 8)
    q = rng.standard_normal((1, 2, 8))
    o = OA.attend(q, k, v, [[2]], [0])
    assert np.allclose(o[0], v[2, 0, 0])


def test_decode_is_attend_of_one_token_and_chains_are_causal():
    k, v, rng = cache(3, 6, 4, 2, 8)
    table, lens = [[5, 0, 2], [1, 3, 4]], [6, 3]
    q = rng.standard_normal((2, 4, 8))
    assert np.allclose(OA.attend(q, k, v, table, lens, scale=0.3), OA.attend(q, k, v, table, lens, [0, 1, 2], np.array([[1], [1]]), 0.3))
    q = rng.standard_normal((7, 4, 8))
    chain = np.array([[(2 << i) - 1] for i in (0, 1, 2, 3, 0, 1, 2)])
    assert np.allclose(OA.attend(q, k, v, table, lens, [0, 4, 7], None), OA.attend(q, k, v, table, lens, [0, 4, 7], chain))


def test_empty_rows_and_unused_requests_are_zero():
    k, v, rng = cache(4, 2, 4, 1, 8)
    q = rng.standard_normal((3, 1, 8))
    o = OA.attend(q, k, v, [[0], [1]], [0, -1], [0, 2, 3], np.array([[0], [2], [1]]))
    assert not o[0].any() and o[1].any() and not o[2].any()


def test_a_commit_then_decode_sees_the_accepted_path():
    # attending from a tree's leaf under its mask is attending after its path has been committed
    k, v, rng = cache(5, 4, 4, 1, 8)
    table, path = [[3, 1, 0, 2]], [0, 2, 5]
    mask = np.zeros((6, 1), dtype=np.int64)
    mask[5] = sum(1 << j for j in path)
    q = rng.standard_normal((6, 1, 8))
    before = OA.attend(q, k, v, table, [7], [0, 6], mask)[5]
    kc, vc, new = OA.commit(k, v, table, [7], [0, 3], path)
    assert new.tolist() == [10]
    assert np.allclose(OA.attend(q[5:], kc, vc, table, [9])[0], before)


def test_append_places_depths_and_leaves_the_rest():
    k, v, rng = cache(6, 3, 2, 1, 4)
    x = rng.standard_normal((3, 1, 4))
    angle = np.arange(9)[:, None] * np.array([1.0, 0.1])
    cos_sin = np.concatenate([np.cos(angle), np.sin(angle)], axis=1)
    q, kc, vc = OA.append(x, x, x, k, v, [[2, 0, 1]], [1], [0, 3], depth=[1, 2, 2], cos_sin=cos_sin)
    where = [(2, 1), (0, 0), (0, 1)]
    for t, (page, row) in enumerate(where):
        assert np.allclose(kc[page, row], OA.turn(x[t], cos_sin, [1, 2, 2][t])) and np.array_equal(vc[page, row], x[t])
        assert np.allclose(q[t], kc[page, row])
    assert np.array_equal(kc[2, 0], k[2, 0]) and np.array_equal(kc[1], k[1])
