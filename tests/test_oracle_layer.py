"""Pins of the float64 definitions of the layer operators: the token recurrence against the
matrix form, against the tree oracle on a chain, and against itself cut into pieces; the norms
against hand-worked values."""
import numpy as np
import pytest

import oracle
from oracle import layer as OL
from gated_delta_net_gb300 import workloads as W


def _inputs(seed, T, hk=1, hv=2, dk=16, dv=32):
    rng = np.random.default_rng(seed)
    k = rng.standard_normal((T, hk, dk))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return (rng.standard_normal((T, hk, dk)), k, rng.standard_normal((T, hv, dv)), -rng.random((T, hv)),
            rng.random((T, hv)), 0.1 * rng.standard_normal((1, hv, dv, dk)))


@pytest.mark.parametrize("T", [1, 2, 7, 33])
def test_prefill_equals_the_matrix_form(T):
    q, k, v, g, beta, S0 = _inputs(T, T)
    o, S = OL.prefill(q, k, v, g, beta, [0, T], S0=S0, scale=0.5)
    for h in range(2):
        gam = np.cumsum(g[:, h])
        D = np.tril(np.exp(gam[:, None] - gam[None, :]))
        K, Q, V = k[:, 0], q[:, 0], v[:, h]
        X = np.tril(beta[:, h, None] * D * (K @ K.T), -1)
        rhs = beta[:, h, None] * (V - np.exp(gam)[:, None] * (K @ S0[0, h].T))
        U = np.linalg.solve(np.eye(T) + X, rhs)
        ref = 0.5 * (np.exp(gam)[:, None] * (Q @ S0[0, h].T) + np.tril(D * (Q @ K.T)) @ U)
        assert np.allclose(o[:, h], ref, rtol=1e-12, atol=1e-12)
        Sref = np.exp(gam[-1]) * S0[0, h] + (np.exp(gam[-1] - gam)[:, None] * U).T @ K
        assert np.allclose(S[0, h], Sref, rtol=1e-12, atol=1e-12)


def test_prefill_equals_the_tree_oracle_on_a_chain():
    tb = W.custom(3, [W.chain_tree(20)], n_k_heads=1, n_v_heads=2, d=16, qkv_dtype="f32", path_fn=W.path_deepest_leaf)
    o, S = OL.prefill(tb.q, tb.k, tb.v, tb.g, tb.beta, tb.node_offsets, S0=tb.S0)
    assert np.allclose(o, oracle.verify(tb), rtol=1e-12, atol=1e-12)
    assert np.allclose(S, oracle.commit(tb)[0], rtol=1e-12, atol=1e-12)


def test_prefill_in_pieces_and_by_single_tokens_is_the_whole():
    q, k, v, g, beta, S0 = _inputs(9, 12)
    o, S = OL.prefill(q, k, v, g, beta, [0, 12], S0=S0)
    o1, S1 = OL.prefill(q[:7], k[:7], v[:7], g[:7], beta[:7], [0, 7], S0=S0)
    o2, S2 = OL.prefill(q[7:], k[7:], v[7:], g[7:], beta[7:], [0, 5], S0=S1)
    assert np.array_equal(np.concatenate([o1, o2]), o) and np.array_equal(S2, S)
    pool = S0.copy()
    for t in range(12):
        ot, pool = OL.decode(q[t:t + 1], k[t:t + 1], v[t:t + 1], g[t:t + 1], beta[t:t + 1], pool)
        assert np.array_equal(ot[0], o[t])
    assert np.array_equal(pool, S)


def test_full_decay_forgets_and_zero_strength_only_decays():
    q, k, v, g, beta, S0 = _inputs(4, 3)
    g[1] = -np.inf
    _, S = OL.prefill(q, k, v, g, beta, [0, 3], S0=S0)
    _, S2 = OL.prefill(q[1:], k[1:], v[1:], g[1:], beta[1:], [0, 2])
    assert np.allclose(S, S2, rtol=1e-15, atol=0)
    _, S = OL.prefill(q[:1], k[:1], v[:1], g[:1], 0 * beta[:1], [0, 1], S0=S0)
    assert np.allclose(S[0], np.exp(g[0])[:, None, None] * S0[0], rtol=1e-15, atol=0)


def test_norms_by_hand():
    q, k, g, b = OL.qk_gates([[[3.0, 4.0]]], [[[0.0, 2.0]]], [[0.0]], [[0.0]], [np.log(2.0)], [0.0], 0.0)
    assert np.allclose(q, [[[0.6, 0.8]]]) and np.allclose(k, [[[0.0, 1.0]]])
    assert np.allclose(g, [[-2.0 * np.log(2.0)]]) and np.allclose(b, [[0.5]])
    y = OL.norm_gate([[[3.0, 4.0]]], [[[0.0, 1.0]]], [1.0, 2.0], 0.0)
    rms = np.sqrt(12.5)
    assert np.allclose(y, [[[0.0, 8.0 / rms / (1 + np.exp(-1.0))]]])
    h, n = OL.residual_norm([[1.0, 1.0]], [[3.0, 4.0]], [1.0, 1.0], 0.5, [2.0, 1.0], 0.0)
    assert np.allclose(h, [[1.0 + 3.0 / rms, 1.0 + 2.0 / rms]])
    assert np.allclose(n, h / np.sqrt(np.mean(h * h)))
