"""The gated delta rule's and block norms' fp64 oracle: hand-worked cases, central differences, and invariants."""
import numpy as np
import pytest

from oracle import delta_oracle as D


def _seq(T, hk, hv, dk, dv, seed, l2=True):
    r = np.random.default_rng(seed)
    Q, K = r.standard_normal((T, hk * dk)), r.standard_normal((T, hk * dk)) * (1.0 if l2 else dk ** -0.5)
    V = r.standard_normal((T, hv * dv))
    g = -np.abs(r.standard_normal((T, hv))) * 0.3
    beta = 1 / (1 + np.exp(-r.standard_normal((T, hv))))
    S0 = r.standard_normal((hv, dv, dk)) * 0.3
    return Q, K, V, g, beta, S0


def test_a_unit_key_with_beta_one_stores_its_value():
    # g = 0, beta = 1: S k^ = v afterwards, whatever was stored under k^ before, and orthogonal keys stay
    S0 = np.zeros((1, 2, 2))
    K = np.array([[3.0, 0.0], [0.0, 2.0], [5.0, 0.0]])
    V = np.array([[1.0, 2.0], [3.0, 4.0], [7.0, 9.0]])
    O, S = D.delta_rule(K, K, V, np.zeros((3, 1)), np.ones((3, 1)), S0, 1, 1, 1.0)
    assert np.allclose(O, V)
    assert np.allclose(S[0], np.array([[7.0, 3.0], [9.0, 4.0]]))


def test_beta_zero_only_decays():
    Q, K, V, g, beta, S0 = _seq(5, 1, 2, 4, 3, 1)
    _, S = D.delta_rule(Q, K, V, g, np.zeros_like(beta), S0, 1, 2, 1.0)
    assert np.allclose(S, S0 * np.exp(g.sum(0))[:, None, None])


def test_value_heads_share_query_key_heads_in_order():
    Q, K, V, g, beta, S0 = _seq(6, 2, 4, 4, 3, 2)
    O, _ = D.delta_rule(Q, K, V, g, beta, S0, 2, 4, 0.5)
    for h in range(4):
        q, k = Q[:, (h // 2) * 4:(h // 2) * 4 + 4], K[:, (h // 2) * 4:(h // 2) * 4 + 4]
        o, _ = D.delta_rule(q, k, V[:, h * 3:h * 3 + 3], g[:, h:h + 1], beta[:, h:h + 1], S0[h:h + 1], 1, 1, 0.5)
        assert np.allclose(O[:, h * 3:h * 3 + 3], o)


@pytest.mark.parametrize("l2", [True, False])
def test_delta_gradient_against_differences(l2):
    hk, hv, dk, dv, T = 1, 2, 3, 2, 5
    args = list(_seq(T, hk, hv, dk, dv, 3, l2))
    r = np.random.default_rng(4)
    dO, dS = r.standard_normal((T, hv * dv)), r.standard_normal((hv, dv, dk))

    def loss(a):
        O, S = D.delta_rule(*a, hk, hv, 0.7, l2)
        return (O * dO).sum() + (S * dS).sum()

    grad = D.delta_rule_grad(*args, dO, dS, hk, hv, 0.7, l2)
    for i, name in enumerate(("dq", "dk", "dv", "dg", "dbeta", "dS0")):
        num = np.zeros_like(args[i])
        for at in np.ndindex(*args[i].shape):
            for sign in (1, -1):
                a = [x.copy() for x in args]
                a[i][at] += sign * 1e-6
                num[at] += sign * loss(a) / 2e-6
        assert np.allclose(grad[name], num, atol=2e-8, rtol=1e-7), name


def test_gate_gradient_is_a_running_sum():
    # dg_t = <S_0, dS_0> - sum_{i<t} (dO_i . O_i - dV_i . V_i): what the kernels sum per chunk
    Q, K, V, g, beta, S0 = _seq(9, 1, 1, 4, 3, 5)
    r = np.random.default_rng(6)
    dO, dS = r.standard_normal((9, 3)), r.standard_normal((1, 3, 4))
    O, _ = D.delta_rule(Q, K, V, g, beta, S0, 1, 1, 0.7)
    G = D.delta_rule_grad(Q, K, V, g, beta, S0, dO, dS, 1, 1, 0.7)
    w = (dO * O).sum(1) - (G["dv"] * V).sum(1)
    assert np.allclose(G["dg"][:, 0], (S0 * G["dS0"]).sum() - (np.cumsum(w) - w))


@pytest.mark.parametrize("group,res,gate,norm2", [(6, True, True, True), (3, True, True, True), (3, False, True, False),
                                                  (6, True, False, False), (2, False, False, True)])
def test_block_norm_gradient_against_differences(group, res, gate, norm2):
    r = np.random.default_rng(7)
    R, W = 3, 6
    a = {"Y": r.standard_normal((R, W)), "X": r.standard_normal((R, W)) if res else None,
         "Z": r.standard_normal((R, W)) if gate else None, "w_post": r.standard_normal(group),
         "lam": r.standard_normal(W), "w_pre": r.standard_normal(W)}
    dXo, dN = r.standard_normal((R, W)), r.standard_normal((R, W)) if norm2 else None

    def loss(a):
        xo, n = D.block_norm(**a, group=group)
        return (xo * dXo).sum() + (0 if dN is None else (n * dN).sum())

    grad = D.block_norm_grad(a["Y"], dXo, dN, a["X"], a["Z"], a["w_post"], a["lam"], a["w_pre"], group)
    for key, name in (("Y", "dy"), ("X", "dx"), ("Z", "dz"), ("w_post", "dw_post"), ("lam", "dlam"),
                      ("w_pre", "dw_pre")):
        if a[key] is None:
            continue
        num = np.zeros_like(a[key])
        for at in np.ndindex(*a[key].shape):
            for sign in (1, -1):
                b = dict(a)
                b[key] = a[key].copy()
                b[key][at] += sign * 1e-6
                num[at] += sign * loss(b) / 2e-6
        assert np.allclose(grad[name], num, atol=3e-8, rtol=1e-7), name


def test_block_norm_by_hand():
    # y = (3, 4): mean square 12.5; x = (1, 1), gate z = 0 closes p
    xo, n = D.block_norm(np.array([[3.0, 4.0]]), eps=0.0)
    assert np.allclose(xo, np.array([[3.0, 4.0]]) / np.sqrt(12.5)) and np.allclose(n, xo)
    xo, n = D.block_norm(np.array([[3.0, 4.0]]), X=np.array([[1.0, 1.0]]), Z=np.zeros((1, 2)), eps=0.0)
    assert np.allclose(xo, 1.0) and np.allclose(n, 1.0)
