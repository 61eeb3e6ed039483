"""fp64 oracle of the gated delta rule and the block norms: the definitions, token by token and row by row.

State S [dv][dk] per value head, value head h reading query/key head h // (heads_v // heads_qk):
    S~ = exp(g_t) S,  e = v_t - S~ k,  S = S~ + beta_t e k^T,  o_t = scale S q
The gradient reverses these lines; the block norms' gradient is written out below.
"""
from __future__ import annotations

import numpy as np

NORM_EPS = 1e-12


def unit(x):
    return x / np.maximum(np.linalg.norm(x, axis=-1, keepdims=True), NORM_EPS)


def unit_grad(x, grad):
    """Gradient through x / max(||x||, 1e-12)."""
    n = np.linalg.norm(x, axis=-1, keepdims=True)
    u = x / np.maximum(n, NORM_EPS)
    inside = grad - np.where(n > NORM_EPS, u * (u * grad).sum(-1, keepdims=True), 0.0)
    return inside / np.maximum(n, NORM_EPS)


def _heads(x, h):
    return x.reshape(x.shape[0], h, x.shape[1] // h)


def _flat(x):
    return x.reshape(x.shape[0], x.shape[1] * x.shape[2])


def _split(Q, K, V, hk, hv, l2norm):
    q, k, v = _heads(Q, hk), _heads(K, hk), _heads(V, hv)
    if l2norm:
        q, k = unit(q), unit(k)
    rep = hv // hk
    return np.repeat(q, rep, 1), np.repeat(k, rep, 1), v


def delta_rule(Q, K, V, g, beta, S0, hk, hv, scale, l2norm=True):
    """One sequence: (O [T][hv*dv], S [hv][dv][dk])."""
    q, k, v = _split(Q, K, V, hk, hv, l2norm)
    S = S0.copy()
    O = np.zeros_like(v)
    for t in range(v.shape[0]):
        S = S * np.exp(g[t])[:, None, None]
        u = beta[t][:, None] * (v[t] - np.einsum("hvk,hk->hv", S, k[t]))
        S = S + np.einsum("hv,hk->hvk", u, k[t])
        O[t] = scale * np.einsum("hvk,hk->hv", S, q[t])
    return _flat(O), S


def delta_rule_grad(Q, K, V, g, beta, S0, dO, dS, hk, hv, scale, l2norm=True):
    """One sequence: dict of dq, dk, dv, dg, dbeta, dS0 from dO and dS (the gradient of the last state)."""
    T = K.shape[0]
    q, k, v = _split(Q, K, V, hk, hv, l2norm)
    do = _heads(dO, hv)
    held, errs, after = [], [], []
    S = S0.copy()
    for t in range(T):
        h = S * np.exp(g[t])[:, None, None]
        e = v[t] - np.einsum("hvk,hk->hv", h, k[t])
        S = h + np.einsum("hv,hk->hvk", beta[t][:, None] * e, k[t])
        held.append(h)
        errs.append(e)
        after.append(S)
    dS = dS.copy()
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dg, db = np.zeros_like(g), np.zeros_like(beta)
    for t in reversed(range(T)):
        d = scale * do[t]
        dq[t] = np.einsum("hvk,hv->hk", after[t], d)
        dS = dS + np.einsum("hv,hk->hvk", d, q[t])
        du = np.einsum("hvk,hk->hv", dS, k[t])
        db[t] = (du * errs[t]).sum(-1)
        de = beta[t][:, None] * du
        dv[t] = de
        dk[t] = np.einsum("hvk,hv->hk", dS, beta[t][:, None] * errs[t]) - np.einsum("hvk,hv->hk", held[t], de)
        dS = dS - np.einsum("hv,hk->hvk", de, k[t])
        dg[t] = (dS * held[t]).sum((-1, -2))
        dS = dS * np.exp(g[t])[:, None, None]
    rep = hv // hk
    dq, dk = (x.reshape(T, hk, rep, x.shape[2]).sum(2) for x in (dq, dk))
    if l2norm:
        dq = unit_grad(_heads(Q, hk), dq)
        dk = unit_grad(_heads(K, hk), dk)
    return {"dq": _flat(dq), "dk": _flat(dk), "dv": _flat(dv), "dg": dg, "dbeta": db, "dS0": dS}


def _sig(z):
    return 1.0 / (1.0 + np.exp(-z))


def block_norm(Y, X=None, Z=None, w_post=None, lam=None, w_pre=None, group=None, eps=1e-6):
    """(x', n): x' = x + lam * RMSNorm(y) * w_post * SiLU(z), n = RMSNorm(x') * w_pre."""
    R, D = Y.shape
    group = group or D
    y = Y.reshape(R, D // group, group)
    p = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps)
    p = (p * (np.ones(group) if w_post is None else w_post)).reshape(R, D)
    if Z is not None:
        p = p * Z * _sig(Z)
    xo = (p if lam is None else lam * p) + (0.0 if X is None else X)
    n = xo / np.sqrt((xo ** 2).mean(-1, keepdims=True) + eps) * (1.0 if w_pre is None else w_pre)
    return xo, n


def block_norm_grad(Y, dXo, dN, X=None, Z=None, w_post=None, lam=None, w_pre=None, group=None, eps=1e-6):
    """dict of dy, dx, dz, dw_post, dlam, dw_pre; dXo or dN may be None (zero)."""
    R, D = Y.shape
    group = group or D
    wp = np.tile(np.ones(group) if w_post is None else w_post, D // group)
    la = np.ones(D) if lam is None else lam
    wn = np.ones(D) if w_pre is None else w_pre
    mean = lambda a: np.repeat(a.reshape(R, D // group, group).mean(-1), group, 1)  # noqa: E731
    ry = 1.0 / np.sqrt(mean(Y ** 2) + eps)
    yh = Y * ry
    s = np.ones_like(Y) if Z is None else Z * _sig(Z)
    xo, _ = block_norm(Y, X, Z, w_post, lam, w_pre, group, eps)
    d = np.zeros_like(Y) if dXo is None else dXo.copy()
    out = {}
    if dN is not None:
        r = 1.0 / np.sqrt((xo ** 2).mean(-1, keepdims=True) + eps)
        t = dN * wn
        d = d + r * (t - xo * r ** 2 * (t * xo).mean(-1, keepdims=True))
        out["dw_pre"] = (dN * xo * r).sum(0)
    else:
        out["dw_pre"] = np.zeros(D)
    out["dx"] = d
    out["dlam"] = (d * yh * wp * s).sum(0)
    dp = d * la
    out["dw_post"] = (dp * yh * s).reshape(-1, group).sum(0)
    if Z is not None:
        out["dz"] = dp * yh * wp * _sig(Z) * (1 + Z * (1 - _sig(Z)))
    u = dp * wp * s
    out["dy"] = ry * (u - yh * mean(u * yh))
    return out
