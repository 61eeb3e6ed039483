"""The operators as a layer uses them: norm, projections, gated delta rule, gated head norm, output projection, residual
norm -- and back -- against the same layer in fp64; and a state handed from the prefill to decoding steps.

The projections are torch products in bf16 on the test's side (as the user's would be), so every tensor that crosses
between the operators is rounded to bf16: eight such roundings in a row on the way in and out, 2^-8 each at most,
bound the outputs and gradients by 2^-5.
"""
import torch
import pytest

from oracle import delta_oracle as O  # noqa: F401  (the oracle's conventions)
from test_weight_layers_b200 import ttt as T

from _gpu import need_gpu

pytestmark = pytest.mark.gpu
TOL = 2 ** -5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _rel(a, b):
    return float((a.double() - b).norm() / b.norm())


HK, HV, DK, DV, D, LENS = 2, 4, 64, 64, 192, [100, 1, 63]
NQ, NV = HK * DK, HV * DV


def _reference(p):
    """The layer in fp64 with autograd."""
    x, y0 = p["x"], p["y0"]
    rms = lambda a, w: a / torch.sqrt((a * a).mean(-1, keepdim=True) + 1e-6) * w  # noqa: E731
    x1 = x + p["lam0"] * rms(y0, p["wp0"])
    h = rms(x1, p["wn0"])
    qkvz = h @ p["Wqkvz"].T
    q, k, v, z = qkvz.split([NQ, NQ, NV, NV], -1)
    unit = lambda a: a / a.norm(dim=-1, keepdim=True).clamp_min(1e-12)  # noqa: E731
    rep = HV // HK
    q = unit(q.unflatten(-1, (HK, DK))).repeat_interleave(rep, 1)
    k = unit(k.unflatten(-1, (HK, DK))).repeat_interleave(rep, 1)
    v = v.unflatten(-1, (HV, DV))
    outs, at, states = [], 0, []
    for n in LENS:
        S = torch.zeros(HV, DV, DK, dtype=torch.float64, device=x.device)
        for t in range(at, at + n):
            S = S * p["g"][t].exp()[:, None, None]
            u = p["beta"][t][:, None] * (v[t] - (S @ k[t][..., None])[..., 0])
            S = S + u[..., None] * k[t][:, None, :]
            outs.append((S @ q[t][..., None])[..., 0] * DK ** -0.5)
        states.append(S)
        at += n
    o = torch.stack(outs)
    o = rms(o, p["wh"]).flatten(1) * (z * torch.sigmoid(z))
    return x1 + p["lam1"] * rms(o @ p["Wo"].T, p["wp1"]), torch.stack(states)


def test_layer_forward_and_backward():
    gen = torch.Generator(device="cuda").manual_seed(0)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    bf = lambda t: t.bfloat16()  # noqa: E731
    R = sum(LENS)
    x, y0 = bf(rn(R, D)), bf(rn(R, D))
    Wqkvz, Wo = bf(rn(2 * NQ + 2 * NV, D) * D ** -0.5), bf(rn(D, NV) * NV ** -0.5)
    lam0, lam1, wp0, wp1, wn0 = (1 + 0.1 * rn(D) for _ in range(5))
    wh = 1 + 0.1 * rn(DV)
    g, beta = -0.1 * rn(R, HV).abs(), torch.sigmoid(rn(R, HV))
    dout = bf(rn(R, D))

    # forward
    cu = torch.tensor([0, 100, 101, 164], dtype=torch.int32, device="cuda")
    dm, n1 = T.delta_dims(HK, HV, DK, DV), T.norm_cfg(D)
    x1, h = torch.empty_like(x), torch.empty_like(x)
    T.ttt_block_norm(y0, x1, R, n1, X=x, w_post=wp0, res_scale=lam0, w_pre=wn0, N=h)
    qkvz = h @ Wqkvz.T
    ld = qkvz.stride(0)
    q, k, v, z = qkvz.split([NQ, NQ, NV, NV], -1)
    io = T.io_cfg(ld_q=ld, ld_k=ld, ld_v=ld)
    ws = T.delta_workspace(dm, R, len(LENS), T.TTT_BF16, backward=True)
    o = torch.empty((R, NV), dtype=torch.bfloat16, device="cuda")
    S = torch.empty((len(LENS), HV, DV, DK), device="cuda")
    T.ttt_delta_chunked(q, k, v, g, beta, None, S, o, R, dm, io, ws, cu_seqlens=cu, n_seq=3, scale=DK ** -0.5)
    heads = T.norm_cfg(NV, DV, ld_z=ld)
    og = torch.empty_like(o)
    T.ttt_block_norm(o, og, R, heads, Z=z, w_post=wh)
    y1 = og @ Wo.T
    x2 = torch.empty_like(x)
    T.ttt_block_norm(y1, x2, R, n1, X=x1, w_post=wp1, res_scale=lam1)

    # backward
    e = torch.empty_like
    dy1, dx1 = e(y1), e(x)
    dw = {n: torch.empty_like(t) for n, t in (("wp1", wp1), ("lam1", lam1), ("wh", wh), ("wp0", wp0), ("lam0", lam0),
                                              ("wn0", wn0))}
    wsn = T.norm_workspace(R, n1)
    T.ttt_block_norm_backward(y1, dout, dy1, R, n1, wsn, X=x1, w_post=wp1, res_scale=lam1, dX=dx1, dw_post=dw["wp1"],
                              dres_scale=dw["lam1"])
    dog, dWo = dy1 @ Wo, dy1.T @ og
    dqkvz = torch.empty_like(qkvz)
    dq, dk, dv, dz = dqkvz.split([NQ, NQ, NV, NV], -1)
    do = e(o)
    T.ttt_block_norm_backward(o, dog, do, R, heads, T.norm_workspace(R, heads), Z=z, w_post=wh, dZ=dz,
                              dw_post=dw["wh"])
    dg, db = torch.empty_like(g), torch.empty_like(beta)
    T.ttt_delta_chunked_backward(q, k, v, g, beta, None, do, None, dq, dk, dv, dg, db, None, R, dm, io, ws,
                                 cu_seqlens=cu, n_seq=3, scale=DK ** -0.5)
    dh, dWqkvz = dqkvz @ Wqkvz, dqkvz.T @ h
    dy0, dx = e(y0), e(x)
    T.ttt_block_norm_backward(y0, dx1, dy0, R, n1, wsn, X=x, w_post=wp0, res_scale=lam0, w_pre=wn0, dN=dh, dX=dx,
                              dw_post=dw["wp0"], dres_scale=dw["lam0"], dw_pre=dw["wn0"])
    assert T.ttt_poll_status(ws) == T.TTT_OK

    p = {n: t.double().requires_grad_() for n, t in dict(
        x=x, y0=y0, Wqkvz=Wqkvz, Wo=Wo, lam0=lam0, lam1=lam1, wp0=wp0, wp1=wp1, wn0=wn0, wh=wh, g=g, beta=beta).items()}
    ref, states = _reference(p)
    ref.backward(dout.double())
    assert _rel(x2, ref.detach()) < TOL and _rel(S, states.detach()) < TOL
    got = dict(dw, x=dx, y0=dy0, Wqkvz=dWqkvz, Wo=dWo, g=dg, beta=db)
    for name, t in got.items():
        assert _rel(t, p[name].grad) < TOL, name


def test_prefill_hands_its_state_to_decoding():
    gen = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    lens, steps = [130, 0, 17], 5
    dm = T.delta_dims(HK, HV, DK, DV)
    pool = torch.zeros((6, HV, DV, DK), device="cuda")
    toks = [[rn(n + steps, w).bfloat16() for w in (NQ, NQ, NV)] + [-0.1 * rn(n + steps, HV).abs(),
            torch.sigmoid(rn(n + steps, HV))] for n in lens]
    heads = T.norm_cfg(NV, DV)
    wh = 1 + 0.1 * rn(DV)

    def prefill(cut):
        parts = [torch.cat([t[i][:n + cut] for t, n in zip(toks, lens)]) for i in range(5)]
        R = parts[0].shape[0]
        o = torch.empty((R, NV), dtype=torch.bfloat16, device="cuda")
        S = torch.empty((3, HV, DV, DK), device="cuda")
        ends = [0]
        for n in lens:
            ends.append(ends[-1] + n + cut)
        cu = torch.tensor(ends, dtype=torch.int32, device="cuda")
        T.ttt_delta_chunked(*parts, None, S, o, R, dm, T.io_cfg(), T.delta_workspace(dm, R, 3, T.TTT_BF16),
                            cu_seqlens=cu, n_seq=3)
        og = torch.empty_like(o)
        T.ttt_block_norm(o, og, R, heads, w_post=wh)
        return [og[ends[i]:ends[i + 1]] for i in range(3)], S

    long_o, long_s = prefill(steps)
    _, S = prefill(0)
    slots = torch.tensor([4, 1, 2], dtype=torch.int32, device="cuda")
    pool[slots.long()] = S
    for s in range(steps):
        row = [torch.stack([t[i][n + s] for t, n in zip(toks, lens)]) for i in range(5)]
        o, og = (torch.empty((3, NV), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        T.ttt_delta_step(*row, pool, o, 3, dm, T.io_cfg(), slots=slots)
        T.ttt_block_norm(o, og, 3, heads, w_post=wh)
        for i, n in enumerate(lens):
            assert _rel(og[i], long_o[i][n + s].double()) < 2 ** -6  # two bf16 roundings on each side
    assert _rel(pool[slots.long()], long_s.double()) < 1e-4
