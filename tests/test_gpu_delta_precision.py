"""What the chunked gated delta rule keeps of its operands' precision, on the GPU against the fp64 oracle.

Tolerances, from the arithmetic (c terms of a sum, M the sum of their magnitudes):
  - a product of split operands drops 2^-22 of an operand twice and the product of the low parts once, and its sum
    loses 2^-24 per term: SUM(c) = 3 * 2^-22 + c * 2^-24, relative to M; a bf16 output adds half a step, 2^-8.
  - a value off by d before it is rounded to bf16 is rounded to another one with probability |d| / step, and is then
    off by a step of 2^-7 of the value at most: against the rounded oracle the relative Frobenius error is
    sqrt(2^-7 * d).  Outputs that keep 11 bits of their operands are at 1e-3 there.
"""
import numpy as np
import pytest
import torch

from oracle import delta_oracle as D
from test_gpu_delta import TOL_S, Seqs
from test_weight_layers_b200 import ttt as T

from _gpu import f64, need_gpu, rel_fro

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def SUM(c):
    return 3 * 2 ** -22 + c * 2 ** -24


def flip(d):
    return (2 ** -7 * d) ** 0.5


def rounded(x):
    return f64(torch.from_numpy(np.ascontiguousarray(x)).bfloat16())


def overwritten(n, dk, dv, seed):
    """One key, written again and again: a large value first, then values of about one."""
    c = Seqs([n], 1, 1, dk, dv, seed=seed, s0=False, decay=0.0)
    c.K[:] = c.K[0].clone()
    c.V[:] = c.V.float().sign().bfloat16()
    c.V[0] *= 1000
    c.beta[:] = 0.9983
    c.scale = 1.0
    return c


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 40), (192, 64), (256, 64)])
@pytest.mark.parametrize("n", [40, 41, 200])
def test_output_of_an_overwritten_key(n, dk, dv):
    # o = P U: two writes of about 1000 of opposite signs, then what is left of them
    c = overwritten(n, dk, dv, dk)
    c.Q = c.K.clone()
    O, S, _ = c.forward()
    at, args = c._seq(0)
    o, _ = D.delta_rule(*args, 1, 1, c.scale)
    assert np.all(np.abs(f64(O) - o) <= 2 ** -8 * np.abs(o) + SUM(64 + dk) * 2100)


@pytest.mark.parametrize("dk,dv", [(64, 64), (192, 64), (256, 64)])
@pytest.mark.parametrize("n", [40, 41, 200])
def test_output_where_a_large_state_is_overwritten(n, dk, dv):
    # o = e^c S q + P U: the state's read of about 1000 against the write that replaces it
    c = overwritten(n, dk, dv, dk + 1)
    c.Q = c.K.clone()
    c.V[0] /= 1000
    k = c.K[0].float()
    c.S0 = (1000 * k / k.norm()).expand(1, 1, dv, dk).contiguous()
    O, S, _ = c.forward()
    at, args = c._seq(0)
    o, _ = D.delta_rule(*args, 1, 1, c.scale)
    assert np.all(np.abs(f64(O) - o) <= 2 ** -8 * np.abs(o) + SUM(64 + dk) * 2100)


@pytest.mark.parametrize("dk,dv", [(64, 64), (192, 72), (256, 64)])
def test_gradients_of_an_overwritten_key(dk, dv):
    # dq = scale S^T dO with S = the sum of writes of about 1000 that leave about one; the same sums are in dk
    c = overwritten(200, dk, dv, dk + 2)
    c.l2 = c.io.qk_l2norm = 0
    c.K /= c.K[0].float().norm()
    c.Q /= 8
    out, _ = c.backward()
    at, args = c._seq(0)
    z = f64(c.dS[0])
    ref = D.delta_rule_grad(*args, f64(c.dO), z, 1, 1, c.scale, False)
    # terms: sums of |U| of 2100 at most per channel, times |dO| in dq; in dk also times |dS|, which reaches every token
    of_do = np.abs(f64(c.dO)).sum(-1, keepdims=True)
    for name, size in (("dq", of_do), ("dk", of_do + of_do.max() + np.abs(z).sum())):
        err = np.linalg.norm(f64(out[name]) - ref[name], axis=-1, keepdims=True)
        most = 2 ** -8 * np.linalg.norm(ref[name], axis=-1, keepdims=True) + SUM(64 + dv) * 2100 * size
        assert np.all(err <= most), (name, float((err / most).max()))


# lens, heads_qk, heads_v, dk, dv
ROUNDED = [([300, 41], 1, 2, 64, 64), ([200], 2, 4, 128, 128), ([200, 77], 1, 1, 192, 192), ([150], 1, 2, 256, 72),
           ([5000], 1, 1, 64, 64), ([90], 1, 1, 40, 24)]


@pytest.mark.parametrize("lens,hk,hv,dk,dv", ROUNDED)
def test_outputs_are_the_rounded_ones(lens, hk, hv, dk, dv):
    c = Seqs(lens, hk, hv, dk, dv, seed=dk + 7)
    O, S, _ = c.forward()
    ref = np.concatenate([D.delta_rule(*c._seq(i)[1], hk, hv, c.scale)[0] for i in range(c.N)])
    assert rel_fro(f64(O), rounded(ref)) < flip(TOL_S / 3)


@pytest.mark.parametrize("lens,hk,hv,dk,dv", ROUNDED)
def test_gradients_are_the_rounded_ones(lens, hk, hv, dk, dv):
    # dq, dk: two more products in a row than the states' three give
    c = Seqs(lens, hk, hv, dk, dv, seed=dk + 8)
    out, _ = c.backward()
    refs = [D.delta_rule_grad(*c._seq(i)[1], f64(c.dO[c._seq(i)[0]]), f64(c.dS[i]), hk, hv, c.scale)
            for i in range(c.N)]
    for k in ("dq", "dk", "dv"):
        assert rel_fro(f64(out[k]), rounded(np.concatenate([r[k] for r in refs]))) < flip(TOL_S), k


@pytest.mark.parametrize("dk", [64, 256])
def test_gradients_behind_many_resets(dk):
    # the tokens behind 48 resets in a chunk, whose decays do not depend on them
    c = Seqs([64], 1, 1, dk, 64, seed=31)
    c.g[:48] = float("-inf")
    out, _ = c.backward()
    ref = D.delta_rule_grad(*c._seq(0)[1], f64(c.dO), f64(c.dS[0]), 1, 1, c.scale)
    for k in ("dq", "dk", "dv"):
        assert rel_fro(f64(out[k][48:]), rounded(ref[k][48:])) < flip(TOL_S), k
    for k in ("dg", "dbeta"):
        assert rel_fro(f64(out[k][48:]), ref[k][48:]) < 2 * TOL_S, k


@pytest.mark.parametrize("n", [40, 41, 64, 130])
def test_a_reset_before_growth_leaves_nothing(n):
    # g = -inf forgets the state whatever the gates behind it do with it
    c = Seqs([n], 1, 1, 64, 64, seed=32)
    c.beta[:] = 0
    c.g[:] = 0
    c.g[20] = float("-inf")
    c.g[21:24] = 29.0
    O, S, _ = c.forward()
    assert torch.all(S == 0) and torch.all(O[20:] == 0) and torch.all(O[:20].abs().amax(-1) > 0)
    c.dO[21:] = 0
    out, _ = c.backward()
    assert torch.all(out["dS0"].abs().amax() > 0)
    c.dO[:20] = 0
    out, _ = c.backward()
    assert torch.all(out["dS0"] == 0)


def test_states_and_gates_keep_what_is_stated():
    # dk = dv = 128: eight steps of 16 terms twice (leading and low parts) for each of a chunk's three products, each
    # step cutting off 2^-24 of the sum: 48 * 2^-24, and the operands' 3 * 2^-22 a product
    c = Seqs([640, 333], 2, 4, 128, 128, seed=33)
    tol = 48 * 2 ** -24 + 9 * 2 ** -22
    _, S, _ = c.forward()
    ref = np.stack([D.delta_rule(*c._seq(i)[1], 2, 4, c.scale)[1] for i in range(2)])
    assert rel_fro(f64(S), ref) < tol
    out, _ = c.backward()
    refs = [D.delta_rule_grad(*c._seq(i)[1], f64(c.dO[c._seq(i)[0]]), f64(c.dS[i]), 2, 4, c.scale) for i in range(2)]
    assert rel_fro(f64(out["dS0"]), np.stack([r["dS0"] for r in refs])) < tol
    for k in ("dg", "dbeta"):
        assert rel_fro(f64(out[k]), np.concatenate([r[k] for r in refs])) < 2 * tol, k


@pytest.mark.parametrize("dk,dv", [(64, 64), (192, 40)])
def test_gates_of_an_empty_state_have_no_gradient(dk, dv):
    # dg_t is the product of the state before the token with its gradient: exactly zero without one
    for s0 in (False, True):
        c = Seqs([1, 1, 0, 1, 70], 1, 2, dk, dv, seed=34, s0=s0)
        if s0:
            c.S0.zero_()
        out, _ = c.backward()
        assert torch.all(out["dg"][:4] == 0) and torch.all(out["dg"][4:].abs().amax(-1) > 0)
        c.check_backward(out)
    c = Seqs([130], 1, 2, dk, dv, seed=35)
    c.g[:] = float("-inf")
    out, _ = c.backward()
    assert torch.all(out["dg"] == 0)


def test_gates_between_resets():
    # resets at a chunk's first and last tokens, next to each other, on one of the heads only, and none
    c = Seqs([260, 90], 1, 2, 64, 64, seed=36)
    for t in (0, 20, 21, 63, 64, 100, 255, 259, 300):
        c.g[t, 0] = float("-inf")
    c.g[150] = -200.0
    out, _ = c.backward()
    c.check_backward(out)
    assert torch.all(out["dg"][c.g < -104] == 0)
    refs = [D.delta_rule_grad(*c._seq(i)[1], f64(c.dO[c._seq(i)[0]]), f64(c.dS[i]), 1, 2, c.scale) for i in range(2)]
    ref = np.concatenate([r["dg"] for r in refs])
    for h in range(2):
        assert rel_fro(f64(out["dg"])[:, h], ref[:, h]) < 2 * TOL_S
