"""Calls at the borders of what the gated delta rule's documentation allows, on the GPU against the fp64 oracle."""
import pytest
import torch

from test_gpu_delta import Seqs
from test_weight_layers_b200 import ttt as T

from _gpu import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def test_the_outputs_gradient_may_be_the_values():
    c = Seqs([100, 70], 1, 2, 64, 64, seed=40)
    c.dO = c.V.clone()
    want, _ = c.backward()
    c.dO = c.V
    out, ws = c.backward()
    assert T.ttt_poll_status(ws) == T.TTT_OK and all(torch.equal(out[k], want[k]) for k in out)
    c.check_backward(out)


@pytest.mark.parametrize("lens,hk,hv,dk,dv", [([70, 5], 1, 2, 64, 520), ([66], 1, 1, 40, 1024), ([30], 1, 1, 192, 1024),
                                              ([900], 1, 1, 64, 520), ([100], 1, 1, 256, 544)])
def test_many_value_channels(lens, hk, hv, dk, dv):
    # more than 32 slices of 16 channels in the gates' sums
    c = Seqs(lens, hk, hv, dk, dv, seed=dv)
    c.check_forward(*c.forward()[:2])
    c.check_backward(c.backward()[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_step_of_many_value_channels(dtype):
    c = Seqs([1] * 3, 1, 1, 256, 1024, seed=41, dtype=dtype)
    pool, O = c.S0.clone(), torch.zeros((3, 1024), dtype=dtype, device="cuda")
    T.ttt_delta_step(c.Q, c.K, c.V, c.g, c.beta, pool, O, 3, c.dm, c.io, scale=c.scale)
    c.check_forward(O, pool)


@pytest.mark.parametrize("dtype,n", [(torch.bfloat16, 12), (torch.float32, 12), (torch.float32, 70)])
@pytest.mark.parametrize("size", [1e25, 2e38])
def test_rows_too_large_for_a_norm_count_as_zero(dtype, n, size):
    # token by token the norms are summed in fp32: such keys write nothing, such queries read zero
    c = Seqs([n], 1, 2, 64, 64, seed=42, dtype=dtype)
    rows = torch.tensor([2, 3, 7], device="cuda"), torch.tensor([3, 5], device="cuda")
    for t, at in ((c.K, rows[0]), (c.Q, rows[1])):
        t[at] = (t[at].sign().float() * size).to(dtype)
    O, S, _ = c.forward()
    step_pool = c.S0.clone()
    step_O = torch.zeros_like(O)
    for t in range(n):
        at = slice(t, t + 1)
        T.ttt_delta_step(c.Q[at], c.K[at], c.V[at], c.g[at], c.beta[at], step_pool, step_O[at], 1, c.dm, c.io,
                         scale=c.scale)
    c.K[rows[0]] = 0
    c.Q[rows[1]] = 0
    c.check_forward(O, S)
    c.check_forward(step_O, step_pool)


def test_a_pool_without_slots():
    # every row is padding
    c = Seqs([1] * 3, 1, 1, 64, 64, seed=43)
    O = torch.full((3, 64), 77.0, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int32, device="cuda")
    T.ttt_delta_step(c.Q, c.K, c.V, c.g, c.beta, c.S0[:0], O, 3, c.dm, c.io, slots=slots)
    assert torch.all(O == 77)
