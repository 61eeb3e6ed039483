"""Calls at the borders of what the gated delta rule's documentation allows, on the GPU against the fp64 oracle."""
import pytest
import torch

from oracle import delta_oracle as D
from test_gpu_delta import TOL_O, TOL_S, Seqs
from test_weight_layers_b200 import ttt as T

from _gpu import f64, need_gpu, rel_fro

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


def test_many_rows_of_few_slots():
    # 300 rows on 7 slots in turn, some of them padding: each slot's rows are its tokens in order
    B, hv, d = 300, 2, 64
    c = Seqs([B], 1, hv, d, d, seed=44)
    pool = torch.stack([c.S0[0] * (i + 1) / 4 for i in range(7)])
    before = pool.clone()
    which = torch.arange(B) % 9 - 1  # -1, 0 .. 7: the last is past the pool
    O = torch.full((B, hv * d), 77.0, dtype=torch.bfloat16, device="cuda")
    T.ttt_delta_step(c.Q, c.K, c.V, c.g, c.beta, pool, O, B, c.dm, c.io, slots=which.to(torch.int32).cuda(),
                     scale=c.scale)
    torch.cuda.synchronize()
    assert torch.all(O[(which < 0).cuda()] == 77) and torch.all(O[(which > 6).cuda()] == 77)
    for slot in range(7):
        rows = (which == slot).nonzero()[:, 0].cuda()
        args = [f64(t[rows]) for t in (c.Q, c.K, c.V, c.g, c.beta)]
        o, s = D.delta_rule(*args, f64(before[slot]), 1, hv, c.scale)
        assert rel_fro(f64(O[rows]), o) < TOL_O and rel_fro(f64(pool[slot]), s) < TOL_S


def test_two_gradients_at_once_and_in_two_graphs():
    # one is cut into segments; a workspace each
    cs = [Seqs([1800], 1, 1, 64, 64, seed=45), Seqs([300, 0, 41], 1, 4, 128, 64, seed=46)]
    want = [c.backward()[0] for c in cs]
    wss = [c.workspace(True) for c in cs]
    outs = [c.outputs_bwd() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, ws, out, st in zip(cs, wss, outs, streams):
            c.backward(ws=ws, out=out, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o[k], w[k]) for o, w in zip(outs, want) for k in w)
    graphs = []
    for c, ws, out in zip(cs, wss, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.backward(ws=ws, out=out)
        for t in out.values():
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o[k], w[k]) for o, w in zip(outs, want) for k in w)
    assert all(T.ttt_poll_status(ws) == T.TTT_OK for ws in wss)


def test_a_nan_stays_in_its_sequence_on_the_way_back():
    for lens, d in (([70, 70, 70], 64), ([1000, 900, 1100], 64)):   # whole, and cut into segments
        c = Seqs(lens, 1, 1, d, d, seed=47)
        clean, _ = c.backward()
        at = c.starts[1] + 5
        c.V[at, 3] = float("nan")
        c.K[at + 1, 1] = float("inf")
        c.dO[at + 9, 0] = float("inf")
        out, ws = c.backward()
        assert T.ttt_poll_status(ws) == T.TTT_OK
        for i in (0, 2):
            rows = slice(c.starts[i], c.starts[i + 1])
            assert all(torch.equal(out[k][rows], clean[k][rows]) for k in ("dq", "dk", "dv", "dg", "dbeta"))
            assert torch.equal(out["dS0"][i], clean["dS0"][i])
