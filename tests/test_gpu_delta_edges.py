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


def test_short_neighbours_leave_a_long_sequence_cut():
    # whether a sequence is cut goes by the lengths themselves: with and without a few tokens beside it, a long one
    # runs in segments of the same size, to the last bit
    # (the gates hold the state over several segments, so that uncut sums differ from joined ones)
    alone = Seqs([32000], 4, 4, 192, 192, seed=48, decay=1e-4)
    c = Seqs([1, 32000, 0, 1, 1, 1], 4, 4, 192, 192, seed=49)
    for name in ("Q", "K", "V", "g", "beta", "dO"):
        getattr(c, name)[1:32001] = getattr(alone, name)
    for name in ("S0", "dS"):
        getattr(c, name)[1] = getattr(alone, name)[0]
    O, S, _ = alone.forward()
    O2, S2, ws = c.forward()
    assert T.ttt_poll_status(ws) == T.TTT_OK and torch.equal(O2[1:32001], O) and torch.equal(S2[1], S[0])
    out, _ = alone.backward()
    out2, ws = c.backward()
    assert T.ttt_poll_status(ws) == T.TTT_OK and torch.equal(out2["dS0"][1], out["dS0"][0])
    assert all(torch.equal(out2[k][1:32001], out[k]) for k in ("dq", "dk", "dv", "dg", "dbeta"))


@pytest.mark.parametrize("lens,hk,hv,dk,dv", [([3000, 1, 0, 64, 100, 2999], 1, 1, 64, 64),
                                              ([20, 65, 1500, 64, 0, 129], 1, 2, 192, 64),
                                              ([0, 0, 800, 0, 0, 0, 0, 0], 1, 3, 128, 128),
                                              ([768] * 5 + [2500], 1, 1, 40, 16),
                                              ([900, 30], 1, 1, 256, 200)])
def test_ragged_batches_in_segments(lens, hk, hv, dk, dv):
    for s0 in (False, True):
        c = Seqs(lens, hk, hv, dk, dv, seed=50 + dk, s0=s0, lead=2, tail=3, decay=0.003)
        O, S, ws = c.forward()
        assert T.ttt_poll_status(ws) == T.TTT_OK and torch.all(O[:2] == 77) and torch.all(O[-3:] == 77)
        c.check_forward(O, S)
        out, ws = c.backward()
        assert T.ttt_poll_status(ws) == T.TTT_OK
        c.check_backward(out)
    state = c.S0.clone()  # in place
    O2, _, _ = c.forward(S=state, S0=state)
    assert torch.equal(O, O2) and torch.equal(S, state)


def test_equal_sequences_without_offsets_in_segments():
    # two sequences are cut, forty fill the card as they are; without offsets that is known before the launch
    for n, length in ((2, 900), (40, 900), (3, 130)):
        c = Seqs([length] * n, 1, 2, 64, 64, seed=51)
        O, S, _ = c.forward()
        O2, S2, ws = c.forward(cu=None)
        assert T.ttt_poll_status(ws) == T.TTT_OK and torch.equal(O, O2) and torch.equal(S, S2)
        out, _ = c.backward()
        cu, c.cu = c.cu, None
        out2, ws = c.backward()
        c.cu = cu
        assert T.ttt_poll_status(ws) == T.TTT_OK and all(torch.equal(out[k], out2[k]) for k in out)
