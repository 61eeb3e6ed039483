"""The gated delta rule on the GPU against the fp64 oracle, through the C ABI.

Tolerances (relative Frobenius norms), from the arithmetic:
  - a bf16 output is off by half a step of the value, 2^-8 at most, and by the products before it; O's take
    their factors' leading 11 bits (2^-12 each, two factors): 2^-8 + 2^-11.
  - states are products of split operands (2^-22) summed over at most 256 terms in fp32; three of them in
    a row per chunk, each bounded by 256 * 2^-24: 3 * (2^-22 + 2^-16) ~ 4.7e-5.
  - dq, dk: two TF32 products in a row (2^-11 per operand, 4 operands) and the rounding: 2^-8 + 2^-9.
  - dg, dbeta: sums of up to 64 (dg) fp32 terms of a few such products: 2 * the states' bound.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import delta_oracle as D
from test_weight_layers_b200 import ttt as T

from _gpu import f64, need_gpu, rel_fro

pytestmark = pytest.mark.gpu

TOL_S = 3 * (2 ** -22 + 2 ** -16)
TOL_O = 2 ** -8 + 2 ** -11
TOL_QK = 2 ** -8 + 2 ** -9
TOL_V = 2 ** -8 + TOL_S
TOL_G = 2 * TOL_S


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


class Seqs:
    """Packed sequences on the device, with what the calls need."""

    def __init__(self, lens, hk, hv, dk, dv, seed=0, dtype=torch.bfloat16, l2=1, s0=True, packed=False, decay=0.3,
                 lead=0, tail=0, vscale=1.0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.lens, self.hk, self.hv, self.dk, self.dv, self.l2 = list(lens), hk, hv, dk, dv, l2
        self.N, self.T, self.lead = len(lens), lead + sum(lens) + tail, lead
        nq, nv = hk * dk, hv * dv
        x = rn(self.T, 2 * nq + nv)
        if not l2:
            x[:, :2 * nq] *= dk ** -0.5
        x[:, 2 * nq:] *= vscale
        x = x.to(dtype)
        parts = (x[:, :nq], x[:, nq:2 * nq], x[:, 2 * nq:])
        self.Q, self.K, self.V = parts if packed else tuple(p.contiguous() for p in parts)
        self.g = -decay * rn(self.T, hv).abs()
        self.beta = torch.sigmoid(rn(self.T, hv))
        self.S0 = rn(self.N, hv, dv, dk) * 0.3 if s0 else None
        self.dO, self.dS = rn(self.T, nv).to(dtype), rn(self.N, hv, dv, dk) * 0.3
        self.starts = [lead + sum(lens[:i]) for i in range(self.N + 1)]
        self.cu = torch.tensor(self.starts, dtype=torch.int32, device="cuda")
        self.scale = dk ** -0.5
        self.dm = T.delta_dims(hk, hv, dk, dv)
        self.io = T.io_cfg(qk_l2norm=l2, ld_q=self.Q.stride(0) if self.T > 1 else 0,
                           ld_k=self.K.stride(0) if self.T > 1 else 0, ld_v=self.V.stride(0) if self.T > 1 else 0)
        self.code = T.dtype_code(dtype)

    def workspace(self, backward=False):
        return T.delta_workspace(self.dm, self.T, self.N, self.code, backward)

    def forward(self, ws=None, O=None, S=None, S0="own", cu="own", stream=None):
        ws = self.workspace() if ws is None else ws
        O = torch.full((self.T, self.hv * self.dv), 77.0, dtype=self.V.dtype, device="cuda") if O is None else O
        S = torch.full((self.N, self.hv, self.dv, self.dk), 77.0, device="cuda") if S is None else S
        S0 = self.S0 if isinstance(S0, str) else S0
        T.ttt_delta_chunked(self.Q, self.K, self.V, self.g, self.beta, S0, S, O, self.T, self.dm, self.io, ws,
                            cu_seqlens=self.cu if isinstance(cu, str) else cu, n_seq=self.N, scale=self.scale,
                            stream=stream)
        return O, S, ws

    def outputs_bwd(self):
        out = {}
        for name, t in (("dq", self.Q), ("dk", self.K), ("dv", self.V)):
            n = t.stride(0) if self.T > 1 else t.shape[1]
            out[name] = torch.full((self.T, n), 77.0, dtype=t.dtype, device="cuda")[:, :t.shape[1]]
        out["dg"], out["dbeta"] = torch.full_like(self.g, 77.0), torch.full_like(self.beta, 77.0)
        out["dS0"] = torch.full((self.N, self.hv, self.dv, self.dk), 77.0, device="cuda")
        return out

    def backward(self, ws=None, out=None, dS="own", stream=None):
        ws = self.workspace(True) if ws is None else ws
        out = self.outputs_bwd() if out is None else out
        T.ttt_delta_chunked_backward(self.Q, self.K, self.V, self.g, self.beta, self.S0, self.dO,
                                     self.dS if isinstance(dS, str) else dS, out["dq"], out["dk"], out["dv"],
                                     out["dg"], out["dbeta"], out["dS0"], self.T, self.dm, self.io, ws,
                                     cu_seqlens=self.cu, n_seq=self.N, scale=self.scale, stream=stream)
        return out, ws

    def _seq(self, i):
        a, b = self.starts[i], self.starts[i + 1]
        S0 = np.zeros((self.hv, self.dv, self.dk)) if self.S0 is None else f64(self.S0[i])
        return slice(a, b), [f64(t[a:b]) for t in (self.Q, self.K, self.V, self.g, self.beta)] + [S0]

    def check_forward(self, O, S):
        ref_o, got_o, ref_s = [], [], []
        for i in range(self.N):
            at, args = self._seq(i)
            o, s = D.delta_rule(*args, self.hk, self.hv, self.scale, bool(self.l2))
            ref_o.append(o)
            got_o.append(f64(O[at]))
            ref_s.append(s)
        tol = TOL_O if O.dtype == torch.bfloat16 else TOL_S
        if self.T:
            assert rel_fro(np.concatenate(got_o), np.concatenate(ref_o)) < tol
        assert rel_fro(f64(S), np.stack(ref_s)) < TOL_S

    def check_backward(self, out, dS="own"):
        ref = {}
        for i in range(self.N):
            at, args = self._seq(i)
            d = f64(self.dS[i]) if isinstance(dS, str) else np.zeros((self.hv, self.dv, self.dk))
            r = D.delta_rule_grad(*args, f64(self.dO[at]), d, self.hk, self.hv, self.scale, bool(self.l2))
            for k, v in r.items():
                ref.setdefault(k, []).append(v)
        live = slice(self.starts[0], self.starts[-1])
        for k, tol in (("dq", TOL_QK), ("dk", TOL_QK), ("dv", TOL_V), ("dg", TOL_G), ("dbeta", TOL_G)):
            assert rel_fro(f64(out[k][live]), np.concatenate(ref[k])) < tol, k
        assert rel_fro(f64(out["dS0"]), np.stack(ref["dS0"])) < TOL_S


# lens, heads_qk, heads_v, dk, dv, qk_l2norm, initial state, q/k/v as slices of one buffer
SHAPES = [
    ([1], 1, 1, 64, 64, 1, False, False),
    ([64], 1, 2, 64, 64, 1, True, False),
    ([65, 0, 1, 63, 130], 2, 4, 128, 128, 1, True, True),
    ([200], 2, 2, 192, 192, 1, True, False),
    ([129, 3], 1, 1, 256, 256, 1, False, True),
    ([150], 1, 3, 40, 72, 1, True, True),        # padded key and value widths, odd head count
    ([100, 28], 3, 3, 96, 16, 0, True, False),   # without the key norm
    ([70], 1, 1, 8, 8, 1, True, False),
    ([300], 1, 1, 64, 264, 1, False, False),     # more value channels than keys, past four blocks of 64
    ([0, 0], 1, 1, 64, 64, 1, True, False),
    ([40], 2, 4, 192, 128, 1, True, True),       # the longest call that runs token by token, and the next
    ([41], 2, 4, 192, 128, 1, True, True),
    ([7, 0, 1, 20], 1, 3, 256, 40, 0, True, False),
    ([5000], 1, 1, 64, 64, 1, True, False),      # few heads and long: cut into segments
    ([1500, 0, 2100, 30, 1], 1, 1, 192, 192, 1, True, True),
    ([1000, 1], 1, 2, 256, 64, 1, True, False),
    ([1700, 800], 1, 2, 128, 72, 1, False, False),
    ([1024, 1025], 2, 2, 40, 16, 0, True, False),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{max(s[0])}-{s[1]}.{s[2]}-{s[3]}.{s[4]}")
def test_forward(shape):
    lens, hk, hv, dk, dv, l2, s0, packed = shape
    c = Seqs(lens, hk, hv, dk, dv, seed=dk + dv, l2=l2, s0=s0, packed=packed)
    O, S, ws = c.forward()
    assert T.ttt_poll_status(ws) == T.TTT_OK
    c.check_forward(O, S)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{max(s[0])}-{s[1]}.{s[2]}-{s[3]}.{s[4]}")
def test_backward(shape):
    lens, hk, hv, dk, dv, l2, s0, packed = shape
    if not sum(lens):
        c = Seqs(lens, hk, hv, dk, dv)
        out, ws = c.backward()
        assert T.ttt_poll_status(ws) == T.TTT_OK and torch.equal(out["dS0"], c.dS)
        return
    c = Seqs(lens, hk, hv, dk, dv, seed=dk + dv + 1, l2=l2, s0=s0, packed=packed)
    out, ws = c.backward()
    assert T.ttt_poll_status(ws) == T.TTT_OK
    c.check_backward(out)


@pytest.mark.parametrize("lens,hk,hv,dk,dv", [([64, 64], 1, 1, 64, 64), ([1, 0, 37], 2, 4, 192, 128),
                                              ([90], 1, 1, 40, 24), ([20], 1, 2, 256, 64)])
def test_forward_fp32(lens, hk, hv, dk, dv):
    c = Seqs(lens, hk, hv, dk, dv, seed=9, dtype=torch.float32, packed=True)
    O, S, ws = c.forward()
    assert T.ttt_poll_status(ws) == T.TTT_OK
    c.check_forward(O, S)


@pytest.mark.parametrize("decay", [0.0, 30.0])
def test_no_decay_and_full_decay(decay):
    c = Seqs([200, 64], 1, 2, 64, 64, seed=3, decay=decay)
    c.check_forward(*c.forward()[:2])
    out, _ = c.backward()
    c.check_backward(out)


def test_closed_and_open_writes():
    # beta = 0 writes nothing, beta = 1 replaces; whole rows of each
    c = Seqs([130], 1, 2, 64, 64, seed=4)
    c.beta[::3] = 0.0
    c.beta[1::3] = 1.0
    c.check_forward(*c.forward()[:2])
    c.check_backward(c.backward()[0])


@pytest.mark.parametrize("scale", [1e-18, 1e18])
def test_range_of_values(scale):
    # states and errors are scaled by powers of two per row: the values' magnitude does not matter
    c = Seqs([140], 1, 1, 64, 64, seed=5, vscale=scale, s0=False)
    c.check_forward(*c.forward()[:2])
    c.dS *= 0
    c.check_backward(c.backward()[0])


def test_keys_of_any_magnitude_and_zero_keys():
    c = Seqs([140], 1, 1, 64, 64, seed=6)
    c.K[::2] = (c.K[::2].float() * 1e15).bfloat16()
    c.Q[1::2] = (c.Q[1::2].float() * 1e-10).bfloat16()
    c.K[7] = 0
    c.Q[70] = 0
    c.check_forward(*c.forward()[:2])


def test_large_state_with_small_writes():
    c = Seqs([140], 1, 1, 64, 64, seed=7, vscale=1e-30, decay=1e-3)
    c.S0 *= 1e6
    c.beta *= 1e-30
    c.check_forward(*c.forward()[:2])


@pytest.mark.parametrize("low", [float("-inf"), torch.finfo(torch.float32).min, -1e6])
def test_gates_that_forget(low):
    # a reset inside a chunk, at its border, twice in a row; the tokens behind it keep their own decays
    c = Seqs([200, 70], 1, 2, 64, 64, seed=25)
    for t in (0, 10, 11, 63, 64, 130, 205):
        c.g[t] = low
    c.check_forward(*c.forward()[:2])
    out, _ = c.backward()
    c.check_backward(out)
    pool, O = c.S0.clone(), torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 205], device="cuda")
    d = Seqs([1, 1], 1, 2, 64, 64, seed=25)
    d.Q, d.K, d.V, d.g, d.beta = (t[rows].contiguous() for t in (c.Q, c.K, c.V, c.g, c.beta))
    d.S0 = c.S0
    T.ttt_delta_step(d.Q, d.K, d.V, d.g, d.beta, pool, O, 2, d.dm, d.io, scale=d.scale)
    d.check_forward(O, pool)


def test_long_sequence_in_place():
    # cut into segments: the last one may end before the first has read the state that it overwrites
    c = Seqs([20000], 1, 1, 64, 64, seed=26)
    O, S, _ = c.forward()
    state = c.S0.clone()
    O2, _, ws = c.forward(S=state, S0=state)
    assert T.ttt_poll_status(ws) == T.TTT_OK
    assert torch.equal(O, O2) and torch.equal(S, state)


def test_workspace_of_a_larger_call():
    # sized for 16 sequences that are not cut, used for one that is
    big, c = Seqs([250] * 16, 4, 4, 64, 64, seed=29), Seqs([4000], 4, 4, 64, 64, seed=30)
    want, want_s, _ = c.forward()
    ws, wsb = big.workspace(), big.workspace(True)
    big.forward(ws=ws)
    O, S, _ = c.forward(ws=ws)
    assert torch.equal(O, want) and torch.equal(S, want_s)
    big.backward(ws=wsb)
    out, _ = c.backward(ws=wsb)
    ref, _ = c.backward()
    assert T.ttt_poll_status(wsb) == T.TTT_OK and all(torch.equal(out[k], ref[k]) for k in out)


def test_gradients_of_zero_and_tiny_rows():
    # x / max(||x||, 1e-12): a zero row passes 1e12 times the gradient, a tiny one 1 / ||x|| times its part across x
    c = Seqs([80], 1, 1, 64, 64, seed=27)
    c.K[5] = 0
    c.Q[70] = 0
    c.K[40] = (c.K[40].float() * 1e-9).bfloat16()
    out, _ = c.backward()
    at, args = c._seq(0)
    ref = D.delta_rule_grad(*args, f64(c.dO), f64(c.dS[0]), 1, 1, c.scale)
    for k, tol in (("dq", TOL_QK), ("dk", TOL_QK)):
        for rows in ([5], [40], [70], [i for i in range(80) if i not in (5, 40, 70)]):
            assert rel_fro(f64(out[k][rows]), ref[k][rows]) < tol, (k, rows)
    assert rel_fro(f64(out["dg"]), ref["dg"]) < TOL_G and rel_fro(f64(out["dbeta"]), ref["dbeta"]) < TOL_G


def test_many_sequences():
    # more than the chunk table sorts, lengths of 0 to 3
    lens = [i % 4 for i in range(1500)]
    c = Seqs(lens, 1, 1, 64, 64, seed=28)
    c.check_forward(*c.forward()[:2])
    c.check_backward(c.backward()[0])


def test_growing_gate():
    c = Seqs([100], 1, 1, 64, 64, seed=8)
    c.g = c.g.abs() * 0.3
    c.check_forward(*c.forward()[:2])
    c.check_backward(c.backward()[0])


def test_rows_outside_the_sequences_stay():
    c = Seqs([70, 5], 1, 2, 64, 64, seed=10, lead=3, tail=9)
    O, S, _ = c.forward()
    c.check_forward(O, S)
    assert torch.all(O[:3] == 77) and torch.all(O[-9:] == 77)
    out, _ = c.backward()
    c.check_backward(out)
    for k in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.all(out[k][:3] == 77) and torch.all(out[k][-9:] == 77), k


def test_equal_sequences_without_offsets():
    c = Seqs([48, 48, 48], 1, 1, 64, 64, seed=11)
    a, sa, _ = c.forward()
    b, sb, _ = c.forward(cu=None)
    assert torch.equal(a, b) and torch.equal(sa, sb)


def test_resuming_from_the_state_in_place():
    c = Seqs([256], 1, 2, 64, 64, seed=12)
    O, S, _ = c.forward()
    whole = c.__dict__.copy()
    state = c.S0.clone()
    parts = []
    for a, b in ((0, 128), (128, 256)):
        d = Seqs([b - a], 1, 2, 64, 64)
        d.Q, d.K, d.V, d.g, d.beta = (whole[n][a:b].contiguous() for n in ("Q", "K", "V", "g", "beta"))
        parts.append(d.forward(S=state, S0=state)[0])
    assert rel_fro(f64(torch.cat(parts)), f64(O)) < 2 * TOL_O
    assert rel_fro(f64(state), f64(S)) < TOL_S


@pytest.mark.parametrize("cu", [[0, 80, 60, 100], [0, 30, 60, 101], [-1, 30, 60, 100]])
def test_bad_offsets_write_nothing(cu):
    c = Seqs([30, 30, 40], 1, 1, 64, 64, seed=13)
    bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
    O, S, ws = c.forward(cu=bad)
    assert T.ttt_poll_status(ws) == T.TTT_ERR_INVALID
    assert torch.all(O == 77) and torch.all(S == 77)
    c.forward(ws=ws, O=O, S=S)  # while the error is recorded, calls on the workspace write nothing
    torch.cuda.synchronize()
    assert torch.all(O == 77)
    T.ttt_reset_status(ws)
    c.forward(ws=ws, O=O, S=S)
    assert T.ttt_poll_status(ws) == T.TTT_OK
    c.check_forward(O, S)


def test_a_nan_stays_in_its_sequence():
    c = Seqs([70, 70, 70], 1, 2, 64, 64, seed=14)
    clean, sc, _ = c.forward()
    c.V[75, 3] = float("nan")
    c.K[76, 1] = float("inf")
    O, S, ws = c.forward()
    assert T.ttt_poll_status(ws) == T.TTT_OK
    for i in (0, 2):
        at = slice(c.starts[i], c.starts[i + 1])
        assert torch.equal(O[at], clean[at]) and torch.equal(S[i], sc[i])


def test_deterministic_and_replayed_from_a_graph_on_another_stream():
    c = Seqs([65, 1, 200], 2, 4, 128, 128, seed=15)
    O, S, _ = c.forward()
    out, _ = c.backward()
    ws, wsb = c.workspace(), c.workspace(True)
    O2, S2 = torch.zeros_like(O), torch.zeros_like(S)
    out2 = c.outputs_bwd()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.forward(ws=ws, O=O2, S=S2)
        c.backward(ws=wsb, out=out2)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(O, O2) and torch.equal(S, S2) and all(torch.equal(out[k], out2[k]) for k in out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.forward(ws=ws, O=O2, S=S2)
        c.backward(ws=wsb, out=out2)
    c.V.mul_(2)
    want, ws_want, _ = c.forward()
    want_b, _ = c.backward()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, O2) and torch.equal(ws_want, S2) and all(torch.equal(want_b[k], out2[k]) for k in out)


def test_two_calls_at_once():
    a, b = Seqs([500], 2, 2, 64, 64, seed=16), Seqs([300, 200], 1, 4, 128, 64, seed=17)
    want = [c.forward()[:2] for c in (a, b)]
    wss = [c.workspace() for c in (a, b)]
    outs = [(torch.zeros_like(o), torch.zeros_like(s)) for o, s in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for c, ws, (o, s), st in zip((a, b), wss, outs, streams):
            c.forward(ws=ws, O=o, S=s, stream=st)
    torch.cuda.synchronize()
    for (o, s), (wo, wsn) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(s, wsn)


def test_offsets_past_32_bits():
    # rows 20,480 elements apart: the last tokens lie past 2^31 elements
    T_, ld = 110_000, 20_480
    buf = torch.zeros((T_, ld), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(18)
    x = torch.randn((T_, 192), generator=gen, device="cuda").bfloat16()
    buf[:, :192] = x
    c = Seqs([1], 1, 1, 64, 64)
    lens = [T_ - 100, 100]
    g = -torch.rand((T_, 1), generator=gen, device="cuda")
    beta = torch.rand((T_, 1), generator=gen, device="cuda")
    cu = torch.tensor([0, T_ - 100, T_], dtype=torch.int32, device="cuda")
    ws = T.delta_workspace(c.dm, T_, 2, T.TTT_BF16)
    S = [torch.zeros((2, 1, 64, 64), device="cuda") for _ in range(2)]
    O = torch.zeros((T_, 64), dtype=torch.bfloat16, device="cuda")
    io = T.io_cfg(ld_q=ld, ld_k=ld, ld_v=ld, ld_o=ld)
    T.ttt_delta_chunked(buf[:, :64], buf[:, 64:128], buf[:, 128:192], g, beta, None, S[0], buf[:, 192:256], T_, c.dm,
                        io, ws, cu_seqlens=cu, n_seq=len(lens))
    q, k, v = (x[:, i * 64:(i + 1) * 64].contiguous() for i in range(3))
    T.ttt_delta_chunked(q, k, v, g, beta, None, S[1], O, T_, c.dm, T.io_cfg(), ws, cu_seqlens=cu, n_seq=2)
    assert torch.equal(buf[:, 192:256], O) and torch.equal(S[0], S[1])
    assert torch.all(buf[:, 256:260] == 0)


# ---- one token at a time


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,hk,hv,dk,dv", [(1, 4, 4, 192, 192), (5, 2, 4, 128, 128), (3, 1, 1, 256, 40),
                                           (2, 1, 2, 40, 72), (17, 1, 1, 64, 8)])
def test_step(dtype, B, hk, hv, dk, dv):
    c = Seqs([1] * B, hk, hv, dk, dv, seed=20, dtype=dtype, packed=True)
    n = B + 3
    pool = torch.full((n, hv, dv, dk), 5.0, device="cuda")
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32)
    pool[slots.long().cuda()] = c.S0
    O = torch.full((B, hv * dv), 77.0, dtype=dtype, device="cuda")
    T.ttt_delta_step(c.Q, c.K, c.V, c.g, c.beta, pool, O, B, c.dm, c.io, slots=slots.cuda(), scale=c.scale)
    c.check_forward(O, pool[slots.long().cuda()])
    rest = sorted(set(range(n)) - set(slots.tolist()))
    assert torch.all(pool[rest] == 5)


def test_step_padding_and_repeated_slots():
    hv, d = 2, 64
    c = Seqs([6], 1, hv, d, d, seed=21)   # rows 0..5
    pool = torch.stack([c.S0[0], c.S0[0] * 2, c.S0[0] * 3])
    # rows 0, 2 and 5 are consecutive tokens of slot 1; rows 1 and 3 are padding; row 4 has slot 0
    slots = torch.tensor([1, -1, 1, 3, 0, 1], dtype=torch.int32, device="cuda")
    O = torch.full((6, hv * d), 77.0, dtype=torch.bfloat16, device="cuda")
    before = pool.clone()
    T.ttt_delta_step(c.Q, c.K, c.V, c.g, c.beta, pool, O, 6, c.dm, c.io, slots=slots, scale=c.scale)
    torch.cuda.synchronize()
    assert torch.all(O[[1, 3]] == 77) and torch.equal(pool[2], before[2])
    for rows, slot in (([0, 2, 5], 1), ([4], 0)):
        args = [f64(t[rows]) for t in (c.Q, c.K, c.V, c.g, c.beta)]
        o, s = D.delta_rule(*args, f64(before[slot]), 1, hv, c.scale)
        assert rel_fro(f64(O[rows]), o) < TOL_O and rel_fro(f64(pool[slot]), s) < TOL_S


def test_step_without_slots_and_none():
    c = Seqs([1, 1], 1, 1, 64, 64, seed=22)
    pool = c.S0.clone()
    O = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")
    T.ttt_delta_step(c.Q, c.K, c.V, c.g, c.beta, pool, O, 2, c.dm, c.io, scale=c.scale)
    c.check_forward(O, pool)
    T.ttt_delta_step(c.Q[:0], c.K[:0], c.V[:0], c.g[:0], c.beta[:0], pool, O[:0], 0, c.dm, c.io)


def test_prefill_then_steps_is_the_long_prefill():
    c = Seqs([75], 2, 4, 64, 128, seed=23)
    O, S, _ = c.forward()
    pool = torch.empty_like(S)
    Op = torch.zeros_like(O)
    cu = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    c.forward(O=Op, S=pool, cu=cu)
    for t in range(70, 75):
        at = slice(t, t + 1)
        T.ttt_delta_step(c.Q[at], c.K[at], c.V[at], c.g[at], c.beta[at], pool, Op[at], 1, c.dm, c.io, scale=c.scale)
    c.check_forward(Op, pool)
    assert rel_fro(f64(pool), f64(S)) < TOL_S


def test_step_in_a_graph():
    c = Seqs([1] * 4, 1, 2, 64, 64, seed=24)
    pool, want = c.S0.clone(), c.S0.clone()
    O = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    step = lambda p: T.ttt_delta_step(c.Q, c.K, c.V, c.g, c.beta, p, O, 4, c.dm, c.io, slots=slots)  # noqa: E731
    step(want.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(pool)
    for _ in range(3):
        graph.replay()
        step(want)
    torch.cuda.synchronize()
    assert torch.equal(pool, want)
