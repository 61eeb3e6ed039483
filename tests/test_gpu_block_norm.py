"""Block norms on the GPU against the fp64 oracle, through the C ABI.

Tolerances (relative Frobenius norms): a bf16 output is rounded once (2^-8 at most) from fp32 sums; an fp32 one is
off by its sums' rounding, D / 8 terms per thread and a tree over the threads: below 2^-24 * (8192 / 256 + 16) < 3e-6.
The weights' gradients sum up to 4096 fp32 products per thread and block: taken as 4 times that.
"""
import numpy as np
import pytest
import torch

from oracle import delta_oracle as D
from test_weight_layers_b200 import ttt as T

from _gpu import f64, need_gpu, rel_fro

pytestmark = pytest.mark.gpu

TOL = {torch.bfloat16: 2 ** -8 + 3e-6, torch.float32: 3e-6}
TOL_W = 1.2e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


class Rows:
    def __init__(self, R, W, group=None, dtype=torch.bfloat16, res=True, gate=True, weights=True, pad=0, shift=0, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.R, self.W, self.group, self.dtype, self.pad, self.shift = R, W, group or W, dtype, pad, shift
        rows = lambda s=1.0: self.blank().copy_((rn(R, W) * s).to(dtype))  # noqa: E731
        self.Y, self.X, self.Z = rows(2.0), rows() if res else None, rows() if gate else None
        self.w_post = 1 + 0.2 * rn(self.group) if weights else None
        self.lam = 0.5 + 0.1 * rn(W) if weights and (res or self.group == W) else None
        self.w_pre = 1 + 0.2 * rn(W) if weights else None
        self.dXo, self.dN = rows(), rows()
        ld = W + pad
        self.cfg = T.norm_cfg(W, self.group, 1e-6, ld, ld, ld, ld, ld)

    def blank(self, fill=77.0):
        buf = torch.full((self.R * (self.W + self.pad) + self.shift,), fill, dtype=self.dtype, device="cuda")
        return buf[self.shift:].view(self.R, self.W + self.pad)[:, :self.W]

    def forward(self, xo=True, n=True, lam=True):
        Xo, N = self.blank() if xo else None, self.blank() if n else None
        T.ttt_block_norm(self.Y, Xo, self.R, self.cfg, X=self.X, Z=self.Z, w_post=self.w_post,
                         res_scale=self.lam if lam else None, w_pre=self.w_pre if n else None, N=N)
        return Xo, N

    def args(self, lam=True):
        o = lambda t: None if t is None else f64(t)  # noqa: E731
        return o(self.X), o(self.Z), o(self.w_post), o(self.lam) if lam else None, o(self.w_pre), self.group

    def backward(self, dxo=True, dn=True):
        e = lambda t: None if t is None else torch.full_like(t, 77.0)  # noqa: E731
        out = {"dy": self.blank(), "dx": self.blank() if self.X is not None else None,
               "dz": self.blank() if self.Z is not None else None, "dw_post": e(self.w_post), "dlam": e(self.lam),
               "dw_pre": e(self.w_pre)}
        ws = T.norm_workspace(self.R, self.cfg)
        T.ttt_block_norm_backward(self.Y, self.dXo if dxo else None, out["dy"], self.R, self.cfg, ws, X=self.X,
                                  Z=self.Z, w_post=self.w_post, res_scale=self.lam, w_pre=self.w_pre,
                                  dN=self.dN if dn else None, dX=out["dx"], dZ=out["dz"], dw_post=out["dw_post"],
                                  dres_scale=out["dlam"], dw_pre=out["dw_pre"])
        return out


# rows, D, group, dtype, residual, gate, weights, row padding, element shift of the first row
SHAPES = [
    (1, 1, None, torch.float32, True, True, True, 0, 0),
    (3, 7, None, torch.bfloat16, True, True, True, 0, 0),
    (7, 768, None, torch.float32, True, True, True, 0, 0),
    (33, 768, 192, torch.bfloat16, True, True, True, 0, 0),      # four means to a row, with the second norm
    (33, 768, 192, torch.bfloat16, False, True, True, 8, 0),
    (5, 777, None, torch.bfloat16, True, False, True, 3, 1),     # odd width, stride and alignment
    (600, 1000, None, torch.bfloat16, True, True, False, 0, 0),  # no weights
    (40, 2048, 64, torch.float32, True, True, True, 0, 0),
    (9, 2056, None, torch.bfloat16, False, False, True, 24, 8),
    (6, 8192, None, torch.bfloat16, True, True, True, 0, 0),
    (3, 8192, 1024, torch.float32, True, False, True, 0, 0),
    (2000, 64, None, torch.bfloat16, True, True, True, 0, 0),
]
IDS = [f"{s[0]}x{s[1]}-{s[2]}-{str(s[3])[6:]}-{int(s[4])}{int(s[5])}{int(s[6])}" for s in SHAPES]


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward(shape):
    c = Rows(*shape, seed=shape[0] + shape[1])
    xo, n = D.block_norm(f64(c.Y), *c.args())
    for want_xo, want_n in ((True, True), (True, False), (False, True)):
        Xo, N = c.forward(want_xo, want_n)
        if want_xo:
            assert rel_fro(f64(Xo), xo) < TOL[c.dtype]
        if want_n:
            assert rel_fro(f64(N), n) < TOL[c.dtype]
        for t in (Xo, N):
            if t is not None and c.pad and c.R > 1:  # what lies between the rows stays
                assert torch.all(t.as_strided((c.R - 1, c.pad), (c.W + c.pad, 1), t.storage_offset() + c.W) == 77)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_backward(shape):
    c = Rows(*shape, seed=shape[0] + shape[1] + 1)
    for dxo, dn in ((True, True), (False, True), (True, False)):
        out = c.backward(dxo, dn)
        X, Z, wp, lam, wn, group = c.args()
        ref = D.block_norm_grad(f64(c.Y), f64(c.dXo) if dxo else None, f64(c.dN) if dn else None, X, Z, wp, lam, wn,
                                group)
        for k, t in out.items():
            if t is not None:
                if np.linalg.norm(ref[k]) == 0:
                    assert torch.all(t == 0), k
                else:
                    # D = 1: a norm of one value is +-1, and its gradient cancels to about eps
                    tol = (TOL_W if k.startswith(("dw", "dl")) else TOL[c.dtype]) if c.W > 1 else 1.0
                    assert rel_fro(f64(t), ref[k]) < tol, (k, dxo, dn)


def test_head_norm_without_second_norm_runs_groups_as_rows():
    c = Rows(50, 512, 128, res=False, seed=5)
    c.lam = None
    Xo, _ = c.forward(n=False)
    assert rel_fro(f64(Xo), D.block_norm(f64(c.Y), *c.args())[0]) < TOL[c.dtype]
    out = torch.zeros(128, device="cuda")
    dy, dz = c.blank(), c.blank()
    T.ttt_block_norm_backward(c.Y, c.dXo, dy, c.R, c.cfg, T.norm_workspace(c.R, c.cfg), Z=c.Z, w_post=c.w_post, dZ=dz,
                              dw_post=out)
    ref = D.block_norm_grad(f64(c.Y), f64(c.dXo), None, None, f64(c.Z), f64(c.w_post), None, None, 128)
    for t, k in ((dy, "dy"), (dz, "dz")):
        assert rel_fro(f64(t), ref[k]) < TOL[c.dtype]
    assert rel_fro(f64(out), ref["dw_post"]) < TOL_W


def test_in_place_residual_stream():
    c = Rows(100, 768, seed=6)
    Xo, N = c.forward()
    x = c.X.clone()
    N2 = c.blank()
    T.ttt_block_norm(c.Y, x, c.R, c.cfg, X=x, Z=c.Z, w_post=c.w_post, res_scale=c.lam, w_pre=c.w_pre, N=N2)
    assert torch.equal(x, Xo) and torch.equal(N, N2)
    want = c.backward()
    d = c.dXo.clone()  # the stream's gradient in place
    dy, dz = c.blank(), c.blank()
    T.ttt_block_norm_backward(c.Y, d, dy, c.R, c.cfg, None, X=c.X, Z=c.Z, w_post=c.w_post, res_scale=c.lam,
                              w_pre=c.w_pre, dN=c.dN, dX=d, dZ=dz)
    assert torch.equal(d, want["dx"]) and torch.equal(dy, want["dy"]) and torch.equal(dz, want["dz"])


def test_no_rows():
    c = Rows(4, 64, seed=7)
    c.R = 0
    T.ttt_block_norm(c.Y, c.blank(), 0, c.cfg)
    out = torch.full((64,), 77.0, device="cuda")
    T.ttt_block_norm_backward(c.Y, c.dXo, None, 0, c.cfg, T.norm_workspace(0, c.cfg), dw_pre=out)
    torch.cuda.synchronize()
    assert torch.all(out == 0)


def test_zero_and_non_finite_rows_stay_by_themselves():
    c = Rows(64, 768, seed=8)
    Xo, N = c.forward()
    c.Y[3] = 0
    c.X[3] = 0
    c.Y[9, 5] = float("nan")
    c.X[20, 1] = float("inf")
    c.Z[30] = -3e38  # SiLU underflows to zero: p = 0
    Xo2, N2 = c.forward()
    keep = [i for i in range(64) if i not in (3, 9, 20, 30)]
    assert torch.equal(Xo[keep], Xo2[keep]) and torch.equal(N[keep], N2[keep])
    assert torch.all(Xo2[3] == 0) and torch.all(N2[3] == 0) and torch.equal(Xo2[30], c.X[30])


def test_rows_past_32_bits_deterministic_and_in_a_graph():
    R, W, ld = 270_000, 64, 8192  # the last rows lie past 2^31 elements
    buf = torch.zeros((R, ld), dtype=torch.bfloat16, device="cuda")
    y = torch.randn((R, W), generator=torch.Generator(device="cuda").manual_seed(9), device="cuda").bfloat16()
    buf[:, :W] = y
    far, near = T.norm_cfg(W, ld_y=ld, ld_xout=ld), T.norm_cfg(W)
    w = torch.rand(W, device="cuda")
    T.ttt_block_norm(buf[:, :W], buf[:, W:2 * W], R, far, w_post=w)
    out = torch.zeros_like(y)
    T.ttt_block_norm(y, out, R, near, w_post=w)
    assert torch.equal(buf[:, W:2 * W], out)
    ws = T.norm_workspace(R, near)
    grads = []
    for _ in range(2):
        dy, dw = torch.zeros_like(y), torch.zeros_like(w)
        T.ttt_block_norm_backward(y, out, dy, R, near, ws, w_post=w, dw_post=dw)
        grads.append((dy, dw))
    assert torch.equal(grads[0][0], grads[1][0]) and torch.equal(grads[0][1], grads[1][1])
    graph = torch.cuda.CUDAGraph()
    dy, dw = torch.zeros_like(y), torch.zeros_like(w)
    with torch.cuda.graph(graph):
        T.ttt_block_norm_backward(y, out, dy, R, near, ws, w_post=w, dw_post=dw)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dy, grads[0][0]) and torch.equal(dw, grads[0][1])
