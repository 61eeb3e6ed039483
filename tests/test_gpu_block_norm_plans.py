"""Block norms over every split of a row (threads to a row, chunks of 8 columns to a thread), in both types, on the GPU
against the fp64 oracle; and rows of one column, whose norm's gradient cancels.

Tolerances as derived for the block norms' tests: half a step of the output's type and 3e-6 for the sums; 1.2e-5 for the
weights' gradients, sums over the rows.
"""
import numpy as np
import pytest
import torch

from oracle import delta_oracle as D
from test_gpu_block_norm import TOL, TOL_W, Rows
from test_weight_layers_b200 import ttt as T

from _gpu import f64, need_gpu, rel_fro

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


# rows, D, group: with more rows than fill the card, a warp to a row up to 1024 columns, 128 threads up to 4096, 256
# above; the gradient 32, 128, 256 and 512 threads
PLANS = [(700, 200, None), (700, 512, None), (700, 768, None), (700, 1024, None), (600, 1536, None), (600, 2048, None),
         (600, 2600, None), (600, 4096, None), (600, 5000, None), (600, 8192, None), (700, 512, 128), (700, 768, 192),
         (600, 2048, 256), (600, 4096, 512), (600, 8192, 64), (300, 1000, 8)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("R,W,group", PLANS)
def test_forward_plans(R, W, group, dtype):
    c = Rows(R, W, group, dtype, seed=W + R)
    xo, n = D.block_norm(f64(c.Y), *c.args())
    Xo, N = c.forward()
    assert rel_fro(f64(Xo), xo) < TOL[dtype] and rel_fro(f64(N), n) < TOL[dtype]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("R,W,group", PLANS)
def test_backward_plans(R, W, group, dtype):
    c = Rows(R, W, group, dtype, seed=W + R + 1)
    X, Z, wp, lam, wn, grp = c.args()
    ref = D.block_norm_grad(f64(c.Y), f64(c.dXo), f64(c.dN), X, Z, wp, lam, wn, grp)
    for k, t in c.backward().items():
        assert rel_fro(f64(t), ref[k]) < (TOL_W if k.startswith(("dw", "dl")) else TOL[dtype]), k


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_unaligned_rows_of_many_columns(dtype):
    # element by element: odd strides and first elements
    for W, group in ((777, None), (2601, None), (1024, 128)):
        c = Rows(601, W, group, dtype, pad=3, shift=1, seed=W)
        X, Z, wp, lam, wn, grp = c.args()
        xo, n = D.block_norm(f64(c.Y), X, Z, wp, lam, wn, grp)
        Xo, N = c.forward()
        assert rel_fro(f64(Xo), xo) < TOL[dtype] and rel_fro(f64(N), n) < TOL[dtype]
        ref = D.block_norm_grad(f64(c.Y), f64(c.dXo), f64(c.dN), X, Z, wp, lam, wn, grp)
        for k, t in c.backward().items():
            assert rel_fro(f64(t), ref[k]) < (TOL_W if k.startswith(("dw", "dl")) else TOL[dtype]), k


def test_rows_of_one_column():
    """D = 1: the norm is +-1 up to eps.  What passes through it is u (1 - yh^2) r: the difference of two terms of size
    r u, each off by 2^-20 at most (twice yh's 2^-22 of the reciprocal root and 2^-24 of its product, and three roundings);
    everything else is held to the ordinary tolerances."""
    c = Rows(5, 1, None, torch.float32, seed=11)
    X, Z, wp, lam, wn, group = c.args()
    Y, dXo, dN = f64(c.Y), f64(c.dXo), f64(c.dN)
    tol = TOL[torch.float32]
    xo, _ = D.block_norm(Y, X, Z, wp, lam, wn, group)
    ry, r = 1 / np.sqrt(Y ** 2 + 1e-6), 1 / np.sqrt(xo ** 2 + 1e-6)
    silu = Z / (1 + np.exp(-Z))
    for dxo, dn in ((True, False), (True, True), (False, True)):
        ref = D.block_norm_grad(Y, dXo if dxo else None, dN if dn else None, X, Z, wp, lam, wn, group)
        out = {k: f64(t) for k, t in c.backward(dxo, dn).items()}
        off = 2 ** -20 * np.abs(r * dN * wn) if dn else 0 * Y      # in dx
        assert np.all(np.abs(out["dx"] - ref["dx"]) <= off + tol * np.abs(ref["dx"]))
        for k, factor in (("dz", np.abs(ref["dz"]) / np.maximum(np.abs(ref["dx"]), 1e-30)),):
            assert np.all(np.abs(out[k] - ref[k]) <= off * factor + 4 * tol * np.abs(ref[k])), k
        u = np.abs(lam * wp * silu)
        assert np.all(np.abs(out["dy"] - ref["dy"]) <= ry * u * (2 ** -20 * np.abs(ref["dx"]) + off))
        for k, factor in (("dw_post", np.abs(lam * silu)), ("dlam", np.abs(wp * silu))):
            assert np.all(np.abs(out[k] - ref[k]) <= (off * factor).sum() + TOL_W * np.abs(ref["dx"] * factor).sum()), k
        if dn:
            assert np.all(np.abs(out["dw_pre"] - ref["dw_pre"]) <= TOL_W * np.abs(dN).sum())
        else:
            assert np.all(out["dw_pre"] == 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_groups_as_rows_with_a_residual(dtype):
    # no second norm and no residual scale: the groups of strided rows are taken as rows of their own
    c = Rows(601, 512, 128, dtype, pad=8, seed=12)
    c.lam = c.w_pre = None
    ref, _ = D.block_norm(f64(c.Y), *c.args())
    Xo, _ = c.forward(n=False)
    assert rel_fro(f64(Xo), ref) < TOL[dtype]
    assert torch.all(Xo.as_strided((c.R - 1, c.pad), (c.W + c.pad, 1), Xo.storage_offset() + c.W) == 77)
    X, Z, wp, lam, wn, group = c.args()
    want = D.block_norm_grad(f64(c.Y), f64(c.dXo), None, X, Z, wp, lam, wn, group)
    dy, dz, dx, dw = c.blank(), c.blank(), c.blank(), torch.zeros(128, device="cuda")
    T.ttt_block_norm_backward(c.Y, c.dXo, dy, c.R, c.cfg, T.norm_workspace(c.R, c.cfg), X=c.X, Z=c.Z, w_post=c.w_post,
                              dX=dx, dZ=dz, dw_post=dw)
    for t, k in ((dy, "dy"), (dz, "dz"), (dx, "dx")):
        assert rel_fro(f64(t), want[k]) < TOL[dtype], k
    assert rel_fro(f64(dw), want["dw_post"]) < TOL_W


@pytest.mark.parametrize("shape", [(650, 768, None), (650, 768, 192), (9, 2600, None), (650, 8192, None)])
def test_every_output_on_an_input(shape):
    c = Rows(*shape, dtype=torch.float32, seed=13)
    Xo, N = c.forward()
    y, z = c.Y.clone(), c.Z.clone()
    T.ttt_block_norm(y, y, c.R, c.cfg, X=c.X, Z=z, w_post=c.w_post, res_scale=c.lam, w_pre=c.w_pre, N=z)
    assert torch.equal(y, Xo) and torch.equal(z, N)
    want = c.backward()
    y, z, x = c.Y.clone(), c.Z.clone(), c.X.clone()
    T.ttt_block_norm_backward(y, c.dXo, y, c.R, c.cfg, None, X=x, Z=z, w_post=c.w_post, res_scale=c.lam, w_pre=c.w_pre,
                              dN=c.dN, dX=x, dZ=z)
    assert torch.equal(y, want["dy"]) and torch.equal(z, want["dz"]) and torch.equal(x, want["dx"])


def test_one_weight_gradient_at_a_time():
    c = Rows(700, 768, None, seed=14)
    want = c.backward()
    ws = T.norm_workspace(c.R, c.cfg)
    for arg, k in (("dw_post", "dw_post"), ("dres_scale", "dlam"), ("dw_pre", "dw_pre")):
        out = torch.full((768,), 77.0, device="cuda")
        T.ttt_block_norm_backward(c.Y, c.dXo, None, c.R, c.cfg, ws, X=c.X, Z=c.Z, w_post=c.w_post, res_scale=c.lam,
                                  w_pre=c.w_pre, dN=c.dN, **{arg: out})
        assert torch.equal(out, want[k]), k


def test_two_gradients_at_once_and_in_two_graphs():
    cs = [Rows(700, 768, None, seed=15), Rows(400, 2048, 256, seed=16)]
    want = [c.backward() for c in cs]

    def call(c, ws, out):
        T.ttt_block_norm_backward(c.Y, c.dXo, out["dy"], c.R, c.cfg, ws, X=c.X, Z=c.Z, w_post=c.w_post,
                                  res_scale=c.lam, w_pre=c.w_pre, dN=c.dN, dX=out["dx"], dZ=out["dz"],
                                  dw_post=out["dw_post"], dres_scale=out["dlam"], dw_pre=out["dw_pre"])

    wss = [T.norm_workspace(c.R, c.cfg) for c in cs]
    outs = [{k: torch.zeros_like(t) for k, t in w.items()} for w in want]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, ws, out, st in zip(cs, wss, outs, streams):
            with torch.cuda.stream(st):
                call(c, ws, out)
    torch.cuda.synchronize()
    assert all(torch.equal(o[k], w[k]) for o, w in zip(outs, want) for k in w)
    graphs = []
    for c, ws, out in zip(cs, wss, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(c, ws, out)
        for t in out.values():
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o[k], w[k]) for o, w in zip(outs, want) for k in w)
