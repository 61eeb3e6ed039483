"""Host-side refusals of the gated delta rule and block norm entry points: documented codes before any device work."""
import ctypes

import pytest
import torch

from test_weight_layers_b200 import build as B
from test_weight_layers_b200 import ttt as T

FAKE = [ctypes.c_void_p((i + 1) << 24) for i in range(20)]  # aligned, never dereferenced
OK, INV, UNS, WS, AL = (T.TTT_OK, T.TTT_ERR_INVALID, T.TTT_ERR_UNSUPPORTED, T.TTT_ERR_WORKSPACE, T.TTT_ERR_ALIGN)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return T.lib()


def _fwd(lib, dm=None, dt=T.TTT_BF16, T_=256, n_seq=2, io=None, ws_bytes=1 << 40, cu=FAKE[10], Q=FAKE[0], O=FAKE[7],
         S0=FAKE[5], g=FAKE[3], ws=FAKE[11]):
    dm = dm or T.delta_dims(2, 4, 128, 64)
    io = io or T.io_cfg()
    return lib.ttt_delta_chunked(Q, FAKE[1], FAKE[2], g, FAKE[4], S0, FAKE[6], O, cu, n_seq, T_, 1.0, dm,
                                 ctypes.byref(io), dt, ws, ws_bytes, None)


def _bwd(lib, dm=None, dt=T.TTT_BF16, T_=256, n_seq=2, ws_bytes=1 << 40, dQ=FAKE[8], dg=FAKE[9]):
    dm = dm or T.delta_dims(2, 4, 128, 64)
    return lib.ttt_delta_chunked_backward(FAKE[0], FAKE[1], FAKE[2], FAKE[3], FAKE[4], None, FAKE[5], None, dQ,
                                          FAKE[12], FAKE[13], dg, FAKE[14], None, FAKE[10], n_seq, T_, 1.0, dm,
                                          ctypes.byref(T.io_cfg()), dt, FAKE[11], ws_bytes, None)


def _step(lib, dm=None, dt=T.TTT_BF16, B_=4, slots=FAKE[10], n_slots=8, S=FAKE[6], O=FAKE[7], io=None):
    dm = dm or T.delta_dims(2, 4, 128, 64)
    io = io or T.io_cfg()
    return lib.ttt_delta_step(FAKE[0], FAKE[1], FAKE[2], FAKE[3], FAKE[4], S, n_slots, slots, O, B_, 1.0, dm,
                              ctypes.byref(io), dt, None)


def test_delta_shapes(lib):
    for bad in ((0, 1, 64, 64), (2, 3, 64, 64), (1, 1, 0, 64), (1, 1, 64, -8)):
        assert _fwd(lib, T.delta_dims(*bad)) == INV, bad
        assert lib.ttt_delta_workspace_bytes(T.delta_dims(*bad), 10, 1, T.TTT_BF16, 0) == 0
    for uns in ((1, 1, 60, 64), (1, 1, 264, 64), (1, 1, 64, 12), (1, 1, 64, 1032), (1, 8192, 64, 64)):
        assert _fwd(lib, T.delta_dims(*uns)) == UNS, uns
        assert _step(lib, T.delta_dims(*uns)) == UNS, uns
        assert _bwd(lib, T.delta_dims(*uns)) == UNS, uns
        assert lib.ttt_delta_workspace_bytes(T.delta_dims(*uns), 10, 1, T.TTT_BF16, 0) == 0
    assert _fwd(lib, dt=5) == INV and _step(lib, dt=5) == INV and _bwd(lib, dt=5) == INV
    assert _bwd(lib, dt=T.TTT_FP32) == UNS
    assert _fwd(lib, T_=1 << 31) == UNS and _fwd(lib, T_=-1) == INV and _fwd(lib, n_seq=-1) == INV


def test_delta_arguments(lib):
    assert _fwd(lib, Q=None) == INV and _fwd(lib, g=None) == INV and _fwd(lib, O=FAKE[2]) == INV
    assert _fwd(lib, Q=ctypes.c_void_p((1 << 24) + 2)) == AL
    assert _fwd(lib, S0=ctypes.c_void_p((1 << 24) + 4)) == AL
    assert _fwd(lib, io=T.io_cfg(ld_k=100)) == INV            # ld < heads * dk
    assert _fwd(lib, io=T.io_cfg(ld_v=260)) == AL             # 520-byte rows
    assert _fwd(lib, cu=None, n_seq=3) == INV                 # 256 tokens in 3 equal sequences
    assert _fwd(lib, cu=None, n_seq=0) == INV
    assert _fwd(lib, n_seq=0, T_=256) == OK                   # offsets of no sequence: nothing to do
    assert _fwd(lib, n_seq=(1 << 24) + 1) == UNS
    assert lib.ttt_delta_chunked_backward(*FAKE[:5], None, FAKE[5], FAKE[6], FAKE[8], FAKE[12], FAKE[13], FAKE[9],
                                          FAKE[14], FAKE[6], FAKE[10], 2, 256, 1.0, T.delta_dims(2, 4, 128, 64),
                                          ctypes.byref(T.io_cfg()), T.TTT_BF16, FAKE[11], 1 << 40, None) == INV  # dS0 = dS
    assert _bwd(lib, dQ=None) == INV and _bwd(lib, dg=None) == INV and _bwd(lib, dQ=FAKE[0]) == INV
    assert _step(lib, slots=None, B_=9) == INV                # more rows than slots
    assert _step(lib, S=None) == INV and _step(lib, O=FAKE[0]) == INV and _step(lib, B_=-1) == INV
    assert _step(lib, B_=0) == OK


def test_delta_workspace(lib):
    dm = T.delta_dims(2, 4, 128, 64)
    for dt in (T.TTT_BF16, T.TTT_FP32):
        need = lib.ttt_delta_workspace_bytes(dm, 256, 2, dt, 0)
        assert need > 0 and _fwd(lib, dt=dt, ws_bytes=need - 1) == WS
    need = lib.ttt_delta_workspace_bytes(dm, 256, 2, T.TTT_BF16, 1)
    assert need > lib.ttt_delta_workspace_bytes(dm, 256, 2, T.TTT_BF16, 0)
    assert _bwd(lib, ws_bytes=need - 1) == WS
    assert _fwd(lib, ws=None) == WS and _fwd(lib, ws=ctypes.c_void_p((1 << 24) + 128)) == WS


def test_delta_workspace_serves_every_smaller_call(lib):
    # long sequences of few heads are cut, which takes room that more or shorter ones do not need
    for dims in ((4, 4, 192, 192), (1, 1, 64, 64), (8, 16, 128, 128), (2, 2, 256, 40)):
        dm = T.delta_dims(*dims)
        for back in (0, 1):
            size = lambda t, n: lib.ttt_delta_workspace_bytes(dm, t, n, T.TTT_BF16, back)  # noqa: E731, B023
            grid = [(t, n) for t in (0, 40, 700, 705, 768, 1374, 5000, 9999, 40000, 131072) for n in (1, 2, 3, 7, 16, 50, 400)]
            for t, n in grid:
                assert all(size(t, n) >= size(u, m) for u, m in grid if u <= t and m <= n), (dims, t, n)
            # ... and each call's own need is within its query
            for t, n in grid:
                if t:
                    rc = _fwd(lib, dm, T_=t, n_seq=n, ws_bytes=size(t, n), Q=ctypes.c_void_p((1 << 24) + 2))
                    assert rc == AL, (dims, t, n)  # past the workspace check, stopped at Q's alignment


def _norm(lib, cfg, dt=T.TTT_BF16, Y=FAKE[0], Xo=FAKE[1], N=FAKE[2], X=FAKE[3], T_=8, w=FAKE[4]):
    return lib.ttt_block_norm(X, Y, None, w, None, None, Xo, N, T_, ctypes.byref(cfg), dt, None)


def _norm_bwd(lib, cfg, dt=T.TTT_BF16, dXo=FAKE[1], dN=FAKE[2], X=FAKE[3], Z=None, dX=FAKE[5], dY=FAKE[6], dZ=None,
              dw=FAKE[7], T_=8, ws_bytes=1 << 40, ws=FAKE[8]):
    return lib.ttt_block_norm_backward(X, FAKE[0], Z, FAKE[4], None, None, dXo, dN, dX, dY, dZ, dw, None, None, T_,
                                       ctypes.byref(cfg), dt, ws, ws_bytes, None)


def test_block_norm_refusals(lib):
    for call in (_norm, _norm_bwd):
        assert call(lib, T.norm_cfg(768, 100)) == INV          # group does not divide D
        assert call(lib, T.norm_cfg(0)) == INV and call(lib, T.norm_cfg(768, eps=-1.0)) == INV
        assert call(lib, T.norm_cfg(8200)) == UNS
        assert call(lib, T.norm_cfg(768, 12)) == UNS           # several groups, not of a multiple of 8
        assert call(lib, T.norm_cfg(768), dt=3) == INV and call(lib, T.norm_cfg(768), T_=-1) == INV
        assert call(lib, T.norm_cfg(768, ld_x=700)) == INV
    assert _norm(lib, T.norm_cfg(768), Y=None) == INV and _norm(lib, T.norm_cfg(768), Xo=None, N=None) == INV
    assert _norm(lib, T.norm_cfg(768), Y=ctypes.c_void_p((1 << 24) + 1)) == AL
    assert _norm(lib, T.norm_cfg(768), w=ctypes.c_void_p((1 << 24) + 2)) == AL
    assert _norm(lib, T.norm_cfg(768), T_=0) == OK
    cfg = T.norm_cfg(768)
    assert _norm_bwd(lib, cfg, dXo=None, dN=None) == INV and _norm_bwd(lib, cfg, X=None) == INV
    assert _norm_bwd(lib, cfg, dZ=FAKE[9]) == INV              # dZ without Z
    need = lib.ttt_block_norm_workspace_bytes(ctypes.byref(cfg), 8)
    assert need > 0 and _norm_bwd(lib, cfg, ws_bytes=need - 1) == WS and _norm_bwd(lib, cfg, ws=None) == WS
    assert lib.ttt_block_norm_workspace_bytes(ctypes.byref(T.norm_cfg(768, 100)), 8) == 0


def test_binding_refuses_tensors_that_do_not_match():
    q, bad = torch.zeros(4, 256), torch.zeros(4, 250)
    with pytest.raises(ValueError):
        T._rows("Q", bad, 4, 256, 0, torch.float32)            # too few columns
    with pytest.raises(ValueError):
        T._rows("Q", q, 5, 256, 0, torch.float32)              # too few rows
    with pytest.raises(ValueError):
        T._rows("Q", q, 4, 256, 0, torch.bfloat16)
    with pytest.raises(ValueError):
        T._rows("Q", torch.zeros(4, 512)[:, :256], 4, 256, 0, torch.float32)  # stride the call does not say
    T._rows("Q", torch.zeros(4, 512)[:, :256], 4, 256, 512, torch.float32)
    with pytest.raises(ValueError):
        T._dense("g", torch.zeros(4, 3), (4, 2))
    with pytest.raises(ValueError):
        T._dense("g", torch.zeros(2, 4).t(), (4, 2))
