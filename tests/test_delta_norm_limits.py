"""Host-side limits of the gated delta rule's entry points: what is documented as allowed is not refused."""
import ctypes

import pytest

from test_weight_layers_b200 import build as B
from test_weight_layers_b200 import ttt as T

FAKE = [ctypes.c_void_p((i + 1) << 24) for i in range(20)]  # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 24) + 2)
OK, INV, UNS, WS, AL = (T.TTT_OK, T.TTT_ERR_INVALID, T.TTT_ERR_UNSUPPORTED, T.TTT_ERR_WORKSPACE, T.TTT_ERR_ALIGN)
DM = T.delta_dims(2, 2, 64, 64)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return T.lib()


@pytest.mark.parametrize("same", [0, 1, 2])
def test_the_outputs_gradient_may_be_an_input(lib, same):
    # dO is read only; a misaligned dbeta stops the call behind the check of the inputs
    call = lambda dO, dV: lib.ttt_delta_chunked_backward(  # noqa: E731
        *FAKE[:5], None, dO, None, FAKE[8], FAKE[12], dV, FAKE[9], ODD, None, FAKE[10], 2, 256, 1.0, DM,
        ctypes.byref(T.io_cfg()), T.TTT_BF16, FAKE[11], 1 << 40, None)
    assert call(FAKE[same], FAKE[13]) == AL          # stopped at dbeta's alignment
    good = lambda dO, dV: lib.ttt_delta_chunked_backward(  # noqa: E731
        *FAKE[:5], None, dO, None, FAKE[8], FAKE[12], dV, FAKE[9], FAKE[14], None, FAKE[10], 2, 256, 1.0, DM,
        ctypes.byref(T.io_cfg()), T.TTT_BF16, FAKE[11], 1 << 40, None)
    assert good(FAKE[same], FAKE[same]) == INV       # an output on an input is refused
    assert good(FAKE[5], FAKE[5]) == INV             # ... and on dO


def test_outputs_on_inputs_are_refused(lib):
    io = ctypes.byref(T.io_cfg())
    for same in range(3):
        assert lib.ttt_delta_chunked(*FAKE[:5], None, None, FAKE[same], FAKE[10], 2, 256, 1.0, DM, io, T.TTT_BF16,
                                     FAKE[11], 1 << 40, None) == INV
        assert lib.ttt_delta_step(*FAKE[:5], FAKE[6], 8, FAKE[10], FAKE[same], 4, 1.0, DM, io, T.TTT_BF16, None) == INV


def test_an_empty_pool(lib):
    # NULL is what an empty tensor has; every row is padding, so nothing is launched
    step = lambda S, n, slots: lib.ttt_delta_step(  # noqa: E731
        *FAKE[:5], S, n, slots, FAKE[7], 4, 1.0, DM, ctypes.byref(T.io_cfg()), T.TTT_BF16, None)
    assert step(None, 0, FAKE[10]) == OK and step(FAKE[6], 0, FAKE[10]) == OK
    assert step(None, 8, FAKE[10]) == INV and step(None, 0, None) == INV


def test_the_largest_calls(lib):
    # the documented limits themselves are taken (stopped at Q's alignment), one more is not
    def fwd(t, n, cu=FAKE[10]):
        return lib.ttt_delta_chunked(ODD, *FAKE[1:5], None, None, FAKE[7], cu, n, t, 1.0, DM, ctypes.byref(T.io_cfg()),
                                     T.TTT_BF16, FAKE[11], 1 << 62, None)
    top, most = 2 ** 31 - 65, 1 << 24
    assert fwd(top, 1) == AL and fwd(top + 1, 1) == UNS
    assert fwd(256, most) == AL and fwd(256, most + 1) == UNS
    for t, n, some in ((top, 1, True), (top + 1, 1, False), (256, most, True), (256, most + 1, False)):
        assert (lib.ttt_delta_workspace_bytes(DM, t, n, T.TTT_BF16, 0) > 0) == some
