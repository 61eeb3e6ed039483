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
