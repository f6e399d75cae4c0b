"""Decay calls on the tensor-core path without tokens pass the states on (GPU)."""
import pytest
import torch

import chunked_gated_delta_07_gb300 as gdr
from test_decay_gpu import inputs, ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_07_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("lens", [None, [0, 0]])
@pytest.mark.parametrize("path", ["auto", "tc", "simt"])
def test_states_go_through(lens, path):
    x = inputs(2, 0, 3, 128, 64, "bf16", 860, lens=lens)
    out, hT = gdr.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], cu_seqlens=x["cu"], path=path)
    dq, dk, dv, dh0 = gdr.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["dout"], dhT=x["dhT"], h0=x["h0"],
                                    cu_seqlens=x["cu"], path=path)
    ok()
    assert torch.equal(hT, x["h0"]) and torch.equal(dh0, x["dhT"])
    assert out.shape == x["v"].shape and dq.shape == dk.shape == x["q"].shape and dv.shape == x["v"].shape
