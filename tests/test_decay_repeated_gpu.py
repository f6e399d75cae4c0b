"""Decay linear attention called again and again: every call's results equal the first call's bit
for bit (GPU; the other tests compare single calls with the definition).

The kernels' warps hand tiles, products and units to each other through shared and tensor memory.
Where one of them came too early or too late, it would show in a call now and then, so every
call's results are looked at and not the last one's alone.  Segments make the local pass run; short
last tiles its zeroed rows, and the outputs' stores row by row.
"""
import pytest
import torch

import chunked_gated_delta_07_gb300 as gdr
from test_decay_gpu import inputs, ok, seg_tiles  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu
LENS = [1 + (37 * i) % 300 for i in range(60)] + [2000, 3000]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_07_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)


def differing(call, first, times):
    """Values that differ from the first call's, over so many calls."""
    n = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(times):
        for a, c in zip(call(), first):
            n += (a != c).sum()
    ok()   # no wait ran out either
    return int(n)


@pytest.mark.parametrize("seg_tiles", [0, 1, 3], indirect=True)
@pytest.mark.parametrize("dk,dv,H,lens", [(64, 64, 16, LENS), (128, 128, 8, LENS), (128, 64, 8, LENS), (128, 128, 16, None),
                                          (64, 64, 16, None)])
def test_every_backward_call_gives_the_same(seg_tiles, dk, dv, H, lens):  # noqa: F811
    x = inputs(2, 3001, H, dk, dv, "bf16", 710, lens=lens)
    call = lambda: gdr.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["dout"], dhT=x["dhT"], h0=x["h0"],  # noqa: E731
                                 cu_seqlens=x["cu"], scale=0.5)
    assert differing(call, call(), 200) == 0


@pytest.mark.parametrize("seg_tiles", [0, 1, 3], indirect=True)
@pytest.mark.parametrize("dk,dv,H,lens", [(64, 64, 32, LENS), (128, 128, 16, LENS), (64, 128, 16, LENS),
                                          (128, 128, 16, None), (64, 64, 16, None)])
def test_every_forward_call_gives_the_same(seg_tiles, dk, dv, H, lens):  # noqa: F811
    x = inputs(2, 3001, H, dk, dv, "bf16", 720, lens=lens)
    call = lambda: gdr.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], cu_seqlens=x["cu"], scale=0.5)  # noqa: E731
    assert differing(call, call(), 500) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [LENS, None])
def test_every_call_on_the_cuda_cores_gives_the_same(dtype, lens):
    x = inputs(2, 1001, 3, 128, 64, dtype, 730, lens=lens)
    call = lambda: gdr.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["dout"], dhT=x["dhT"], h0=x["h0"],  # noqa: E731
                                 cu_seqlens=x["cu"], scale=0.5, path="simt")
    assert differing(call, call(), 100) == 0


@pytest.mark.parametrize("T", [1, 5, 20])
def test_every_decoding_call_gives_the_same(T):
    x = inputs(64, T, 16, 128, 128, "bf16", 740)

    def call():
        state = x["h0"].clone()
        return gdr.decay_recurrent_fwd(x["q"], x["k"], x["v"], x["g"], state, scale=0.5), state

    assert differing(call, call(), 200) == 0
