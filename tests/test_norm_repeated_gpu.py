"""Layer norm backward, called again and again: the weights' gradients of every call equal the
first call's bit for bit, and that one the formula in 64 bits (GPU).

A block adds up its groups' partial sums through the shared memory that held the ring of rows; a
row copy that arrived there late would drop a group's sums from one call and not from the next.
So the shapes have several groups to a block (rows of up to 2048 elements in 16-byte pieces),
a few steps of the ring or many, and ends at which no group, some or all are past the last row.
"""
import pytest
import torch

import chunked_gated_delta_07_gb300 as gdr
import decay_ref as ref
from test_norm_gpu import BOUND32, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_07_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("shape,per_head", [
    ((1, 128), False), ((33, 128), False), ((20011, 128), False), ((700, 16, 128), True), ((4096, 3, 64), True),
    ((6007, 256), False), ((3001, 1024), False), ((1500, 2048), False)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_call_gives_the_same_sums(shape, per_head, dtype):
    x, dy, w, b = inputs(shape, per_head, dtype, 900 + len(shape))
    _, mean, rstd = gdr.layer_norm_fwd(x, w, b)
    dx, dw, db = gdr.layer_norm_bwd(dy, x, mean, rstd, w)
    _, rw, rb = ref.norm_bwd(dy, x, mean, rstd, w, per_head)
    assert ref.rel(dw, rw) <= BOUND32 and ref.rel(db, rb) <= BOUND32
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        got = gdr.layer_norm_bwd(dy, x, mean, rstd, w)
        for a, c in zip(got, (dx, dw, db)):
            differ += (a != c).sum()
    assert int(differ) == 0
