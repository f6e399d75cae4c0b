"""Layer norm with very many weight rows: as many as the calls accept, more than a grid's second axis
counts (GPU; the 64-bit formula runs on the GPU too, for its size).  Bounds as in test_norm_gpu."""
import pytest
import torch

import chunked_gated_delta_07_gb300 as gdr
from test_norm_gpu import BOUND16, BOUND32, DT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_07_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)


def rel(a, r):
    return float((a.double() - r).norm() / r.norm())


@pytest.mark.parametrize("shape,dtype", [((1, 65537, 2056), "bf16"), ((1, 70000, 4099), "bf16"), ((2, 66000, 1028), "f32"),
                                         ((1, 131073, 1024), "bf16"), ((1, 1 << 20, 8), "bf16"), ((3, 1 << 20, 5), "f32")])
def test_weight_rows(shape, dtype):
    gen = torch.Generator(device="cuda").manual_seed(shape[1])
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, dy = (rnd(*shape) * 1.5 + 0.3).to(DT[dtype]), rnd(*shape).to(DT[dtype])
    w, b = 1 + 0.2 * rnd(*shape[1:]), 0.1 * rnd(*shape[1:])
    y, mean, rstd = gdr.layer_norm_fwd(x, w, b)
    dx, dw, db = gdr.layer_norm_bwd(dy, x, mean, rstd, w)
    bound = BOUND16 if dtype == "bf16" else BOUND32
    xd = x.double()
    m = xd.mean(-1, keepdim=True)
    r = ((xd - m).square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    assert rel(y, (xd - m) * r * w + b) <= bound
    assert rel(mean, m[..., 0]) <= BOUND32 and rel(rstd, r[..., 0]) <= BOUND32
    m, r, dyd = mean.double()[..., None], rstd.double()[..., None], dy.double()
    xh = (xd - m) * r
    wdy = dyd * w
    want = r * (wdy - wdy.mean(-1, keepdim=True) - xh * (wdy * xh).mean(-1, keepdim=True))
    far = float((dx.double() - want).norm())
    assert far <= (BOUND16 * float(want.norm()) if dtype == "bf16" else 0.0) + BOUND32 * float((r * wdy).norm())
    assert rel(dw, (dyd * xh).sum(0)) <= BOUND32 and rel(db, dyd.sum(0)) <= BOUND32
