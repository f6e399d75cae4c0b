"""norm_gate at gates where exp(-z) overflows or vanishes: outputs and gradients, element by element.

Nothing in the definition overflows fp32 at |z| of 1e30, so everything is finite.  Each result is held against
the size of the terms that it is made of: fp32 within 1e-5; bf16, whose sigmoids are off by up to (4 + 1.2 |z|) 2^-23,
1.2e-5 at z = -80, within 2e-5 and half a step, 2^-8 of the value.  Sigmoids below 2^-126 (z below -87.3)
may be taken for 0: FLOOR, 90 * 1.2e-38 of the other factors, which are below 30 here.  The sigmoid's derivative
g (1 - g) takes 1 - g from a g that is off by 2^-22.
"""
import pytest
import torch

import block_norm_ref as ref
import chunked_gated_delta_07_gb300 as gdr

pytestmark = pytest.mark.gpu
FLOOR = 30 * 90 * 1.2e-38


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_07_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("big", [1e30, -1e30, 90.0, 3.0])
def test_extremes(big, kind, act, dtype):
    gen = torch.Generator(device="cuda").manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    z = torch.tensor([-200.0, -90.0, -88.0, -87.5, -80.0, -20.0, -1e30, 0.0, 17.0, 88.0, 200.0, 1.0, -1.0, 0.5, -0.5, big],
                     device="cuda").repeat(12, 1).to(dtype)
    x, dy = rnd(12, 16).to(dtype), rnd(12, 16).to(dtype)
    w, b = 1 + 0.2 * rnd(16), 0.1 * rnd(16)
    y, mean, rstd = gdr.norm_gate_fwd(x, z, w, b, kind=kind, act=act)
    dx, dz, dw, db = gdr.norm_gate_bwd(dy, x, z, rstd, mean, weight=w, bias=b, kind=kind, act=act, want_dbias=True)
    torch.cuda.synchronize()
    assert gdr.gdr_get_status() == gdr.GDR_OK
    assert all(t.isfinite().all() for t in (y, dx, dz, dw, db))

    X, Z, DY, W, B, rs = (t.double() for t in (x, z, dy, w, b, rstd[:, None]))
    xh = (X if mean is None else X - mean.double()[:, None]) * rs
    n, a, g, left = xh * W + B, ref.act(Z, act)[0], torch.sigmoid(Z), torch.sigmoid(-Z)
    n_size, a_size = (xh * W).abs() + B.abs(), a.abs()
    if act == "silu":   # g (1 + z (1 - g))
        slope, slope_size = g + g * Z * left, g + g * Z.abs() * left
    else:
        slope, slope_size = g * left, g * left + 2.0 ** -22 / 1e-5 * g
    dn = DY * a * W
    k = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    layer = kind == "layer"
    want_dx = rs * (dn - xh * k(dn * xh) - (k(dn) if layer else 0))
    dx_size = rs * (dn.abs() + xh.abs() * k((dn * xh).abs()) + (k(dn.abs()) if layer else 0))
    fine = 1e-5 if dtype == torch.float32 else 2e-5
    step = 0.0 if dtype == torch.float32 else 2.0 ** -8
    for name, got, want, size, rounding in (
            ("y", y, n * a, n_size * a_size, step), ("dx", dx, want_dx, dx_size, step),
            ("dgate", dz, DY * n * slope, DY.abs() * n_size * slope_size, step),
            ("dweight", dw, (DY * a * xh).sum(0), (DY * a * xh).abs().sum(0), 0.0),
            ("dbias", db, (DY * a).sum(0), (DY * a).abs().sum(0), 0.0)):
        off = (got.double() - want).abs() / (fine * size + rounding * want.abs() + 12 * FLOOR)
        assert float(off.max()) <= 1, f"{name}: {float(off.max()):.2f} of its bound at {int(off.argmax())}"
