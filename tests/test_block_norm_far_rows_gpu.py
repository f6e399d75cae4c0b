"""Norms around a block on rows whose mean is large against their spread (kind "layer").

Backward, against the formulas in 64 bits with the statistics that the call is given.  BOUND, 2-norm of
the error over the 2-norm of the result: the terms of a weight's sum are off by a few roundings each (the
mean taken off, the scaling, the products: 4 * 2^-24, a sigmoid within 2^-22 more; in the bf16 kernels
within (4 + 1.2 |z|) 2^-23, 7e-7 in the mean square at |z| of 2), of independent signs, and 512 of them added one by one by
sqrt(512 / 2) 2^-24 = 9.5e-7 at the most: 2e-6, and 3e-6 leaves room for the roundings of the rows' own
sums.  None of them grows with the mean.  bf16 outputs: one rounding, BOUND16 as for other rows.

Forward, against statistics in 64 bits: the mean, a sum of up to 2048 terms in a tree and a product, is
off by less than 8 * 2^-24 of itself, which every element of the row shares.
"""
import pytest
import torch

import block_norm_ref as ref
import chunked_gated_delta_07_gb300 as gdr

pytestmark = pytest.mark.gpu
BOUND, BOUND32, BOUND16, EPS = 3e-6, 1e-5, 4e-3, 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_07_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)


def close(got, want, bound, what):
    far = (got.double() - want).norm() / want.norm()
    assert float(far) <= bound, f"{what}: {float(far):.2e} > {bound}"


# (bf16: 400 + a spread of 1 in steps of 2)
@pytest.mark.parametrize("dtype,mean", [(torch.float32, 1000.0), (torch.float32, -100.0), (torch.bfloat16, 400.0)])
@pytest.mark.parametrize("shape,heads", [((512, 1000), False), ((300, 2047), False), ((256, 3, 128), True)])
def test_gradients(shape, heads, dtype, mean):
    gen = torch.Generator(device="cuda").manual_seed(shape[0])
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, z, dy, dr = (t.to(dtype) for t in (mean + rnd(*shape), 2 * rnd(*shape), rnd(*shape), rnd(*shape)))
    wshape = shape[-2:] if heads else shape[-1:]
    w, b = 1 + 0.2 * rnd(*wshape), 0.1 * rnd(*wshape)
    m, s = (t.float() for t in ref.stats(x.double(), "layer", EPS))
    tol = BOUND if dtype == torch.float32 else BOUND16
    got = gdr.add_norm_bwd(dy, x, s, m, dr=dr, weight=w, scale=0.5, kind="layer", want_dbias=True)
    want = ref.add_back(dy.double(), dr.double(), x.double(), m.double(), s.double(), w.double(), 0.5, "layer", wshape)
    for name, p, q, t in zip(("dx", "dresidual", "dweight", "dbias"), got, want, (tol, tol, BOUND, BOUND)):
        close(p, q, t, name)
    got = gdr.norm_gate_bwd(dy, x, z, s, m, weight=w, bias=b, scale=0.5, kind="layer", want_dbias=True)
    want = ref.gate_back(dy.double(), x.double(), z.double(), m.double(), s.double(), w.double(), b.double(), 0.5, "layer",
                         "silu", wshape)
    for name, p, q, t in zip(("dx", "dgate", "dweight", "dbias"), got, want, (tol, tol, BOUND, BOUND)):
        close(p, q, t, name)
    assert gdr.gdr_get_status() == gdr.GDR_OK


@pytest.mark.parametrize("D", [1000, 2047, 128])
def test_forward(D):
    gen = torch.Generator(device="cuda").manual_seed(D)
    x, z = 1000.0 + torch.randn(64, D, generator=gen, device="cuda"), torch.randn(64, D, generator=gen, device="cuda")
    tol = BOUND32 + 8 * 2.0 ** -24 * 1000
    y, r, mean, _ = gdr.add_norm_fwd(x, torch.zeros_like(x), kind="layer")
    assert torch.equal(r, x)
    close(y, ref.norm(x.double(), None, None, "layer", EPS), tol, "add_norm")
    close(mean, x.double().mean(-1), 8 * 2.0 ** -24, "mean")
    y = gdr.norm_gate_fwd(x, z, kind="layer")[0]
    close(y, ref.gate(x.double(), z.double(), None, None, None, 1.0, "layer", "silu", EPS), tol, "norm_gate")
    assert gdr.gdr_get_status() == gdr.GDR_OK
