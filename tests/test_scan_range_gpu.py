"""The gated scan at both ends of fp32: what decays below it, and inputs, states and gradients of 1e-25 to 1e30.

A stretch of tokens is passed as h -> A h + B with A the product of its decays, so what a state leaves is off
by half of fp32's least number, 2^-150, of it for each of the stretches that it passes (at most 40 here), besides
roundings in proportion.
"""
import numpy as np
import pytest
import torch

import chunked_gated_delta_07_gb300 as gdr
import scan_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_07_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)


def run(x, a, h0, dout, dhT, lens, **form):
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    out, hT, states = gdr.gated_scan_fwd(x[None], a[None], h0=h0, cu_seqlens=cu, want_states=True, **form)
    dx, da, dh0 = gdr.gated_scan_bwd(x[None], a[None], dout[None], dhT, h0, states, cu, **form)
    torch.cuda.synchronize()
    assert gdr.gdr_get_status() == gdr.GDR_OK
    return out[0], hT, dx[0], da[0], dh0


@pytest.mark.parametrize("scale", [2.0 ** -83, 2.0 ** 99])   # 1e-25, 6e29
def test_every_size_of_values(scale):
    """Inputs, states and gradients times a power of two: results times it, within roundings near fp32's ends."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    lens, D = [300, 33, 700, 1], 40
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, a, h0, dout, dhT = rnd(1034, D), rnd(1034, D) - 2, rnd(4, D), rnd(1034, D), rnd(4, D)
    for source in ("plain", "convex", "variance"):
        one = run(x, a, h0, dout, dhT, lens, source=source)
        other = run(x * scale, a, h0 * scale, dout, dhT, lens, source=source)   # (da has both factors: its values too)
        for p, q, k in zip(one, other, (scale, scale, 1.0, scale, 1.0)):
            assert ((q.double() / k - p.double()).abs() <= 1e-6 * p.double().abs() + 1e-6).all()
        other = run(x, a, h0, dout * scale, dhT * scale, lens, source=source)
        for p, q, k in zip(one, other, (1.0, 1.0, scale, scale, scale)):
            assert ((q.double() / k - p.double()).abs() <= 1e-6 * p.double().abs() + 1e-6).all()


def test_what_decays_out_of_range():
    """softplus(57) = 57: two such tokens leave 1e-50 of a state, which a stretch's product cannot hold."""
    T, D = 200, 32
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, dout = torch.zeros(T, D, device="cuda"), torch.randn(T, D, generator=gen, device="cuda")
    for at in ((5,), (5, 6), (20, 21), (20, 40), (20, 150), (130, 131)):
        a = torch.full((T, D), -3.0, device="cuda")
        a[list(at)] = 57.0
        h0, dhT = torch.full((1, D), 1e30, device="cuda"), torch.randn(1, D, generator=gen, device="cuda")
        got = run(x, a, h0, dout, dhT, [T], gate="softplus")
        h, last = ref.forward(x, a, h0, [T], 0.0, "softplus", "plain")
        gx, ga, g0 = ref.backward(x, a, h0, dout, dhT, [T], 0.0, "softplus", "plain")
        lost = 40 * 2.0 ** -150
        # Decays within 3 * 2^-22, 200 of them.  l, a sum of terms of both signs, is off by up to 1e-6, that of terms of
        # size 1 (dx is l here); da = l (alpha h_{t-1}) g', whose second factor is h_t, by that times |h_t g'| too:
        # where the terms of l cancel, the error in proportion to da alone would be less than l's own.
        by_l = 1e-6 * h.abs() * torch.sigmoid(a.double().cpu())
        for p, q, size, more in zip(got, (h, last, gx, ga, g0), (1e30, 1e30, 8.0, 8e30, 8.0), (0.0, 0.0, 1e-6, by_l, 1e-6)):
            off = (p.double().cpu() - q).abs()
            assert (off <= 200 * 3 * 2.0 ** -22 * q.abs() + lost * size + more).all(), at
