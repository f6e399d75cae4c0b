"""The gated scan's decay and weight, element by element.

One token: from h0 = 1 and x = 0 the state is alpha, with dout = 1 the gradient of h0 is; from nothing
and x = 1 the convex source leaves 1 - alpha.  In units of U = 2^-22, relative to the value, with s the
sigmoid, q = 1 - s, n = b s, from the error bounds of the special-function unit (an exponential of base
two within U, a reciprocal within U / 2) and half a step, U / 4, for every other operation:

fp32 tensors.  e^-a: 1.25 (the argument's rounding error is put back, with a rounding or two of its own).  s: q 1.25 + 1/4
  + 1/2, n: 1/4 more.  alpha is off by what n is off by, n (1.25 q + 1), and by an exponential of its own, 1.75
  (from n = 1/2 on; below that 1 - alpha <= 0.4 comes from a polynomial, and alpha's own part is less).
  1 - alpha: below n = 1/2 n's part, at most 2.25, and the polynomial's, 1; from there on alpha's error
  times alpha / (1 - alpha), which is at most 0.77 / n and 1.54, 0.77 * 2.25 + 1.54 * 1.75 = 4.4.
  Softplus: 1.25 + 1/4 + 1/2 + 1/4 = 2.25 on either side of 0, and a rounding.
bf16 tensors.  e^-a has its argument's error too, |a| / 2; bounds of at most 2 take 1 - alpha from one polynomial,
  off by 3.6e-8 and the roundings of its terms, which alpha >= e^-2 shows 7.4 times: 21 * 2^-24 at b = 2.
"""
import math

import pytest
import torch

import chunked_gated_delta_07_gb300 as gdr

pytestmark = pytest.mark.gpu
U = 2.0 ** -22


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_07_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)


def gates(D, dtype, b, gate):
    """a and, in 64 bits, alpha, 1 - alpha and the bound of alpha's error."""
    a = torch.linspace(-16, 16, D, device="cuda").to(dtype).reshape(1, 1, D)
    e = a.double().reshape(1, D)
    if gate == "softplus":
        bound = torch.full_like(e, 3 * U) if dtype == torch.float32 else (3 + e.abs() / 2) * U
        return a, torch.sigmoid(-e), torch.sigmoid(e), bound
    n, q = b * torch.sigmoid(e), torch.sigmoid(-e)
    if dtype == torch.float32:
        bound = (n * (1.25 * q + 1) + 1.75) * U
    else:
        bound = (n * (q * (1 + e.abs() / 2) + 1.5) + (21 / 4 if b <= 2 else 2)) * U
    return a, torch.exp(-n), -torch.expm1(-n), bound


def within(got, want, bound, what):
    off = (got.double().reshape(want.shape) / want - 1).abs() / bound
    assert float(off.max()) <= 1, f"{what}: {float(off.max()):.2f} of its bound"


@pytest.mark.parametrize("D", [4096, 4095])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate,b", [("bounded", 0.25), ("bounded", 1.0), ("bounded", 2.0), ("bounded", 3.0), ("bounded", 8.0),
                                    ("softplus", 0.0)])
def test_decay(gate, b, dtype, D):
    a, alpha, _, bound = gates(D, dtype, b, gate)
    h0, zero, one = torch.ones(1, D, device="cuda"), torch.zeros_like(a), torch.ones_like(a)
    for source in ("plain", "variance"):
        form = dict(b=b, gate=gate, source=source)
        within(gdr.gated_scan_fwd(zero, a, h0=h0, **form)[1], alpha, bound, "hT")
        within(gdr.gated_scan_bwd(zero, a, one, h0=h0, **form)[2], alpha, bound, "dh0")
        state = h0.clone()
        gdr.gated_scan_recurrent_fwd(zero, a, state, **form)
        within(state, alpha, bound, "state")
    assert gdr.gdr_get_status() == gdr.GDR_OK


@pytest.mark.parametrize("gate,b", [("bounded", 0.25), ("bounded", 1.0), ("bounded", 2.0), ("bounded", 8.0), ("softplus", 0.0)])
def test_weight(gate, b):
    """fp32: also where a memory is long and 1 - alpha 2e-7."""
    D = 4096
    a, _, left, _ = gates(D, torch.float32, b, gate)
    form = dict(b=b, gate=gate, source="convex")
    bound = torch.full_like(left, 5 * U)
    within(gdr.gated_scan_fwd(torch.ones_like(a), a, **form)[1], left, bound, "hT")
    within(gdr.gated_scan_bwd(torch.zeros_like(a), a, torch.ones_like(a), **form)[0], left, bound, "dx")
    assert gdr.gdr_get_status() == gdr.GDR_OK


def test_decays_add_up():
    """What the decay of fp32 tensors is off by at the bound's end, alpha = e^-2 (1 + d), stays within its
    bound over tokens of the same gate: h = x / (1 - alpha) in the end."""
    a = torch.full((1, 64, 32), 20.0, device="cuda")
    out, _, _ = gdr.gated_scan_fwd(torch.ones_like(a), a, source="plain")
    want = 1 / (1 - math.exp(-2.0 / (1 + math.exp(-20.0))))
    # alpha's bound times alpha / (1 - alpha) = 0.157, and the rounding of each step, 2^-24 / (1 - alpha)
    assert float((out[0, -1].double() / want - 1).abs().max()) <= 0.157 * 3.75 * U + 2 * 2.0 ** -24
    assert gdr.gdr_get_status() == gdr.GDR_OK
