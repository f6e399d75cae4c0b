"""The gated scan over many tiles and clusters of up to 16 blocks, element by element.

A result is a sum over its memory, up to a thousand tokens, each term off by its roundings: sqrt(1000) * 3 *
2^-24 = 5.7e-6 of the channel's root mean square in the mean square, seven times that at the worst of some
10^7 elements: 4e-5 of |value| + rms.  bf16 outputs have one more rounding, half a step, 2^-8 of the value at the most.  A single
wrong element, a misplaced cut or a lost first or last token is off by the order of the rms.
"""
import numpy as np
import pytest
import torch

import chunked_gated_delta_07_gb300 as gdr
import scan_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_07_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)


def each(got, want, what):
    """rms: of the channel, over tokens or sequences."""
    step = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    got = got.double().cpu().reshape(want.shape)
    rms = want.square().mean(0, keepdim=True).sqrt()
    off = (got - want).abs() / (step * want.abs() + 4e-5 * (want.abs() + rms) + 1e-30)
    at = np.unravel_index(int(off.argmax()), off.shape)
    assert float(off.max()) <= 1, f"{what} at {at}: {float(got[at]):.6g}, {float(want[at]):.6g}"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,D", [([20000], 64), ([9000, 1, 4000], 256), ([1] * 3000, 32), ([5] * 700, 1024),
                                    ([4097, 0, 33, 8000, 1, 127, 129, 128, 0, 2047], 63), ([33] * 300, 130),
                                    ([16] * 40 + [15] * 40 + [17] * 40 + [3000], 48)])
@pytest.mark.parametrize("packed", [True, False])
def test_elements(lens, D, dtype, packed):
    if not packed and len(set(lens)) > 1:
        lens = [max(lens)] * 3
    gen = torch.Generator(device="cuda").manual_seed(D)
    total, N = sum(lens), len(lens)
    shape = (1, total, D) if packed else (N, lens[0], D)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    far = 7.0 * torch.rand(D, generator=gen, device="cuda") - 6.0
    x, a, dout = (t.to(DT[dtype]) for t in (rnd(*shape), rnd(*shape) + far, rnd(*shape)))
    h0, dhT = rnd(N, D), rnd(N, D)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda") if packed else None
    out, hT, states = gdr.gated_scan_fwd(x, a, h0=h0, cu_seqlens=cu, source="variance", want_states=True)
    dx, da, dh0 = gdr.gated_scan_bwd(x, a, dout, dhT, h0, states, cu, source="variance")
    torch.cuda.synchronize()
    assert gdr.gdr_get_status() == gdr.GDR_OK
    flat = [t.reshape(-1, D) for t in (x, a, dout)]
    form = dict(b=2.0, gate="bounded", source="variance")
    h, last = ref.forward(flat[0], flat[1], h0, lens, **form)
    gx, ga, g0 = ref.backward(flat[0], flat[1], h0, flat[2], dhT, lens, **form)
    each(out, h, "out")
    each(states, h[127::128], "states")
    each(dx, gx, "dx")
    each(da, ga, "da")
    rms = h.square().mean(0, keepdim=True).sqrt()   # (one sequence: its state may be anywhere below that)
    assert ((hT.double().cpu() - last).abs() <= 4e-5 * (last.abs() + rms)).all()
    assert ((dh0.double().cpu() - g0).abs() <= 4e-5 * (g0.abs() + (gx.square().mean(0, keepdim=True).sqrt()))).all()
