"""Large and small magnitudes in the decay linear attention (GPU).

The CUDA cores scale values by up to lam^-15 inside a block of tokens, at most e^15 = 2^22, so products
scale k v below 2^104 overflow nowhere.  The tensor cores divide a tile's outputs by factors f >= 2^-64
while they add them up, which allows |scale q.k| and |out / scale| up to 2^62, and take 2^-64 of
scale S^T q into outputs that the decay leaves less of the entering state S.  Results within
those limits are as exact, relative to their size, as at usual magnitudes: bounds as in test_decay_gpu.
"""
import pytest
import torch

import chunked_gated_delta_07_gb300 as gdr
from test_decay_gpu import check_bwd, check_fwd, inputs, seg_tiles  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu
SLOPES = [3.9, 0.9, 0.3, 0.01]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_07_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)


def scaled(x, **by):
    return {n: t * by[n] if n in by and t is not None else t for n, t in x.items()}


@pytest.mark.parametrize("seg_tiles", [0, 1], indirect=True)
@pytest.mark.parametrize("size", [1e14, 1e25, 1e30, 1e-25])
@pytest.mark.parametrize("dtype,path", [("bf16", "auto"), ("bf16", "simt"), ("f32", "auto")])
def test_values(seg_tiles, size, dtype, path):  # noqa: F811
    """Values, and so states and outputs, of this size; in the backward pass dout and dhT."""
    if path == "auto" and dtype == "bf16" and size > 2.0 ** 62:
        pytest.skip("beyond the tensor cores' range")
    x = inputs(2, 333, 4, 128, 128, dtype, 500, slopes=SLOPES)
    check_fwd(scaled(x, v=size, h0=size), path)
    check_bwd(scaled(x, dout=size, dhT=size), path)


@pytest.mark.parametrize("dtype,path", [("bf16", "auto"), ("bf16", "simt"), ("f32", "auto")])
def test_keys(dtype, path):
    """q.k of 1e18 = 2^60."""
    x = inputs(2, 333, 4, 128, 128, dtype, 510, slopes=SLOPES)
    check_fwd(scaled(x, q=1e9, k=1e9, h0=1e9), path)


@pytest.mark.parametrize("dtype,path", [("bf16", "auto"), ("bf16", "simt"), ("f32", "auto")])
def test_entering_state(dtype, path):
    """A state 2^40 times the size of what is written: once it has faded, 2^-24 of an output is left of
    it on the tensor cores where there should be nothing."""
    x = inputs(2, 333, 4, 128, 128, dtype, 520, slopes=SLOPES)
    faded = scaled(x, h0=2.0 ** 40)
    out, _ = gdr.decay_fwd(faded["q"], faded["k"], faded["v"], faded["g"], h0=faded["h0"], scale=0.5, path=path)
    want, _ = gdr.decay_fwd(x["q"], x["k"], x["v"], x["g"], scale=0.5, path=path)
    torch.cuda.synchronize()
    # the fastest head, from where lam^i 2^40 is below 2^-24
    far = (out[:, 20:, 0].double() - want[:, 20:, 0].double()).abs()
    assert float(far.max()) <= 2.0 ** -22 + (2.0 ** -7 * want[:, 20:, 0].double().abs()).max() * (dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_single_tokens(dtype):
    x = inputs(3, 20, 4, 128, 128, dtype, 530, slopes=SLOPES)
    for T in (1, 4, 20):
        y = {n: x[n][:, :T].contiguous() * (1e30 if n == "v" else 1) for n in ("q", "k", "v")}
        state = x["h0"] * 1e30
        want_state = state.clone()
        out = gdr.decay_recurrent_fwd(y["q"], y["k"], y["v"], x["g"], state)
        small = x["h0"].clone()
        want = gdr.decay_recurrent_fwd(y["q"], y["k"], (y["v"].double() / 1e30).to(y["v"].dtype), x["g"], small)
        torch.cuda.synchronize()
        assert out.isfinite().all() and state.isfinite().all() and not torch.equal(state, want_state)
        # the same numbers in other units: roundings differ where 1e30 is not a power of two
        assert float((out.double() / 1e30 - want.double()).norm() / want.double().norm()) <= 1e-2
        assert float((state.double() / 1e30 - small.double()).norm() / small.double().norm()) <= 1e-2


@pytest.mark.parametrize("seg_tiles", [0, 1], indirect=True)
@pytest.mark.parametrize("dtype,path", [("bf16", "auto"), ("bf16", "simt"), ("f32", "auto")])
def test_heads_that_grow(seg_tiles, dtype, path):  # noqa: F811
    """Log-decays above 0: 200 tokens take the state to e^2, e^20 and e^80 of itself."""
    x = inputs(2, 200, 3, 128, 64, dtype, 540, slopes=[-0.01, -0.1, -0.4])
    check_fwd(x, path)
    check_bwd(x, path)
