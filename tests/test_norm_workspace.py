"""The scratch of the layer norm's backward pass: the caller's own, so that it can run on a stream beside
other calls that need scratch (refusals on the CPU, the results on the GPU)."""
import pytest
import torch

import chunked_gated_delta_07_gb300 as gdr
from chunked_gated_delta_07_gb300 import _build
from test_decay_gpu import inputs as decay_inputs
from test_norm_gpu import inputs as norm_inputs


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()


def nbwd(**kw):
    a = dict(dy=1 << 20, x=2 << 20, mean=3 << 20, rstd=4 << 20, weight=5 << 20, dx=6 << 20, dweight=7 << 20,
             dbias=8 << 20, rows=8, G=2, D=128, dtype=gdr.GDR_BF16, workspace=9 << 20, workspace_bytes=1 << 20, stream=0)
    a.update(kw)
    return gdr.gdr_layer_norm_bwd_ex(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(workspace=(9 << 20) + 8), gdr.GDR_ERR_INVALID_ARG), (dict(rows=7), gdr.GDR_ERR_INVALID_ARG),
    (dict(dy=None), gdr.GDR_ERR_INVALID_ARG), (dict(dx=3 << 20), gdr.GDR_ERR_INVALID_ARG),
    (dict(D=16385), gdr.GDR_ERR_UNSUPPORTED)])
def test_refusals(kw, code):
    assert nbwd(**kw) == code


def test_sizes():
    size = gdr.gdr_layer_norm_bwd_workspace_size
    assert size(0, 1, 128) == 0 and size(7, 2, 128) == 0 and size(8, 2, 0) == 0 and size(8, 2, 16385) == 0
    # two partial sums at least, and no more than two for every resident block
    assert 2 * 4 * 2048 <= size(8191, 1, 2048) <= 2 * 4 * 2048 * 4 * 160
    assert size(8, 2, 128, gdr.GDR_F32) >= 2 * 4 * 2 * 128


def test_workspace_must_be_on_the_device_and_contiguous():
    t = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        gdr.layer_norm_bwd(t, t, t[:, 0].contiguous(), t[:, 0].contiguous(), workspace=torch.zeros(1 << 16))


@pytest.fixture
def cuda():
    torch.cuda.set_device(0)


def sized(rows, G, D, dtype=gdr.GDR_BF16):
    return torch.empty(gdr.gdr_layer_norm_bwd_workspace_size(rows, G, D, dtype), dtype=torch.uint8, device="cuda")


@pytest.mark.gpu
def test_too_small(cuda):
    x, dy, w, b = norm_inputs((500, 256), False, "bf16", 1)
    _, mean, rstd = gdr.layer_norm_fwd(x, w, b)
    for n in (0, 16, gdr.gdr_layer_norm_bwd_workspace_size(500, 1, 256) - 16):
        with pytest.raises(gdr.GdrError) as e:
            gdr.layer_norm_bwd(dy, x, mean, rstd, w, workspace=torch.empty(max(n, 1), dtype=torch.uint8, device="cuda"))
        assert e.value.code == gdr.GDR_ERR_NO_WORKSPACE
    # no gradients of the weights: no scratch
    gdr.layer_norm_bwd(dy, x, mean, rstd, w, want_dweight=False, want_dbias=False, workspace=sized(500, 1, 256)[:16])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [128, 1000, 999, 2048])
def test_streams_side_by_side(cuda, D):
    """Two norms and a decay backward on three streams, each with its own scratch, again and again: all
    equal what they give alone."""
    rows, calls = 20000, []
    for seed in (1, 2):
        x, dy, w, b = norm_inputs((rows, D), False, "bf16", seed)
        _, mean, rstd = gdr.layer_norm_fwd(x, w, b)
        ws = sized(rows, 1, D)
        calls.append(lambda s, x=x, dy=dy, w=w, m=mean, r=rstd, ws=ws: gdr.layer_norm_bwd(dy, x, m, r, w, stream=s,
                                                                                         workspace=ws))
    y = decay_inputs(1, 9000, 4, 128, 128, "bf16", 3)
    ws = torch.empty(gdr.gdr_decay_workspace_size(1, 9000, 4, 128, 128, backward=True), dtype=torch.uint8, device="cuda")
    calls.append(lambda s: gdr.decay_bwd(y["q"], y["k"], y["v"], y["g"], y["dout"], dhT=y["dhT"], h0=y["h0"], stream=s,
                                         workspace=ws))
    alone = [c(None) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    differ = [torch.zeros((), dtype=torch.int64, device="cuda") for _ in calls]
    torch.cuda.synchronize()
    for _ in range(30):
        for i, (c, s) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(s):   # (the outputs' memory belongs to the stream too)
                for a, e in zip(c(s), alone[i]):
                    differ[i] += (a != e).sum()
    torch.cuda.synchronize()
    assert [int(d) for d in differ] == [0, 0, 0] and gdr.gdr_get_status() == gdr.GDR_OK
