"""The reference gradients of the norms around a block against differences, and what the calls
refuse (CPU only)."""
import pytest
import torch

import block_norm_ref as ref
import chunked_gated_delta_07_gb300 as gdr
from chunked_gated_delta_07_gb300 import _build

INV, UNS = gdr.GDR_ERR_INVALID_ARG, gdr.GDR_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()


def difference(loss, args, k, way):
    ends = []
    for e in (1e-5, -1e-5):
        moved = list(args)
        moved[k] = moved[k] + e * way
        ends.append(float(loss(*moved)))
    return (ends[0] - ends[1]) / 2e-5


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gradients_against_differences(kind, act):
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, res, z, dy, dr, w, b = rnd(6, 9), rnd(6, 9), rnd(6, 9), rnd(6, 9), rnd(6, 9), rnd(9), rnd(9)
    scale, eps = 0.5, 1e-5
    r = res + scale * x
    mean, rstd = ref.stats(r, kind, eps)
    add = ref.add_back(dy, dr, r, mean, rstd, w, scale, kind, (9,))

    def loss_add(x, res, w, b):
        s = res + scale * x
        return (dy * ref.norm(s, w, b, kind, eps) + dr * s).sum()

    mean, rstd = ref.stats(x, kind, eps)
    gate = ref.gate_back(dy, x, z, mean, rstd, w, b, scale, kind, act, (9,))
    loss_gate = lambda x, z, w, b: (dy * ref.gate(x, z, w, b, res, scale, kind, act, eps)).sum()  # noqa: E731
    for loss, args, grads in ((loss_add, (x, res, w, b), add), (loss_gate, (x, z, w, b), gate)):
        for k, g in enumerate(grads):
            way = rnd(*g.shape)
            # the central difference is off by e^2 times a third derivative, and by 2^-53 / e of the loss
            assert abs(difference(loss, args, k, way) - float((g * way).sum())) < 1e-7 * (1 + float((g * way).abs().sum()))


def call(fn, base):
    return lambda **kw: fn(**{**base, **kw})


SIZES = dict(rows=8, G=2, D=128, scale=0.5, kind=gdr.GDR_NORM_RMS, dtype=gdr.GDR_BF16, stream=0)
WS = dict(workspace=30 << 20, workspace_bytes=1 << 24)
add_fwd = call(gdr.gdr_add_norm_fwd, dict(x=1 << 20, residual=2 << 20, weight=3 << 20, bias=4 << 20, sum=5 << 20, y=6 << 20,
                                          mean=None, rstd=8 << 20, eps=1e-5, **SIZES))
add_bwd = call(gdr.gdr_add_norm_bwd, dict(dy=1 << 20, dsum=2 << 20, sum=3 << 20, mean=None, rstd=5 << 20, weight=6 << 20,
                                          dx=7 << 20, dresidual=8 << 20, dweight=9 << 20, dbias=10 << 20, **SIZES, **WS))
gate_fwd = call(gdr.gdr_norm_gate_fwd, dict(x=1 << 20, gate=2 << 20, weight=3 << 20, bias=4 << 20, residual=5 << 20, y=6 << 20,
                                            mean=None, rstd=8 << 20, eps=1e-5, act=gdr.GDR_ACT_SILU, **SIZES))
gate_bwd = call(gdr.gdr_norm_gate_bwd, dict(dy=1 << 20, x=2 << 20, gate=3 << 20, mean=None, rstd=5 << 20, weight=6 << 20,
                                            bias=11 << 20, dx=7 << 20, dgate=8 << 20, dweight=9 << 20, dbias=10 << 20,
                                            act=gdr.GDR_ACT_SILU, **SIZES, **WS))
COMMON = [(dict(rows=-2), INV), (dict(rows=7), INV), (dict(G=0), INV), (dict(D=0), INV), (dict(D=16385), UNS),
          (dict(dtype=3), INV), (dict(kind=2), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
          (dict(rows=1 << 41), UNS), (dict(mean=20 << 20), INV)]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(x=None), INV), (dict(residual=None), INV), (dict(sum=None), INV),
    (dict(y=None), INV), (dict(sum=1 << 20), INV), (dict(y=2 << 20), INV), (dict(sum=(2 << 20) + 2), INV),
    (dict(y=(1 << 20) + 2), INV), (dict(y=5 << 20), INV), (dict(y=3 << 20), INV), (dict(rstd=1 << 20), INV),
    (dict(kind=gdr.GDR_NORM_LAYER, mean=8 << 20), INV)])
def test_add_forward_refuses(kw, code):
    assert add_fwd(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(dy=None), INV), (dict(sum=None), INV), (dict(rstd=None), INV), (dict(dresidual=None), INV), (dict(dx=8 << 20), INV),
    (dict(dx=(1 << 20) + 2), INV), (dict(dx=5 << 20), INV), (dict(dweight=1 << 20), INV), (dict(dbias=9 << 20), INV),
    (dict(dweight=6 << 20), INV), (dict(kind=gdr.GDR_NORM_LAYER), INV), (dict(workspace=(30 << 20) + 8), INV)])
def test_add_backward_refuses(kw, code):
    assert add_bwd(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(act=2), INV), (dict(eps=float("inf")), INV), (dict(x=None), INV), (dict(gate=None), INV), (dict(y=None), INV),
    (dict(y=(1 << 20) + 2), INV), (dict(y=(5 << 20) + 2), INV), (dict(y=4 << 20), INV), (dict(rstd=2 << 20), INV)])
def test_gate_forward_refuses(kw, code):
    assert gate_fwd(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(act=-1), INV), (dict(dy=None), INV), (dict(x=None), INV), (dict(gate=None), INV), (dict(rstd=None), INV),
    (dict(dx=None), INV), (dict(dgate=None), INV), (dict(dgate=7 << 20), INV), (dict(dx=(3 << 20) + 2), INV),
    (dict(dx=11 << 20), INV), (dict(dweight=3 << 20), INV), (dict(kind=gdr.GDR_NORM_LAYER), INV),
    (dict(workspace=(30 << 20) + 4), INV)])
def test_gate_backward_refuses(kw, code):
    assert gate_bwd(**kw) == code


def test_sizes():
    size = gdr.gdr_block_norm_bwd_workspace_size
    assert size(0, 1, 128) == 0 and size(7, 2, 128) == 0 and size(8, 2, 0) == 0 and size(8, 2, 16385) == 0
    assert 2 * 4 * 2048 <= size(8191, 1, 2048) <= 2 * 4 * 2048 * 4 * 160


def test_tensors():
    x = torch.zeros(4, 3, 8)
    st = torch.zeros(4, 3)
    assert gdr.check_block_norm_inputs(x, torch.zeros(3, 8), gate=x, dy=None) == (12, 3, 8)
    for kw in (dict(weight=torch.zeros(7)), dict(gate=torch.zeros(4, 3, 7)), dict(dy=x.bfloat16()), dict(rstd=torch.zeros(4)),
               dict(kind="batch"), dict(residual=torch.zeros(3, 4, 8).transpose(0, 1))):
        with pytest.raises(ValueError):
            gdr.check_block_norm_inputs(x, **kw)
    for fn in (lambda: gdr.add_norm_fwd(x, x), lambda: gdr.add_norm_bwd(x, x, st), lambda: gdr.norm_gate_fwd(x, x),
               lambda: gdr.norm_gate_bwd(x, x, x, st)):
        with pytest.raises(ValueError, match="CUDA"):
            fn()
    for fn in (lambda: gdr.add_norm_fwd(x, None), lambda: gdr.add_norm_bwd(None, x, st), lambda: gdr.add_norm_bwd(x, x, None),
               lambda: gdr.add_norm_bwd(x, x, st, mean=st), lambda: gdr.add_norm_bwd(x, x, st, kind="layer"),
               lambda: gdr.norm_gate_fwd(x, None), lambda: gdr.norm_gate_fwd(x, x, act="relu"),
               lambda: gdr.norm_gate_bwd(x, x, None, st), lambda: gdr.norm_gate_bwd(x, x, x, st, act="relu"),
               lambda: gdr.add_norm_bwd(st[0], st[0], st[0, 0], per_head=True)):
        with pytest.raises(ValueError):
            fn()
