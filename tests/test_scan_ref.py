"""The scan's reference gradients against differences, and what its calls refuse (CPU only)."""
import pytest
import torch

import chunked_gated_delta_07_gb300 as gdr
import scan_ref as ref
from chunked_gated_delta_07_gb300 import _build

INV, UNS = gdr.GDR_ERR_INVALID_ARG, gdr.GDR_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()


@pytest.mark.parametrize("gate", ["bounded", "softplus"])
@pytest.mark.parametrize("source", ["plain", "convex", "variance"])
def test_gradients_against_differences(gate, source):
    gen = torch.Generator().manual_seed(1)
    lens, D = [5, 0, 9], 3
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, a, h0, dout, dhT = rnd(14, D), rnd(14, D), rnd(3, D), rnd(14, D), rnd(3, D)
    grads = ref.backward(x, a, h0, dout, dhT, lens, 2.0, gate, source)

    def loss(*args):
        out, hT = ref.forward(*args, lens, 2.0, gate, source)
        return float((dout * out).sum() + (dhT * hT).sum())

    for k, g in enumerate(grads):
        way = rnd(*g.shape)
        step = [x, a, h0]
        ends = []
        for e in (1e-5, -1e-5):
            moved = list(step)
            moved[k] = moved[k] + e * way
            ends.append(loss(*moved))
        # the central difference is off by e^2 times a third derivative, and by 2^-53 / e of the loss
        assert abs((ends[0] - ends[1]) / 2e-5 - float((g * way).sum())) < 1e-7 * (1 + float((g * way).abs().sum()))


def fwd(**kw):
    a = dict(x=1 << 20, a=2 << 20, h0=None, out=5 << 20, hT=None, states=None, cu_seqlens=None, B=1, T=64, D=128, b=2.0,
             dtype=gdr.GDR_BF16, gate=gdr.GDR_GATE_BOUNDED, source=gdr.GDR_SOURCE_PLAIN, stream=0)
    a.update(kw)
    return gdr.gdr_gated_scan_fwd(**a)


def bwd(**kw):
    a = dict(x=1 << 20, a=2 << 20, h0=None, states=None, dout=3 << 20, dhT=None, dx=5 << 20, da=6 << 20, dh0=None,
             cu_seqlens=None, B=1, T=64, D=128, b=2.0, dtype=gdr.GDR_BF16, gate=gdr.GDR_GATE_BOUNDED,
             source=gdr.GDR_SOURCE_PLAIN, workspace=None, workspace_bytes=0, stream=0)
    a.update(kw)
    return gdr.gdr_gated_scan_bwd(**a)


def step(**kw):
    a = dict(x=1 << 20, a=2 << 20, state=3 << 20, out=5 << 20, N=1, T=1, D=128, b=2.0, dtype=gdr.GDR_BF16,
             gate=gdr.GDR_GATE_BOUNDED, source=gdr.GDR_SOURCE_PLAIN, stream=0)
    a.update(kw)
    return gdr.gdr_gated_scan_recurrent_fwd(**a)


COMMON = [(dict(T=-1), INV), (dict(D=0), INV), (dict(b=0.0), INV), (dict(b=float("nan")), INV), (dict(b=float("inf")), INV),
          (dict(dtype=5), INV), (dict(gate=2), INV), (dict(source=3), INV), (dict(x=None), INV), (dict(a=None), INV),
          (dict(T=1 << 31), UNS), (dict(T=1 << 30, D=1 << 11), UNS),
          (dict(T=(1 << 31) - 4096), UNS), (dict(D=(1 << 22) + 1), UNS)]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(B=0), INV), (dict(out=None), INV), (dict(out=1 << 20), INV), (dict(out=(2 << 20) + 2), INV),
    (dict(hT=(1 << 20) + 4), INV), (dict(h0=9 << 20, hT=(9 << 20) + 4), INV), (dict(h0=(5 << 20) + 8), INV),
    (dict(T=128, states=(1 << 20) + 8), INV), (dict(cu_seqlens=7 << 20, hT=7 << 20), INV), (dict(B=1 << 16, T=1 << 15), UNS)])
def test_forward_refuses(kw, code):
    assert fwd(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(B=0), INV), (dict(dout=None), INV), (dict(dx=None), INV), (dict(da=None), INV), (dict(dx=3 << 20), INV),
    (dict(da=5 << 20), INV), (dict(dh0=9 << 20, dhT=9 << 20), INV), (dict(dh0=9 << 20, h0=(9 << 20) + 4), INV),
    (dict(workspace=(9 << 20) + 8), INV), (dict(T=128, states=5 << 20), INV)])
def test_backward_refuses(kw, code):
    assert bwd(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(N=0), INV), (dict(state=None), INV), (dict(out=None), INV), (dict(out=2 << 20), INV), (dict(state=1 << 20), INV),
    (dict(out=3 << 20), INV)])
def test_single_tokens_refuse(kw, code):
    assert step(**kw) == code


def test_the_bound_is_not_looked_at_without_it():
    assert fwd(gate=gdr.GDR_GATE_SOFTPLUS, b=0.0, x=None) == INV   # (for x)
    assert fwd(gate=gdr.GDR_GATE_SOFTPLUS, b=0.0, T=0) == gdr.GDR_OK


def test_workspace_sizes():
    size = gdr.gdr_gated_scan_bwd_workspace_size
    assert size(0, 5, 8) == size(1, -1, 8) == size(1, 5, 0) == 0
    assert size(1, 127, 8) == 0 and size(1, 128, 8) == 32 and size(3, 100, 8) == 64 and size(3, 100, 8, True) == 0


def _x(B=2, T=5, D=8, dtype=torch.bfloat16):
    return dict(x=torch.zeros(B, T, D, dtype=dtype), a=torch.zeros(B, T, D, dtype=dtype))


def test_tensors_that_are_accepted():
    assert gdr.check_scan_inputs(**_x()) == (5, 8, 2)
    cu = torch.tensor([0, 2, 2, 5], dtype=torch.int32)
    assert gdr.check_scan_inputs(**_x(B=1), cu_seqlens=cu, h0=torch.zeros(3, 8))[2] == 3
    assert gdr.check_scan_inputs(**_x(T=130), states=torch.zeros(2, 8)) == (130, 8, 2)


@pytest.mark.parametrize("change", [
    dict(a=torch.zeros(2, 5, 9, dtype=torch.bfloat16)), dict(a=torch.zeros(2, 5, 8)), dict(a=None), dict(x=None),
    dict(x=torch.zeros(2, 5, 8, dtype=torch.float16)), dict(x=torch.zeros(10, 8, dtype=torch.bfloat16)),
    dict(a=torch.zeros(5, 2, 8, dtype=torch.bfloat16).transpose(0, 1)), dict(h0=torch.zeros(1, 8)),
    dict(hT=torch.zeros(2, 8, dtype=torch.bfloat16)), dict(dhT=torch.zeros(2, 9)), dict(out=torch.zeros(2, 5, 8)),
    dict(dout=torch.zeros(2, 5, 7, dtype=torch.bfloat16)), dict(states=torch.zeros(1, 8)),
    dict(cu_seqlens=torch.tensor([0, 5], dtype=torch.int32))])
def test_mismatched_tensors(change):
    with pytest.raises(ValueError):
        gdr.check_scan_inputs(**{**_x(), **change})


def test_cpu_tensors_and_unknown_names():
    x = _x()
    for call in (lambda: gdr.gated_scan_fwd(**x), lambda: gdr.gated_scan_bwd(**x, dout=x["x"]),
                 lambda: gdr.gated_scan_recurrent_fwd(**x, state=torch.zeros(2, 8))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError):
        gdr.gated_scan_bwd(**x, dout=None)
    with pytest.raises(ValueError):
        gdr.gated_scan_recurrent_fwd(**x, state=None)
    for names in (dict(gate="tanh", source="plain"), dict(gate="bounded", source="mean")):
        with pytest.raises(ValueError):
            gdr._scan_form(**names)
