"""What the decay attention's and the layer norm's calls refuse before they launch anything
(CPU only): at the C boundary by status code, at the tensor level with ValueError."""
import pytest
import torch

import chunked_gated_delta_07_gb300 as gdr
from chunked_gated_delta_07_gb300 import _build

INV, UNS = gdr.GDR_ERR_INVALID_ARG, gdr.GDR_ERR_UNSUPPORTED
FAR = {n: (i + 1) << 52 for i, n in enumerate(("q", "k", "v", "out", "dout", "dq", "dk", "dv"))}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()


def fwd(**kw):
    a = dict(q=1 << 20, k=2 << 20, v=3 << 20, log_decay=4 << 20, h0=None, out=5 << 20, hT=None, cu_seqlens=None,
             B=1, T=64, H=2, dk=128, dv=128, scale=1.0, dtype=gdr.GDR_BF16, path=gdr.GDR_PATH_AUTO,
             workspace=None, workspace_bytes=0, stream=0)
    a.update(kw)
    return gdr.gdr_decay_fwd(**a)


def bwd(**kw):
    a = dict(q=1 << 20, k=2 << 20, v=3 << 20, log_decay=4 << 20, h0=None, dout=5 << 20, dhT=None, dq=6 << 20,
             dk=7 << 20, dv=8 << 20, dh0=None, cu_seqlens=None, B=1, T=64, H=2, dk_dim=128, dv_dim=128, scale=1.0,
             dtype=gdr.GDR_BF16, path=gdr.GDR_PATH_AUTO, workspace=None, workspace_bytes=0, stream=0)
    a.update(kw)
    return gdr.gdr_decay_bwd(**a)


def step(**kw):
    a = dict(q=1 << 20, k=2 << 20, v=3 << 20, log_decay=4 << 20, state=8 << 20, out=5 << 20, N=1, T=1, H=2, dk=128,
             dv=128, scale=1.0, dtype=gdr.GDR_BF16, stream=0)
    a.update(kw)
    return gdr.gdr_decay_recurrent_fwd(**a)


COMMON = [(dict(H=0), INV), (dict(T=-1), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
          (dict(dtype=5), INV), (dict(log_decay=None), INV), (dict(q=None), INV), (dict(T=(1 << 40) + 1), UNS)]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(B=0), INV), (dict(path=9), INV), (dict(dk=96), UNS), (dict(dv=256), UNS), (dict(dv=0), INV),
    (dict(out=None), INV), (dict(out=1 << 20), INV), (dict(hT=(3 << 20) + 16), INV),
    (dict(h0=9 << 20, hT=(9 << 20) + 16), INV), (dict(h0=(9 << 20) + 4), INV), (dict(hT=(9 << 20) + 8), INV),
    (dict(out=4 << 20), INV), (dict(workspace=(9 << 20) + 8), INV),
    (dict(path=gdr.GDR_PATH_TC, dtype=gdr.GDR_F32), UNS), (dict(path=gdr.GDR_PATH_TC, k=(2 << 20) + 2), UNS),
    (dict(q=FAR["q"], k=FAR["k"], v=FAR["v"], out=FAR["out"], T=1 << 40, H=1 << 22), UNS)])
def test_forward(kw, code):
    assert fwd(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(B=0), INV), (dict(path=-1), INV), (dict(dk_dim=32), UNS), (dict(dv_dim=100), UNS), (dict(dout=None), INV),
    (dict(dq=None), INV), (dict(dq=5 << 20), INV), (dict(dk=6 << 20), INV), (dict(dv=1 << 20), INV),
    (dict(dhT=(9 << 20) + 4), INV), (dict(dh0=(9 << 20) + 4), INV), (dict(dhT=9 << 20, dh0=9 << 20), INV),
    (dict(h0=9 << 20, dh0=9 << 20), INV), (dict(path=gdr.GDR_PATH_TC, dq=(6 << 20) + 2), UNS)])
def test_backward(kw, code):
    assert bwd(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(N=0), INV), (dict(dk=16), UNS), (dict(state=None), INV), (dict(state=(8 << 20) + 4), INV),
    (dict(out=3 << 20), INV), (dict(out=8 << 20), INV), (dict(state=1 << 20), INV)])
def test_single_tokens(kw, code):
    assert step(**kw) == code


def nfwd(**kw):
    a = dict(x=1 << 20, weight=2 << 20, bias=3 << 20, y=4 << 20, mean=5 << 20, rstd=6 << 20, rows=8, G=2, D=128,
             eps=1e-5, dtype=gdr.GDR_BF16, stream=0)
    a.update(kw)
    return gdr.gdr_layer_norm_fwd(**a)


def nbwd(**kw):
    a = dict(dy=1 << 20, x=2 << 20, mean=3 << 20, rstd=4 << 20, weight=5 << 20, dx=6 << 20, dweight=7 << 20,
             dbias=8 << 20, rows=8, G=2, D=128, dtype=gdr.GDR_BF16, stream=0)
    a.update(kw)
    return gdr.gdr_layer_norm_bwd(**a)


NORM = [(dict(rows=-2), INV), (dict(rows=7), INV), (dict(G=0), INV), (dict(D=0), INV), (dict(D=16385), UNS),
        (dict(dtype=3), INV), (dict(x=None), INV), (dict(rows=1 << 41), UNS)]


@pytest.mark.parametrize("kw,code", NORM + [
    (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(y=None), INV), (dict(y=(1 << 20) + 2), INV),
    (dict(y=2 << 20), INV), (dict(mean=1 << 20), INV), (dict(rstd=5 << 20), INV)])
def test_norm_forward(kw, code):
    assert nfwd(**kw) == code


@pytest.mark.parametrize("kw,code", NORM + [
    (dict(dy=None), INV), (dict(mean=None), INV), (dict(dx=None), INV), (dict(dx=(2 << 20) + 2), INV),
    (dict(dweight=5 << 20), INV), (dict(dweight=1 << 20), INV), (dict(dbias=7 << 20), INV), (dict(dx=3 << 20), INV)])
def test_norm_backward(kw, code):
    assert nbwd(**kw) == code


def test_workspace_sizes():
    size = gdr.gdr_decay_workspace_size
    assert size(8, 4096, 0, 128, 128) == 0 and size(8, 4096, 16, 96, 128) == 0
    # a lone long sequence is cut: at least one state per head and boundary
    # (and direction: forward states, and backward their gradients too)
    one = 16 * 128 * 128 * 4
    assert size(1, 1 << 18, 16, 128, 128) >= one
    assert size(1, 1 << 18, 16, 128, 128, backward=True) >= 2 * one
    assert size(1, 1 << 18, 16, 128, 128) >= size(1, 1 << 18, 16, 128, 128, path=gdr.GDR_PATH_SIMT)
    assert size(37, 65536, 32, 64, 64, packed=True) >= 3 * 8 * 38


# ---- tensors ----------------------------------------------------------------------------
def _x(B=2, T=5, H=3, dk=64, dv=128, dtype=torch.bfloat16):
    return dict(q=torch.zeros(B, T, H, dk, dtype=dtype), k=torch.zeros(B, T, H, dk, dtype=dtype),
                v=torch.zeros(B, T, H, dv, dtype=dtype), log_decay=torch.zeros(H))


def test_tensors_that_are_accepted():
    assert gdr.check_decay_inputs(**_x()) == (2, 5, 3, 64, 128, 2)
    cu = torch.tensor([0, 2, 5], dtype=torch.int32)
    assert gdr.check_decay_inputs(**_x(B=1), cu_seqlens=cu, h0=torch.zeros(2, 3, 64, 128))[5] == 2
    assert gdr.check_norm_inputs(torch.zeros(4, 3, 8), torch.zeros(3, 8), torch.zeros(3, 8)) == (12, 3, 8)
    assert gdr.check_norm_inputs(torch.zeros(4, 3, 8), torch.zeros(8)) == (12, 1, 8)


@pytest.mark.parametrize("change", [
    dict(k=torch.zeros(2, 5, 3, 128, dtype=torch.bfloat16)), dict(v=torch.zeros(2, 5, 4, 128, dtype=torch.bfloat16)),
    dict(k=torch.zeros(2, 5, 3, 64)), dict(q=torch.zeros(2, 5, 3, 64, dtype=torch.float16)),
    dict(q=torch.zeros(5, 3, 64, dtype=torch.bfloat16)), dict(v=None), dict(log_decay=torch.zeros(4)),
    dict(log_decay=torch.zeros(3, dtype=torch.bfloat16)), dict(log_decay=None),
    dict(k=torch.zeros(5, 2, 3, 64, dtype=torch.bfloat16).transpose(0, 1)),
    dict(h0=torch.zeros(1, 3, 64, 128)), dict(h0=torch.zeros(2, 3, 128, 64)),
    dict(dhT=torch.zeros(2, 3, 64, 128, dtype=torch.bfloat16)), dict(dout=torch.zeros(2, 5, 3, 64, dtype=torch.bfloat16)),
    dict(cu_seqlens=torch.tensor([0, 5], dtype=torch.int32))])
def test_mismatched_tensors(change):
    with pytest.raises(ValueError):
        gdr.check_decay_inputs(**{**_x(), **change})


def test_offsets():
    for cu in (torch.tensor([0, 2, 5]), torch.tensor([0], dtype=torch.int32), torch.zeros((2, 2), dtype=torch.int32)):
        with pytest.raises(ValueError):
            gdr.check_decay_inputs(**_x(B=1), cu_seqlens=cu)


@pytest.mark.parametrize("kw", [
    dict(weight=torch.zeros(7)), dict(weight=torch.zeros(4, 8)), dict(weight=torch.zeros(8, dtype=torch.bfloat16)),
    dict(weight=torch.zeros(3, 8), bias=torch.zeros(8)), dict(dy=torch.zeros(4, 3, 7)), dict(mean=torch.zeros(4)),
    dict(rstd=torch.zeros(4, 3, dtype=torch.float64)), dict(x=torch.zeros(4, 3, 8, dtype=torch.float16)),
    dict(x=torch.zeros(4, 3, 0)), dict(x=None)])
def test_mismatched_norm_tensors(kw):
    with pytest.raises(ValueError):
        gdr.check_norm_inputs(**{"x": torch.zeros(4, 3, 8), **kw})


def test_cpu_tensors_and_unknown_names():
    x = _x(dk=128)
    t = torch.zeros(4, 8)
    for call in (lambda: gdr.decay_fwd(**x), lambda: gdr.decay_bwd(**x, dout=x["v"]),
                 lambda: gdr.decay_recurrent_fwd(**x, state=torch.zeros(2, 3, 128, 128)),
                 lambda: gdr.layer_norm_fwd(t), lambda: gdr.layer_norm_bwd(t, t, t[:, 0].contiguous(), t[:, 0].contiguous())):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError):
        gdr.decay_bwd(**x, dout=None)
    with pytest.raises(ValueError):
        gdr.decay_recurrent_fwd(**x, state=None)
    with pytest.raises(ValueError):
        gdr.layer_norm_bwd(t, t, None, None)
