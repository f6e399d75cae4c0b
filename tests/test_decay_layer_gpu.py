"""The example layer (norm, decay attention, norm per head): gradients against the same layer
in plain fp64 torch, packed against separate sequences, and single tokens against the whole.

Bounds: bf16 activations pass through some ten roundings of 2^-8 at most (1.7e-3 in the mean
square) each between input and gradient; as squares 10 * (1.7e-3)^2 is (5.4e-3)^2.  The norm per
head divides by a spread that both sides round differently; BOUND = 3e-2 leaves a factor of five.
"""
import importlib.util
import os

import pytest
import torch

import chunked_gated_delta_07_gb300 as gdr

pytestmark = pytest.mark.gpu
BOUND = 3e-2
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    from chunked_gated_delta_07_gb300 import _build
    _build.build()
    spec = importlib.util.spec_from_file_location("decay_layer", os.path.join(ROOT, "examples", "decay_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    torch.manual_seed(3)
    return m


def plain(layer, x, p):
    """The layer in fp64 with torch's own gradients: the attention as a masked product."""
    norm = lambda z, w, b: ((z - z.mean(-1, keepdim=True))  # noqa: E731
                            * (z.var(-1, correction=0, keepdim=True) + 1e-5).rsqrt() * w + b)
    y = norm(x, p["norm_w"], p["norm_b"])
    B, T = x.shape[:2]
    q, k, v = ((y @ p[w]).view(B, T, layer.heads, layer.head_dim).transpose(1, 2) for w in ("w_q", "w_k", "w_v"))
    n = torch.arange(T, device=x.device)
    n = (n[:, None] - n[None, :]).double()
    decay = torch.exp(layer.log_decay.double()[:, None, None] * n.clamp(min=0)) * (n >= 0)
    o = layer.scale * ((q @ k.transpose(-1, -2)) * decay) @ v
    o = norm(o.transpose(1, 2), p["head_w"], p["head_b"])
    return x + o.reshape(B, T, -1) @ p["w_o"]


def far(a, b):
    return float((a.double() - b).norm() / b.norm())


def test_gradients(ex):
    layer = ex.DecayLayer(width=256, heads=3)
    x = torch.randn(2, 200, 256, device="cuda").bfloat16().requires_grad_()
    dy = torch.randn(2, 200, 256, device="cuda").bfloat16()
    layer(x).backward(dy)
    p = {n: t.detach().double().requires_grad_() for n, t in layer.named_parameters()}
    x64 = x.detach().double().requires_grad_()
    plain(layer, x64, p).backward(dy.double())
    got = {n: far(t.grad, p[n].grad) for n, t in layer.named_parameters()}
    got["x"] = far(x.grad, x64.grad)
    assert max(got.values()) <= BOUND, got
    assert gdr.gdr_get_status() == gdr.GDR_OK


def test_packed_equals_separate_sequences(ex):
    layer = ex.DecayLayer(width=256, heads=2)
    lens = [100, 1, 227]
    x = torch.randn(1, sum(lens), 256, device="cuda").bfloat16()
    cu = torch.tensor([0, 100, 101, 328], dtype=torch.int32, device="cuda")
    packed = layer(x, cu)
    parts = [layer(s.contiguous()) for s in x.split(lens, 1)]
    assert far(torch.cat(parts, 1), packed.double()) <= BOUND


def test_prompt_and_single_tokens_equal_the_whole(ex):
    layer = ex.DecayLayer(width=256, heads=4)
    x = torch.randn(3, 140, 256, device="cuda").bfloat16()
    whole = layer(x).detach()
    y, state = layer.prefill(x[:, :130].contiguous())
    rows = [y] + [layer.step(x[:, t:t + 1].contiguous(), state) for t in range(130, 140)]
    assert far(torch.cat(rows, 1), whole.double()) <= BOUND


def test_training_learns(ex):
    losses = ex.train(ex.DecayLayer(), steps=25)
    assert losses[-1] < 0.5 * losses[0]
