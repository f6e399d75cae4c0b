"""The gated scan and the norms around a block together, as a model uses them: gradients through two
blocks of examples/recurrent_block.py against the same blocks in 64 bits, and serving against the
whole sequence.

Bounds: in fp32 every operator is within 1e-5 of its definition (and the library's matrix products
within 2^-24 sqrt(256) of theirs); two blocks of five operators each, forward and backward, with
gradients a few times their factors: 20 * 1e-5 * 5 = 1e-3.  In bf16 the same tokens served in other
pieces meet the same values up to the roundings of some ten intermediate tensors, 2^-8 each at the
most, 1.7e-3 in the mean square: sqrt(20) * 1.7e-3 = 7.6e-3 for two blocks, 1.5e-2.
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import chunked_gated_delta_07_gb300 as gdr  # noqa: E402
import recurrent_block as ex  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_07_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)


def plain(block, u, r, lens):
    """A block by torch's own operations, in the type of its inputs (64 bits)."""
    w = {k: v.detach().double().requires_grad_(True) for k, v in block.named_parameters()}
    r = r + block.scale * u
    y = r * (r.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w["norm"]
    x, a = y @ w["w_x"], y @ w["w_a"] + w["far"]
    g = -block.b * torch.sigmoid(a)
    alpha, s = torch.exp(g), torch.sqrt(-torch.expm1(2 * g))
    rows, at = [], 0
    for m in lens:
        h = torch.zeros_like(x[0, 0])
        for t in range(at, at + m):
            h = alpha[0, t] * h + s[0, t] * x[0, t]
            rows.append(h)
        at += m
    h = torch.stack(rows)[None].unflatten(-1, (block.heads, -1))
    z = (y @ w["w_z"]).unflatten(-1, (block.heads, -1))
    o = h * (h.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w["head_norm"] * torch.nn.functional.silu(z)
    return o.flatten(-2) @ w["w_o"], r, w


@pytest.fixture
def exact_products():
    was = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    yield
    torch.backends.cuda.matmul.allow_tf32 = was


@pytest.mark.parametrize("lens", [[150], [70, 0, 1, 130]])
def test_gradients_of_two_blocks(lens, exact_products):
    torch.manual_seed(1)
    blocks = [ex.RecurrentBlock(width=64, heads=2, head_dim=32, dtype=torch.float32) for _ in range(2)]
    T = sum(lens)
    cu = torch.tensor([sum(lens[:n]) for n in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    u, r, du, dr = (torch.randn(1, T, 64, device="cuda") for _ in range(4))
    u.requires_grad_(True)
    r.requires_grad_(True)
    pu, pr = u, r
    for block in blocks:
        pu, pr = block(pu, pr, cu)
    ((pu * du).sum() + (pr * dr).sum()).backward()
    assert gdr.gdr_get_status() == gdr.GDR_OK
    eu, er = u.detach().double().requires_grad_(True), r.detach().double().requires_grad_(True)
    qu, qr, weights = eu, er, []
    for block in blocks:
        qu, qr, w = plain(block, qu, qr, lens)
        weights.append(w)
    ((qu * du.double()).sum() + (qr * dr.double()).sum()).backward()
    pairs = [("u", pu.detach(), qu), ("r", pr.detach(), qr), ("du", u.grad, eu.grad), ("dr", r.grad, er.grad)]
    for n, (block, w) in enumerate(zip(blocks, weights)):
        pairs += [(f"{n} {k}", v.grad, w[k].grad) for k, v in block.named_parameters()]
    for name, got, want in pairs:
        far = float((got.double() - want.detach()).norm() / want.detach().norm())
        assert far <= 1e-3, f"{name}: {far:.1e}"


def test_served_in_pieces():
    torch.manual_seed(2)
    blocks = [ex.RecurrentBlock() for _ in range(2)]
    x = torch.randn(3, 140, 256, device="cuda").bfloat16()
    with torch.no_grad():
        u, r = torch.zeros_like(x), x
        for block in blocks:
            u, r = block(u, r)
    whole = (u + r).float()
    states = [torch.zeros(3, 256, device="cuda") for _ in blocks]
    rows = []
    for lo, hi in [(0, 100), (100, 101), (101, 130)] + [(t, t + 1) for t in range(130, 140)]:
        r = x[:, lo:hi].contiguous()
        u = torch.zeros_like(r)
        for block, state in zip(blocks, states):
            u, r = block.serve(u, r, state)
        rows.append((u + r).float())
    assert gdr.gdr_get_status() == gdr.GDR_OK
    assert float((torch.cat(rows, 1) - whole).norm() / whole.norm()) <= 1.5e-2


def test_the_example_runs():
    torch.manual_seed(0)
    losses = ex.train([ex.RecurrentBlock() for _ in range(2)], steps=3, batch=2, tokens=130)
    assert len(losses) == 3 and all(v == v and v < float("inf") for v in losses)
    assert gdr.gdr_get_status() == gdr.GDR_OK


def test_tensors_of_another_device_are_refused(monkeypatch):
    x, h, w = torch.zeros(1, 4, 8, device="cuda"), torch.zeros(1, 8, device="cuda"), torch.ones(1, 4, device="cuda")
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for call in (lambda: gdr.gated_scan_fwd(x, x), lambda: gdr.gated_scan_bwd(x, x, x),
                 lambda: gdr.gated_scan_recurrent_fwd(x, x, h), lambda: gdr.add_norm_fwd(x, x),
                 lambda: gdr.add_norm_bwd(x, x, w), lambda: gdr.norm_gate_fwd(x, x), lambda: gdr.norm_gate_bwd(x, x, x, w)):
        with pytest.raises(ValueError, match="current"):
            call()
