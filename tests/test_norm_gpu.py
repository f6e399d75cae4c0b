"""GPU parity of the layer norm (gdr_layer_norm_*) against its formula in 64 bits.

Bounds (relative 2-norm): bf16 results are rounded once, to 8 significant bits, 2^-8; fp32
results, statistics and the weights' gradients are sums in fp32 over at most some ten
thousand terms in a fixed tree of partial sums, each term with a few roundings: below
64 * 2^-24 = 3.8e-6; BOUND32 = 5e-6.  dx is a difference of terms of the size of rstd w dy (for
D = 2 it cancels down to eps rstd^2 of them), so its fp32 error is measured against those.
Where the mean is far larger than the spread, the mean's own rounding, 2^-24 |mean| / spread,
comes on top.
"""
import numpy as np
import pytest
import torch

import chunked_gated_delta_07_gb300 as gdr
import decay_ref as ref

pytestmark = pytest.mark.gpu
BOUND32, BOUND16 = 5e-6, 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_07_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)


def inputs(shape, per_head, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    ws = shape[-2:] if per_head else shape[-1:]
    return ((rnd(*shape) * 1.5 + 0.3).to(DT[dtype]), rnd(*shape).to(DT[dtype]), 1 + 0.2 * rnd(*ws), 0.1 * rnd(*ws))


def check(x, dy, w, b, eps=1e-5, per_head=False):
    bound = BOUND16 if x.dtype == torch.bfloat16 else BOUND32
    y, mean, rstd = gdr.layer_norm_fwd(x, w, b, eps=eps)
    dx, dw, db = gdr.layer_norm_bwd(dy, x, mean, rstd, w, per_head=per_head)
    torch.cuda.synchronize()
    ry, rm, rr = ref.norm_fwd(x, w, b, eps)
    assert ref.rel(y, ry) <= bound and ref.rel(rstd, rr) <= BOUND32
    assert np.abs(ref.np64(mean) - rm).max() <= BOUND32 * np.abs(ref.np64(x)).max()
    rx, rw, rb = ref.norm_bwd(dy, x, mean, rstd, w, per_head)
    terms = np.linalg.norm(ref.np64(rstd)[..., None] * ref.np64(dy) * (1.0 if w is None else ref.np64(w)))
    far = np.linalg.norm(ref.np64(dx) - rx), ref.rel(dw, rw), ref.rel(db, rb)
    assert far[0] <= (BOUND16 * np.linalg.norm(rx) if bound == BOUND16 else 0.0) + BOUND32 * terms, far
    assert max(far[1:]) <= BOUND32, far
    assert dw.shape == rw.shape
    return y, mean, rstd, dx, dw, db


WIDTHS = [2, 7, 8, 31, 64, 100, 128, 250, 256, 257, 512, 1000, 1024, 1025, 2048, 4096, 5000, 8192, 9999, 16384]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 13])
def test_widths(D, dtype, rows):
    check(*inputs((rows, D), False, dtype, D + rows))


@pytest.mark.parametrize("shape", [(5, 3, 128), (700, 16, 128), (3, 40, 64), (2, 11, 5, 96), (1, 1, 33), (9, 70, 1000),
                                   (4, 2, 3000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_weight_per_head(shape, dtype):
    check(*inputs(shape, True, dtype, sum(shape)), per_head=True)


@pytest.mark.parametrize("shape", [(20011, 128), (6007, 1000), (1500, 4096), (70001, 5)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows(shape, dtype):
    """More rows than resident blocks take in one step: every block adds up several."""
    check(*inputs(shape, False, dtype, 3 + shape[1]))


def test_without_weight_and_with_parts_not_wanted():
    x, dy, w, b = inputs((40, 6, 128), True, "bf16", 5)
    check(x, dy, None, None)
    check(x, dy, None, None, per_head=True)
    y, mean, rstd = gdr.layer_norm_fwd(x, w, b)
    only, m, r = gdr.layer_norm_fwd(x, w, b, want_stats=False)
    assert m is None and r is None and torch.equal(only, y)
    dx, dw, db = gdr.layer_norm_bwd(dy, x, mean, rstd, w)
    for want in ((True, False), (False, True), (False, False)):
        got = gdr.layer_norm_bwd(dy, x, mean, rstd, w, want_dweight=want[0], want_dbias=want[1])
        assert torch.equal(got[0], dx)
        for g, full, on in zip(got[1:], (dw, db), want):
            assert (g is None) if not on else torch.equal(g, full)


@pytest.mark.parametrize("D", [128, 1000, 5000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_unaligned_rows(D, dtype):
    """Tensors one element past a 16-byte boundary take the element-wise kernels."""
    x, dy, w, b = inputs((9, D), False, dtype, D)
    moved = []
    for t in (x, dy):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:].copy_(t.flatten())
        moved.append(buf[1:].view(t.shape))
    check(moved[0], moved[1], w, b)


def test_in_place():
    x, dy, w, b = inputs((100, 512), False, "bf16", 6)
    y, mean, rstd, dx, _, _ = check(x, dy, w, b)
    z = x.clone()
    assert torch.equal(gdr.layer_norm_fwd(z, w, b, out=z)[0], y) and torch.equal(z, y)


def test_constant_and_far_rows():
    """A constant row has variance 0: y = bias exactly where the mean is exact; a row far from
    zero loses no more than its mean's rounding (two passes, no difference of squares)."""
    x = torch.full((4, 256), 3.0, device="cuda")
    w, b = torch.ones(256, device="cuda"), torch.linspace(-1, 1, 256, device="cuda")
    y, mean, rstd = gdr.layer_norm_fwd(x, w, b)
    assert torch.equal(y, b.expand(4, -1)) and (mean == 3).all()
    assert torch.allclose(rstd, torch.full((4,), 1e-5, device="cuda").rsqrt())
    gen = torch.Generator(device="cuda").manual_seed(9)
    far = 1000.0 + torch.randn((8, 1000), generator=gen, device="cuda")
    y, _, _ = gdr.layer_norm_fwd(far)
    ry, _, _ = ref.norm_fwd(far)
    assert ref.rel(y, ry) <= BOUND32 + 8 * 2.0 ** -24 * 1000


def test_a_bad_row_stays_alone():
    x, dy, w, b = inputs((70, 128), False, "bf16", 7)
    y, mean, rstd, dx, _, _ = check(x, dy, w, b)
    x[33] = float("nan")
    x[50, 3] = float("inf")
    got = gdr.layer_norm_fwd(x, w, b)[0]
    keep = [r for r in range(70) if r not in (33, 50)]
    assert torch.equal(got[keep], y[keep]) and got[33].isnan().all()


def test_gradient_against_differences():
    """Along a random direction, central differences of the fp64 formula: the third-order
    term at a step of 1e-4 is about 1e-8 of the value."""
    x, dy, w, b = inputs((6, 100), False, "f32", 8)
    _, _, _, dx, dw, db = check(x, dy, w, b)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for n, t, grad in ((0, x, dx), (1, w, dw), (2, b, db)):
        d = torch.randn(t.shape, generator=gen, device="cuda")
        side = []
        for e in (1e-4, -1e-4):
            a = [x.double(), w.double(), b.double()]
            a[n] = a[n] + e * d.double()
            side.append((ref.norm_fwd(*a)[0] * ref.np64(dy)).sum())
        want, have = (side[0] - side[1]) / 2e-4, (ref.np64(grad) * ref.np64(d)).sum()
        assert abs(want - have) <= 2 * BOUND32 * np.linalg.norm(ref.np64(grad)) * np.linalg.norm(ref.np64(d)), n


def test_same_result_every_time_and_no_rows():
    x, dy, w, b = inputs((5000, 256), False, "bf16", 10)
    a, c = check(x, dy, w, b), check(x, dy, w, b)
    assert all(torch.equal(p, q) for p, q in zip(a, c))
    y, mean, rstd = gdr.layer_norm_fwd(x[:0], w, b)
    dx, dw, db = gdr.layer_norm_bwd(dy[:0], x[:0], mean, rstd, w)
    assert y.shape == (0, 256) and dx.shape == (0, 256) and not dw.any() and not db.any()
