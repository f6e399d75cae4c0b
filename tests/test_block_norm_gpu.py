"""GPU parity of the norms around a block (gdr_add_norm_*, gdr_norm_gate_*) against their
definitions in 64 bits.

Bounds (2-norm of the error over the 2-norm of the result), from the roundings:
  fp32 tensors, statistics and the weights' sums: a reciprocal root within 2^-22, a sigmoid within
    2^-20, sums of up to 2^14 terms in partial sums of a few hundred, sqrt(2^14) 2^-24 = 7.6e-6 at
    the most: BOUND32 = 1e-5.
  bf16 outputs: one rounding, 2^-8 of the value at the most and 1.7e-3 in the mean square:
    BOUND16 = 4e-3.
y of add_norm is held against the norm of the sum as the call stored it.
"""
import itertools

import pytest
import torch

import block_norm_ref as ref
import chunked_gated_delta_07_gb300 as gdr

pytestmark = pytest.mark.gpu
BOUND32, BOUND16, EPS = 1e-5, 4e-3, 1e-5
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_07_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)


def ok():
    torch.cuda.synchronize()
    st = gdr.gdr_get_status()
    assert st == gdr.GDR_OK, gdr.gdr_status_string(st)


def close(got, want, bound, what=""):
    assert got.shape == want.shape, what
    far = (got.double() - want).norm() / want.norm().clamp(min=1e-30)
    assert float(far) <= bound, f"{what}: {float(far):.2e} > {bound}"


def inputs(shape, heads, dtype, seed, shift=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731

    def rows(std=1.0, mean=0.0):
        t = (rnd(*shape) * std + mean).to(DT[dtype])
        if not shift:
            return t
        flat = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
        return flat[shift:].view(shape).copy_(t)

    wshape = shape[-2:] if heads else shape[-1:]
    return dict(x=rows(1.5, 0.3), z=rows(2.0), res=rows(2.0), dy=rows(), dr=rows(), w=1 + 0.2 * rnd(*wshape),
                b=0.1 * rnd(*wshape))


def d(t):
    return None if t is None else t.double()


def check_add(i, dtype, kind, scale, with_dr=True, bias=True):
    tol = BOUND16 if dtype == "bf16" else BOUND32
    b = i["b"] if bias else None
    y, r, mean, rstd = gdr.add_norm_fwd(i["x"], i["res"], i["w"], b, scale=scale, kind=kind, eps=EPS)
    dr = i["dr"] if with_dr else None
    got = gdr.add_norm_bwd(i["dy"], r, rstd, mean, dr=dr, weight=i["w"], scale=scale, kind=kind, want_dbias=True)
    ok()
    close(r, d(i["res"]) + scale * d(i["x"]), tol, "r")
    m, s = ref.stats(d(r), kind, EPS)
    assert (mean is None) == (kind == "rms")
    if mean is not None:
        close(mean, m, BOUND32, "mean")
    close(rstd, s, BOUND32, "rstd")
    close(y, ref.norm(d(r), d(i["w"]), d(b), kind, EPS), tol, "y")
    want = ref.add_back(d(i["dy"]), d(dr), d(r), m, d(rstd), d(i["w"]), scale, kind, i["w"].shape)
    for name, p, q, t in zip(("dx", "dresidual", "dweight", "dbias"), got, want, (tol, tol, BOUND32, BOUND32)):
        close(p, q, t, name)
    assert (got[0] is got[1]) == (scale == 1.0)


def check_gate(i, dtype, kind, act, scale, with_res=True, bias=True):
    tol = BOUND16 if dtype == "bf16" else BOUND32
    b, res = i["b"] if bias else None, i["res"] if with_res else None
    y, mean, rstd = gdr.norm_gate_fwd(i["x"], i["z"], i["w"], b, residual=res, scale=scale, kind=kind, act=act, eps=EPS)
    got = gdr.norm_gate_bwd(i["dy"], i["x"], i["z"], rstd, mean, weight=i["w"], bias=b, scale=scale, kind=kind, act=act,
                            want_dbias=True)
    ok()
    m, s = ref.stats(d(i["x"]), kind, EPS)
    if mean is not None:
        close(mean, m, BOUND32, "mean")
    close(rstd, s, BOUND32, "rstd")
    close(y, ref.gate(d(i["x"]), d(i["z"]), d(i["w"]), d(b), d(res), scale, kind, act, EPS), tol, "y")
    want = ref.gate_back(d(i["dy"]), d(i["x"]), d(i["z"]), m, s, d(i["w"]), d(b), scale, kind, act, i["w"].shape)
    for name, p, q, t in zip(("dx", "dgate", "dweight", "dbias"), got, want, (tol, tol, BOUND32, BOUND32)):
        close(p, q, t, name)


WIDTHS = [(5, 3), (33, 8), (1, 64), (700, 100), (257, 128), (64, 255), (3, 999), (600, 1000), (300, 2048), (17, 4097),
          (20, 8192), (9, 8200), (5, 16384)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", WIDTHS)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_widths(shape, dtype, kind):
    i = inputs(shape, False, dtype, sum(shape))
    check_add(i, dtype, kind, 0.5)
    check_gate(i, dtype, kind, "silu", 0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(300, 16, 128), (7, 3, 64), (2, 50, 5, 96), (41, 3, 33), (1, 1, 256), (3, 70, 2048)])
def test_heads(shape, dtype):
    i = inputs(shape, True, dtype, 3)
    check_add(i, dtype, "rms", 1.0)
    check_gate(i, dtype, "layer", "sigmoid", 2.0)


@pytest.mark.parametrize("kind,act,with_res,bias,scale", list(itertools.product(
    ["rms", "layer"], ["silu", "sigmoid"], [True, False], [True, False], [1.0, -0.25])))
def test_options(kind, act, with_res, bias, scale):
    for dtype in ("bf16", "f32"):
        i = inputs((130, 72), False, dtype, 5)
        check_gate(i, dtype, kind, act, scale, with_res, bias)
        check_add(i, dtype, kind, scale, with_res, bias)


@pytest.mark.parametrize("dtype,D", [("bf16", 256), ("bf16", 250), ("f32", 256), ("f32", 250)])
@pytest.mark.parametrize("shift", [1, 4])
def test_alignment(dtype, D, shift):
    i = inputs((90, D), False, dtype, 6, shift)
    check_add(i, dtype, "rms", 0.5)
    check_gate(i, dtype, "layer", "silu", 0.5)


def test_without_weights():
    i = inputs((60, 4, 64), True, "f32", 8)
    y, r, _, rstd = gdr.add_norm_fwd(i["x"], i["res"], eps=EPS)
    g = gdr.add_norm_bwd(i["dy"], r, rstd, per_head=True)
    y2, _, rstd2 = gdr.norm_gate_fwd(i["x"], i["z"], eps=EPS)
    g2 = gdr.norm_gate_bwd(i["dy"], i["x"], i["z"], rstd2, want_dweight=False)
    ok()
    zero = torch.zeros_like(d(rstd))
    close(y, ref.norm(d(r), None, None, "rms", EPS), BOUND32)
    for p, q in zip(g, ref.add_back(d(i["dy"]), None, d(r), zero, d(rstd), None, 1.0, "rms", (4, 64))):
        if p is not None:
            close(p, q, BOUND32)
    assert g[2].shape == (4, 64) and g[3] is None and g2[2] is None
    close(y2, ref.gate(d(i["x"]), d(i["z"]), None, None, None, 1.0, "rms", "silu", EPS), BOUND32)
    close(g2[0], ref.gate_back(d(i["dy"]), d(i["x"]), d(i["z"]), zero, d(rstd2), None, None, 1.0, "rms", "silu", (64,))[0],
          BOUND32)
    assert gdr.add_norm_fwd(i["x"], i["res"], want_stats=False)[2:] == (None, None)


@pytest.mark.parametrize("shape", [(500, 128), (40, 2048), (30, 999)])
def test_in_place(shape):
    i = inputs(shape, False, "bf16", 4)
    y, r, _, rstd = gdr.add_norm_fwd(i["x"], i["res"], i["w"], scale=0.5)
    x, res = i["x"].clone(), i["res"].clone()
    got = gdr.add_norm_fwd(x, res, i["w"], scale=0.5, out=x, sum_out=res)
    assert torch.equal(x, y) and torch.equal(res, r) and torch.equal(got[3], rstd)
    for which in ("x", "z", "res"):
        j = {k: i[k].clone() for k in ("x", "z", "res")}
        want = gdr.norm_gate_fwd(i["x"], i["z"], i["w"], residual=i["res"])[0]
        gdr.norm_gate_fwd(j["x"], j["z"], i["w"], residual=j["res"], out=j[which])
        assert torch.equal(j[which], want)
    # the gradients over their inputs, at the C boundary
    rows, D = shape
    want = gdr.norm_gate_bwd(i["dy"], i["x"], i["z"], rstd, weight=i["w"])
    j = {k: i[k].clone() for k in ("dy", "x", "z")}
    dw = torch.empty_like(i["w"])
    rc = gdr.gdr_norm_gate_bwd(j["dy"], j["x"], j["z"], None, rstd, i["w"], None, j["x"], j["dy"], dw, None, rows, 1, D, 1.0,
                               gdr.GDR_NORM_RMS, gdr.GDR_ACT_SILU, gdr.GDR_BF16)
    assert rc == gdr.GDR_OK and torch.equal(j["x"], want[0]) and torch.equal(j["dy"], want[1]) and torch.equal(dw, want[2])
    want = gdr.add_norm_bwd(i["dy"], r, rstd, dr=i["dr"], weight=i["w"], scale=0.5)
    j = {"dy": i["dy"].clone(), "dr": i["dr"].clone()}
    rc = gdr.gdr_add_norm_bwd(j["dy"], j["dr"], r, None, rstd, i["w"], j["dy"], j["dr"], dw, None, rows, 1, D, 0.5,
                              gdr.GDR_NORM_RMS, gdr.GDR_BF16)
    assert rc == gdr.GDR_OK and torch.equal(j["dy"], want[0]) and torch.equal(j["dr"], want[1]) and torch.equal(dw, want[2])
    ok()


def test_values_that_are_not_finite_stay_in_their_row():
    i = inputs((90, 200), False, "f32", 2)
    j = {k: v.clone() for k, v in i.items()}
    j["x"][40, 3], j["z"][50, 7], j["res"][60, 9] = float("nan"), float("inf"), float("-inf")
    clean = torch.ones(90, dtype=torch.bool, device="cuda")
    clean[[40, 50, 60]] = False
    for call in (lambda s: gdr.add_norm_fwd(s["x"], s["res"], s["w"], s["b"], kind="layer"),
                 lambda s: gdr.norm_gate_fwd(s["x"], s["z"], s["w"], s["b"], residual=s["res"], kind="layer")):
        for p, q in zip(call(i), call(j)):
            assert torch.equal(p[clean], q[clean])
    y = gdr.norm_gate_fwd(j["x"], j["z"], act="sigmoid")[0]
    assert y[40].isnan().all() and y[50].isfinite().all()   # the sigmoid of an infinity is 1
    ok()


def test_large_and_tiny_gates():
    """Gates where exp(-z) overflows or vanishes."""
    z = torch.tensor([-200.0, -90.0, -88.0, -1e30, 0.0, 90.0, 200.0, 1e30], device="cuda").repeat(4, 1)
    for dtype in ("f32", "bf16"):
        i = inputs((4, 8), False, dtype, 2)
        zz = z.to(DT[dtype])
        for act in ("silu", "sigmoid"):
            y, _, rstd = gdr.norm_gate_fwd(i["x"], zz, act=act)
            dx, dz, _, _ = gdr.norm_gate_bwd(i["dy"], i["x"], zz, rstd, act=act)
            ok()
            assert all(t.isfinite().all() for t in (y, dx, dz)) or act == "silu" and y[:, 7].abs().max() > 1e29
            keep = slice(0, 7)
            want = ref.gate(d(i["x"]), d(zz), None, None, None, 1.0, "rms", act, EPS)
            close(y[:, keep], want[:, keep], BOUND16 if dtype == "bf16" else BOUND32)


def test_no_rows():
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    y, r, _, rstd = gdr.add_norm_fwd(x, x, w)
    assert y.shape == r.shape == x.shape
    for dx, other, dw, db in (gdr.add_norm_bwd(x, r, rstd, weight=w, want_dbias=True),
                              gdr.norm_gate_bwd(x, x, x, rstd, weight=w, want_dbias=True)):
        assert dx.shape == other.shape == x.shape and not dw.any() and not db.any()
    ok()


def test_same_results_on_every_call():
    i = inputs((3001, 16, 128), True, "bf16", 9)
    first = None
    for _ in range(60):
        y, r, _, rstd = gdr.add_norm_fwd(i["x"], i["res"], i["w"], scale=0.5)
        y2, _, rstd2 = gdr.norm_gate_fwd(i["x"], i["z"], i["w"])
        got = (y, r, rstd, y2, rstd2) + gdr.add_norm_bwd(i["dy"], r, rstd, dr=i["dr"], weight=i["w"], scale=0.5)[:3] + \
            gdr.norm_gate_bwd(i["dy"], i["x"], i["z"], rstd2, weight=i["w"])[:3]
        if first is None:
            first = got
        assert all(torch.equal(p, q) for p, q in zip(first, got))
    ok()


def test_workspaces_streams_and_graphs():
    sets = [inputs((700 + n, 256), False, "bf16", n) for n in range(3)]
    rstd = [gdr.norm_gate_fwd(i["x"], i["z"])[2] for i in sets]
    call = lambda i, s, **kw: gdr.norm_gate_bwd(i["dy"], i["x"], i["z"], s, weight=i["w"], **kw)  # noqa: E731
    want = [call(i, s) for i, s in zip(sets, rstd)]
    ws = [torch.empty(gdr.gdr_block_norm_bwd_workspace_size(700 + n, 1, 256), dtype=torch.uint8, device="cuda") for n in range(3)]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [call(i, s, stream=st, workspace=w) for i, s, st, w in zip(sets, rstd, streams, ws)]
        torch.cuda.synchronize()
        for p, q in zip(want, got):
            assert all(torch.equal(u, v) for u, v in zip(p[:3], q[:3]))
    with pytest.raises(gdr.GdrError) as e:
        call(sets[0], rstd[0], workspace=ws[0][:-16])
    assert e.value.code == gdr.GDR_ERR_NO_WORKSPACE
    i = {k: v.clone() for k, v in sets[0].items()}
    r = rstd[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(i, r, workspace=ws[0])
    for k, v in sets[1].items():
        i[k].copy_(v[:700] if v.dim() == 2 else v)
    r.copy_(rstd[1][:700])
    graph.replay()
    want = call(i, r)
    ok()
    assert all(torch.equal(u, v) for u, v in zip(got[:3], want[:3]))


def test_forward_on_streams_and_captured():
    sets = [inputs((700 + n, D), False, "bf16", n) for n, D in enumerate((256, 250, 2048))]
    call = lambda i: gdr.add_norm_fwd(i["x"], i["res"], i["w"], i["b"], kind="layer") + \
        gdr.norm_gate_fwd(i["x"], i["z"], i["w"], residual=i["res"])[::2]  # noqa: E731
    want = [call(i) for i in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for i, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(call(i))
        torch.cuda.synchronize()
        for p, q in zip(want, got):
            assert all(torch.equal(u, v) for u, v in zip(p, q))
    i = {k: torch.zeros_like(v) for k, v in sets[1].items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(i)
    for k, v in sets[1].items():
        i[k].copy_(v)
    graph.replay()
    ok()
    assert all(torch.equal(u, v) for u, v in zip(got, want[1]))


@pytest.mark.parametrize("D", [2048, 1001])
def test_offsets_beyond_32_bits(D):
    """More than 2^31 elements: the first and the last rows, and what lies around the outputs left alone."""
    rows = (1 << 31) // D + 300
    gen = torch.Generator(device="cuda").manual_seed(7)
    x, z, dy = (torch.empty(rows, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(3))
    w = torch.randn(D, generator=gen, device="cuda")
    flat = torch.full(((rows + 2) * D,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = flat[D:-D].view(rows, D)
    y, _, rstd = gdr.norm_gate_fwd(x, z, w, out=out)
    assert (flat[:D] == 7).all() and (flat[-D:] == 7).all()
    dx, dz, _, _ = gdr.norm_gate_bwd(dy, x, z, rstd, weight=w)
    ok()
    for part in (slice(0, 50), slice(rows - 50, rows)):
        f = lambda t: d(t[part])  # noqa: E731
        close(y[part], ref.gate(f(x), f(z), d(w), None, None, 1.0, "rms", "silu", 1e-5), BOUND16, "y")
        s = ref.stats(f(x), "rms", 1e-5)
        want = ref.gate_back(f(dy), f(x), f(z), *s, d(w), None, 1.0, "rms", "silu", w.shape)
        close(dx[part], want[0], BOUND16, "dx")
        close(dz[part], want[1], BOUND16, "dgate")
    del dx, dz
    y, r, _, rstd = gdr.add_norm_fwd(x, z, w, scale=0.5)
    dx, dres, _, _ = gdr.add_norm_bwd(dy, r, rstd, weight=w, scale=0.5)
    ok()
    for part in (slice(0, 50), slice(rows - 50, rows)):
        f = lambda t: d(t[part])  # noqa: E731
        close(r[part], f(z) + 0.5 * f(x), BOUND16, "r")
        m, s = ref.stats(f(r), "rms", 1e-5)
        close(y[part], ref.norm(f(r), d(w), None, "rms", 1e-5), BOUND16, "y")
        want = ref.add_back(f(dy), None, f(r), m, s, d(w), 0.5, "rms", w.shape)
        close(dx[part], want[0], BOUND16, "dx")
        close(dres[part], want[1], BOUND16, "dresidual")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(900, 65), (700, 127), (301, 501), (150, 1025), (260, 2047), (90, 4095), (41, 6001)])
def test_odd_widths(shape, dtype):
    """Single elements, every number of threads to a row."""
    i = inputs(shape, False, dtype, sum(shape))
    check_add(i, dtype, "layer", 0.5)
    check_gate(i, dtype, "rms", "silu", 0.5)
    check_gate(inputs((shape[0] // 5 + 1, 3, shape[1]), True, dtype, 1), dtype, "layer", "sigmoid", 1.0)
