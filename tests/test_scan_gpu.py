"""GPU parity of the gated scan (gdr_gated_scan_*) against its definition in 64 bits.

Bounds (2-norm of the error over the 2-norm of the result), from the roundings:
  fp32 tensors and all states: a decay is off by at most 3 * 2^-24 (its exponential within two
    units, a rounding), a weight or a factor of a gradient by 2^-20 of itself; over a memory of up
    to a thousand tokens, of independent signs, sqrt(1000) * 3 * 2^-24 = 5.7e-6; BOUND32 = 1e-5.
  bf16 outputs: one rounding of the result, at most 2^-9 + the above (half a step is 2^-8 of the
    lower end of a binade, 1.7e-3 in the mean square); BOUND16 = 4e-3.
"""
import numpy as np
import pytest
import torch

import chunked_gated_delta_07_gb300 as gdr
import scan_ref as ref

pytestmark = pytest.mark.gpu
BOUND32, BOUND16 = 1e-5, 4e-3
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_07_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)


def inputs(lens, D, dtype, seed, packed=True, states=True, shift=0):
    """shift: elements that the tensors start behind an aligned address."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    total, N = int(sum(lens)), len(lens)

    def place(t):
        if not shift:
            return t
        flat = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
        return flat[shift:].view(t.shape).copy_(t)

    shape = (1, total, D) if packed else (N, lens[0], D)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    far = 7.0 * torch.rand(D, generator=gen, device="cuda") - 6.0
    x, a, dout = rnd(*shape), rnd(*shape) + far, rnd(*shape)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda") if packed else None
    return dict(x=place(x.to(DT[dtype])), a=place(a.to(DT[dtype])), dout=place(dout.to(DT[dtype])), cu=cu,
                h0=rnd(N, D) if states else None, dhT=rnd(N, D) if states else None, lens=list(lens))


def ok():
    torch.cuda.synchronize()
    st = gdr.gdr_get_status()
    assert st == gdr.GDR_OK, gdr.gdr_status_string(st)


def close(got, want, bound, what=""):
    got = got.detach().double().cpu().reshape(want.shape)
    far = (got - want).norm() / want.norm().clamp(min=1e-30)
    assert float(far) <= bound, f"{what}: {float(far):.2e} > {bound}"


def check(i, dtype, b=2.0, gate="bounded", source="plain", kept=True):
    form = dict(b=b, gate=gate, source=source)
    out, hT, states = gdr.gated_scan_fwd(i["x"], i["a"], h0=i["h0"], cu_seqlens=i["cu"], want_states=True, **form)
    dx, da, dh0 = gdr.gated_scan_bwd(i["x"], i["a"], i["dout"], dhT=i["dhT"], h0=i["h0"],
                                     states=states if kept else None, cu_seqlens=i["cu"], **form)
    ok()
    D = i["x"].shape[-1]
    flat = {k: i[k].reshape(-1, D) for k in ("x", "a", "dout")}
    tol = BOUND16 if dtype == "bf16" else BOUND32
    h, last = ref.forward(flat["x"], flat["a"], i["h0"], i["lens"], **form)
    close(out, h, tol, "out")
    close(hT, last, BOUND32, "hT")
    if states.numel():
        close(states, h[127::128], BOUND32, "states")
    gx, ga, g0 = ref.backward(flat["x"], flat["a"], i["h0"], flat["dout"], i["dhT"], i["lens"], **form)
    close(dx, gx, tol, "dx")
    close(da, ga, tol, "da")
    close(dh0, g0, BOUND32, "dh0")
    return out, hT, dx, da, dh0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["bounded", "softplus"])
@pytest.mark.parametrize("source", ["plain", "convex", "variance"])
def test_forms(dtype, gate, source):
    check(inputs([300, 1, 129], 72, dtype, 1), dtype, gate=gate, source=source, b=8.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (1, 2, 2), (3, 127, 31), (1, 128, 32), (2, 129, 33), (1, 1100, 8), (5, 33, 64),
                                   (70, 17, 40), (1, 257, 1000), (2, 640, 65), (9, 128, 96), (4, 300, 34)])
def test_dense(B, T, D, dtype):
    check(inputs([T] * B, D, dtype, B + T + D, packed=False), dtype, source="variance")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[1] * 40, [0, 5, 0, 0, 300, 0], [128, 128, 1, 127], [2000], [17, 600, 3, 3, 900, 1, 0, 64],
                                  [0, 0, 7], [129] * 9])
def test_packed(lens, dtype):
    check(inputs(lens, 40, dtype, len(lens)), dtype, source="convex", kept=False)


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 63), ("bf16", 62), ("f32", 64), ("f32", 63)])
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_alignment(dtype, D, shift):
    check(inputs([200, 150], D, dtype, shift, shift=shift), dtype, source="variance", gate="softplus")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_states(dtype):
    i = inputs([260, 40], 24, dtype, 3, states=False)
    check(i, dtype)
    out, hT, states = gdr.gated_scan_fwd(i["x"], i["a"], cu_seqlens=i["cu"], want_state=False)
    assert hT is None and states is None
    assert gdr.gated_scan_bwd(i["x"], i["a"], i["dout"], cu_seqlens=i["cu"], want_dh0=False)[2] is None


def test_kept_states_change_nothing():
    i = inputs([700, 0, 333], 96, "bf16", 5)
    states = gdr.gated_scan_fwd(i["x"], i["a"], h0=i["h0"], cu_seqlens=i["cu"], want_states=True)[2]
    with_, without = (gdr.gated_scan_bwd(i["x"], i["a"], i["dout"], i["dhT"], i["h0"], st, i["cu"]) for st in (states, None))
    ok()
    for p, q in zip(with_, without):
        assert torch.equal(p, q)


@pytest.mark.parametrize("lens", [None, [50, 0, 200, 1]])
def test_state_in_place(lens):
    i = inputs(lens or [251] * 3, 40, "f32", 6, packed=lens is not None)
    want = gdr.gated_scan_fwd(i["x"], i["a"], h0=i["h0"], cu_seqlens=i["cu"])
    state = i["h0"].clone()
    out, hT, _ = gdr.gated_scan_fwd(i["x"], i["a"], h0=state, hT=state, cu_seqlens=i["cu"])
    ok()
    assert hT is state and torch.equal(state, want[1]) and torch.equal(out, want[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,T,D", [(1, 1, 1), (5, 1, 1000), (3, 7, 129), (200, 2, 64)])
def test_single_tokens(N, T, D, dtype):
    for gate, source in (("bounded", "variance"), ("softplus", "convex")):
        i = inputs([T] * N, D, dtype, N + T, packed=False)
        state = i["h0"].clone()
        out = gdr.gated_scan_recurrent_fwd(i["x"], i["a"], state, b=5.0, gate=gate, source=source)
        ok()
        h, hT = ref.forward(i["x"].reshape(-1, D), i["a"].reshape(-1, D), i["h0"], i["lens"], 5.0, gate, source)
        close(out, h, BOUND16 if dtype == "bf16" else BOUND32, "out")
        close(state, hT, BOUND32, "state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_in_pieces_then_single_tokens(dtype):
    i = inputs([500] * 2, 72, dtype, 9, packed=False)
    whole, hT, _ = gdr.gated_scan_fwd(i["x"], i["a"], h0=i["h0"], source="convex")
    state, outs = i["h0"].clone(), []
    for lo, hi in ((0, 130), (130, 131), (131, 490)):
        cut = lambda t: t[:, lo:hi].contiguous()  # noqa: E731
        outs.append(gdr.gated_scan_fwd(cut(i["x"]), cut(i["a"]), h0=state, hT=state, source="convex")[0])
    for t in range(490, 500):
        cut = lambda v: v[:, t:t + 1].contiguous()  # noqa: E731
        outs.append(gdr.gated_scan_recurrent_fwd(cut(i["x"]), cut(i["a"]), state, source="convex"))
    ok()
    close(torch.cat(outs, 1), whole.double().cpu(), 2 * BOUND16 if dtype == "bf16" else 2 * BOUND32)
    close(state, hT.double().cpu(), 2 * BOUND32)


@pytest.mark.parametrize("lens,D", [([20000], 64), ([9000, 1, 4000], 256), ([1] * 3000, 32), ([5] * 700, 1024)])
def test_many_tiles(lens, D):
    """Clusters of eight blocks, many steps."""
    check(inputs(lens, D, "bf16", 11), "bf16", source="variance")


@pytest.mark.parametrize("dtype,D", [("bf16", 40), ("f32", 33)])
def test_very_many_empty_sequences(dtype, D):
    """What holds tokens is as without them, bit for bit, and an empty sequence passes its state on."""
    lens, at = [], []
    for n, gap in ((5, 50000), (300, 3), (1, 70001), (2, 1), (900, 30000), (129, 2), (7, 9000)):
        at.append(len(lens))
        lens += [n] + [0] * gap
    i = inputs(lens, D, dtype, 21)
    full = {k: i[k] for k in ("h0", "dhT")}
    cu = torch.tensor(np.concatenate([[0], np.cumsum([lens[n] for n in at])]), dtype=torch.int32, device="cuda")
    rows = torch.tensor(at, device="cuda")
    few = {k: v[rows].contiguous() for k, v in full.items()}
    res = []
    for c, st in ((cu, few), (i["cu"], full)):
        out, hT, kept = gdr.gated_scan_fwd(i["x"], i["a"], h0=st["h0"], cu_seqlens=c, want_states=True, source="variance")
        res.append((out, hT, kept) + gdr.gated_scan_bwd(i["x"], i["a"], i["dout"], st["dhT"], st["h0"], kept, c, source="variance"))
    ok()
    (out, hT, kept, dx, da, dh0), (out2, hT2, kept2, dx2, da2, dh02) = res
    for p, q in ((out, out2), (kept, kept2), (dx, dx2), (da, da2), (hT, hT2[rows]), (dh0, dh02[rows])):
        assert torch.equal(p, q)
    empty = torch.ones(len(lens), dtype=torch.bool, device="cuda")
    empty[rows] = False
    assert torch.equal(hT2[empty], full["h0"][empty]) and torch.equal(dh02[empty], full["dhT"][empty])


def test_long_memory():
    """Decays of 1 - 1e-4 to 1 - 1e-7, fp32 states: the decay keeps the relative accuracy of 1 - alpha.
    Inputs of one sign, so that an error of the decay does not average out."""
    T, D = 6000, 32
    gen = torch.Generator(device="cuda").manual_seed(2)
    a = torch.linspace(-16, -9, D, device="cuda").expand(1, T, D).contiguous()
    x = torch.rand(1, T, D, generator=gen, device="cuda") + 0.5
    h0 = torch.rand(1, D, generator=gen, device="cuda")
    for source in ("plain", "convex", "variance"):
        out, hT, _ = gdr.gated_scan_fwd(x, a, h0=h0, source=source)
        ok()
        h, last = ref.forward(x[0], a[0], h0, [T], 2.0, "bounded", source)
        # each of 6000 steps rounds the state to 2^-24 of itself, of either sign, and the decay,
        # which is the same throughout, to 2^-25: 6000 * 2^-25 = 1.8e-4 of a state that lives that
        # long at the most; 2e-4
        close(out, h, 2e-4, "out")
        close(hT, last, 2e-4, "hT")


# ---- what is not finite --------------------------------------------------------------------
@pytest.mark.parametrize("where", ["x", "a", "h0", "dout", "dhT"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_not_finite_stays_in_its_sequence_and_channel(where, value):
    lens = [100, 300, 0, 61, 140]
    i = inputs(lens, 40, "f32", 13)
    j = {k: v.clone() if torch.is_tensor(v) else v for k, v in i.items()}
    if where in ("h0", "dhT"):
        j[where][1, 5] = value
    else:
        j[where][0, 180, 5] = value   # token 80 of sequence 1
    res = []
    for s in (i, j):
        out, hT, st = gdr.gated_scan_fwd(s["x"], s["a"], h0=s["h0"], cu_seqlens=s["cu"], source="variance", want_states=True)
        res.append((out, hT) + gdr.gated_scan_bwd(s["x"], s["a"], s["dout"], s["dhT"], s["h0"], st, s["cu"], source="variance"))
    ok()
    for name, p, q in zip(("out", "hT", "dx", "da", "dh0"), *res):
        hit = torch.zeros_like(p, dtype=torch.bool)
        if name in ("hT", "dh0"):
            hit[1, 5] = True
        else:
            hit[0, 100:400, 5] = True
        assert torch.equal(p[~hit], q[~hit]), name
    out, hT, dx, da, dh0 = res[1]
    if value != value:   # a NaN reaches everything behind it (of a gradient: in front of it)
        if where in ("x", "a"):
            assert out[0, 180:400, 5].isnan().all() and hT[1, 5].isnan()
        if where == "h0":
            assert out[0, 100:400, 5].isnan().all() and hT[1, 5].isnan()
        if where in ("dout", "a"):
            assert dx[0, 100:180, 5].isnan().all() and dh0[1, 5].isnan()
        if where == "dhT":
            assert dx[0, 100:400, 5].isnan().all() and dh0[1, 5].isnan()


def test_gates_at_their_ends():
    """a of -inf keeps the state, +inf decays by the bound (bounded) or forgets (softplus)."""
    a = torch.tensor([float("-inf"), -1e30, -100.0, 1e30, float("inf")], device="cuda").reshape(1, 1, 5)
    x, h0 = torch.full((1, 1, 5), 2.0, device="cuda"), torch.full((1, 5), 3.0, device="cuda")
    for gate, least in (("bounded", float(np.exp(-2.0))), ("softplus", 0.0)):
        for source in ("plain", "convex", "variance"):
            alpha = torch.tensor([1.0, 1.0, 1.0, least, least], dtype=torch.float64)
            w = {"plain": torch.ones(5, dtype=torch.float64), "convex": 1 - alpha, "variance": (1 - alpha ** 2).sqrt()}[source]
            for out in (gdr.gated_scan_fwd(x, a, h0=h0, gate=gate, source=source)[0],
                        gdr.gated_scan_recurrent_fwd(x, a, h0.clone(), gate=gate, source=source)):
                close(out[0, 0], 3 * alpha + 2 * w, 1e-6, f"{gate} {source}")
            dx, da, dh0 = gdr.gated_scan_bwd(x, a, torch.ones_like(x), h0=h0, gate=gate, source=source)
            close(dx[0, 0], w, 1e-6, "dx")
            close(dh0[0], alpha, 1e-6, "dh0")
            assert da.isfinite().all() and float(da[..., :2].abs().max()) < 1e-12
    ok()


# ---- calls --------------------------------------------------------------------------------
@pytest.mark.parametrize("cu", [[0, 5, 3, 10], [1, 4, 10], [0, 4, 9], [0, 4, 11], [0, -1, 10]])
def test_bad_offsets_write_nothing(cu):
    i = inputs([10], 24, "f32", 1)
    off = torch.tensor(cu, dtype=torch.int32, device="cuda")
    N = len(cu) - 1
    out, hT = torch.full_like(i["x"], 7.0), torch.full((N, 24), 7.0, device="cuda")
    gdr.gated_scan_fwd(i["x"], i["a"], cu_seqlens=off, out=out, hT=hT)
    assert gdr.gdr_get_status() == gdr.GDR_ERR_BAD_SEQLENS
    assert (out == 7).all() and (hT == 7).all()
    dx, da, dh0 = torch.full_like(out, 7.0), torch.full_like(out, 7.0), torch.full_like(hT, 7.0)
    rc = gdr.gdr_gated_scan_bwd(i["x"], i["a"], None, None, i["dout"], None, dx, da, dh0, off, N, 10, 24, 2.0, gdr.GDR_F32,
                                gdr.GDR_GATE_BOUNDED, gdr.GDR_SOURCE_PLAIN)
    assert rc == gdr.GDR_OK and gdr.gdr_get_status() == gdr.GDR_ERR_BAD_SEQLENS
    assert (dx == 7).all() and (da == 7).all() and (dh0 == 7).all()
    ok()


def test_no_tokens():
    x, h0 = torch.empty(2, 0, 24, device="cuda"), torch.randn(2, 24, device="cuda")
    assert torch.equal(gdr.gated_scan_fwd(x, x, h0=h0)[1], h0) and not gdr.gated_scan_fwd(x, x)[1].any()
    assert torch.equal(gdr.gated_scan_bwd(x, x, x, dhT=h0)[2], h0) and not gdr.gated_scan_bwd(x, x, x)[2].any()
    x, cu = x[:1], torch.zeros(3, dtype=torch.int32, device="cuda")
    assert torch.equal(gdr.gated_scan_fwd(x, x, h0=h0, cu_seqlens=cu)[1], h0)
    assert torch.equal(gdr.gated_scan_bwd(x, x, x, dhT=h0, cu_seqlens=cu)[2], h0)
    state = h0.clone()
    gdr.gated_scan_recurrent_fwd(torch.empty(2, 0, 24, device="cuda"), torch.empty(2, 0, 24, device="cuda"), state)
    assert torch.equal(state, h0)
    ok()


def test_same_results_on_every_call():
    i = inputs([3001, 77, 1500], 200, "bf16", 4)
    first = None
    for _ in range(60):
        out, hT, st = gdr.gated_scan_fwd(i["x"], i["a"], h0=i["h0"], cu_seqlens=i["cu"], want_states=True, source="variance")
        got = (out, hT, st) + gdr.gated_scan_bwd(i["x"], i["a"], i["dout"], i["dhT"], i["h0"], st, i["cu"], source="variance")
        if first is None:
            first = got
        for p, q in zip(first, got):
            assert torch.equal(p, q)
    ok()


def test_side_by_side_on_streams():
    sets = [inputs([900 + 100 * n, 50], 72, "f32", n) for n in range(3)]
    want = [gdr.gated_scan_bwd(i["x"], i["a"], i["dout"], i["dhT"], i["h0"], None, i["cu"]) for i in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    scratch = [torch.empty(gdr.gdr_gated_scan_bwd_workspace_size(2, sum(i["lens"]), 72, True), dtype=torch.uint8, device="cuda")
               for i in sets]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [gdr.gated_scan_bwd(i["x"], i["a"], i["dout"], i["dhT"], i["h0"], None, i["cu"], stream=st, workspace=w)
               for i, st, w in zip(sets, streams, scratch)]
        torch.cuda.synchronize()
        for p, q in zip(want, got):
            assert all(torch.equal(u, v) for u, v in zip(p, q))
    ok()


def test_workspace_too_small():
    i = inputs([900], 72, "f32", 1)
    need = gdr.gdr_gated_scan_bwd_workspace_size(1, 900, 72, True)
    assert need == 7 * 72 * 4
    with pytest.raises(gdr.GdrError) as e:
        gdr.gated_scan_bwd(i["x"], i["a"], i["dout"], cu_seqlens=i["cu"],
                           workspace=torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == gdr.GDR_ERR_NO_WORKSPACE


def test_captured_and_replayed():
    i = inputs([700, 20], 72, "bf16", 8)
    out, hT = torch.empty_like(i["x"]), torch.empty_like(i["h0"])
    ws = torch.empty(gdr.gdr_gated_scan_bwd_workspace_size(2, 720, 72, True), dtype=torch.uint8, device="cuda")

    def step():
        gdr.gated_scan_fwd(i["x"], i["a"], h0=i["h0"], cu_seqlens=i["cu"], out=out, hT=hT)
        return gdr.gated_scan_bwd(i["x"], i["a"], i["dout"], i["dhT"], i["h0"], None, i["cu"], workspace=ws)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = step()
    other = inputs([700, 20], 72, "bf16", 9)
    for k in ("x", "a", "dout", "h0", "dhT"):
        i[k].copy_(other[k])
    graph.replay()
    want = gdr.gated_scan_fwd(other["x"], other["a"], h0=other["h0"], cu_seqlens=other["cu"])
    gwant = gdr.gated_scan_bwd(other["x"], other["a"], other["dout"], other["dhT"], other["h0"], None, other["cu"])
    ok()
    assert torch.equal(out, want[0]) and torch.equal(hT, want[1])
    assert all(torch.equal(p, q) for p, q in zip(grads, gwant))


@pytest.mark.parametrize("D", [64, 63])
def test_waits_that_run_out_are_reported(monkeypatch, D):
    """GDR_TC_WAIT_NS=0: a wait not satisfied at once gives up (for the tile's copy, or for the other
    blocks of a cluster).  The call returns, and the next one is right."""
    i = inputs([5000], D, "bf16", 3)
    want = gdr.gated_scan_fwd(i["x"], i["a"], h0=i["h0"], cu_seqlens=i["cu"], want_states=True)
    grads = gdr.gated_scan_bwd(i["x"], i["a"], i["dout"], i["dhT"], i["h0"], want[2], i["cu"])
    ok()
    monkeypatch.setenv("GDR_TC_WAIT_NS", "0")
    gdr.gated_scan_fwd(i["x"], i["a"], h0=i["h0"], cu_seqlens=i["cu"])
    assert gdr.gdr_get_status() == gdr.GDR_ERR_TIMEOUT
    gdr.gated_scan_bwd(i["x"], i["a"], i["dout"], i["dhT"], i["h0"], want[2], i["cu"])
    assert gdr.gdr_get_status() == gdr.GDR_ERR_TIMEOUT
    monkeypatch.delenv("GDR_TC_WAIT_NS")
    got = gdr.gated_scan_fwd(i["x"], i["a"], h0=i["h0"], cu_seqlens=i["cu"], want_states=True)
    again = gdr.gated_scan_bwd(i["x"], i["a"], i["dout"], i["dhT"], i["h0"], got[2], i["cu"])
    ok()
    assert all(torch.equal(p, q) for p, q in zip(want + grads, got + again))


@pytest.mark.parametrize("B,T,D", [(1, 131072, 96), (3, 30001, 40)])
def test_long(B, T, D):
    """Long sequences, in 64 bits on the GPU by blocks of tokens (the state carried from block to block)."""
    i = inputs([T] * B, D, "f32", 17, packed=False)
    out, hT, _ = gdr.gated_scan_fwd(i["x"], i["a"], h0=i["h0"], source="convex")
    ok()
    alpha, w, _, _ = ref.gates(i["a"].double(), 2.0, "bounded", "convex")
    u, h = w * i["x"].double(), i["h0"].double()
    for t in range(T):
        h = torch.addcmul(u[:, t], alpha[:, t], h, out=u[:, t])
    close(out, u.cpu(), BOUND32, "out")
    close(hT, h.cpu(), BOUND32, "hT")


@pytest.mark.parametrize("D", [65536, 65537])
def test_offsets_beyond_32_bits(D):
    """More than 2^31 elements: the first and the last channels, in 64 bits, and rows behind the tokens left alone."""
    T = 33000
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, a, dout = (torch.empty(1, T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(3))
    flat = torch.full(((T + 2) * D,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = flat[D:-D].view(1, T, D)
    h0, dhT = (torch.randn(1, D, generator=gen, device="cuda") for _ in range(2))
    _, hT, states = gdr.gated_scan_fwd(x, a, h0=h0, out=out, want_states=True, source="convex")
    dx, da, dh0 = gdr.gated_scan_bwd(x, a, dout, dhT, h0, states, source="convex")
    ok()
    assert (flat[:D] == 7).all() and (flat[-D:] == 7).all()
    for cols in (slice(0, 2), slice(D - 3, D)):
        one = lambda t: t[..., cols].reshape(-1, t[..., cols].shape[-1])  # noqa: E731
        form = dict(b=2.0, gate="bounded", source="convex")
        h, last = ref.forward(one(x), one(a), one(h0), [T], **form)
        close(one(out), h, BOUND16, "out")
        close(one(hT), last, BOUND32, "hT")
        close(one(states), h[127::128], BOUND32, "states")
        gx, ga, g0 = ref.backward(one(x), one(a), one(h0), one(dout), one(dhT), [T], **form)
        close(one(dx), gx, BOUND16, "dx")
        close(one(da), ga, BOUND16, "da")
        close(one(dh0), g0, BOUND32, "dh0")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_most_channels(dtype):
    """2^22 channels, one more refused."""
    D, T = 1 << 22, 130
    i = inputs([T], D, dtype, 3, packed=False)
    out, hT, states = gdr.gated_scan_fwd(i["x"], i["a"], h0=i["h0"], want_states=True)
    dx, da, dh0 = gdr.gated_scan_bwd(i["x"], i["a"], i["dout"], i["dhT"], i["h0"], states)
    ok()
    for cols in (slice(0, 33), slice(D - 33, D)):
        one = lambda t: t[..., cols].reshape(-1, 33)  # noqa: E731
        form = dict(b=2.0, gate="bounded", source="plain")
        h, last = ref.forward(one(i["x"]), one(i["a"]), one(i["h0"]), [T], **form)
        tol = BOUND16 if dtype == "bf16" else BOUND32
        close(one(out), h, tol, "out")
        close(one(hT), last, BOUND32, "hT")
        gx, ga, g0 = ref.backward(one(i["x"]), one(i["a"]), one(i["h0"]), one(i["dout"]), one(i["dhT"]), [T], **form)
        close(one(dx), gx, tol, "dx")
        close(one(da), ga, tol, "da")
        close(one(dh0), g0, BOUND32, "dh0")
    x = torch.zeros(1, 1, D + 1, device="cuda")
    with pytest.raises(gdr.GdrError) as e:
        gdr.gated_scan_fwd(x, x)
    assert e.value.code == gdr.GDR_ERR_UNSUPPORTED


@pytest.mark.parametrize("dtype,D", [("bf16", 63), ("f32", 63), ("f32", 64)])
def test_captured_forms(dtype, D):
    """Rows and pairs, with the states kept, and single tokens behind the prompt, in one graph."""
    i, other = inputs([900, 0, 150], D, dtype, 8), inputs([900, 0, 150], D, dtype, 9)
    tok = [torch.randn(3, 1, D, device="cuda").to(DT[dtype]) for _ in range(2)]

    def step(i):
        out, hT, states = gdr.gated_scan_fwd(i["x"], i["a"], h0=i["h0"], cu_seqlens=i["cu"], want_states=True)
        grads = gdr.gated_scan_bwd(i["x"], i["a"], i["dout"], i["dhT"], i["h0"], states, i["cu"])
        return (out, hT.clone(), states, gdr.gated_scan_recurrent_fwd(*tok, hT), hT) + grads

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(i)
    for k in ("x", "a", "dout", "h0", "dhT"):
        i[k].copy_(other[k])
    for _ in range(2):
        graph.replay()
    want = step(other)
    ok()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
