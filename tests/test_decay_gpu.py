"""GPU parity of the linear attention with one constant decay per head (gdr_decay_*)
against its definition in 64 bits.

Bounds (2-norm of the error over the 2-norm of the result), derived from the roundings:
  fp32 tensors and all states: products and sums in fp32 over up to some thousand terms,
    and powers exp(n g) with a relative error of about n |g| 2^-24 (n |g| < 16 where they
    matter): below 16 * 2^-24 + sqrt(4096) * 2^-24 = 4.8e-6; BOUND32 = 1e-5.
  bf16 outputs: the in-tile weights or the state once, and the result once, to 8 significant
    bits: at most 2^-8, and 1.7e-3 in the mean square over many values; two such errors
    give 2.4e-3; BOUND16 = 4e-3.
"""
import os

import numpy as np
import pytest
import torch

import chunked_gated_delta_07_gb300 as gdr
import decay_ref as ref

pytestmark = pytest.mark.gpu
BOUND32, BOUND16 = 1e-5, 4e-3
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_07_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)


@pytest.fixture
def seg_tiles(request):
    """GDR_DECAY_SEG_TILES for one test: the sequences are cut every so many 128-token tiles."""
    n = request.param
    if n:
        os.environ["GDR_DECAY_SEG_TILES"] = str(n)
    yield n
    os.environ.pop("GDR_DECAY_SEG_TILES", None)


def inputs(B, T, H, dk, dv, dtype, seed, lens=None, states=True, slopes=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    cu = None
    if lens is not None:
        B, T = 1, int(sum(lens))
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    N = B if lens is None else len(lens)
    unit = lambda x: torch.nn.functional.normalize(x, dim=-1).to(DT[dtype])  # noqa: E731
    slopes = slopes or [2.0 ** (-8 * (h + 1) / H) for h in range(H)]
    return dict(q=unit(rnd(B, T, H, dk)), k=unit(rnd(B, T, H, dk)), v=rnd(B, T, H, dv).to(DT[dtype]),
                dout=rnd(B, T, H, dv).to(DT[dtype]), g=torch.tensor([-s for s in slopes], device="cuda"),
                h0=rnd(N, H, dk, dv) * 0.5 if states else None, dhT=rnd(N, H, dk, dv) * 0.5 if states else None,
                cu=cu)


def ok():
    torch.cuda.synchronize()
    st = gdr.gdr_get_status()
    assert st == gdr.GDR_OK, gdr.gdr_status_string(st)


def check_fwd(x, path="auto", scale=0.5, **kw):
    out, hT = gdr.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], cu_seqlens=x["cu"], scale=scale,
                            path=path, **kw)
    ok()
    ro, rh = ref.decay_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"], x["cu"], scale)
    b = BOUND16 if x["q"].dtype == torch.bfloat16 else BOUND32
    assert ref.rel(out, ro) <= b and ref.rel(hT, rh) <= BOUND32, (ref.rel(out, ro), ref.rel(hT, rh))
    return out, hT


def check_bwd(x, path="auto", scale=0.5, **kw):
    got = gdr.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["dout"], dhT=x["dhT"], h0=x["h0"], cu_seqlens=x["cu"],
                        scale=scale, path=path, **kw)
    ok()
    want = ref.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["dout"], x["dhT"], x["h0"], x["cu"], scale)
    b = BOUND16 if x["q"].dtype == torch.bfloat16 else BOUND32
    far = [ref.rel(a, r) for a, r in zip(got, want)]
    assert max(far[:3]) <= b and far[3] <= BOUND32, far
    return got


LENGTHS = [1, 2, 15, 16, 17, 127, 128, 129, 255, 300]


@pytest.mark.parametrize("T", LENGTHS)
@pytest.mark.parametrize("dtype,path", [("bf16", "auto"), ("bf16", "simt"), ("f32", "auto")])
def test_forward_lengths(T, dtype, path):
    check_fwd(inputs(2, T, 3, 128, 128, dtype, 10 + T), path)


@pytest.mark.parametrize("T", LENGTHS)
@pytest.mark.parametrize("dtype,path", [("bf16", "auto"), ("bf16", "simt"), ("f32", "auto")])
def test_backward_lengths(T, dtype, path):
    check_bwd(inputs(2, T, 2, 128, 128, dtype, 40 + T), path)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9])
@pytest.mark.parametrize("path", ["auto", "tc"])
def test_short_sequences_on_either_path(T, path):
    """At most 8 tokens run on the CUDA cores unless the tensor cores are asked for."""
    x = inputs(3, T, 2, 128, 64, "bf16", 60 + T)
    check_fwd(x, path)
    check_bwd(x, path)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("dtype,path", [("bf16", "auto"), ("bf16", "simt"), ("f32", "auto")])
def test_widths(dk, dv, dtype, path):
    x = inputs(2, 333, 3, dk, dv, dtype, 70 + dk + dv)
    check_fwd(x, path)
    check_bwd(x, path)


@pytest.mark.parametrize("states", [True, False])
@pytest.mark.parametrize("dtype,path", [("bf16", "auto"), ("bf16", "simt"), ("f32", "auto")])
def test_packed_with_empty_and_short_sequences(states, dtype, path):
    x = inputs(1, 0, 3, 128, 128, dtype, 90, lens=[0, 1, 130, 0, 128, 7, 257, 0], states=states)
    check_fwd(x, path)
    check_bwd(x, path)


@pytest.mark.parametrize("seg_tiles", [1, 2, 3], indirect=True)
@pytest.mark.parametrize("lens", [None, [700, 5, 1300, 0, 129]])
@pytest.mark.parametrize("dtype,path", [("bf16", "auto"), ("bf16", "simt"), ("f32", "auto")])
def test_segments(seg_tiles, lens, dtype, path):
    """Sequences cut into segments whose states are chained, the last segment partial; decays
    from those that forget within a tile to those that remember everything."""
    x = inputs(2, 1100, 3, 128, 64, dtype, 100 + seg_tiles, lens=lens, slopes=[0.9, 0.02, 0.0])
    check_fwd(x, path)
    check_bwd(x, path)


@pytest.mark.parametrize("seg_tiles", [8, 11, 12], indirect=True)
@pytest.mark.parametrize("B,T", [(1, 5000), (2, 3333)])
def test_segments_summed_in_parts(seg_tiles, B, T):
    """Segments of 8 tiles or more are summed in parts, for the heads that remember that far:
    memories of all parts, some of them and the last few tokens alone."""
    x = inputs(B, T, 5, 64, 128, "bf16", 160 + seg_tiles, slopes=[0.0, 0.002, 0.1, 0.2, 3.0])
    check_fwd(x)
    check_bwd(x)


@pytest.mark.parametrize("path", ["auto", "simt"])
def test_long_sequence_uses_segments(path):
    x = inputs(1, 9000, 1, 128, 128, "bf16", 130, slopes=[0.004])
    check_fwd(x, path)
    check_bwd(x, path)


@pytest.mark.parametrize("dtype,path", [("bf16", "auto"), ("f32", "auto")])
def test_extreme_decays(dtype, path):
    """No decay, a decay below fp32's range within a token, and -inf: only the own token remains."""
    x = inputs(2, 200, 4, 128, 128, dtype, 140, slopes=[0.0, 3.0, 200.0, 1e-7])
    check_fwd(x, path)
    check_bwd(x, path)
    y = dict(x, g=torch.full((4,), -float("inf"), device="cuda"))
    out, hT = gdr.decay_fwd(y["q"], y["k"], y["v"], y["g"], h0=y["h0"], path=path)
    ok()
    own = (ref.np64(y["q"]) * ref.np64(y["k"])).sum(-1, keepdims=True) * ref.np64(y["v"])
    b = BOUND16 if dtype == "bf16" else BOUND32
    assert ref.rel(out, own) <= b
    last = ref.np64(y["k"][:, -1])[..., :, None] * ref.np64(y["v"][:, -1])[..., None, :]
    assert ref.rel(hT, last) <= BOUND32


@pytest.mark.parametrize("seg_tiles", [0, 8], indirect=True)
@pytest.mark.parametrize("g", [0.0, -1e-4, -2e-3])
def test_weak_decays_keep_states_in_full_precision(g, seg_tiles):
    """States that remember thousands of tokens.  The tensor cores add a tile's products 16 tokens
    and one of three terms at a time, 24 sums that are cut off and not rounded: half a unit in the
    last place (2^-24) each on average, always towards zero, 24 * 2^-24 = 1.4e-6 for the tile's
    part.  Adding the parts up must not add to that but what rounding does, 2^-24 at random."""
    x = inputs(1, 4096, 2, 128, 128, "bf16", 140, slopes=[-g, -g])
    bound = 1.5e-6
    _, hT = gdr.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"])
    dh0 = gdr.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["dout"], dhT=x["dhT"], h0=x["h0"])[3]
    ok()
    far = ref.rel(hT, ref.decay_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"], None)[1])
    far0 = ref.rel(dh0, ref.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["dout"], x["dhT"], x["h0"], None)[3])
    assert far <= bound and far0 <= bound, (far, far0)


@pytest.mark.parametrize("path", ["auto", "simt"])
def test_unaligned_pointers_take_the_general_path(path):
    """Tensors one element past a 16-byte boundary."""
    x = inputs(2, 150, 2, 128, 128, "bf16", 150)
    for n in ("q", "k", "v", "dout"):
        buf = torch.empty(x[n].numel() + 1, dtype=torch.bfloat16, device="cuda")
        buf[1:].copy_(x[n].flatten())
        x[n] = buf[1:].view(x[n].shape)
    check_fwd(x, path)
    check_bwd(x, path)
    with pytest.raises(gdr.GdrError):
        gdr.decay_fwd(x["q"], x["k"], x["v"], x["g"], path="tc")


@pytest.mark.parametrize("path", ["auto", "simt"])
def test_neighbours_do_not_leak(path):
    """NaN and infinities of one packed sequence reach no other one: equal to the call alone."""
    x = inputs(1, 0, 2, 128, 128, "bf16", 160, lens=[100, 200, 77])
    clean = check_fwd(x, path)
    grads = check_bwd(x, path)
    for n, bad in (("k", float("nan")), ("v", float("inf")), ("q", float("nan")), ("dout", -float("inf"))):
        x[n] = x[n].clone()
        x[n][:, 100:300] = bad
    out, hT = gdr.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], cu_seqlens=x["cu"], scale=0.5, path=path)
    got = gdr.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["dout"], dhT=x["dhT"], h0=x["h0"], cu_seqlens=x["cu"],
                        scale=0.5, path=path)
    ok()
    for a, c in ((out, clean[0]), *zip(got[:3], grads[:3])):
        assert torch.equal(a[:, :100], c[:, :100]) and torch.equal(a[:, 300:], c[:, 300:])
    for a, c in ((hT, clean[1]), (got[3], grads[3])):
        assert torch.equal(a[0], c[0]) and torch.equal(a[2], c[2])


@pytest.mark.parametrize("seg_tiles", [0, 1], indirect=True)
@pytest.mark.parametrize("path", ["auto", "simt"])
def test_state_carried_in_place_and_in_pieces(seg_tiles, path):
    """hT may be h0; two calls with the state carried over equal one over all tokens."""
    x = inputs(2, 515, 3, 128, 128, "bf16", 170)
    out, hT = check_fwd(x, path)
    state = x["h0"].clone()
    outs = []
    for a, b in ((0, 260), (260, 515)):
        p = [x[n][:, a:b].contiguous() for n in ("q", "k", "v")]
        o, s = gdr.decay_fwd(*p, x["g"], h0=state, hT=state, scale=0.5, path=path)
        assert s is state
        outs.append(o)
    ok()
    assert ref.rel(state, ref.np64(hT)) <= BOUND32
    assert ref.rel(torch.cat(outs, 1), ref.np64(out)) <= 2 * BOUND16   # two rounded results


@pytest.mark.parametrize("path", ["auto", "simt"])
def test_deterministic_and_on_another_stream(path):
    x = inputs(3, 400, 3, 128, 128, "bf16", 180)
    a = check_fwd(x, path) + check_bwd(x, path)
    ws = torch.empty(max(16, gdr.gdr_decay_workspace_size(3, 400, 3, 128, 128, backward=True)), dtype=torch.uint8,
                     device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    b = gdr.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], scale=0.5, path=path, stream=side, workspace=ws)
    b += gdr.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["dout"], dhT=x["dhT"], h0=x["h0"], scale=0.5, path=path,
                       stream=side, workspace=ws)
    side.synchronize()
    assert all(torch.equal(p, r) for p, r in zip(a, b))


@pytest.mark.parametrize("d,H", [(64, 32), (128, 16)])
def test_many_calls_neither_stall_nor_differ(d, H):
    """Packed sequences with many short last tiles, whose rows are stored one by one while the next
    tiles are under way: no call may run into a wait's limit or give another result."""
    lens = [1 + (37 * i) % 300 for i in range(60)] + [2000, 3000]
    x = inputs(1, 0, H, d, d, "bf16", 700, lens=lens)
    out, hT = check_fwd(x)
    for _ in range(300):
        o, h = gdr.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], cu_seqlens=x["cu"], scale=0.5)
    ok()
    assert torch.equal(o, out) and torch.equal(h, hT)


def test_gradients_against_differences():
    """The gradients along a random direction against central differences of the fp64 forward:
    bilinear in each input, so a difference in one input is exact up to rounding."""
    x = inputs(1, 40, 2, 64, 64, "f32", 190)
    got = dict(zip(("q", "k", "v", "h0"), check_bwd(x)))
    gen = torch.Generator(device="cuda").manual_seed(7)
    for n, grad in got.items():
        d = torch.randn(x[n].shape, generator=gen, device="cuda")
        side = []
        for e in (1.0, -1.0):
            y = dict(x, **{n: x[n] + e * d})
            o, h = ref.decay_fwd(y["q"], y["k"], y["v"], y["g"], y["h0"], None, 0.5)
            side.append((o * ref.np64(x["dout"])).sum() + (h * ref.np64(x["dhT"])).sum())
        want = (side[0] - side[1]) / 2
        have = (ref.np64(grad) * ref.np64(d)).sum()
        size = np.linalg.norm(ref.np64(grad)) * np.linalg.norm(ref.np64(d))
        assert abs(have - want) <= BOUND32 * size, (n, have, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("N,T", [(1, 1), (5, 1), (3, 2), (2, 7), (1, 40)])
def test_single_tokens(dtype, dk, dv, N, T):
    x = inputs(N, T, 3, dk, dv, dtype, 200 + T + N)
    state = x["h0"].clone()
    out = gdr.decay_recurrent_fwd(x["q"], x["k"], x["v"], x["g"], state, scale=0.25)
    ok()
    ro, rh = ref.decay_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"], None, 0.25)
    # only the result is rounded: 1.7e-3 in the mean square over the outputs
    assert ref.rel(out, ro) <= (2.0 ** -9 if dtype == "bf16" else BOUND32) and ref.rel(state, rh) <= BOUND32


def test_prompt_then_single_tokens():
    x = inputs(2, 150, 4, 128, 128, "bf16", 230)
    out, state = gdr.decay_fwd(*(x[n][:, :140].contiguous() for n in ("q", "k", "v")), x["g"], h0=x["h0"])
    outs = [out]
    for t in range(140, 150):
        outs.append(gdr.decay_recurrent_fwd(*(x[n][:, t:t + 1].contiguous() for n in ("q", "k", "v")), x["g"], state))
    ok()
    ro, rh = ref.decay_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"])
    assert ref.rel(torch.cat(outs, 1), ro) <= BOUND16 and ref.rel(state, rh) <= BOUND32


def test_no_tokens():
    x = inputs(2, 0, 3, 128, 128, "bf16", 240)
    out, hT = gdr.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"])
    assert out.shape == (2, 0, 3, 128) and torch.equal(hT, x["h0"])
    assert not gdr.decay_fwd(x["q"], x["k"], x["v"], x["g"])[1].any()
    dh0 = gdr.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["dout"], dhT=x["dhT"])[3]
    assert torch.equal(dh0, x["dhT"])
    state = x["h0"].clone()
    gdr.decay_recurrent_fwd(x["q"], x["k"], x["v"], x["g"], state)
    assert torch.equal(state, x["h0"])
    y = inputs(1, 0, 3, 128, 128, "bf16", 241, lens=[0, 0])
    out, hT = gdr.decay_fwd(y["q"], y["k"], y["v"], y["g"], h0=y["h0"], cu_seqlens=y["cu"])
    ok()
    assert torch.equal(hT, y["h0"])


@pytest.mark.parametrize("path", ["auto", "simt"])
@pytest.mark.parametrize("offsets", [[0, 50, 40, 100], [1, 50, 100], [0, 50, 99], [0, -5, 100]])
def test_bad_offsets_are_reported_and_write_nothing(offsets, path):
    x = inputs(1, 100, 2, 128, 128, "bf16", 250)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    out = torch.full_like(x["v"], 7.0)
    hT = torch.full((len(offsets) - 1, 2, 128, 128), 7.0, device="cuda")
    gdr.decay_fwd(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, out=out, hT=hT, path=path)
    torch.cuda.synchronize()
    assert gdr.gdr_get_status() == gdr.GDR_ERR_BAD_SEQLENS
    assert (out == 7.0).all() and (hT == 7.0).all()
    ok()   # the status was cleared


@pytest.mark.parametrize("seg_tiles", [0, 2], indirect=True)
@pytest.mark.parametrize("lens", [None, [300, 0, 129, 500]])
def test_waits_that_run_out_report_a_timeout_and_unwind(seg_tiles, lens, monkeypatch):
    """Every wait of the tensor-core kernels is bounded.  With the limit at 0 each looks once: the
    first one not yet satisfied sets the status and the block unwinds (its copies drained, its
    tensor memory freed), so the next call at the default limit is right."""
    x = inputs(2, 600, 3, 128, 128, "bf16", 600, lens=lens)
    ok()
    monkeypatch.setenv("GDR_TC_WAIT_NS", "0")
    gdr.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], cu_seqlens=x["cu"])
    assert gdr.gdr_get_status() == gdr.GDR_ERR_TIMEOUT
    gdr.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["dout"], dhT=x["dhT"], h0=x["h0"], cu_seqlens=x["cu"])
    assert gdr.gdr_get_status() == gdr.GDR_ERR_TIMEOUT
    monkeypatch.delenv("GDR_TC_WAIT_NS")
    for _ in range(2):
        check_fwd(x)
        check_bwd(x)
