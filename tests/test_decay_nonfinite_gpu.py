"""A NaN or an infinity of one token in the decay linear attention: which results it reaches (GPU).

By the recurrence S_t = lam S_{t-1} + k_t v_t^T a NaN in k_t or v_t makes elements of the state NaN, an
infinity infinite or NaN, and lam times those stays so, however fast the head forgets: every later output of
the head that reads them and the last state are not finite.  Long sequences are cut into segments, of which
a fast head's local sums read the last tokens alone, so the token is planted where they skip it.  Rows and
columns that it does not touch, tokens before its 128-token tile, other heads and other sequences keep
their values, bit for bit where they are computed the same way.
"""
import pytest
import torch

import chunked_gated_delta_07_gb300 as gdr
import decay_ref as ref
from test_decay_gpu import BOUND16, BOUND32, inputs, ok, seg_tiles  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
AT, TILE = 300, 256   # the token and the start of its 128-token tile
D, E = 5, 70          # its channel of k (q), of v (dout)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_07_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)


def make(dtype, lens, seed):
    # heads that forget within a tile, within some and never
    return inputs(2, 2500, 3, 128, 128, dtype, seed, lens=lens, slopes=[2.0, 0.3, 0.0])


def plant(x, name, value, head, channel, at):
    x = dict(x)
    x[name] = x[name].clone()
    x[name][0, at, head, channel] = value
    return x


LENS = [None, [2500, 77, 1300]]


@pytest.mark.parametrize("seg_tiles", [0, 4, 6], indirect=True)
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("head", [0, 1, 2])
@pytest.mark.parametrize("name,value", [("k", NAN), ("v", NAN), ("v", INF), ("k", -INF)])
@pytest.mark.parametrize("dtype,path", [("bf16", "auto"), ("bf16", "simt"), ("f32", "auto")])
def test_forward(seg_tiles, lens, head, name, value, dtype, path):  # noqa: F811
    x = make(dtype, lens, 800)
    call = lambda y: gdr.decay_fwd(y["q"], y["k"], y["v"], y["g"], h0=y["h0"], cu_seqlens=y["cu"],  # noqa: E731
                                   scale=0.5, path=path)
    out, hT = call(x)
    bad, hbad = call(plant(x, name, value, head, D if name == "k" else E, AT))
    ok()
    # the sequence's later outputs: all columns for a row of the state, one for a column
    cols = slice(None) if name == "k" else E
    assert not bad[0, AT:2500, head, cols].isfinite().any()
    assert not (hbad[0, head, D] if name == "k" else hbad[0, head, :, E]).isfinite().any()
    if name == "v":
        rest = [e for e in range(128) if e != E]
        assert bad[0, :2500, head][:, rest].isfinite().all() and hbad[0, head][:, rest].isfinite().all()
    else:
        assert hbad[0, head, [d for d in range(128) if d != D]].isfinite().all()
    # before its tile, other heads, other sequences
    others = [h for h in range(3) if h != head]
    assert torch.equal(bad[0, :TILE], out[0, :TILE]) and torch.equal(bad[0, :2500, others], out[0, :2500, others])
    assert torch.equal(bad[0, 2500:], out[0, 2500:]) and torch.equal(bad[1:], out[1:])
    assert torch.equal(hbad[0, others], hT[0, others]) and torch.equal(hbad[1:], hT[1:])


@pytest.mark.parametrize("seg_tiles", [0, 4], indirect=True)
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("head", [0, 1, 2])
@pytest.mark.parametrize("name", ["k", "v", "q", "dout"])
@pytest.mark.parametrize("dtype,path", [("bf16", "auto"), ("bf16", "simt"), ("f32", "auto")])
def test_backward(seg_tiles, lens, head, name, dtype, path):  # noqa: F811
    """k and v reach the dq of later tokens through the state; q and dout the dk and dv of earlier
    tokens and dh0 through the state's gradient."""
    x = make(dtype, lens, 810)
    call = lambda y: gdr.decay_bwd(y["q"], y["k"], y["v"], y["g"], y["dout"], dhT=y["dhT"], h0=y["h0"],  # noqa: E731
                                   cu_seqlens=y["cu"], scale=0.5, path=path)
    at = AT if name in ("k", "v") else 2499 - AT
    end = (at // 128 + 1) * 128   # of its tile
    c = D if name in ("k", "q") else E
    dq, dk, dv, dh0 = call(x)
    bq, bk, bv, bh = call(plant(x, name, NAN, head, c, at))
    ok()
    if name in ("k", "v"):   # dq_t = scale S_t dout_t
        assert bq[0, at:2500, head, c if name == "k" else slice(None)].isnan().all()
        assert torch.equal(bq[0, :at // 128 * 128], dq[0, :at // 128 * 128])
        assert torch.equal(bh, dh0)
    else:                    # dk_t = dS_t v_t, dv_t = dS_t^T k_t
        rows, cols = (c, slice(None)) if name == "q" else (slice(None), c)
        assert bk[0, :at + 1, head, rows].isnan().all() and bv[0, :at + 1, head, cols].isnan().all()
        assert bh[0, head, rows, cols].isnan().all()
        assert torch.equal(bk[0, end:], dk[0, end:]) and torch.equal(bv[0, end:], dv[0, end:])
        assert torch.equal(bq[0, end:], dq[0, end:])
    others = [h for h in range(3) if h != head]
    for a, b in ((bq, dq), (bk, dk), (bv, dv)):
        assert torch.equal(a[0, :2500, others], b[0, :2500, others])
        assert torch.equal(a[0, 2500:], b[0, 2500:]) and torch.equal(a[1:], b[1:])
    assert torch.equal(bh[0, others], dh0[0, others]) and torch.equal(bh[1:], dh0[1:])


@pytest.mark.parametrize("seg_tiles", [4], indirect=True)
def test_clean_columns_keep_their_values(seg_tiles):  # noqa: F811
    """The columns of v beside the planted one are right, not only finite."""
    x = make("bf16", None, 820)
    bad, hbad = gdr.decay_fwd(*(plant(x, "v", NAN, 0, E, AT)[n] for n in ("q", "k", "v")), x["g"], h0=x["h0"], scale=0.5)
    ok()
    ro, rh = ref.decay_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"], None, 0.5)
    rest = [e for e in range(128) if e != E]
    assert ref.rel(bad[..., rest], ro[..., rest]) <= BOUND16 and ref.rel(hbad[..., rest], rh[..., rest]) <= BOUND32


@pytest.mark.parametrize("seg_tiles", [0, 4], indirect=True)
def test_state_in_place(seg_tiles):  # noqa: F811
    """hT = h0 with a NaN that the local sums skip: the states entered are the first ones all the same."""
    x = plant(make("bf16", None, 830), "v", NAN, 0, E, AT)
    _, hT = gdr.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], scale=0.5)
    state = x["h0"].clone()
    gdr.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=state, hT=state, scale=0.5)
    ok()
    assert torch.equal(state.nan_to_num(7.0), hT.nan_to_num(7.0)) and state[0, 0, :, E].isnan().all()


@pytest.mark.parametrize("seg_tiles", [0, 4], indirect=True)
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("lens", LENS)
def test_other_widths(seg_tiles, dk, dv, lens):  # noqa: F811
    x = inputs(2, 2500, 3, dk, dv, "bf16", 840, lens=lens, slopes=[2.0, 0.3, 0.0])
    out, hT = gdr.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], cu_seqlens=x["cu"], scale=0.5)
    y = plant(x, "v", NAN, 0, 9, AT)
    bad, hbad = gdr.decay_fwd(y["q"], y["k"], y["v"], y["g"], h0=y["h0"], cu_seqlens=y["cu"], scale=0.5)
    args = dict(dhT=y["dhT"], h0=y["h0"], cu_seqlens=y["cu"], scale=0.5)
    dq = gdr.decay_bwd(y["q"], y["k"], y["v"], y["g"], y["dout"], **args)[0]
    z = plant(x, "q", NAN, 0, 9, 2499 - AT)
    _, dk_, dv_, dh0 = gdr.decay_bwd(z["q"], z["k"], z["v"], z["g"], z["dout"], **args)
    ok()
    assert bad[0, AT:2500, 0, 9].isnan().all() and hbad[0, 0, :, 9].isnan().all()
    assert torch.equal(bad[0, :2500, 1:], out[0, :2500, 1:]) and torch.equal(hbad[0, 1:], hT[0, 1:])
    assert torch.equal(bad[0, 2500:], out[0, 2500:]) and torch.equal(hbad[1:], hT[1:])
    assert dq[0, AT:2500, 0].isnan().all() and dq[0, :TILE].isfinite().all() and dq[0, :2500, 1:].isfinite().all()
    assert dk_[0, :2500 - AT, 0, 9].isnan().all() and dv_[0, :2500 - AT, 0].isnan().all()
    assert dh0[0, 0, 9].isnan().all() and dh0[0, 1:].isfinite().all() and dh0[1:].isfinite().all()


@pytest.mark.parametrize("T", [1, 5, 40, 300])
@pytest.mark.parametrize("dtype,path", [("bf16", "auto"), ("bf16", "tc"), ("bf16", "simt"), ("f32", "auto")])
def test_log_decay_that_is_no_number(T, dtype, path):
    """Every output and state of its head is NaN, from the first token on; other heads are untouched."""
    x = inputs(2, T, 3, 128, 128, dtype, 850)
    g = x["g"].clone()
    g[1] = NAN
    for h0 in (x["h0"], None):
        out, hT = gdr.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=h0, path=path)
        bad, hbad = gdr.decay_fwd(x["q"], x["k"], x["v"], g, h0=h0, path=path)
        dq = gdr.decay_bwd(x["q"], x["k"], x["v"], g, x["dout"], h0=h0, path=path)[0]
        ok()
        assert bad[:, :, 1].isnan().all() and hbad[:, 1].isnan().all() and dq[:, :, 1].isnan().all()
        assert torch.equal(bad[:, :, ::2], out[:, :, ::2]) and torch.equal(hbad[:, ::2], hT[:, ::2])
        assert dq[:, :, ::2].isfinite().all()
    state = x["h0"].clone()
    out = gdr.decay_recurrent_fwd(x["q"], x["k"], x["v"], g, state)
    ok()
    assert out[:, :, 1].isnan().all() and state[:, 1].isnan().all() and out[:, :, ::2].isfinite().all()
