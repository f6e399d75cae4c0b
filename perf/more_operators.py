"""Cases of the gated scan and of the norms around a block, with their plain forms.

Gated scan, one decay per token and channel, per (sequence, channel):

    alpha_t = exp(g(a_t)),  g(a) = -b sigmoid(a) or -softplus(a)
    h_t = alpha_t h_{t-1} + w(alpha_t) x_t
    w = 1 (plain), 1 - alpha (convex) or sqrt(1 - alpha^2) (variance)

over a prompt (scan_fwd: every h_t, the last one, and after every 128 tokens of the batch the
fp32 state that the backward pass starts from), its gradients (scan_bwd), and token by token
with the state updated in place (scan_step).

Norms around a block, N(x) = xh w + bias, xh = x rstd (rms) or (x - mean) rstd (layer), with
one weight for all rows or one per group of rows (per head):

    before it:  r = residual + scale x,   y = N(r)                       (add_norm)
    behind it:  y = residual + scale N(x) act(z), act silu or sigmoid    (norm_gate)

forward, and backward from the forward's statistics.

`run` computes a case in its plain form (elementary torch operations in 32 bits) where
`own` is false and by the library's calls where it is true.
"""
import math

import numpy as np
import torch

own = False   # set from outside: False for the plain forms, True for the library's calls

EVERY = 128   # tokens from one kept state to the next
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases ------------------------------------------------------------------------
def _scan(name, op, B, T, D, dtype, gate="bounded", source="plain", b=2.0, packed=0, state=True, kept=False):
    return {"name": name, "op": op, "B": B, "T": T, "D": D, "dtype": dtype, "gate": gate, "source": source, "b": b,
            "packed": packed, "state": state, "kept": kept}


def _norm(name, op, rows, groups, D, dtype, kind="rms", act="silu", scale=1.0, extra=True):
    return {"name": name, "op": op, "rows": rows, "groups": groups, "D": D, "dtype": dtype, "kind": kind, "act": act,
            "scale": scale, "extra": extra}


def listed():
    return [
        # the next piece of a chat's prompt, the state carried in and out: latency counts
        _scan("scan_prompt_33", "scan_fwd", 1, 33, 2048, "bf16", source="variance"),
        # one layer's forward pass of a training step, 8 sequences of 4096 tokens
        _scan("scan_train_8x4096", "scan_fwd", 8, 4096, 2048, "bf16", source="variance", state=False, kept=True),
        # a long document, one sequence
        _scan("scan_document_256k", "scan_fwd", 1, 262144, 2048, "bf16"),
        # a serving engine's batch of prompts of unequal lengths, a narrower model
        _scan("scan_prompts_packed_64k", "scan_fwd", 1, 65536, 1000, "bf16", source="convex", packed=37),
        # the training step's backward pass, from the states that its forward pass kept
        _scan("scan_grad_8x4096", "scan_bwd", 8, 4096, 2048, "bf16", source="variance", state=False, kept=True),
        # a small run in fp32: packed sequences, odd width, initial states and their gradients,
        # nothing kept from the forward pass
        _scan("scan_grad_packed_f32", "scan_bwd", 1, 5003, 333, "f32", gate="softplus", source="convex", packed=7),
        # one token of each of 256 conversations served together
        _scan("scan_step_256", "scan_step", 256, 1, 2048, "bf16"),
        # the residual stream's sum and the norm in front of a block, the training step's tokens
        _norm("add_norm_32k", "add_norm_fwd", 8 * 4096, 1, 2048, "bf16", scale=0.5),
        # a few tokens' rows, a width that is no power of two, fp32, layer norm with a bias
        _norm("add_norm_small", "add_norm_fwd", 7, 1, 1000, "f32", kind="layer"),
        # its backward pass, ragged row count
        _norm("add_norm_grad_8k", "add_norm_bwd", 8191, 1, 2048, "bf16", scale=0.5),
        # the gated norm of every head's output behind the mixing layer of the training step
        _norm("norm_gate_heads", "norm_gate_fwd", 8 * 4096 * 16, 16, 128, "bf16", extra=False),
        # its backward pass
        _norm("norm_gate_grad_heads", "norm_gate_bwd", 8 * 4096 * 16, 16, 128, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step", "add_norm_fwd", "add_norm_bwd",
                     "norm_gate_fwd", "norm_gate_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if not op.startswith("scan"):
        D = _log_int(rng, 8, 8192)
        groups = rng.choice([1, 1, 3, 16]) if D <= 256 else 1
        rows = _log_int(rng, 1, max(1, min(1 << 19, (1 << 25) // D) // groups)) * groups
        case = _norm("", op, rows, groups, D, dtype, rng.choice(["rms", "rms", "layer"]),
                     rng.choice(["silu", "silu", "sigmoid"]), rng.choice([1.0, 0.5, 0.125]), rng.choice([True, False]))
        return {k: v for k, v in case.items() if k != "name"}
    D = _log_int(rng, 8, 4096)
    gate, source = rng.choice(["bounded", "bounded", "softplus"]), rng.choice(["plain", "convex", "variance"])
    b, state, kept = rng.choice([2.0, 2.0, 5.0, 8.0]), rng.choice([True, False]), rng.choice([True, False])
    if op == "scan_step":
        B, T, packed, state, kept = _log_int(rng, 1, 1024), rng.choice([1, 1, 1, 2, 4]), 0, True, False
    else:
        total = _log_int(rng, 1, min(1 << 17, (1 << 26) // D))   # tokens over all sequences
        packed = rng.choice([0, 0, _log_int(rng, 1, 64)])
        B = 1 if packed else _log_int(rng, 1, max(1, min(64, total)))
        T = max(1, total // B)
    case = _scan("", op, B, T, D, dtype, gate, source, b, packed, state, kept)
    return {k: v for k, v in case.items() if k != "name"}


# ---- the inputs -----------------------------------------------------------------------
def _lengths(case, seed):
    """Lengths of the packed sequences: spread over a factor of 64, some may be empty."""
    w = np.exp(np.random.RandomState(seed).uniform(0.0, math.log(64.0), case["packed"]))
    ends = np.floor(np.cumsum(w) / w.sum() * case["T"]).astype(np.int64)
    ends[-1] = case["T"]
    return np.diff(np.concatenate([[0], ends]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = TYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * std

    s = dict(case)
    if not case["op"].startswith("scan"):
        rows, G, D = case["rows"], case["groups"], case["D"]
        shape = (rows // G, G, D) if G > 1 else (rows, D)
        s["x"] = (normal(*shape) * 1.5 + 0.3).to(dt)
        s["weight"] = 1.0 + normal(*shape[len(shape) - (2 if G > 1 else 1):], std=0.2)
        s["bias"] = normal(*s["weight"].shape, std=0.1) if case["kind"] == "layer" else None
        if case["op"].startswith("norm_gate"):
            s["z"] = normal(*shape).to(dt)
        if case["op"] == "add_norm_fwd" or case["op"] == "norm_gate_fwd" and case["extra"]:
            s["residual"] = normal(*shape, std=2.0).to(dt)
        if case["op"].endswith("bwd"):
            s["dy"] = normal(*shape).to(dt)
            if case["op"] == "add_norm_bwd" and case["extra"]:
                s["dr"] = normal(*shape).to(dt)   # the gradient along the residual stream
            s["mean"], s["rstd"] = _stats(s["x"].float(), case["kind"])   # saved by the forward pass
        return s
    B, T, D = case["B"], case["T"], case["D"]
    N = case["packed"] or B
    s["x"] = normal(B, T, D).to(dt)
    # each channel has its own usual memory, from about a token to some hundreds
    far = 7.0 * torch.rand(D, generator=gen, device="cuda") - 6.0
    s["a"] = normal(B, T, D).add_(far).to(dt)
    s["cu"] = None
    if case["packed"]:
        ends = np.concatenate([[0], np.cumsum(_lengths(case, seed))])
        s["cu"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    if case["op"] == "scan_step":
        s["h"] = normal(N, D)
        return s
    s["h0"] = normal(N, D) if case["state"] else None
    if case["op"] == "scan_bwd":
        s["dout"] = normal(B, T, D).to(dt)
        s["dhT"] = normal(N, D) if case["state"] else None
        s["states"] = _plain_scan_fwd(s)[2] if case["kept"] else None   # kept by the forward pass
    return s


# ---- the plain forms --------------------------------------------------------------------
def _gate(s):
    """alpha, w and what the gradients take: dw/dg and dg/da, in 32 bits."""
    a = s["a"].float()
    if s["gate"] == "bounded":
        g = -s["b"] * torch.sigmoid(a)
        slope = g * torch.sigmoid(-a)
    else:
        g = -(a.clamp(min=0) + torch.log1p(torch.exp(-a.abs())))
        slope = -torch.sigmoid(a)
    alpha = torch.exp(g)
    if s["source"] == "plain":
        return alpha, torch.ones_like(a), torch.zeros_like(a), slope
    if s["source"] == "convex":
        return alpha, -torch.expm1(g), -alpha, slope
    w = torch.sqrt(-torch.expm1(2 * g))
    return alpha, w, -alpha * alpha / w, slope


def _ends(s):
    """First and last tokens of the sequences that have any, and their numbers, on [B T] tokens."""
    B, T = s["x"].shape[:2]
    if s["cu"] is None:
        first = torch.arange(B, device="cuda") * T
        return first, first + T - 1, torch.arange(B, device="cuda"), B
    cu = s["cu"].long()
    has = torch.nonzero(cu[1:] > cu[:-1]).squeeze(1)
    return cu[:-1][has], cu[1:][has] - 1, has, cu.numel() - 1


def _sweep(A, U):
    """h_t = A_t h_{t-1} + U_t along the first axis from h = 0, by doubling; overwrites both."""
    d = 1
    while d < U.shape[0]:
        U[d:] = U[d:] + A[d:] * U[:-d]
        A[d:] = A[d:] * A[:-d]
        d *= 2
    return U


def _plain_states(s, alpha, w):
    """Every h_t in 32 bits; all tensors [B T, D]."""
    first, _, seq, _ = _ends(s)
    alpha, u = alpha.clone(), w * s["x"].flatten(0, 1).float()
    if s["h0"] is not None:
        u[first] = u[first] + alpha[first] * s["h0"][seq]
    alpha[first] = 0
    return _sweep(alpha, u)


def _plain_scan_fwd(s):
    alpha, w, _, _ = (v.flatten(0, 1) for v in _gate(s))
    h = _plain_states(s, alpha, w)
    _, last, seq, N = _ends(s)
    hT = h.new_zeros((N, h.shape[1])) if s["h0"] is None else s["h0"].clone()
    hT[seq] = h[last]
    return h.reshape(s["x"].shape).to(s["x"].dtype), hT, h[EVERY - 1::EVERY].clone()


def _plain_scan_bwd(s):
    """With l_t the gradient of h_t: l_t = dout_t + alpha_{t+1} l_{t+1} (the last one holds dhT
    too), dx = w l, da = l (alpha h_{t-1} + w'(g) x) g'(a), dh0 = alpha_1 l_1."""
    alpha, w, dw, slope = (v.flatten(0, 1) for v in _gate(s))
    first, last, seq, N = _ends(s)
    h = _plain_states(s, alpha, w)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[first] = 0 if s["h0"] is None else s["h0"][seq]
    lam = s["dout"].flatten(0, 1).float()
    if s["dhT"] is not None:
        lam = lam.index_add(0, last, s["dhT"][seq])
    after = torch.cat([alpha[1:], torch.zeros_like(alpha[:1])])
    after[last] = 0
    lam = _sweep(after.flip(0), lam.flip(0)).flip(0)
    x = s["x"].flatten(0, 1).float()
    dx, da = w * lam, lam * (alpha * before + dw * x) * slope
    dh0 = h.new_zeros((N, h.shape[1])) if s["dhT"] is None else s["dhT"].clone()
    dh0[seq] = alpha[first] * lam[first]
    shape, dt = s["x"].shape, s["x"].dtype
    return dx.reshape(shape).to(dt), da.reshape(shape).to(dt), dh0


def _plain_scan_step(s):
    alpha, w, _, _ = _gate(s)
    x = s["x"].float()
    out = torch.empty_like(s["x"])
    for t in range(x.shape[1]):
        s["h"].mul_(alpha[:, t]).add_(w[:, t] * x[:, t])
        out[:, t] = s["h"].to(out.dtype)
    return out, s["h"]


def _stats(x, kind):
    if kind == "rms":
        return None, torch.rsqrt(x.square().mean(-1) + EPS)
    mean = x.mean(-1)
    return mean, torch.rsqrt((x - mean[..., None]).square().mean(-1) + EPS)


def _centred(x, s):
    return x if s["mean"] is None else x - s["mean"][..., None]


def _act(z, act):
    """act(z) and its derivative."""
    g = torch.sigmoid(z)
    if act == "sigmoid":
        return g, g * (1 - g)
    return z * g, g * (1 + z * (1 - g))


def _affine(xh, s):
    y = xh * s["weight"]
    return y if s["bias"] is None else y + s["bias"]


def _plain_norm_fwd(s):
    x, dt = s["x"].float(), s["x"].dtype
    if s["op"] == "add_norm_fwd":
        r = (s["residual"].float() + s["scale"] * x).to(dt)   # the stream is kept in its type
        x = r.float()
    mean, rstd = _stats(x, s["kind"])
    y = _affine((x if mean is None else x - mean[..., None]) * rstd[..., None], s)
    if s["op"] == "add_norm_fwd":
        return y.to(dt), r, mean, rstd
    y = s["scale"] * y * _act(s["z"].float(), s["act"])[0]
    if s["extra"]:
        y = y + s["residual"].float()
    return y.to(dt), mean, rstd


def _through(dn, xh, s):
    """The gradient through N's statistics, dn that of xh."""
    d = dn - xh * (dn * xh).mean(-1, keepdim=True)
    if s["kind"] == "layer":
        d = d - dn.mean(-1, keepdim=True)
    return d * s["rstd"][..., None]


def _plain_norm_bwd(s):
    dy, dt = s["dy"].float(), s["dy"].dtype
    xh = _centred(s["x"].float(), s) * s["rstd"][..., None]
    dz = None
    if s["op"] == "norm_gate_bwd":
        act, slope = _act(s["z"].float(), s["act"])
        dz = (s["scale"] * dy * _affine(xh, s) * slope).to(dt)
        dy = s["scale"] * dy * act
    d = _through(dy * s["weight"], xh, s)
    dw, db = (dy * xh).sum(0), dy.sum(0) if s["kind"] == "layer" else None
    if dz is not None:
        return d.to(dt), dz, dw, db
    if s["extra"]:
        d = d + s["dr"].float()
    return (s["scale"] * d).to(dt), d.to(dt), dw, db


def run(s):
    op = s["op"]
    if own:
        import chunked_gated_delta_07_gb300 as gdr
        if op.startswith("scan"):
            form = {"b": s["b"], "gate": s["gate"], "source": s["source"]}
            if op == "scan_fwd":
                return gdr.gated_scan_fwd(s["x"], s["a"], h0=s["h0"], cu_seqlens=s["cu"], want_states=s["kept"], **form)
            if op == "scan_bwd":
                return gdr.gated_scan_bwd(s["x"], s["a"], s["dout"], dhT=s["dhT"], h0=s["h0"], states=s["states"],
                                          cu_seqlens=s["cu"], **form)
            return gdr.gated_scan_recurrent_fwd(s["x"], s["a"], s["h"], **form), s["h"]
        form = {"scale": s["scale"], "kind": s["kind"]}
        if op == "add_norm_fwd":
            return gdr.add_norm_fwd(s["x"], s["residual"], s["weight"], s["bias"], eps=EPS, **form)
        if op == "add_norm_bwd":
            return gdr.add_norm_bwd(s["dy"], s["x"], s["rstd"], s["mean"], dr=s.get("dr"), weight=s["weight"],
                                    want_dbias=s["bias"] is not None, **form)
        if op == "norm_gate_fwd":
            return gdr.norm_gate_fwd(s["x"], s["z"], s["weight"], s["bias"], residual=s.get("residual"), act=s["act"],
                                     eps=EPS, **form)
        return gdr.norm_gate_bwd(s["dy"], s["x"], s["z"], s["rstd"], s["mean"], weight=s["weight"], bias=s["bias"],
                                 act=s["act"], want_dbias=s["bias"] is not None, **form)
    if op == "scan_fwd":
        out, hT, states = _plain_scan_fwd(s)
        return out, hT, states if s["kept"] else None
    if op == "scan_bwd":
        return _plain_scan_bwd(s)
    if op == "scan_step":
        return _plain_scan_step(s)
    return _plain_norm_fwd(s) if op.endswith("fwd") else _plain_norm_bwd(s)


# ---- what a pass cannot do without -----------------------------------------------------
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if not op.startswith("scan"):
        n, wb = case["rows"] * case["D"], 4 * case["groups"] * case["D"]
        layer = case["kind"] == "layer"
        stats, affine = 4 * case["rows"] * (2 if layer else 1), wb * (2 if layer else 1)
        if op == "add_norm_fwd":     # x, residual -> y, r
            return {"bytes": 4 * n * es + stats + affine, "flops": 8 * n}
        if op == "add_norm_bwd":     # dy, r, (dr) -> dx, dresidual
            return {"bytes": (5 if case["extra"] else 4) * n * es + stats + 2 * affine, "flops": 13 * n}
        if op == "norm_gate_fwd":    # x, z, (residual) -> y
            return {"bytes": (4 if case["extra"] else 3) * n * es + stats + affine, "flops": 12 * n}
        return {"bytes": 5 * n * es + stats + 2 * affine, "flops": 26 * n}   # dy, x, z -> dx, dz
    n, D = case["B"] * case["T"] * case["D"], case["D"]
    states = 4 * (case["B"] * case["T"] // EVERY) * D if case["kept"] else 0
    st = 4 * (case["packed"] or case["B"]) * D
    if op == "scan_bwd":             # x, a, dout -> dx, da
        return {"bytes": 5 * n * es + states + st * (3 if case["state"] else 1), "flops": 30 * n}
    return {"bytes": 3 * n * es + states + st * (2 if case["state"] else 1), "flops": 12 * n}


# ---- the definition in 64 bits -----------------------------------------------------------
def _padded(x, lens):
    """[1, total, D] in packed order -> [longest, N, D] in fp64, zero past each end."""
    x = x.double().flatten(0, 1)
    return torch.nn.utils.rnn.pad_sequence(list(torch.split(x, lens)))


def _unpadded(x, lens, shape):
    return torch.cat([x[:m, n] for n, m in enumerate(lens)]).reshape(shape)


def _exact_scan(case, s, lens):
    x, a = _padded(s["x"], lens), _padded(s["a"], lens)
    T, N, D = x.shape
    left = torch.tensor(lens, device=x.device)[:, None]
    sig = 1.0 / (1.0 + torch.exp(-a))
    if case["gate"] == "bounded":
        alpha, dg = torch.exp(-case["b"] * sig), -case["b"] * sig * (1.0 - sig)
    else:
        alpha, dg = 1.0 / (1.0 + torch.exp(a)), -sig   # exp(-log(1 + e^a))
    w = {"plain": lambda: torch.ones_like(alpha), "convex": lambda: 1.0 - alpha,
         "variance": lambda: ((1.0 - alpha) * (1.0 + alpha)).sqrt()}[case["source"]]()
    h = s["h"] if case["op"] == "scan_step" else s["h0"]
    h = torch.zeros((N, D), dtype=torch.float64, device=x.device) if h is None else h.double()
    u, states = w * x, torch.empty((T + 1, N, D), dtype=torch.float64, device=x.device)
    states[0] = h
    ragged = min(lens) < T
    for t in range(T):   # a sequence past its end keeps its state
        torch.addcmul(u[t], alpha[t], states[t], out=states[t + 1])
        if ragged:
            states[t + 1] = torch.where(left > t, states[t + 1], states[t])
    after, h = states[1:], states[T]
    if case["op"] == "scan_step":
        return _unpadded(after, lens, s["x"].shape), h
    if case["op"] == "scan_fwd":
        out = _unpadded(after, lens, s["x"].shape)
        return out, h, out.flatten(0, 1)[EVERY - 1::EVERY] if case["kept"] else None
    dout = _padded(s["dout"], lens)
    r = torch.zeros_like(h) if s["dhT"] is None else s["dhT"].double()   # the gradient of h_{t-1}, of hT at first
    lam = torch.zeros_like(x)
    for t in reversed(range(T)):
        live = left > t
        lam[t] = torch.where(live, dout[t] + r, 0.0)
        r = torch.where(live, alpha[t] * lam[t], r)
    if case["source"] == "plain":
        dwx = 0.0
    elif case["source"] == "convex":
        dwx = -alpha * x
    else:
        dwx = -alpha.square() * x / w
    da = lam * (alpha * states[:-1] + dwx) * dg
    return _unpadded(w * lam, lens, s["x"].shape), _unpadded(da, lens, s["x"].shape), r


def _exact_norm(case, s):
    x, w = s["x"].double(), s["weight"].double()
    b = 0.0 if s["bias"] is None else s["bias"].double()
    layer, scale = case["kind"] == "layer", case["scale"]
    if "norm_gate" in case["op"]:
        z = s["z"].double()
        sig = 1.0 / (1.0 + torch.exp(-z))
        act, dact = (sig, sig * (1 - sig)) if case["act"] == "sigmoid" else (z * sig, sig + z * sig * (1 - sig))
    if case["op"].endswith("fwd"):
        r = None
        if case["op"] == "add_norm_fwd":
            r = s["residual"].double() + scale * x
            x = r.to(s["x"].dtype).double()   # the norm is that of the stream as it is stored
        mean = torch.mean(x, -1, keepdim=True) if layer else torch.zeros_like(x[..., :1])
        rstd = ((x - mean).square().mean(-1, keepdim=True) + EPS) ** -0.5
        y = (x - mean) * rstd * w + b
        stats = (mean.squeeze(-1) if layer else None, rstd.squeeze(-1))
        if r is not None:
            return (y, r) + stats
        y = scale * y * act
        return (y + s["residual"].double() if case["extra"] else y,) + stats
    dy, rstd = s["dy"].double(), s["rstd"].double()[..., None]
    xh = ((x - s["mean"].double()[..., None]) if layer else x) * rstd
    first = ()
    if case["op"] == "norm_gate_bwd":
        first = (scale * dy * (xh * w + b) * dact,)
        dy = scale * dy * act
    D = x.shape[-1]
    n = dy * w
    d = rstd * (n - xh * ((n * xh).sum(-1, keepdim=True) / D) - (n.sum(-1, keepdim=True) / D if layer else 0.0))
    sums = (torch.sum(dy * xh, 0), torch.sum(dy, 0) if layer else None)
    if case["op"] == "norm_gate_bwd":
        return (d,) + first + sums
    if case["extra"]:
        d = d + s["dr"].double()
    return (scale * d, d) + sums


def exact(case, seed):
    s = prepare(case, seed)
    if not case["op"].startswith("scan"):
        return _exact_norm(case, s)
    lens = _lengths(case, seed) if case["packed"] else np.full(case["B"], case["T"])
    lens = [int(n) for n in lens]
    if len(lens) * max(lens) * case["D"] > 1 << 30:
        return None   # the padded tensors in 64 bits would take the card's memory
    if not case["packed"]:
        s["x"], s["a"] = s["x"].reshape(1, -1, case["D"]), s["a"].reshape(1, -1, case["D"])
        out = _exact_scan(case, s, lens)
        whole = (case["B"], case["T"], case["D"])
        return tuple(v.reshape(whole) if v is not None and v.dim() == 3 else v for v in out)
    return _exact_scan(case, s, lens)
