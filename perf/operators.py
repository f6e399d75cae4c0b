"""Cases of the decay linear attention and layer norm operators, with their plain forms.

Decay linear attention, one log-decay g_h <= 0 per head, per (sequence, head):

    S_t = exp(g_h) S_{t-1} + k_t v_t^T,    o_t = scale * S_t^T q_t

over a prompt (decay_fwd), its gradients (decay_bwd), and token by token with the state
updated in place (decay_step).  Layer norm over the last axis, with one weight and bias
for all rows or one per group of rows (per head), forward and backward.

`run` computes a case in its plain form (elementary torch operations in 32 bits) where
`own` is false and by the library's calls where it is true.
"""
import math

import numpy as np
import torch

own = False   # set from outside: False for the plain forms, True for the library's calls

CHUNK = 128   # tokens per block of the plain chunked form
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases ------------------------------------------------------------------------
def _decay(name, op, B, T, H, dk, dv, dtype, packed=0, state=True):
    return {"name": name, "op": op, "B": B, "T": T, "H": H, "dk": dk, "dv": dv, "dtype": dtype,
            "packed": packed, "state": state}


def _norm(name, op, rows, groups, D, dtype):
    return {"name": name, "op": op, "rows": rows, "groups": groups, "D": D, "dtype": dtype}


def listed():
    return [
        # the next piece of a chat's prompt, with the state carried in: latency counts
        _decay("prompt_33", "decay_fwd", 1, 33, 16, 128, 128, "bf16"),
        # one layer's forward pass of a training step: 8 sequences of 4096 tokens
        _decay("train_8x4096", "decay_fwd", 8, 4096, 16, 128, 128, "bf16", state=False),
        # a long document, one sequence: 16 heads are all the parallelism it has by itself
        _decay("document_256k", "decay_fwd", 1, 262144, 16, 128, 128, "bf16"),
        # a serving engine's batch of prompts of unequal lengths, narrow heads
        _decay("prompts_packed_64k", "decay_fwd", 1, 65536, 32, 64, 64, "bf16", packed=37),
        # the same training step's backward pass
        _decay("grad_8x4096", "decay_bwd", 8, 4096, 16, 128, 128, "bf16", state=False),
        # a small run in fp32 on packed sequences with initial states and their gradients
        _decay("grad_packed_f32", "decay_bwd", 1, 5003, 2, 64, 64, "f32", packed=7),
        # one token of one conversation
        _decay("step_1", "decay_step", 1, 1, 16, 128, 128, "bf16"),
        # one token of each of 256 conversations served together
        _decay("step_256", "decay_step", 256, 1, 16, 128, 128, "bf16"),
        # the norm of every head's output after the attention of the training step
        _norm("norm_heads", "norm_fwd", 8 * 4096 * 16, 16, 128, "bf16"),
        # a few tokens' rows, an odd width, fp32
        _norm("norm_small", "norm_fwd", 7, 1, 1000, "f32"),
        # the backward pass of the norm of every head's output
        _norm("norm_grad_heads", "norm_bwd", 8 * 4096 * 16, 16, 128, "bf16"),
        # the backward pass of the norm in front of a layer 16 x 128 wide, ragged row count
        _norm("norm_grad_wide", "norm_bwd", 8191, 1, 2048, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decay_fwd", "decay_fwd", "decay_bwd", "decay_bwd", "decay_step", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        D = _log_int(rng, 8, 8192)
        groups = rng.choice([1, 1, 3, 16]) if D <= 256 else 1
        rows = _log_int(rng, 1, max(1, min(1 << 19, (1 << 25) // D) // groups)) * groups
        return {k: v for k, v in _norm("", op, rows, groups, D, dtype).items() if k != "name"}
    H = rng.choice([1, 2, 5, 16, 32])
    dk, dv = rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
    if op == "decay_step":
        B, T, packed, state = _log_int(rng, 1, 256), rng.choice([1, 1, 1, 2, 4]), 0, True
    else:
        most = (1 << 19 if dtype == "bf16" else 1 << 16) // H   # tokens over all sequences
        total = _log_int(rng, 1, most)
        packed = rng.choice([0, 0, _log_int(rng, 1, 64)])
        B = 1 if packed else _log_int(rng, 1, max(1, min(16, total)))
        T, state = max(1, total // B), rng.choice([True, False])
    return {k: v for k, v in _decay("", op, B, T, H, dk, dv, dtype, packed, state).items() if k != "name"}


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

    s = {"op": case["op"]}
    if case["op"].startswith("norm"):
        rows, G, D = case["rows"], case["groups"], case["D"]
        shape = (rows // G, G, D) if G > 1 else (rows, D)
        x = (normal(*shape) * 1.5 + 0.3).to(dt)
        s.update(x=x, weight=1.0 + normal(*shape[len(shape) - (2 if G > 1 else 1):], std=0.2))
        s["bias"] = normal(*s["weight"].shape, std=0.1)
        if case["op"] == "norm_bwd":
            s["dy"] = normal(*shape).to(dt)
            xf = x.float()   # the statistics that the forward pass saved
            s["mean"] = xf.mean(-1)
            s["rstd"] = torch.rsqrt((xf - s["mean"][..., None]).square().mean(-1) + EPS)
        return s
    B, T, H, dk, dv = (case[n] for n in ("B", "T", "H", "dk", "dv"))
    N = case["packed"] or B
    # unit-norm q and k, as after the layer's key normalisation
    s["q"] = torch.nn.functional.normalize(normal(B, T, H, dk), dim=-1).to(dt)
    s["k"] = torch.nn.functional.normalize(normal(B, T, H, dk), dim=-1).to(dt)
    s["v"] = normal(B, T, H, dv).to(dt)
    # one decay per head, geometric from half a token's to some hundred tokens' memory
    slope = 2.0 ** (-8.0 * (torch.arange(H, device="cuda") + 1) / H)
    s["log_decay"] = -slope * (0.8 + 0.4 * torch.rand(H, generator=gen, device="cuda"))
    s["scale"] = 0.5
    if case["op"] == "decay_step":
        s["state"] = normal(N, H, dk, dv, std=0.5)
        return s
    s["h0"] = normal(N, H, dk, dv, std=0.5) if case["state"] else None
    s["cu"] = None
    if case["packed"]:
        ends = np.concatenate([[0], np.cumsum(_lengths(case, seed))])
        s["cu"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    if case["op"] == "decay_bwd":
        s["dout"] = normal(B, T, H, dv).to(dt)
        s["dhT"] = normal(N, H, dk, dv, std=0.5) if case["state"] else None
    return s


# ---- the plain forms --------------------------------------------------------------------
class _Blocks:
    """The packed tokens in blocks of CHUNK that restart at every sequence start."""

    def __init__(self, cu, total, N, device):
        lens = (cu[1:] - cu[:-1]).long()
        last = torch.cumsum((lens + CHUNK - 1) // CHUNK, 0)      # blocks up to each sequence's end
        self.nc = total // CHUNK + N                             # an upper bound: no look at the values
        c = torch.arange(self.nc, device=device)
        used = c < last[-1]
        self.seq = torch.searchsorted(last, c, right=True).clamp(max=N - 1)
        first = last[self.seq] - (lens[self.seq] + CHUNK - 1) // CHUNK
        self.start = torch.where(used, (c - first) * CHUNK, 0)   # within the sequence
        self.len = torch.where(used, (lens[self.seq] - self.start).clamp(0, CHUNK), 0)
        self.end = self.start + self.len
        self.seq_len = lens
        self.pos = torch.arange(CHUNK, device=device)
        self.ok = self.pos[None, :] < self.len[:, None]
        self.at = torch.where(self.ok, cu[:-1].long()[self.seq][:, None] + self.start[:, None] + self.pos, total)
        # reversed order: token i of a block is the sequence's (start + i)-th from its end
        back = cu[1:].long()[self.seq][:, None] - 1 - self.start[:, None] - self.pos
        self.at_back = torch.where(self.ok, back, total)
        self.total, self.N = total, N

    def take(self, x, at):
        """[tokens, H, d] -> [H, blocks, CHUNK, d] in fp32, zero past a block's end."""
        x = torch.cat([x.float(), x.new_zeros((1,) + x.shape[1:], dtype=torch.float32)])
        return x[at].permute(2, 0, 1, 3)

    def put(self, y, at):
        """The inverse of take: [H, blocks, CHUNK, d] -> [tokens, H, d]."""
        out = y.new_empty((self.total + 1, y.shape[0], y.shape[-1]))
        out[at] = y.permute(1, 2, 0, 3)
        return out[:-1]


def _plain_pass(b, q, k, v, g, s0, at):
    """o_t = S_t^T q_t and the last S, S_t = e^g S_{t-1} + k_t v_t^T, tokens in the order of `at`."""
    q, k, v = b.take(q, at), b.take(k, at), b.take(v, at)
    gh = g.float()[:, None, None]
    n = b.pos[:, None] - b.pos[None, :]
    mask = torch.exp(gh * n.clamp(min=0)) * (n >= 0)                              # [H, C, C]
    out = ((q @ k.transpose(-1, -2)) * mask[:, None]) @ v
    left = (b.len[:, None] - 1 - b.pos).clamp(min=0)
    kv = (k * (torch.exp(gh * left) * b.ok)[..., None]).transpose(-1, -2) @ v     # [H, nc, dk, dv]
    H, nc, dk, dv = kv.shape
    kv = kv.reshape(H, nc, dk * dv)
    gap = b.start[:, None] - b.end[None, :]
    before = (b.seq[:, None] == b.seq[None, :]) & (gap >= 0) & (b.len[None, :] > 0)
    s_in = (torch.exp(gh * gap.clamp(min=0)) * before) @ kv                       # [H, nc, dk dv]
    rest = b.seq_len[:, None] - b.end[None, :]
    mine = torch.arange(b.N, device=g.device)[:, None] == b.seq[None, :]
    s_T = (torch.exp(gh * rest.clamp(min=0)) * (mine & (b.len > 0))) @ kv         # [H, N, dk dv]
    if s0 is not None:
        s0 = s0.transpose(0, 1).reshape(H, b.N, dk * dv)
        s_in = s_in + torch.exp(gh * b.start[None, :, None]) * s0[:, b.seq]
        s_T = s_T + torch.exp(gh * b.seq_len[None, :, None]) * s0
    s_in = s_in.reshape(H, nc, dk, dv)
    out = out + torch.exp(gh * (b.pos + 1)[None, None, :])[..., None] * (q @ s_in)
    return b.put(out, at), s_T.reshape(H, b.N, dk, dv).transpose(0, 1)


def _blocks_of(s):
    B, T = s["q"].shape[:2]
    cu = s.get("cu")
    N = B if cu is None else cu.numel() - 1
    if cu is None:
        cu = torch.arange(B + 1, device=s["q"].device) * T
    return _Blocks(cu, B * T, N, s["q"].device)


def _plain_decay_fwd(s, h0):
    q, v = s["q"], s["v"]
    b = _blocks_of(s)
    out, hT = _plain_pass(b, q.flatten(0, 1), s["k"].flatten(0, 1), v.flatten(0, 1), s["log_decay"], h0, b.at)
    return (out * s["scale"]).reshape(v.shape).to(q.dtype), hT


def _plain_decay_bwd(s):
    """With dS_t the gradient of S_t: dq = scale S do, dS_t = e^g dS_{t+1} + scale q_t do_t^T,
    dk = dS v, dv = dS^T k, dh0 = e^g dS_1; the last token's dS holds dhT too."""
    b = _blocks_of(s)
    q, k, v, do = (s[n].flatten(0, 1) for n in ("q", "k", "v", "dout"))
    g, scale, h0, dhT = s["log_decay"], s["scale"], s["h0"], s["dhT"]
    dq, _ = _plain_pass(b, do, v, k, g, None if h0 is None else h0.transpose(-1, -2), b.at)
    dk, _ = _plain_pass(b, v, do, q, g, None, b.at_back)
    dv, dS = _plain_pass(b, k, q, do, g, None, b.at_back)
    dq, dk, dv = dq * scale, dk * scale, dv * scale
    gh = g.float()[None, :, None, None]
    dh0 = torch.exp(gh) * scale * dS
    if dhT is not None:
        w = torch.exp(g.float()[:, None, None] * (b.start[:, None] + b.pos))[..., None]   # [H, nc, C, 1]
        d = dhT[b.seq].transpose(0, 1)                                                    # [H, nc, dk, dv]
        dk = dk + b.put((w * b.take(v, b.at_back)) @ d.transpose(-1, -2), b.at_back)
        dv = dv + b.put((w * b.take(k, b.at_back)) @ d, b.at_back)
        dh0 = dh0 + torch.exp(gh * b.seq_len[:, None, None, None]) * dhT
    dt = s["q"].dtype
    return (dq.reshape(s["q"].shape).to(dt), dk.reshape(s["k"].shape).to(dt),
            dv.reshape(s["v"].shape).to(dt), dh0)


def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(-1)
    rstd = torch.rsqrt((x - mean[..., None]).square().mean(-1) + EPS)
    y = (x - mean[..., None]) * rstd[..., None] * s["weight"] + s["bias"]
    return y.to(s["x"].dtype), mean, rstd


def _plain_norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    xh = (x - s["mean"][..., None]) * s["rstd"][..., None]
    wdy = dy * s["weight"]
    dx = (wdy - wdy.mean(-1, keepdim=True) - xh * (wdy * xh).mean(-1, keepdim=True)) * s["rstd"][..., None]
    return dx.to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0)


def run(s):
    op = s["op"]
    if own:
        import chunked_gated_delta_07_gb300 as gdr
        if op == "decay_fwd":
            return gdr.decay_fwd(s["q"], s["k"], s["v"], s["log_decay"], h0=s["h0"], cu_seqlens=s["cu"],
                                 scale=s["scale"])
        if op == "decay_bwd":
            return gdr.decay_bwd(s["q"], s["k"], s["v"], s["log_decay"], dout=s["dout"], dhT=s["dhT"],
                                 h0=s["h0"], cu_seqlens=s["cu"], scale=s["scale"])
        if op == "decay_step":
            out = gdr.decay_recurrent_fwd(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=s["scale"])
            return out, s["state"]
        if op == "norm_fwd":
            return gdr.layer_norm_fwd(s["x"], s["weight"], s["bias"], eps=EPS)
        return gdr.layer_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
    if op == "decay_fwd":
        return _plain_decay_fwd(s, s["h0"])
    if op == "decay_bwd":
        return _plain_decay_bwd(s)
    if op == "decay_step":
        if s["q"].shape[1] > 1:
            out, state = _plain_decay_fwd(s, s["state"])
            s["state"].copy_(state)
            return out, s["state"]
        q, k, v = (s[n][:, 0].float() for n in ("q", "k", "v"))
        s["state"].mul_(torch.exp(s["log_decay"])[None, :, None, None])
        s["state"].add_(k[..., :, None] * v[..., None, :])
        out = s["scale"] * (q[..., None, :] @ s["state"]).squeeze(-2)
        return out[:, None].to(s["q"].dtype), s["state"]
    return _plain_norm_fwd(s) if op == "norm_fwd" else _plain_norm_bwd(s)


# ---- what a pass cannot do without -----------------------------------------------------
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        n, rows, wb = case["rows"] * case["D"], case["rows"], 4 * case["groups"] * case["D"]
        if case["op"] == "norm_fwd":   # x -> y, the statistics; weight and bias
            return {"bytes": 2 * n * es + 8 * rows + 2 * wb, "flops": 8 * n}
        return {"bytes": 3 * n * es + 8 * rows + 3 * wb, "flops": 14 * n}
    B, T, H, dk, dv = (case[n] for n in ("B", "T", "H", "dk", "dv"))
    N = case["packed"] or B
    rows, state = B * T * H, 4 * N * H * dk * dv
    if case["op"] == "decay_bwd":   # q, k, v, dout -> dq, dk, dv, dh0; two states, three products with them
        return {"bytes": rows * (4 * dk + 3 * dv) * es + state * (3 if case["state"] else 1),
                "flops": 10 * rows * dk * dv}
    return {"bytes": rows * (2 * dk + 2 * dv) * es + state * (2 if case["state"] else 1),
            "flops": 4 * rows * dk * dv}


# ---- the definition in 64 bits -----------------------------------------------------------
def _padded(x, lens):
    """[1, total, ...] in packed order -> [N, longest, ...] in fp64, zero past each end."""
    x = x.double().flatten(0, 1)
    return torch.nn.utils.rnn.pad_sequence(list(torch.split(x, list(lens))), batch_first=True)


def _unpadded(x, lens, shape):
    return torch.cat([x[n, :m] for n, m in enumerate(lens)]).reshape(shape)


def exact(case, seed):
    if case["op"].startswith("decay") and case["T"] > 100000:
        return None   # token by token: too long
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        x, w = s["x"].double(), s["weight"].double()
        if case["op"] == "norm_fwd":
            var, mean = torch.var_mean(x, -1, correction=0)
            rstd = 1.0 / torch.sqrt(var + EPS)
            return (x - mean[..., None]) * rstd[..., None] * w + s["bias"].double(), mean, rstd
        dy, mean, rstd = s["dy"].double(), s["mean"].double()[..., None], s["rstd"].double()[..., None]
        xh, D = (x - mean) * rstd, x.shape[-1]
        a, c = (w * dy).sum(-1, keepdim=True) / D, (w * dy * xh).sum(-1, keepdim=True) / D
        return rstd * (w * dy - a - c * xh), torch.sum(dy * xh, 0), torch.sum(dy, 0)
    lens = _lengths(case, seed) if case["packed"] else np.full(case["B"], case["T"])
    lens = [int(n) for n in lens]
    q, k, v = (_padded(s[n], lens) for n in ("q", "k", "v"))
    N, T, H, dk = q.shape
    dv, scale = v.shape[-1], s["scale"]
    left = torch.tensor(lens, device=q.device)
    lam = torch.exp(s["log_decay"].double())[None, :, None, None]
    h = s.get("h0") if case["op"] != "decay_step" else s["state"]
    S = torch.zeros((N, H, dk, dv), dtype=torch.float64, device=q.device) if h is None else h.double()
    if case["op"] != "decay_bwd":
        out = torch.zeros_like(v)
        for t in range(T):   # k is zero past a sequence's end, where the state stays
            live = (left > t)[:, None, None, None]
            S = torch.where(live, lam * S, S) + k[:, t, :, :, None] * v[:, t, :, None, :]
            out[:, t] = scale * (q[:, t, :, None, :] @ S).squeeze(-2)
        return _unpadded(out, lens, s["v"].shape), S
    do = _padded(s["dout"], lens)
    dq, dk_, dv_ = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for t in range(T):
        S = lam * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        dq[:, t] = scale * (S @ do[:, t, :, :, None]).squeeze(-1)
    dS = torch.zeros_like(S) if s["dhT"] is None else s["dhT"].double()
    for t in reversed(range(T)):   # dS holds e^g dS_{t+1} here (dhT at a sequence's last token)
        live = (left > t)[:, None, None, None]
        now = dS + scale * q[:, t, :, :, None] * do[:, t, :, None, :]
        dk_[:, t] = (now @ v[:, t, :, :, None]).squeeze(-1)
        dv_[:, t] = (k[:, t, :, None, :] @ now).squeeze(-2)
        dS = torch.where(live, lam * now, dS)
    return (_unpadded(dq, lens, s["q"].shape), _unpadded(dk_, lens, s["k"].shape),
            _unpadded(dv_, lens, s["v"].shape), dS)
