"""The gated scan, its gradients and its gates from their definitions, in 64 bits on the CPU."""
import torch


def gates(a, b, gate, source):
    """alpha, w, dw/dg, dg/da of a (float64)."""
    sig = torch.sigmoid(a)
    if gate == "bounded":
        g, slope = -b * sig, -b * sig * torch.sigmoid(-a)
    else:
        g, slope = -torch.nn.functional.softplus(a, threshold=1e9), -sig
    alpha, left = torch.exp(g), -torch.expm1(g)
    if source == "plain":
        return alpha, torch.ones_like(a), torch.zeros_like(a), slope
    if source == "convex":
        return alpha, left, -alpha, slope
    w = (left * (1 + alpha)).sqrt()
    return alpha, w, -alpha * alpha / w, slope


def pieces(x, lens):
    """The sequences' slices of a token axis."""
    at, out = 0, []
    for n in lens:
        out.append(x[at:at + n])
        at += n
    return out


def forward(x, a, h0, lens, b, gate, source):
    """x, a [total, D]; h0 [N, D] or None.  Returns (h [total, D], hT [N, D])."""
    x, a = x.double().cpu(), a.double().cpu()
    alpha, w, _, _ = gates(a, b, gate, source)
    out, hT, at = torch.empty_like(x), torch.zeros(len(lens), x.shape[1], dtype=torch.float64), 0
    for n, m in enumerate(lens):
        h = torch.zeros(x.shape[1], dtype=torch.float64) if h0 is None else h0[n].double().cpu()
        for t in range(at, at + m):
            h = alpha[t] * h + w[t] * x[t]
            out[t] = h
        hT[n] = h
        at += m
    return out, hT


def backward(x, a, h0, dout, dhT, lens, b, gate, source):
    """Returns (dx, da, dh0)."""
    out, _ = forward(x, a, h0, lens, b, gate, source)
    x, a, dout = x.double().cpu(), a.double().cpu(), dout.double().cpu()
    alpha, w, dw, slope = gates(a, b, gate, source)
    dx, da, dh0, at = torch.empty_like(x), torch.empty_like(x), torch.zeros(len(lens), x.shape[1], dtype=torch.float64), 0
    for n, m in enumerate(lens):
        r = torch.zeros(x.shape[1], dtype=torch.float64) if dhT is None else dhT[n].double().cpu()
        for t in reversed(range(at, at + m)):
            before = out[t - 1] if t > at else torch.zeros_like(r) if h0 is None else h0[n].double().cpu()
            lam = dout[t] + r
            dx[t] = w[t] * lam
            da[t] = lam * (alpha[t] * before + dw[t] * x[t]) * slope[t]
            r = alpha[t] * lam
        dh0[n] = r
        at += m
    return dx, da, dh0
