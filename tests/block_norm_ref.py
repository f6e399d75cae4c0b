"""The norms around a block and their gradients from their definitions, in 64 bits."""
import torch


def act(z, name):
    """act(z) and its derivative."""
    g = torch.sigmoid(z)
    return (g, g * (1 - g)) if name == "sigmoid" else (z * g, g * (1 + z * (1 - g)))


def stats(x, kind, eps):
    mean = x.mean(-1) if kind == "layer" else torch.zeros_like(x[..., 0])
    return mean, ((x - mean[..., None]).square().mean(-1) + eps) ** -0.5


def norm(x, w, b, kind, eps):
    mean, rstd = stats(x, kind, eps)
    y = (x - mean[..., None]) * rstd[..., None]
    y = y if w is None else y * w
    return y if b is None else y + b


def gate(x, z, w, b, res, scale, kind, name, eps):
    y = scale * norm(x, w, b, kind, eps) * act(z, name)[0]
    return y if res is None else y + res


def sums(t, like):
    return t.reshape(-1, *like).sum(0)


def norm_back(dn, x, mean, rstd, w, kind):
    """dx, xh of the norm's statistics; dn is the gradient of N's output."""
    xh = (x - mean[..., None]) * rstd[..., None]
    n = dn if w is None else dn * w
    d = n - xh * (n * xh).mean(-1, keepdim=True)
    if kind == "layer":
        d = d - n.mean(-1, keepdim=True)
    return d * rstd[..., None], xh


def add_back(dy, dr, r, mean, rstd, w, scale, kind, like):
    d, xh = norm_back(dy, r, mean, rstd, w, kind)
    d = d if dr is None else d + dr
    return scale * d, d, sums(dy * xh, like), sums(dy, like)


def gate_back(dy, x, z, mean, rstd, w, b, scale, kind, name, like):
    xh = (x - mean[..., None]) * rstd[..., None]
    n = xh if w is None else xh * w
    n = n if b is None else n + b
    a, slope = act(z, name)
    dn = scale * dy * a
    return norm_back(dn, x, mean, rstd, w, kind)[0], scale * dy * n * slope, sums(dn * xh, like), sums(dn, like)
