"""The decay linear attention and layer norm of the operator tests in 64 bits, from their
definitions: token by token in numpy, nothing shared with the library."""
from __future__ import annotations

import numpy as np


def np64(t):
    return t.detach().cpu().double().numpy()


def bounds_of(q, cu):
    """(sequence, start, end) of every sequence, as rows of the flattened token axis."""
    B, T = q.shape[:2]
    if cu is None:
        return [(n, n * T, (n + 1) * T) for n in range(B)]
    c = [int(x) for x in cu]
    return [(n, c[n], c[n + 1]) for n in range(len(c) - 1)]


def decay_fwd(q, k, v, g, h0=None, cu=None, scale=1.0):
    """out (v's shape) and hT [N, H, dk, dv] in fp64."""
    seqs = bounds_of(q, cu)
    qf, kf, vf = (np64(x).reshape(-1, *x.shape[2:]) for x in (q, k, v))
    lam = np.exp(np64(g))[:, None, None]
    H, dk, dv = qf.shape[1], qf.shape[2], vf.shape[2]
    out, hT = np.zeros_like(vf), np.zeros((len(seqs), H, dk, dv))
    for n, a, b in seqs:
        S = np.zeros((H, dk, dv)) if h0 is None else np64(h0[n])
        for t in range(a, b):
            S = lam * S + kf[t][:, :, None] * vf[t][:, None, :]
            out[t] = scale * np.einsum("hd,hde->he", qf[t], S)
        hT[n] = S
    return out.reshape(v.shape), hT


def decay_bwd(q, k, v, g, dout, dhT=None, h0=None, cu=None, scale=1.0):
    """dq, dk, dv, dh0 of <dout, out> + <dhT, hT> in fp64."""
    seqs = bounds_of(q, cu)
    qf, kf, vf, of = (np64(x).reshape(-1, *x.shape[2:]) for x in (q, k, v, dout))
    lam = np.exp(np64(g))[:, None, None]
    H, dk, dv = qf.shape[1], qf.shape[2], vf.shape[2]
    dq, dkk, dvv, dh0 = np.zeros_like(qf), np.zeros_like(kf), np.zeros_like(vf), np.zeros((len(seqs), H, dk, dv))
    for n, a, b in seqs:
        S = np.zeros((H, dk, dv)) if h0 is None else np64(h0[n])
        for t in range(a, b):
            S = lam * S + kf[t][:, :, None] * vf[t][:, None, :]
            dq[t] = scale * np.einsum("hde,he->hd", S, of[t])
        E = np.zeros((H, dk, dv)) if dhT is None else np64(dhT[n])
        for t in range(b - 1, a - 1, -1):
            R = E + scale * qf[t][:, :, None] * of[t][:, None, :]
            dkk[t] = np.einsum("hde,he->hd", R, vf[t])
            dvv[t] = np.einsum("hde,hd->he", R, kf[t])
            E = lam * R
        dh0[n] = E
    return dq.reshape(q.shape), dkk.reshape(k.shape), dvv.reshape(v.shape), dh0


def norm_fwd(x, w=None, b=None, eps=1e-5):
    x = np64(x)
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    if w is not None:
        y = y * np64(w)
    if b is not None:
        y = y + np64(b)
    return y, mean, rstd


def norm_bwd(dy, x, mean, rstd, w=None, per_head=False):
    dy, x = np64(dy), np64(x)
    mean, rstd = np64(mean)[..., None], np64(rstd)[..., None]
    xh = (x - mean) * rstd
    wdy = dy if w is None else dy * np64(w)
    dx = rstd * (wdy - wdy.mean(-1, keepdims=True) - xh * (wdy * xh).mean(-1, keepdims=True))
    keep = 2 if per_head or (w is not None and w.dim() == 2) else 1
    axes = tuple(range(x.ndim - keep))
    return dx, (dy * xh).sum(axes), dy.sum(axes)


def rel(x, ref):
    """2-norm of the difference over the 2-norm of the result."""
    x = np64(x) if hasattr(x, "detach") else np.asarray(x, np.float64)
    d, n = np.linalg.norm(x - ref), np.linalg.norm(ref)
    return d / n if n > 0 else d
