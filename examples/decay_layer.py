"""One layer built from the decay linear attention and the layer norm, trained and served.

    x -> norm -> q, k, v projections -> decay attention -> norm of every head -> projection -> + x

The attention S_t = exp(g_h) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t has no normaliser: its
outputs grow with a head's memory, so each head's output is normed with its own weight.  The
layer trains with the chunked forward and backward passes, reads a prompt with the chunked
forward pass, which leaves the state, and continues token by token on that state.

    python examples/decay_layer.py        # a short training run, then a prompt and single tokens
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_gated_delta_07_gb300 as gdr  # noqa: E402


class DecayAttention(torch.autograd.Function):
    """out of gdr.decay_fwd; q, k [B,T,H,dk], v [B,T,H,dv], log_decay [H] (a constant)."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, cu_seqlens, scale):
        out, _ = gdr.decay_fwd(q, k, v, log_decay, cu_seqlens=cu_seqlens, scale=scale, want_state=False)
        ctx.save_for_backward(q, k, v, log_decay)
        ctx.cu_seqlens, ctx.scale = cu_seqlens, scale
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, log_decay = ctx.saved_tensors
        dq, dk, dv, _ = gdr.decay_bwd(q, k, v, log_decay, dout.contiguous(), cu_seqlens=ctx.cu_seqlens,
                                      scale=ctx.scale, want_dh0=False)
        return dq, dk, dv, None, None, None


class LayerNorm(torch.autograd.Function):
    """y of gdr.layer_norm_fwd; weight and bias fp32, [D] or [G, D] (one per head)."""

    @staticmethod
    def forward(ctx, x, weight, bias):
        y, mean, rstd = gdr.layer_norm_fwd(x, weight, bias)
        ctx.save_for_backward(x, mean, rstd, weight)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, mean, rstd, weight = ctx.saved_tensors
        return gdr.layer_norm_bwd(dy.contiguous(), x, mean, rstd, weight)


class DecayLayer(torch.nn.Module):
    def __init__(self, width=512, heads=4, head_dim=128, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.heads, self.head_dim, self.scale = heads, head_dim, head_dim ** -0.5
        inner = heads * head_dim
        lin = lambda i, o: torch.nn.Parameter(torch.randn(i, o, device=device, dtype=dtype) * i ** -0.5)  # noqa: E731
        self.w_q, self.w_k, self.w_v, self.w_o = lin(width, inner), lin(width, inner), lin(width, inner), lin(inner, width)
        vec = lambda f, *s: torch.nn.Parameter(f(*s, device=device, dtype=torch.float32))  # noqa: E731
        self.norm_w, self.norm_b = vec(torch.ones, width), vec(torch.zeros, width)
        self.head_w, self.head_b = vec(torch.ones, heads, head_dim), vec(torch.zeros, heads, head_dim)
        # from half a token's memory to some hundred tokens'
        slope = 2.0 ** (-8.0 * (torch.arange(heads, device=device) + 1) / heads)
        self.register_buffer("log_decay", -slope)

    def _qkv(self, x):
        y = LayerNorm.apply(x, self.norm_w, self.norm_b)
        shape = (*x.shape[:2], self.heads, self.head_dim)
        return tuple((y @ w).view(shape) for w in (self.w_q, self.w_k, self.w_v))

    def _out(self, x, o):
        o = LayerNorm.apply(o, self.head_w, self.head_b)
        return x + o.reshape(*x.shape[:2], -1) @ self.w_o

    def forward(self, x, cu_seqlens=None):
        """Training: x [B, T, width], or packed sequences [1, total, width] with cu_seqlens."""
        q, k, v = self._qkv(x)
        return self._out(x, DecayAttention.apply(q, k, v, self.log_decay, cu_seqlens, self.scale))

    @torch.no_grad()
    def prefill(self, x):
        """A prompt [B, T, width]: its outputs and the state [B, heads, head_dim, head_dim] fp32."""
        q, k, v = self._qkv(x)
        o, state = gdr.decay_fwd(q, k, v, self.log_decay, scale=self.scale)
        return self._out(x, o), state

    @torch.no_grad()
    def step(self, x, state):
        """One more token of every sequence, x [B, 1, width]; the state is updated in place."""
        q, k, v = self._qkv(x)
        return self._out(x, gdr.decay_recurrent_fwd(q, k, v, self.log_decay, state, scale=self.scale))


def train(layer, steps=60, batch=4, tokens=256, width=512, seed=0):
    """Learn a running average: target y_t = 0.9 y_{t-1} + 0.1 x_t.  Returns the losses."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    powers = 0.1 * 0.9 ** (torch.arange(tokens, device="cuda")[:, None] - torch.arange(tokens, device="cuda")[None, :])
    mix = powers.tril()
    opt = torch.optim.Adam(layer.parameters(), lr=2e-3)
    losses = []
    for _ in range(steps):
        x = torch.randn(batch, tokens, width, generator=gen, device="cuda")
        loss = (layer(x.bfloat16()).float() - x - mix @ x).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return [float(v) for v in losses]


def main():
    torch.manual_seed(0)
    layer = DecayLayer()
    losses = train(layer)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} after {len(losses)} steps")
    x = torch.randn(2, 300, 512, device="cuda").bfloat16()
    with torch.no_grad():
        whole = layer(x)
    y, state = layer.prefill(x[:, :290].contiguous())
    rows = [y] + [layer.step(x[:, t:t + 1].contiguous(), state) for t in range(290, 300)]
    far = (torch.cat(rows, 1).float() - whole.float()).norm() / whole.float().norm()
    print(f"prompt of 290 tokens and 10 single ones against all 300 at once: rel {float(far):.1e}")
    assert gdr.gdr_get_status() == gdr.GDR_OK


if __name__ == "__main__":
    main()
