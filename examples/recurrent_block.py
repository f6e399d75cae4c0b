"""Recurrent blocks built from the gated scan and the norms around a block, trained and served.

    r = r + scale u,  y = norm(r)                 the stream's sum and the norm in front (add_norm)
    x, a, z = y W_x, y W_a, y W_z
    h_t = alpha_t h_{t-1} + sqrt(1 - alpha_t^2) x_t, alpha_t = exp(-b sigmoid(a_t))   (gated_scan)
    u = (norm of every head of h, silu(z)) W_o    the norm behind, with its gate (norm_gate)

and so on with the next block's sum.  A block trains on whole or packed sequences; served, it reads a
prompt, which leaves one vector of state per sequence, and goes on token by token.

    python examples/recurrent_block.py    # a short training run, then a prompt and single tokens
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_gated_delta_07_gb300 as gdr  # noqa: E402


class AddNorm(torch.autograd.Function):
    """(y, r) of gdr.add_norm_fwd, rms; weight fp32 [D]."""

    @staticmethod
    def forward(ctx, u, residual, weight, scale):
        y, r, _, rstd = gdr.add_norm_fwd(u, residual, weight, scale=scale)
        ctx.save_for_backward(r, rstd, weight)
        ctx.scale = scale
        return y, r

    @staticmethod
    def backward(ctx, dy, dr):
        r, rstd, weight = ctx.saved_tensors
        du, dres, dw, _ = gdr.add_norm_bwd(dy.contiguous(), r, rstd, dr=dr.contiguous(), weight=weight, scale=ctx.scale)
        return du, dres, dw, None


class NormGate(torch.autograd.Function):
    """y of gdr.norm_gate_fwd, rms and silu; x, z [.., G, D], weight fp32 [G, D]."""

    @staticmethod
    def forward(ctx, x, z, weight):
        y, _, rstd = gdr.norm_gate_fwd(x, z, weight)
        ctx.save_for_backward(x, z, rstd, weight)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, z, rstd, weight = ctx.saved_tensors
        return gdr.norm_gate_bwd(dy.contiguous(), x, z, rstd, weight=weight)[:3]


class GatedScan(torch.autograd.Function):
    """out of gdr.gated_scan_fwd; x, a [B, T, D]."""

    @staticmethod
    def forward(ctx, x, a, cu_seqlens, b):
        out, _, states = gdr.gated_scan_fwd(x, a, cu_seqlens=cu_seqlens, b=b, source="variance", want_state=False,
                                            want_states=True)
        ctx.save_for_backward(x, a, states)
        ctx.cu_seqlens, ctx.b = cu_seqlens, b
        return out

    @staticmethod
    def backward(ctx, dout):
        x, a, states = ctx.saved_tensors
        dx, da, _ = gdr.gated_scan_bwd(x, a, dout.contiguous(), states=states, cu_seqlens=ctx.cu_seqlens, b=ctx.b,
                                       source="variance", want_dh0=False)
        return dx, da, None, None


class RecurrentBlock(torch.nn.Module):
    def __init__(self, width=256, heads=4, head_dim=64, scale=0.5, b=2.0, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.heads, self.scale, self.b = heads, scale, b
        inner = heads * head_dim
        lin = lambda i, o: torch.nn.Parameter(torch.randn(i, o, device=device, dtype=dtype) * i ** -0.5)  # noqa: E731
        self.w_x, self.w_a, self.w_z, self.w_o = lin(width, inner), lin(width, inner), lin(width, inner), lin(inner, width)
        self.norm = torch.nn.Parameter(torch.ones(width, device=device))
        self.head_norm = torch.nn.Parameter(torch.ones(heads, head_dim, device=device))
        # the channels' usual memories, from a token to some hundreds
        self.far = torch.nn.Parameter(torch.linspace(-6, 1, inner, device=device).to(dtype))

    def _heads(self, t):
        return t.unflatten(-1, (self.heads, -1))

    def forward(self, u, r, cu_seqlens=None):
        """u, r [B, T, width] (packed: [1, total, width]): the block's input and the stream."""
        y, r = AddNorm.apply(u, r, self.norm, self.scale)
        h = GatedScan.apply(y @ self.w_x, y @ self.w_a + self.far, cu_seqlens, self.b)
        o = NormGate.apply(self._heads(h), self._heads(y @ self.w_z), self.head_norm)
        return o.flatten(-2) @ self.w_o, r

    @torch.no_grad()
    def serve(self, u, r, state):
        """A prompt or single tokens: u, r [B, T, width], state [B, heads head_dim] fp32; r and state are
        updated in place.  Returns (u, r)."""
        y, _, _, _ = gdr.add_norm_fwd(u, r, self.norm, scale=self.scale, sum_out=r, want_stats=False)
        x, a = y @ self.w_x, y @ self.w_a + self.far
        if u.shape[1] == 1:
            h = gdr.gated_scan_recurrent_fwd(x, a, state, b=self.b, source="variance")
        else:
            h = gdr.gated_scan_fwd(x, a, h0=state, hT=state, b=self.b, source="variance")[0]
        z = self._heads(y @ self.w_z)
        o = gdr.norm_gate_fwd(self._heads(h), z, self.head_norm, out=z, want_stats=False)[0]
        return o.flatten(-2) @ self.w_o, r


def train(blocks, steps=40, batch=4, tokens=192, width=256, seed=0):
    """Learn a running average: target y_t = 0.9 y_{t-1} + 0.1 x_t.  Returns the losses."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    at = torch.arange(tokens, device="cuda")
    mix = (0.1 * 0.9 ** (at[:, None] - at[None, :])).tril()
    opt = torch.optim.Adam([p for b in blocks for p in b.parameters()], lr=2e-3)
    losses = []
    for _ in range(steps):
        x = torch.randn(batch, tokens, width, generator=gen, device="cuda")
        u, r = torch.zeros_like(x, dtype=torch.bfloat16), x.bfloat16()
        for block in blocks:
            u, r = block(u, r)
        loss = ((u + r).float() - x - mix @ x).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return [float(v) for v in losses]


def main():
    torch.manual_seed(0)
    blocks = [RecurrentBlock() for _ in range(2)]
    losses = train(blocks)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} after {len(losses)} steps")
    x = torch.randn(2, 300, 256, device="cuda").bfloat16()
    with torch.no_grad():
        u, r = torch.zeros_like(x), x
        for block in blocks:
            u, r = block(u, r)
        whole = u + r
    states = [torch.zeros(2, 256, device="cuda") for _ in blocks]
    rows = []
    for lo, hi in [(0, 290)] + [(t, t + 1) for t in range(290, 300)]:
        r = x[:, lo:hi].contiguous()
        u = torch.zeros_like(r)
        for block, state in zip(blocks, states):
            u, r = block.serve(u, r, state)
        rows.append(u + r)
    far = (torch.cat(rows, 1).float() - whole.float()).norm() / whole.float().norm()
    print(f"prompt of 290 tokens and 10 single ones against all 300 at once: rel {float(far):.1e}")
    assert gdr.gdr_get_status() == gdr.GDR_OK


if __name__ == "__main__":
    main()
