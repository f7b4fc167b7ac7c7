"""A retention layer over the library's operators, as an example of their use.

The token mixer is linear attention with a fixed decay for each head and rotary
positions on q and k, in the layer's usual order: residual addition and RMS norm,
one fused projection to q, k, v and the output gate, rotary positions in place on the
projection's output, the mixer, the output epilogue (RMS norm and SiLU gate), the
output projection. ``prefill`` runs a prompt in the chunked form and leaves the
states; ``step`` continues token by token from them. ``mixer_gradients`` is the part
of a training step between the projection and the epilogue.

The projections are plain matrix products; everything else runs in the library.
"""
import torch

from ._binding import rmsnorm_gate
from .layer import (add_rmsnorm, decay_chunk_bwd, decay_chunk_fwd, decay_step, rotary,
                    rotary_table)


class RetentionLayer:
    def __init__(self, width, heads, kv_heads=None, head_dim=128, max_len=4096, eps=1e-6, seed=0,
                 device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.H, self.Hk, self.d = heads, kv_heads or heads, head_dim
        self.eps = eps
        n = (2 * self.Hk + 2 * heads) * head_dim       # q, k, v, output gate
        w = lambda *s: (torch.randn(*s, generator=gen, device=device) * s[0] ** -0.5).to(  # noqa: E731
            torch.bfloat16)
        self.w_in, self.w_out = w(width, n), w(heads * head_dim, width)
        self.norm = torch.ones(width, device=device)
        self.out_norm = torch.ones(head_dim, device=device)
        # decays 1 - 2^-5 ... 1 - 2^-12 over the heads
        self.g = torch.log1p(-torch.exp2(-torch.linspace(5.0, 12.0, heads, device=device)))
        self.cos, self.sin = rotary_table(max_len, head_dim, device=device)

    def _project(self, y):
        """q, k, v and gate as views of one projection of y [B, T, width]."""
        B, T, _ = y.shape
        p = (y.reshape(B * T, -1) @ self.w_in).view(B, T, -1)
        parts, at = [], 0
        for h in (self.Hk, self.Hk, self.H, self.H):
            parts.append(p[..., at:at + h * self.d].unflatten(-1, (h, self.d)))
            at += h * self.d
        return parts

    def prefill(self, x, residual, state=None, start=0):
        """x, residual [B, T, width] bf16 -> (layer output, new residual, states)."""
        y, residual = add_rmsnorm(x, residual, self.norm, self.eps)
        q, k, v, z = self._project(y)
        rotary(q, k, self.cos, self.sin, start=start, q_out=q, k_out=k)
        o, state = decay_chunk_fwd(q, k, v, self.g, state)
        o = rmsnorm_gate(o, z.contiguous(), self.out_norm, self.eps)
        return o.flatten(2) @ self.w_out, residual, state

    def step(self, x, residual, state, position):
        """One token of each sequence: x, residual [B, width]; updates the states."""
        y, residual = add_rmsnorm(x, residual, self.norm, self.eps)
        q, k, v, z = self._project(y[:, None])
        rotary(q, k, self.cos, self.sin, start=position, q_out=q, k_out=k)
        o = decay_step(q[:, 0], k[:, 0], v[:, 0], self.g, state)
        o = rmsnorm_gate(o, z[:, 0].contiguous(), self.out_norm, self.eps)
        return o.flatten(1) @ self.w_out, residual

    def mixer_gradients(self, q, k, v, dO, start=0):
        """Gradients of the mixer's output with respect to the q and k it was given
        before their rotation, and v."""
        qr, kr = rotary(q, k, self.cos, self.sin, start=start)
        grads = decay_chunk_bwd(qr, kr, v, self.g, dO)
        grads["q"], grads["k"] = rotary(grads["q"], grads["k"], self.cos, self.sin, start=start,
                                        inverse=True, q_out=grads["q"], k_out=grads["k"])
        return grads
