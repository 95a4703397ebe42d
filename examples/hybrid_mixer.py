"""A hybrid stack's token mixers on libscan: linear attention with a decay for
each head and sliding-window attention with first tokens that stay visible,
alternating, both fed by normed and rotated queries and keys.

    mixer = HybridMixer(layers=4, channels=2048, heads=16, key_heads=4, window=1024)
    y = mixer(x)                       # training: differentiable, whole rows
    y, cache = mixer.prompt(x, slots)  # serving: the prompt, and what decoding goes on from
    y = mixer.token(x1, cache)         # then one token of each request at a time

Run as a script it feeds a prompt and tokens through the caches, checks that they
give what the whole row gives, and takes a gradient step.
"""

from __future__ import annotations

import os
import sys
from dataclasses import dataclass, field

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import associative_affine_scan_gb300 as scan  # noqa: E402


def _rows(grad):
    """A gradient with a unit stride along D: a sum's, for one, is a broadcast number."""
    return grad if grad.stride(-1) == 1 else grad.contiguous()


class QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos, sin):
        ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin)
        return scan.qk_norm_rope_fwd(q, k, q_weight, k_weight, cos, sin)

    @staticmethod
    def backward(ctx, dq, dk):
        return scan.qk_norm_rope_bwd(*ctx.saved_tensors, _rows(dq), _rows(dk)) + (None, None)


class LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay):
        ctx.save_for_backward(q, k, v, log_decay)
        return scan.linattn_fwd(q, k, v, log_decay, need_state=False)[0]

    @staticmethod
    def backward(ctx, dout):
        return scan.linattn_bwd(*ctx.saved_tensors, _rows(dout), need_dh0=False)[:3] + (None,)


class WindowAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, window, sinks):
        o, lse = scan.window_attn_fwd(q, k, v, window, sinks)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.sizes = window, sinks
        return o

    @staticmethod
    def backward(ctx, dout):
        return scan.window_attn_bwd(*ctx.saved_tensors, _rows(dout), *ctx.sizes) + (None, None)


@dataclass
class Cache:
    """What decoding needs of each layer: a pool of states (linear attention) or
    of rings of keys and values (window attention); a request's slot in them;
    and the position of its next token."""

    slots: torch.Tensor
    positions: torch.Tensor
    layers: list = field(default_factory=list)


class HybridMixer(torch.nn.Module):
    def __init__(self, layers=4, channels=2048, heads=16, key_heads=4, window=1024, sinks=4,
                 positions=8192, dtype=torch.bfloat16, device="cuda", seed=0):
        super().__init__()
        g = torch.Generator().manual_seed(seed)
        D = channels // heads
        self.heads, self.key_heads, self.D, self.window, self.sinks = heads, key_heads, D, window, sinks
        freq = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
        angle = torch.arange(positions, dtype=torch.float64)[:, None] * freq
        self.cos, self.sin = angle.cos().float().to(device), angle.sin().float().to(device)
        # half-lives from one step to a few hundred
        self.log_decay = -(2.0 ** (-8.0 * (torch.arange(heads) + 1.0) / heads)).to(device)

        def matrix(n, m):
            return torch.nn.Parameter((torch.randn(n, m, generator=g) * n ** -0.5).to(dtype).to(device))

        def norm():
            return torch.nn.Parameter(torch.ones(D, device=device))

        self.layers = torch.nn.ModuleList()
        for i in range(layers):
            linear = i % 2 == 0
            kv = heads if linear else key_heads
            layer = torch.nn.ParameterDict({
                "qkv": matrix(channels, (heads + 2 * kv) * D), "out": matrix(channels, channels),
                "q_norm": norm(), "k_norm": norm()})
            layer.linear, layer.kv = linear, kv
            self.layers.append(layer)

    def _project(self, layer, x):
        """q, k, v as slices of the one projection."""
        qkv = (x @ layer["qkv"]).unflatten(-1, (-1, self.D))
        H, K = self.heads, layer.kv
        return qkv[..., :H, :], qkv[..., H:H + K, :], qkv[..., H + K:, :]

    def forward(self, x):
        """[B, T, C] -> [B, T, C], differentiable."""
        for layer in self.layers:
            q, k, v = self._project(layer, x)
            q, k = QkNormRope.apply(q, k, layer["q_norm"], layer["k_norm"], self.cos, self.sin)
            if layer.linear:
                o = LinearAttention.apply(q, k, v, self.log_decay)
            else:
                o = WindowAttention.apply(q, k, v, self.window, self.sinks)
            x = x + o.flatten(-2) @ layer["out"]
        return x

    @torch.no_grad()
    def prompt(self, x, slots, pool=None):
        """The prompts [B, T, C] of B requests, whose states and rings go to
        `slots` (int32 [B], distinct) of pools for `pool` requests."""
        B, T, _ = x.shape
        pool = pool or int(slots.max()) + 1
        cache = Cache(slots, torch.full((B,), T, dtype=torch.int32, device=x.device))
        rows = slots.long()
        for layer in self.layers:
            q, k, v = self._project(layer, x)
            q, k = scan.qk_norm_rope_fwd(q, k, layer["q_norm"], layer["k_norm"], self.cos, self.sin)
            if layer.linear:
                o, state = scan.linattn_fwd(q, k, v, self.log_decay)
                held = torch.zeros(pool, *state.shape[1:], device=x.device)
                held[rows] = state
            else:
                W, S = self.window, self.sinks
                o, _ = scan.window_attn_fwd(q, k, v, W, S)
                # the first tokens and the last W, each to its place in the ring
                t = torch.arange(T, device=x.device)
                t = t[(t < S) | (t >= T - W)]
                place = torch.where(t < S, t, S + (t - S) % W)
                held = tuple(torch.zeros(pool, S + W, layer.kv, self.D, dtype=x.dtype, device=x.device)
                             for _ in range(2))
                for ring, rows_of in zip(held, (k, v)):
                    ring[rows[:, None], place[None]] = rows_of[:, t]
            cache.layers.append(held)
            x = x + o.flatten(-2) @ layer["out"]
        return x, cache

    @torch.no_grad()
    def token(self, x, cache):
        """The next token [B, C] of each request."""
        for layer, held in zip(self.layers, cache.layers):
            q, k, v = self._project(layer, x)
            q, k = scan.qk_norm_rope_fwd(q[:, None], k[:, None], layer["q_norm"], layer["k_norm"],
                                         self.cos, self.sin, cache.positions[:, None])
            q, k = q[:, 0], k[:, 0]
            if layer.linear:
                o = scan.linattn_step(q, k, v, self.log_decay, held, cache.slots)
            else:
                o = scan.window_attn_step(q, k, v, *held, cache.positions, self.window, self.sinks, cache.slots)
            x = x + o.flatten(-2) @ layer["out"]
        cache.positions += 1
        return x


def check(layers=4, channels=512, heads=8, key_heads=2, window=64, T=300, tokens=20, B=3,
          dtype=torch.bfloat16, device="cuda"):
    """How far tokens through the caches are from the whole rows (relative, in the
    2-norm), and the gradient norm of one training step."""
    mixer = HybridMixer(layers, channels, heads, key_heads, window, dtype=dtype, device=device)
    x = torch.randn(B, T + tokens, channels, generator=torch.Generator().manual_seed(1)).to(dtype).to(device)
    with torch.no_grad():
        whole = mixer(x)
    slots = torch.arange(B, dtype=torch.int32, device=device).flip(0) + 1
    y, cache = mixer.prompt(x[:, :T], slots, pool=B + 2)
    got = torch.stack([mixer.token(x[:, T + i], cache) for i in range(tokens)], 1)
    got = torch.cat([y, got], 1)
    rel = float((got - whole).double().norm() / whole.double().norm())
    loss = (mixer(x).float() ** 2).mean()
    loss.backward()
    norm = float(sum(p.grad.double().square().sum() for p in mixer.parameters()) ** 0.5)
    return rel, norm


if __name__ == "__main__":
    print("prompt and tokens against whole rows: %.2e; gradient norm %.3e" % check())
