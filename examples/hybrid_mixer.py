"""A hybrid stack's token mixers on libscan: linear attention with a decay for
each head and sliding-window attention with first tokens that stay visible,
alternating, both fed by normed and rotated queries and keys.

    mixer = HybridMixer(layers=4, channels=2048, heads=16, key_heads=4, window=1024)
    y = mixer(x)                       # training: differentiable, whole rows
    y, cache = mixer.prompt(x, slots)  # serving: the prompt, and what decoding goes on from
    y = mixer.token(x1, cache)         # then one token of each request at a time

With norms=True every mixer is a block with a norm before and a norm, a gate and dropout
after it, and with context=True each layer attends to an encoder's states as well:

    decoder = HybridMixer(layers=4, norms=True, context=True, dropout=0.1)
    y = decoder(x, states, lengths, rng=(seed, step))  # encoders of `lengths` states each
    y, cache = decoder.prompt(x, slots, states=states, lengths=lengths)
    y = decoder.token(x1, cache)

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


class CrossAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, lengths):
        o, lse = scan.cross_attn_fwd(q, k, v, lengths)
        ctx.save_for_backward(q, k, v, o, lse, lengths)
        return o

    @staticmethod
    def backward(ctx, dout):
        *saved, lengths = ctx.saved_tensors
        return scan.cross_attn_bwd(*saved, _rows(dout), lengths) + (None,)


class ResidualNorm(torch.autograd.Function):
    """The stream after a block, and the next block's input."""

    @staticmethod
    def forward(ctx, x, y, post, gate, following, p, rng):
        x_out, n = scan.residual_norm_fwd(x, y, post, gate, following, p=p, rng=rng)
        ctx.save_for_backward(x_out, y, post, gate, following)
        ctx.p, ctx.rng = p, rng
        return x_out, n

    @staticmethod
    def backward(ctx, dx, dn):
        x_out, y, post, gate, following = ctx.saved_tensors
        return scan.residual_norm_bwd(x_out, y, _rows(dx), _rows(dn), post, gate, following, p=ctx.p, rng=ctx.rng) + (None, None)


class FirstNorm(torch.autograd.Function):
    """The first block's input: the norm of the stream as it comes."""

    @staticmethod
    def forward(ctx, x, following, dtype):
        ctx.save_for_backward(x, following)
        return scan.residual_norm_fwd(x, None, next_weight=following, dtype=dtype)[1]

    @staticmethod
    def backward(ctx, dn):
        x, following = ctx.saved_tensors
        grads = scan.residual_norm_bwd(x, None, None, _rows(dn), next_weight=following)
        return grads[0], grads[4], None


class Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, rng):
        ctx.p, ctx.rng = p, rng
        return scan.dropout_fwd(x, p, rng)

    @staticmethod
    def backward(ctx, dy):
        return scan.dropout_bwd(_rows(dy), ctx.p, ctx.rng), None, None


@dataclass
class Cache:
    """What decoding needs of each layer: a pool of states (linear attention) or
    of rings of keys and values (window attention), and its pool of the encoders'
    keys and values; a request's slot in them; the position of its next token; and
    the encoders' lengths."""

    slots: torch.Tensor
    positions: torch.Tensor
    layers: list = field(default_factory=list)
    context: list = field(default_factory=list)
    lengths: torch.Tensor = None


class HybridMixer(torch.nn.Module):
    def __init__(self, layers=4, channels=2048, heads=16, key_heads=4, window=1024, sinks=4,
                 positions=8192, dtype=torch.bfloat16, device="cuda", seed=0, norms=False, context=False,
                 dropout=0.0):
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

        if context and not norms:
            raise ValueError("context=True needs norms=True")
        self.norms, self.context, self.dropout, self.dtype = norms, context, dropout, dtype

        def wide(value=1.0):
            return torch.nn.Parameter(torch.full((channels,), value, device=device))

        if norms:
            self.first = wide()
        self.layers = torch.nn.ModuleList()
        for i in range(layers):
            linear = i % 2 == 0
            kv = heads if linear else key_heads
            layer = torch.nn.ParameterDict({
                "qkv": matrix(channels, (heads + 2 * kv) * D), "out": matrix(channels, channels),
                "q_norm": norm(), "k_norm": norm()})
            if norms:  # after the mixer, and (context) after the attention to the encoder
                for block in ("mixer", "context")[:1 + context]:
                    layer.update({block + "_post": wide(), block + "_gate": wide(0.5), block + "_next": wide()})
            if context:
                layer.update({"ctx_q": matrix(channels, channels), "ctx_kv": matrix(channels, 2 * key_heads * D),
                              "ctx_out": matrix(channels, channels)})
            layer.linear, layer.kv = linear, kv
            self.layers.append(layer)

    def _project(self, layer, x):
        """q, k, v as slices of the one projection."""
        qkv = (x @ layer["qkv"]).unflatten(-1, (-1, self.D))
        H, K = self.heads, layer.kv
        return qkv[..., :H, :], qkv[..., H:H + K, :], qkv[..., H + K:, :]

    def _context_kv(self, layer, states):
        """Keys and values of an encoder's states, slices of one projection."""
        kv = (states @ layer["ctx_kv"]).unflatten(-1, (-1, self.D))
        return kv[..., :self.key_heads, :], kv[..., self.key_heads:, :]

    def _blocks(self, x, mix, attend, rng=None):
        """The stack as blocks with norms: mix(i, layer, n) is a layer's mixer, attend(i,
        layer, n) its attention to the encoder. Each block's dropout has a call number of
        its own."""
        p = self.dropout if rng is not None else 0.0
        seed, call = rng if rng is not None else (0, 0)
        call *= 2 * len(self.layers)
        n = FirstNorm.apply(x, self.first, self.dtype)
        for i, layer in enumerate(self.layers):
            for block, run in (("mixer", mix), ("context", attend))[:1 + self.context]:
                y = run(i, layer, n)
                x, n = ResidualNorm.apply(x, y, layer[block + "_post"], layer[block + "_gate"], layer[block + "_next"],
                                          p, (seed, call))
                call += 1
        return x, n

    def _mix(self, layer, n):
        q, k, v = self._project(layer, n)
        q, k = QkNormRope.apply(q, k, layer["q_norm"], layer["k_norm"], self.cos, self.sin)
        if layer.linear:
            o = LinearAttention.apply(q, k, v, self.log_decay)
        else:
            o = WindowAttention.apply(q, k, v, self.window, self.sinks)
        return o.flatten(-2) @ layer["out"]

    def _attend(self, layer, n, states, lengths):
        q = (n @ layer["ctx_q"]).unflatten(-1, (-1, self.D))
        o = CrossAttention.apply(q, *self._context_kv(layer, states), lengths)
        return o.flatten(-2) @ layer["ctx_out"]

    def forward(self, x, states=None, lengths=None, rng=None):
        """[B, T, C] -> [B, T, C], differentiable. states [B, Tk, C], lengths int32 [B]: the
        encoders'; rng (seed, step): dropout's, of the blocks and of the encoders' states."""
        if self.norms:
            if self.context and rng is not None and self.dropout:
                states = Dropout.apply(states, self.dropout, (rng[0] ^ (1 << 63), rng[1]))
            return self._blocks(x, lambda i, layer, n: self._mix(layer, n),
                                lambda i, layer, n: self._attend(layer, n, states, lengths), rng)[1]
        for layer in self.layers:
            x = x + self._mix(layer, x)
        return x

    @torch.no_grad()
    def prompt(self, x, slots, pool=None, states=None, lengths=None):
        """The prompts [B, T, C] of B requests, whose states and rings go to
        `slots` (int32 [B], distinct) of pools for `pool` requests, as do the keys and
        values of their encoders' states (lengths None: all of them)."""
        B, T, _ = x.shape
        pool = pool or int(slots.max()) + 1
        cache = Cache(slots, torch.full((B,), T, dtype=torch.int32, device=x.device))
        rows = slots.long()
        if self.context:
            cache.lengths = torch.zeros(pool, dtype=torch.int32, device=x.device)
            cache.lengths[rows] = lengths if lengths is not None else states.shape[1]

        def mix(i, layer, x):
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
            return o.flatten(-2) @ layer["out"]

        def attend(i, layer, n):
            k, v = self._context_kv(layer, states)
            held = tuple(torch.zeros(pool, *t.shape[1:], dtype=t.dtype, device=t.device) for t in (k, v))
            for pool_of, rows_of in zip(held, (k, v)):
                pool_of[rows] = rows_of
            cache.context.append(held)
            q = (n @ layer["ctx_q"]).unflatten(-1, (-1, self.D))
            return scan.cross_attn_fwd(q, k, v, lengths)[0].flatten(-2) @ layer["ctx_out"]

        if self.norms:
            return self._blocks(x, mix, attend)[1], cache
        for i, layer in enumerate(self.layers):
            x = x + mix(i, layer, x)
        return x, cache

    @torch.no_grad()
    def token(self, x, cache):
        """The next token [B, C] of each request."""
        def mix(i, layer, x):
            held = cache.layers[i]
            q, k, v = self._project(layer, x)
            q, k = scan.qk_norm_rope_fwd(q[:, None], k[:, None], layer["q_norm"], layer["k_norm"],
                                         self.cos, self.sin, cache.positions[:, None])
            q, k = q[:, 0], k[:, 0]
            if layer.linear:
                o = scan.linattn_step(q, k, v, self.log_decay, held, cache.slots)
            else:
                o = scan.window_attn_step(q, k, v, *held, cache.positions, self.window, self.sinks, cache.slots)
            return o.flatten(-2) @ layer["out"]

        def attend(i, layer, n):
            q = (n @ layer["ctx_q"]).unflatten(-1, (-1, self.D))
            o = scan.cross_attn_step(q, *cache.context[i], cache.lengths, cache.slots)
            return o.flatten(-2) @ layer["ctx_out"]

        if self.norms:
            x = self._blocks(x, mix, attend)[1]
        else:
            for i, layer in enumerate(self.layers):
                x = x + mix(i, layer, x)
        cache.positions += 1
        return x


def check(layers=4, channels=512, heads=8, key_heads=2, window=64, T=300, tokens=20, B=3,
          dtype=torch.bfloat16, device="cuda", context=False):
    """How far tokens through the caches are from the whole rows (relative, in the
    2-norm), and the gradient norm of one training step. context: of blocks with norms
    that attend to encoders of three lengths, with dropout in training."""
    mixer = HybridMixer(layers, channels, heads, key_heads, window, dtype=dtype, device=device, norms=context,
                        context=context, dropout=0.1 if context else 0.0)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(B, T + tokens, channels, generator=g).to(dtype).to(device)
    extra, train = {}, {}
    if context:
        x = x.float()  # the stream; the blocks are of `dtype`
        extra = dict(states=torch.randn(B, 90, channels, generator=g).to(dtype).to(device),
                     lengths=torch.tensor([90 - 40 * b for b in range(B)], dtype=torch.int32, device=device))
        train = dict(rng=(7, 1))
    with torch.no_grad():
        whole = mixer(x, **extra)
    slots = torch.arange(B, dtype=torch.int32, device=device).flip(0) + 1
    y, cache = mixer.prompt(x[:, :T], slots, pool=B + 2, **extra)
    got = torch.stack([mixer.token(x[:, T + i], cache) for i in range(tokens)], 1)
    got = torch.cat([y, got], 1)
    rel = float((got - whole).double().norm() / whole.double().norm())
    loss = (mixer(x, **extra, **train).float() ** 2).mean()
    loss.backward()
    norm = float(sum(p.grad.double().square().sum() for p in mixer.parameters()) ** 0.5)
    return rel, norm


if __name__ == "__main__":
    print("prompt and tokens against whole rows: %.2e; gradient norm %.3e" % check())
    print("with norms and an encoder: %.2e; gradient norm %.3e" % check(context=True))
