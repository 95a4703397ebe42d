"""The token mixers together, as examples/hybrid_mixer.py uses them: prompts and
single tokens through the caches against whole rows, and a training step's
gradients against the same stack written in plain 64-bit operations."""

import os
import sys

import pytest
import torch

import _mixer_ref as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def plain(mixer, params, x):
    """The stack in 64 bits on the CPU, differentiable."""
    B, T, C = x.shape
    H, D = mixer.heads, mixer.D
    cos, sin, g = mixer.cos.double().cpu(), mixer.sin.double().cpu(), mixer.log_decay.double().cpu()
    pos = torch.arange(T).expand(B, T)
    for layer, p in zip(mixer.layers, params):
        K = layer.kv
        qkv = (x @ p["qkv"]).unflatten(-1, (-1, D))
        q, k, v = qkv[:, :, :H], qkv[:, :, H:H + K], qkv[:, :, H + K:]
        q = ref.qk_norm_rope(q, p["q_norm"], cos, sin, pos, 1e-6, False)
        k = ref.qk_norm_rope(k, p["k_norm"], cos, sin, pos, 1e-6, False)
        if layer.linear:
            o, _ = ref.linattn(q, k, v, g, None, None, D ** -0.5)
        else:
            k, v = (t.repeat_interleave(H // K, 2) for t in (k, v))
            s = torch.einsum("bihd,bjhd->bhij", q, k) * D ** -0.5
            s = s.masked_fill(~ref.visible(T, T, mixer.window, mixer.sinks), -torch.inf)
            o = torch.einsum("bhij,bjhd->bihd", torch.softmax(s, -1), v)
        x = x + o.flatten(-2) @ p["out"]
    return x


@pytest.mark.parametrize("dtype,tol", [(torch.bfloat16, 2e-2), (torch.float32, 1e-4)])
def test_prompt_and_tokens_equal_whole_rows(lib, dtype, tol):
    """Four layers, each rounding its output once or twice to bf16 (2^-9.2 each,
    root mean square, times the layers' gain of a few); fp32: sums of 300 terms."""
    import hybrid_mixer
    rel, norm = hybrid_mixer.check(dtype=dtype)
    assert rel <= tol and norm > 0, (rel, norm)


@pytest.mark.parametrize("dtype,tol", [(torch.bfloat16, 5e-2), (torch.float32, 1e-4)])
def test_training_step_against_plain(lib, dtype, tol):
    import hybrid_mixer
    mixer = hybrid_mixer.HybridMixer(layers=2, channels=128, heads=2, key_heads=1, window=40, dtype=dtype)
    x = torch.randn(2, 150, 128, generator=torch.Generator().manual_seed(2)).to(dtype)
    w = torch.randn(2, 150, 128, generator=torch.Generator().manual_seed(3)).double()
    y = mixer(x.to("cuda"))
    (y.float() * w.float().to("cuda")).sum().backward()
    params = [{n: p.detach().double().cpu().requires_grad_() for n, p in layer.items()} for layer in mixer.layers]
    want = plain(mixer, params, x.double())
    (want * w).sum().backward()
    rel = float((y.double().cpu() - want).detach().norm() / want.detach().norm())
    assert rel <= tol, rel
    for layer, p in zip(mixer.layers, params):
        for n in p:
            got, ex = layer[n].grad.double().cpu(), p[n].grad
            rel = float((got - ex).norm() / ex.norm())
            assert rel <= tol, (n, rel)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_broadcast_gradients(lib, dtype):
    """A sum of an operator's outputs: the gradient that comes back is one number,
    broadcast, and counts as the same gradient written out."""
    import hybrid_mixer as hm
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(1, 70, 2, 64, generator=g).to(dtype).to("cuda").requires_grad_() for _ in range(3))
    w = torch.ones(64, device="cuda")
    angle = torch.arange(70.0, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, 64, 2, device="cuda") / 64)
    cos, sin, decay = angle.cos(), angle.sin(), torch.full((2,), -0.1, device="cuda")
    for call in (lambda: hm.QkNormRope.apply(q, k, w, w, cos, sin),
                 lambda: (hm.LinearAttention.apply(q, k, v, decay),),
                 lambda: (hm.WindowAttention.apply(q, k, v, 20, 2),)):
        got = torch.autograd.grad(sum(y.sum() for y in call()), (q, k, v), allow_unused=True)
        out = call()
        want = torch.autograd.grad(out, (q, k, v), [torch.ones_like(y) for y in out], allow_unused=True)
        for a, b in zip(got, want):
            assert (a is None and b is None) or torch.equal(a, b)
