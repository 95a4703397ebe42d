"""Attention to an encoder, the norms around a block and dropout together, as
examples/hybrid_mixer.py's decoder uses them: prompts and single tokens through the
caches against whole rows, and a training step's gradients against the same stack
written in plain 64-bit operations."""

import os
import sys

import pytest
import torch

import _block_ref as block
import _mixer_ref as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def attend(q, k, v, scale, seen):
    """Softmax attention in 64 bits; seen [.., Tq, Tk]: the keys of each query."""
    k, v = (t.repeat_interleave(q.shape[2] // t.shape[2], 2) for t in (k, v))
    s = torch.einsum("bihd,bjhd->bhij", q, k) * scale
    s = s.masked_fill(~seen & seen.any(-1, keepdim=True), -torch.inf)
    p = torch.softmax(s, -1).masked_fill(~seen, 0.0)  # rows that see nothing
    return torch.einsum("bhij,bjhd->bihd", p, v)


def plain(mixer, params, first, x, states, lengths, rng):
    """The stack in 64 bits on the CPU, differentiable."""
    B, T, C = x.shape
    H, D, K = mixer.heads, mixer.D, mixer.key_heads
    cos, sin, decay = mixer.cos.double().cpu(), mixer.sin.double().cpu(), mixer.log_decay.double().cpu()
    pos = torch.arange(T).expand(B, T)
    states = states * block.kept(states.shape, mixer.dropout, (rng[0] ^ (1 << 63), rng[1]))
    seen = (torch.arange(states.shape[1]) < lengths[:, None])[:, None, None, :]
    call = rng[1] * 2 * len(params)
    n = block.rms(x, first, 1e-6)
    for layer, p in zip(mixer.layers, params):
        for kind in ("mixer", "context"):
            if kind == "mixer":
                qkv = (n @ p["qkv"]).unflatten(-1, (-1, D))
                q, k, v = qkv[:, :, :H], qkv[:, :, H:H + layer.kv], qkv[:, :, H + layer.kv:]
                q = ref.qk_norm_rope(q, p["q_norm"], cos, sin, pos, 1e-6, False)
                k = ref.qk_norm_rope(k, p["k_norm"], cos, sin, pos, 1e-6, False)
                if layer.linear:
                    o, _ = ref.linattn(q, k, v, decay, None, None, D ** -0.5)
                else:
                    o = attend(q, k, v, D ** -0.5, ref.visible(T, T, mixer.window, mixer.sinks))
                y = o.flatten(-2) @ p["out"]
            else:
                kv = (states @ p["ctx_kv"]).unflatten(-1, (-1, D))
                o = attend((n @ p["ctx_q"]).unflatten(-1, (-1, D)), kv[:, :, :K], kv[:, :, K:], D ** -0.5, seen)
                y = o.flatten(-2) @ p["ctx_out"]
            keep = block.kept(x.shape, mixer.dropout, (rng[0], call))
            x = block.block(x, y, p[kind + "_post"], p[kind + "_gate"], 1.0, 1e-6, keep)
            n = block.rms(x, p[kind + "_next"], 1e-6)
            call += 1
    return n


# Relative errors in the 2-norm. bf16: each of the four blocks rounds its projections,
# queries, keys, values, output and norm, some eight roundings of 2^-9.2 each (root mean
# square) on a path, four blocks adding in squares: sqrt(32) 2^-9.2 = 0.010, times a gain of
# two for the scores. fp32: the same with 2^-23 a sum: 2e-6, and linear attention's sums of
# 300 terms at its chunked form's tenfold.
@pytest.mark.parametrize("dtype,tol", [(torch.bfloat16, 2e-2), (torch.float32, 1e-4)])
def test_prompt_and_tokens_equal_whole_rows(lib, dtype, tol):
    import hybrid_mixer
    rel, norm = hybrid_mixer.check(dtype=dtype, layers=2, context=True)
    assert rel <= tol and norm > 0, (rel, norm)


def test_norms_without_an_encoder(lib):
    import hybrid_mixer
    mixer = hybrid_mixer.HybridMixer(layers=2, channels=256, heads=4, key_heads=2, window=32, norms=True)
    x = torch.randn(2, 110, 256, generator=torch.Generator().manual_seed(3)).to("cuda")
    with torch.no_grad():
        whole = mixer(x)
    y, cache = mixer.prompt(x[:, :100], torch.tensor([1, 0], dtype=torch.int32, device="cuda"))
    got = torch.cat([y] + [mixer.token(x[:, 100 + i], cache)[:, None] for i in range(10)], 1)
    assert float((got - whole).double().norm() / whole.double().norm()) <= 2e-2
    with pytest.raises(ValueError):
        hybrid_mixer.HybridMixer(layers=1, channels=256, heads=4, key_heads=2, context=True)


# The gradients pass the roundings on the way back as well: three times the forward's.
@pytest.mark.parametrize("dtype,tol", [(torch.bfloat16, 6e-2), (torch.float32, 3e-4)])
def test_training_step_against_plain(lib, dtype, tol):
    import hybrid_mixer
    mixer = hybrid_mixer.HybridMixer(layers=2, channels=128, heads=2, key_heads=1, window=40, dtype=dtype, norms=True,
                                     context=True, dropout=0.2)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(3, 150, 128, generator=g)
    states = torch.randn(3, 70, 128, generator=g).to(dtype)
    w = torch.randn(3, 150, 128, generator=g).to(dtype)
    lengths = torch.tensor([70, 0, 33], dtype=torch.int32)
    dx, ds = x.to("cuda").requires_grad_(), states.to("cuda").requires_grad_()
    y = mixer(dx, ds, lengths.to("cuda"), rng=(11, 3))
    y.backward(w.to("cuda"))
    params = [{n: p.detach().double().cpu().requires_grad_() for n, p in layer.items()} for layer in mixer.layers]
    first = mixer.first.detach().double().cpu().requires_grad_()
    px, ps = x.double().requires_grad_(), states.double().requires_grad_()
    want = plain(mixer, params, first, px, ps, lengths, (11, 3))
    want.backward(w.double())
    pairs = [("y", y.detach(), want.detach()), ("x", dx.grad, px.grad), ("states", ds.grad, ps.grad),
             ("first", mixer.first.grad, first.grad)]
    pairs += [(n, layer[n].grad, p[n].grad) for layer, p in zip(mixer.layers, params) for n in p]
    for name, got, ex in pairs:
        rel = float((got.double().cpu() - ex).norm() / ex.norm())
        assert rel <= tol, (name, rel)
    assert not bool(ds.grad[1].any()) and not bool(ds.grad[2, 33:].any())  # past the encoders' lengths


def test_captured_training_step(lib):
    """A whole step, forward and backward, in a CUDA graph: a replay gives what the call did."""
    import hybrid_mixer
    mixer = hybrid_mixer.HybridMixer(layers=2, channels=256, heads=4, key_heads=2, window=64, norms=True, context=True,
                                     dropout=0.1)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(2, 200, 256, generator=g).to("cuda")
    states = torch.randn(2, 90, 256, generator=g).to(torch.bfloat16).to("cuda")
    lengths = torch.tensor([90, 41], dtype=torch.int32, device="cuda")
    names = [n for n, _ in mixer.named_parameters()]

    def step():
        y = mixer(x, states, lengths, rng=(5, 1))
        return torch.autograd.grad((y.float() ** 2).mean(), list(mixer.parameters()))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            want = [t.clone() for t in step()]
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for name, a, b in zip(names, got, want):
        assert torch.equal(a, b), name
    assert lib.scan_get_device_status(stream=side) == lib.SCAN_OK


def test_draws_follow_the_device_numbers(lib):
    """A captured dropout whose numbers lie on the device: each replay draws what the
    numbers say by then, the same as the call with them as arguments."""
    g = torch.Generator().manual_seed(6)
    x, y = (torch.randn(3, 50, 64, generator=g).to("cuda") for _ in range(2))
    rng = torch.tensor([3, 0], dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lib.residual_norm_bwd(x, y, x, None, p=0.3, rng=rng)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        a = lib.dropout_fwd(x, 0.3, rng)
        b, _ = lib.residual_norm_fwd(x, y, p=0.3, rng=rng)
        c = lib.residual_norm_bwd(x, y, x, None, p=0.3, rng=rng)
    for call in (0, 1, 2 ** 40 + 7):
        rng[1] = call
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, lib.dropout_fwd(x, 0.3, (3, call)))
        assert torch.equal(b, lib.residual_norm_fwd(x, y, p=0.3, rng=(3, call))[0])
        assert torch.equal(c[1], lib.residual_norm_bwd(x, y, x, None, p=0.3, rng=(3, call))[1])
