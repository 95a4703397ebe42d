"""The host side of attention to another sequence, of the norms around a block and of
dropout, without a GPU: argument checks, workspace sizes, refusals, the generator's
published values and the gradients' formulas."""

import math
import struct

import pytest
import torch

import _block_ref as ref
import associative_affine_scan_gb300 as scan

OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4
P = 0x7f0000000000  # never dereferenced: every call below is refused on the host


@pytest.fixture(scope="module")
def lib():
    from associative_affine_scan_gb300 import build_lib
    build_lib.build()
    return scan.lib()


def view(ptr=P, sb=1 << 20, st=1024, sh=128):
    return struct.pack("Pqqq", ptr, sb, st, sh)


V = view()
NULL = view(0)


def cross(lib, q=V, lens=None, cu_q=None, cu_k=None, n=0, o=V, lse=P, B=1, Tq=64, Tk=50, Hq=4, Hk=2, D=64, scale=1.0, dt=1,
          ws=P, nws=1 << 30):
    return lib.cross_attn_fwd(q, V, V, lens, cu_q, cu_k, n, o, lse, B, Tq, Tk, Hq, Hk, D, scale, dt, ws, nws, None)


def test_cross_checks(lib):
    assert cross(lib, dt=2) == INVALID
    assert cross(lib, Tk=-1) == INVALID
    assert cross(lib, Hq=3) == INVALID
    assert cross(lib, Hk=0) == INVALID
    assert cross(lib, scale=0.0) == INVALID
    assert cross(lib, scale=float("nan")) == INVALID
    assert cross(lib, q=NULL) == INVALID
    assert cross(lib, o=None) == INVALID
    assert cross(lib, lse=None) == INVALID
    assert cross(lib, cu_q=P, n=2) == INVALID
    assert cross(lib, cu_k=P, n=2) == INVALID
    assert cross(lib, cu_q=P, cu_k=P, n=2, lens=P) == INVALID
    assert cross(lib, cu_q=P, cu_k=P, n=2, B=2) == INVALID
    assert cross(lib, cu_q=P, cu_k=P, n=0) == INVALID
    assert cross(lib, D=68) == UNSUPPORTED
    assert cross(lib, D=136) == UNSUPPORTED
    assert cross(lib, B=40000) == UNSUPPORTED
    assert cross(lib, ws=None) == WORKSPACE
    assert cross(lib, ws=P + 8) == WORKSPACE
    assert cross(lib, nws=100) == WORKSPACE
    assert cross(lib, Tq=0) == OK
    bwd = lambda dk=V, dout=V, nws=1 << 30, Tq=64: lib.cross_attn_bwd(  # noqa: E731
        V, V, V, V, P, dout, None, None, None, 0, V, dk, V, 1, Tq, 50, 4, 2, 64, 1.0, 1, P, nws, None)
    assert bwd(dk=NULL) == INVALID
    assert bwd(dout=None) == INVALID
    assert bwd(nws=256) == WORKSPACE
    step = lambda kc=V, slots=P, n=4, B=2, D=64, scale=1.0, nws=1 << 30: lib.cross_attn_step(  # noqa: E731
        V, kc, V, P, slots, n, V, B, 50, 4, 2, D, scale, 1, P, nws, None)
    assert step(nws=256) == WORKSPACE
    assert step(kc=NULL) == INVALID
    assert step(n=-1) == INVALID
    assert step(slots=None, n=1) == INVALID
    assert step(scale=math.inf) == INVALID
    assert step(D=12) == UNSUPPORTED
    assert step(B=0) == OK
    assert scan.cross_attn_workspace_bytes(2, 64, 50, 4, 2, 64) == 256
    assert scan.cross_attn_workspace_bytes(2, 64, 50, 4, 2, 64, 0, True) >= 256 + 2 * 64 * 4 * 4
    assert scan.cross_attn_workspace_bytes(2, 64, 50, 4, 2, 136) == 0


def norm(lib, x=V, y=V, wp=P, gt=P, wn=P, xo=V, n=V, B=2, T=3, C=64, row=0, alpha=1.0, eps=1e-6, p=0.0, rng=None, st=0, dt=1):
    return lib.residual_norm_fwd(x, y, wp, gt, wn, xo, n, B, T, C, row, alpha, eps, p, 0, 0, rng, st, dt, None)


def test_norm_checks(lib):
    assert norm(lib, st=2) == INVALID
    assert norm(lib, dt=5) == INVALID
    assert norm(lib, B=-1) == INVALID
    assert norm(lib, C=0) == INVALID
    assert norm(lib, eps=-1.0) == INVALID
    assert norm(lib, eps=math.nan) == INVALID
    assert norm(lib, alpha=math.inf) == INVALID
    assert norm(lib, alpha=math.nan) == INVALID
    assert norm(lib, p=1.5) == INVALID
    assert norm(lib, p=math.nan) == INVALID
    assert norm(lib, x=NULL) == INVALID
    assert norm(lib, xo=None) == INVALID
    assert norm(lib, n=None) == INVALID
    assert norm(lib, y=None) == INVALID  # weights of a block that is not there
    assert norm(lib, y=None, wp=None, gt=None, wn=None) == INVALID
    assert norm(lib, y=None, wp=None, gt=None, alpha=0.5) == INVALID
    assert norm(lib, y=None, wp=None, gt=None, p=0.5) == INVALID
    assert norm(lib, st=1, dt=0) == UNSUPPORTED
    assert norm(lib, C=60) == UNSUPPORTED
    assert norm(lib, C=8200) == UNSUPPORTED
    assert norm(lib, B=1 << 20, T=1 << 12) == UNSUPPORTED
    assert norm(lib, x=view(P + 4)) == ALIGNMENT
    assert norm(lib, x=view(st=1026)) == ALIGNMENT
    assert norm(lib, y=view(st=1028)) == ALIGNMENT
    assert norm(lib, wp=P + 4) == ALIGNMENT
    assert norm(lib, rng=P + 4) == ALIGNMENT
    assert norm(lib, T=0) == OK
    bwd = lambda dxo=V, dn=V, wn=P, dwn=P, gt=P, dg=P, nws=1 << 30: lib.residual_norm_bwd(  # noqa: E731
        V, V, dxo, dn, P, gt, wn, V, V, P, dg, dwn, 2, 3, 64, 0, 1.0, 1e-6, 0.0, 0, 0, None, 0, 1, P, nws, None)
    assert bwd(dn=None) == INVALID
    assert bwd(wn=None) == INVALID  # a gradient for a weight that is not there
    assert bwd(wn=None, dwn=None, dxo=None) == INVALID
    assert bwd(gt=None) == INVALID
    assert bwd(dn=view(P + 2)) == ALIGNMENT
    assert bwd(nws=16) == WORKSPACE
    assert scan.residual_norm_workspace_bytes(2, 3, 64) > 0
    assert scan.residual_norm_workspace_bytes(2, 3, 60) == 0


def test_dropout_checks(lib):
    drop = lambda x=V, y=V, B=2, p=0.1, rng=None, dt=1, T=3: lib.dropout_fwd(  # noqa: E731
        x, y, B, T, 64, p, 0, 0, rng, dt, None)
    assert drop(dt=3) == INVALID
    assert drop(B=-1) == INVALID
    assert drop(p=-0.1) == INVALID
    assert drop(p=1.1) == INVALID
    assert drop(p=math.nan) == INVALID
    assert drop(x=None) == INVALID
    assert drop(y=NULL) == INVALID
    assert drop(rng=P + 4) == ALIGNMENT
    assert drop(B=1 << 40) == UNSUPPORTED
    assert drop(B=0) == OK and drop(T=0) == OK


def test_cpu_tensors_and_bad_arguments_are_refused():
    x, t = torch.zeros(1, 8, 2, 64), torch.zeros(2, 3, 64)
    w = torch.ones(64)
    for call in (
        lambda: scan.cross_attn_fwd(x, x, x),
        lambda: scan.cross_attn_bwd(x, x, x, x, torch.zeros(1, 2, 8), x),
        lambda: scan.cross_attn_step(x[:, 0], x, x),
        lambda: scan.residual_norm_fwd(t, t, w, w, w),
        lambda: scan.residual_norm_bwd(t, t, t, t, w, w, w),
        lambda: scan.dropout_fwd(t, 0.1, (1, 2)),
        lambda: scan.dropout_bwd(t, 0.1, (1, 2)),
    ):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    from associative_affine_scan_gb300 import _binding
    for args in ((None, 0.1), ((1, 2), 1.5), ((1, 2), math.nan), ((-1, 2), 0.1), ((1, 1 << 64), 0.1)):
        with pytest.raises(ValueError):
            _binding._random(*args, None)
    assert _binding._random(None, 0.0, None) == (0.0, 0, 0, None)
    with pytest.raises(TypeError):
        scan.dropout_fwd([1.0], 0.1, (1, 2))


def test_generator_known_values():
    """The published test vectors of Philox 4x32 with ten rounds: counter and key all
    zeros, and all ones."""
    words = lambda h: [h[2 * i] | h[2 * i + 1] << 16 for i in range(4)]  # noqa: E731
    assert words(ref.numbers(8, 0, 0).tolist()) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]


def test_formulas_against_autograd():
    """The gradients as the kernels form them: two column sums serve three weights."""
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    B, T, C, alpha, eps = 3, 4, 8, 0.7, 1e-3
    x, y, wp, gt, wn, dxo, dn = r(B, T, C), r(B, T, C), r(C), r(B, C), r(C), r(B, T, C), r(B, T, C)
    keep = ref.kept((B, T, C), 0.4, (5, 6))
    leaves = [t.requires_grad_() for t in (x, y, wp, gt, wn)]
    xo = ref.block(x, y, wp, gt, alpha, eps, keep)
    loss = (xo * dxo).sum() + (ref.rms(xo, wn, eps) * dn).sum()
    want = torch.autograd.grad(loss, leaves)
    with torch.no_grad():
        q = 1 / torch.sqrt((xo * xo).mean(-1, keepdim=True) + eps)
        e, xq = wn * dn, xo * q
        G = dxo + q * (e - xq * (e * xq).mean(-1, keepdim=True))
        u, s = G * keep, 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        f, yh = wp * gt[:, None] * u, y * s
        h = (u * yh).sum(1)
        got = (alpha * G, s * (f - yh * (f * yh).mean(-1, keepdim=True)), (gt * h).sum(0), wp * h, (dn * xq).sum((0, 1)))
    for a, b in zip(got, want):
        assert torch.allclose(a, b)
    q, k, v, do = r(2, 7, 4, 4), r(2, 9, 2, 4), r(2, 9, 2, 4), r(2, 7, 4, 4)
    lens = torch.tensor([9, 5])
    leaves = [t.requires_grad_() for t in (q, k, v)]
    kk, vv = (t.repeat_interleave(2, 2) for t in leaves[1:])
    s = torch.einsum("bihd,bjhd->bhij", q, kk) * 0.6
    p = torch.softmax(s.masked_fill((torch.arange(9) >= lens[:, None])[:, None, None], -torch.inf), -1)
    want = torch.autograd.grad((torch.einsum("bhij,bjhd->bihd", p, vv) * do).sum(), leaves)
    got, _ = ref.cross_grads(*(t.detach() for t in (q, k, v)), do, 0.6, ref.spans(2, 7, 9, lens))
    for a, b in zip(got, want):
        assert torch.allclose(a, b)


def test_steps_of_many_heads(lib):
    """Single tokens are no blocks of a grid's second axis: 1024 requests of 64 heads pass the
    checks of sizes (and are refused for their workspace)."""
    step = lambda B, Hq, Hk, dt: lib.cross_attn_step(  # noqa: E731
        V, V, V, P, P, 4, V, B, 50, Hq, Hk, 64, 1.0, dt, P, 16, None)
    for dt in (0, 1):
        assert step(1024, 64, 8, dt) == WORKSPACE
        assert step(1, 1 << 20, 1, dt) == WORKSPACE
        assert step(1 << 26, 32, 8, dt) == UNSUPPORTED
        assert step(1 << 40, 1, 1, dt) == UNSUPPORTED
        assert step(1, 1 << 40, 1, dt) == UNSUPPORTED
    assert cross(lib, B=1, Hq=1 << 17, nws=16) == UNSUPPORTED


def test_gradients_of_keys_without_query_heads(lib):
    """They are written, so they and the workspace are asked for."""
    bwd = lambda dk, nws, Tk=50, Hk=2, B=1: lib.cross_attn_bwd(  # noqa: E731
        None, V, V, None, None, None, None, None, None, 0, None, dk, V, B, 64, Tk, 0, Hk, 64, 1.0, 1, P, nws, None)
    assert bwd(NULL, 1 << 30) == INVALID
    assert bwd(V, 16) == WORKSPACE
    assert bwd(V, 1 << 30, B=40000) == UNSUPPORTED
    assert bwd(V, 1 << 30, Hk=1 << 40) == UNSUPPORTED
    assert bwd(NULL, 16, Tk=0) == OK and bwd(NULL, 16, Hk=0) == OK


def test_generator_published_values():
    """The three published test vectors of Philox 4x32 with ten rounds: zeros, ones, and the
    digits of pi, whose words all differ, so that they hold the order of the counter's words (block,
    then call, low word first) and of the key's (the seed, low word first)."""
    for counter, key, want in (
        ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
        ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
        ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
         (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
    ):
        pair = lambda w: w[0] | w[1] << 32  # noqa: E731
        block, call, seed = pair(counter[:2]), pair(counter[2:]), pair(key)
        got = ref.numbers(8, seed, call, first=block).tolist()
        assert got == [h for w in want for h in (w & 0xffff, w >> 16)]
