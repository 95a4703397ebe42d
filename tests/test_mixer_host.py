"""The token mixers' host side without a GPU: argument checks of the C entry
points, workspace sizes, and the binding's refusal of CPU tensors."""

import ctypes
import struct

import pytest
import torch

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


def rope(lib, q=V, k=V, cos=P, sin=P, out=V, B=1, T=8, Hq=2, Hk=2, D=64, R=64, pos=16, eps=1e-6, dt=1):
    return lib.qk_norm_rope_fwd(q, k, None, None, cos, sin, None, out, out, B, T, Hq, Hk, D, R, pos, 0, eps, dt, None)


def test_qk_norm_rope_checks(lib):
    assert rope(lib, dt=2) == INVALID
    assert rope(lib, T=-1) == INVALID
    assert rope(lib, R=72) == INVALID
    assert rope(lib, eps=-1.0) == INVALID
    assert rope(lib, eps=float("nan")) == INVALID
    assert rope(lib, cos=None) == INVALID
    assert rope(lib, pos=0) == INVALID
    assert rope(lib, q=None) == INVALID
    assert rope(lib, k=NULL) == INVALID
    assert rope(lib, out=None) == INVALID
    assert rope(lib, D=60, R=0) == UNSUPPORTED
    assert rope(lib, D=264, R=0) == UNSUPPORTED
    assert rope(lib, R=12) == UNSUPPORTED
    assert rope(lib, q=view(P + 2)) == ALIGNMENT
    assert rope(lib, q=view(st=1025)) == ALIGNMENT
    assert rope(lib, cos=P + 4) == ALIGNMENT
    assert rope(lib, T=0) == OK
    assert lib.qk_norm_rope_workspace_bytes(128) > 0 and lib.qk_norm_rope_workspace_bytes(60) == 0
    st = lib.qk_norm_rope_bwd(V, V, None, None, P, P, None, V, V, V, V, P, P, 1, 8, 2, 2, 64, 64, 16, 0, 1e-6, 1,
                              P, 16, None)
    assert st == WORKSPACE


def lin(lib, q=V, dec=P, cu=None, n=0, o=V, B=1, T=64, H=2, Dk=64, Dv=64, scale=1.0, dt=1, ws=P, nws=1 << 30):
    return lib.linattn_fwd(q, V, V, dec, None, cu, n, o, None, B, T, H, Dk, Dv, scale, dt, ws, nws, None)


def test_linattn_checks(lib):
    assert lin(lib, dt=7) == INVALID
    assert lin(lib, B=-1) == INVALID
    assert lin(lib, scale=0.0) == INVALID
    assert lin(lib, scale=float("inf")) == INVALID
    assert lin(lib, scale=float("nan")) == INVALID
    assert lin(lib, dec=None) == INVALID
    assert lin(lib, q=NULL) == INVALID
    assert lin(lib, o=None) == INVALID
    assert lin(lib, cu=P, n=3, B=2) == INVALID
    assert lin(lib, cu=P, n=0) == INVALID
    assert lin(lib, Dk=20) == UNSUPPORTED
    assert lin(lib, Dv=136) == UNSUPPORTED
    assert lin(lib, ws=None) == WORKSPACE
    assert lin(lib, ws=P + 4) == WORKSPACE
    assert lin(lib, nws=16) == WORKSPACE
    assert lin(lib, B=0) == OK
    step = lambda state=P, slots=P, n=4, B=2, scale=1.0: lib.linattn_step(  # noqa: E731
        V, V, V, P, state, slots, n, V, B, 2, 64, 64, scale, 1, None)
    assert step(state=None) == INVALID
    assert step(n=-1) == INVALID
    assert step(slots=None, n=1) == INVALID
    assert step(scale=-1.0) == INVALID
    assert step(state=P + 4) == ALIGNMENT
    assert step(B=0) == OK


def win(lib, q=V, lse=P, cu=None, n=0, B=1, Tq=64, Tk=64, Hq=4, Hk=2, D=64, W=16, S=2, scale=1.0, dt=1, ws=P,
        nws=1 << 30):
    return lib.window_attn_fwd(q, V, V, cu, n, V, lse, B, Tq, Tk, Hq, Hk, D, W, S, scale, dt, ws, nws, None)


def test_window_checks(lib):
    assert win(lib, dt=-1) == INVALID
    assert win(lib, W=0) == INVALID
    assert win(lib, S=-1) == INVALID
    assert win(lib, Hq=3) == INVALID
    assert win(lib, Hk=0) == INVALID
    assert win(lib, scale=0.0) == INVALID
    assert win(lib, q=NULL) == INVALID
    assert win(lib, lse=None) == INVALID
    assert win(lib, cu=P, n=2, Tk=65) == INVALID
    assert win(lib, cu=P, n=2, B=2) == INVALID
    assert win(lib, cu=P, n=0) == INVALID
    assert win(lib, D=68) == UNSUPPORTED
    assert win(lib, D=136) == UNSUPPORTED
    assert win(lib, B=40000, Hq=4) == UNSUPPORTED
    assert win(lib, ws=None) == WORKSPACE
    assert win(lib, nws=100) == WORKSPACE
    assert win(lib, Tq=0) == OK
    step = lambda kc=P, pos=P, slots=P, n=4, W=16, S=2, D=64, B=2: lib.window_attn_step(  # noqa: E731
        V, V, V, kc, P, pos, slots, n, V, B, 4, 2, D, W, S, 1.0, 1, None)
    assert step(kc=None) == INVALID
    assert step(pos=None) == INVALID
    assert step(slots=None, n=1) == INVALID
    assert step(W=0) == INVALID
    assert step(kc=P + 2) == ALIGNMENT
    assert step(D=12) == UNSUPPORTED
    assert step(W=1 << 31) == UNSUPPORTED
    assert step(B=0) == OK


def test_workspace_sizes():
    """The status word, and partial results that follow the sizes: none where a
    row is not cut."""
    assert scan.linattn_workspace_bytes(64, 256, 16, 128, 128) == 256
    cut = scan.linattn_workspace_bytes(1, 16384, 16, 128, 128)
    assert cut > 256 and (cut - 256) % (128 * 128 * 4) == 0
    assert scan.linattn_workspace_bytes(1, 16384, 16, 256, 128) == 0
    assert scan.linattn_workspace_bytes(1, 9000, 12, 64, 128, 6) > 256
    assert scan.window_attn_workspace_bytes(2, 4096, 4096, 16, 4, 128, 1024, 4) == 256
    whole = scan.window_attn_workspace_bytes(2, 4096, 4096, 16, 4, 128, 1 << 40, 4, 0, True)
    assert whole == 256 + 2 * 16 * 4096 * 4  # a window that holds the row: no tile is cut
    assert scan.window_attn_workspace_bytes(2, 4096, 4096, 16, 4, 128, 1024, 4, 0, True) > whole
    assert scan.window_attn_workspace_bytes(2, 4096, 4096, 16, 4, 128, 0, 4) == 0


def test_cpu_tensors_are_refused():
    x = torch.zeros(1, 8, 2, 64)
    t = x[:, 0]
    table = torch.zeros(8, 32)
    pos = torch.zeros(1, dtype=torch.int32)
    for call in (
        lambda: scan.qk_norm_rope_fwd(x, x, None, None, table, table),
        lambda: scan.qk_norm_rope_bwd(x, x, None, None, table, table, x, x),
        lambda: scan.linattn_fwd(x, x, x, torch.zeros(2)),
        lambda: scan.linattn_bwd(x, x, x, torch.zeros(2), x),
        lambda: scan.linattn_step(t, t, t, torch.zeros(2), torch.zeros(1, 2, 64, 64)),
        lambda: scan.window_attn_fwd(x, x, x, 4),
        lambda: scan.window_attn_bwd(x, x, x, x, torch.zeros(1, 2, 8), x, 4),
        lambda: scan.window_attn_step(t, t, t, x, x, pos, 8),
    ):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(TypeError, match="torch.Tensor"):
        scan.linattn_fwd([0.0], x, x, torch.zeros(2))


def test_formulas_against_autograd():
    """The gradient formulas that the kernels implement, in 64 bits against
    differentiation of the definitions: linear attention's gradients as linear
    attention over the other operands, window attention's from its softmax."""
    import _mixer_ref as ref
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    q, k, v, do, h0, dh = r(1, 9, 2, 4), r(1, 9, 2, 4), r(1, 9, 2, 3), r(1, 9, 2, 3), r(1, 2, 4, 3), r(1, 2, 4, 3)
    dec, sc = torch.tensor([-0.3, -0.9], dtype=torch.float64), 0.7
    dq, dk, dv, dh0 = ref.linattn_grads(q, k, v, dec, do, h0, dh, None, sc)
    got, _ = ref.linattn(do, v, k, dec, h0.transpose(-1, -2), None, sc)
    assert torch.allclose(got, dq)
    flip = lambda t: t.flip(1)  # noqa: E731
    lam = torch.exp(dec)[None, :, None, None]
    # reversed: the state that comes in is the gradient of the last one, not yet decayed
    init = dh / sc / lam
    back, end = ref.linattn(flip(v), flip(do), flip(q), dec, init.transpose(-1, -2), None, sc)
    assert torch.allclose(flip(back), dk)
    back, end = ref.linattn(flip(k), flip(q), flip(do), dec, init, None, sc)
    assert torch.allclose(flip(back), dv) and torch.allclose(end * lam * sc, dh0)
    q, k, v, do = r(1, 7, 4, 4), r(1, 9, 2, 4), r(1, 9, 2, 4), r(1, 7, 4, 4)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    kk, vv = (t.repeat_interleave(2, 2) for t in leaves[1:])
    s = torch.einsum("bihd,bjhd->bhij", leaves[0], kk) * 0.6
    p = torch.softmax(s.masked_fill(~ref.visible(7, 9, 3, 2), -torch.inf), -1)
    want = torch.autograd.grad((torch.einsum("bhij,bjhd->bihd", p, vv) * do).sum(), leaves)
    got, _ = ref.window_grads(q, k, v, do, 3, 2, None, 0.6)
    for a, b in zip(got, want):
        assert torch.allclose(a, b)
