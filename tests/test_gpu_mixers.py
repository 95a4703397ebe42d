"""GPU parity of the token mixers against their definitions in 64 bits
(_mixer_ref), through the binding: sizes from one step up, odd sizes, shared
heads, strides, packed and empty sequences, rows that see no key, idle requests,
and values outside the sequences that must not be used."""

import math

import pytest
import torch

import _mixer_ref as ref
from _mixer_ref import U16, U32, f64, gate

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, dtype=F32, mul=1.0):
    return (mul * torch.randn(shape, generator=g)).to(dtype).to(DEV)


def framed(t, mode):
    """The same values as a slice of a larger tensor that holds NaN around them:
    'wide': longer rows and more heads; 'odd': rows that start off 16 bytes."""
    if mode == "plain":
        return t
    B, T, H, D = t.shape
    extra = 8 if mode == "wide" else 3
    big = torch.full((B, T + 2, H + 2, D + extra), NAN, dtype=t.dtype, device=t.device)
    at = 0 if mode == "wide" else 1
    out = big[:, 1:T + 1, 1:H + 1, at:at + D]
    out.copy_(t)
    return out


def offsets(lengths):
    return torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------------
# norm and rotation
# ---------------------------------------------------------------------------

def tables(P, R):
    if R == 0:
        return None, None
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    a = torch.arange(P, dtype=torch.float64)[:, None] * f
    return a.cos().float().to(DEV), a.sin().float().to(DEV)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,R", [(8, 8), (64, 64), (64, 32), (96, 48), (96, 96), (128, 128), (128, 0),
                                 (200, 104), (256, 256)])
@pytest.mark.parametrize("pairs", [False, True])
def test_qk_norm_rope(lib, dtype, D, R, pairs):
    for (B, T, Hq, Hk), weights, given in (((1, 1, 1, 1), True, False), ((2, 7, 6, 3), True, True),
                                           ((3, 65, 5, 1), False, True)):
        g = gen(D + R + B)
        x = [normal(g, B, T, h, D, dtype=dtype, mul=3.0) for h in (Hq, Hk)]
        dy = [normal(g, B, T, h, D, dtype=dtype) for h in (Hq, Hk)]
        w = [normal(g, D) + 1.0 for _ in range(2)] if weights else [None, None]
        cos, sin = tables(300, R)
        pos = torch.randint(0, 300, (B, T), generator=g).to(torch.int32).to(DEV) if given else None
        y = lib.qk_norm_rope_fwd(framed(x[0], "wide"), x[1], w[0], w[1], cos, sin, pos, interleaved=pairs)
        d = lib.qk_norm_rope_bwd(framed(x[0], "wide"), x[1], w[0], w[1], cos, sin, dy[0],
                                 framed(dy[1], "wide"), pos, interleaved=pairs)
        p = torch.arange(T).expand(B, T) if pos is None else pos.cpu()
        for m in range(2):
            xr = f64(x[m]).requires_grad_()
            wr = torch.ones(D, dtype=torch.float64) if w[m] is None else f64(w[m])
            wr.requires_grad_()
            yr = ref.qk_norm_rope(xr, wr, f64(cos), f64(sin), p, 1e-6, pairs)
            dxr, dwr = torch.autograd.grad((yr * f64(dy[m])).sum(), (xr, wr))
            # terms: the two products of a pair; D of the norm's sum
            n = (xr / torch.sqrt((xr * xr).mean(-1, keepdim=True) + 1e-6)).detach()
            zmag = (n * wr.detach()).abs().amax(-1, keepdim=True)
            gate(y[m], yr.detach(), zmag.expand_as(yr), dtype=dtype, terms=D, name="y")
            r = 1 / torch.sqrt((f64(x[m]) ** 2).mean(-1, keepdim=True) + 1e-6)
            gmag = 2 * f64(dy[m]).abs().amax(-1, keepdim=True) * wr.detach().abs().amax()
            mag = (r * gmag * (1 + n.abs() * n.abs().mean(-1, keepdim=True))).expand_as(dxr)
            gate(d[m], dxr, mag, dtype=dtype, terms=D, name="dx")
            if w[m] is not None:
                dwmag = (2 * f64(dy[m]).abs().amax(-1, keepdim=True) * n.abs()).sum((0, 1, 2))
                gate(d[2 + m], dwr, dwmag, dtype=F32, terms=D, name="dw")


def test_qk_norm_rope_in_place_one_sided_and_bad_positions(lib):
    g = gen(3)
    q, k = normal(g, 2, 9, 4, 64, dtype=BF), normal(g, 2, 9, 2, 64, dtype=BF)
    cos, sin = tables(16, 64)
    want = lib.qk_norm_rope_fwd(q, k, None, None, cos, sin)
    only = lib.qk_norm_rope_fwd(q[:, :, :0], k, None, None, cos, sin)
    assert only[0].numel() == 0 and torch.equal(only[1], want[1])
    got = lib.qk_norm_rope_fwd(q, k, None, None, cos, sin, out=(q, k))
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    pos = torch.tensor([[0, 15, 16, -1] + [3] * 5] * 2, dtype=torch.int32, device=DEV)
    y, _ = lib.qk_norm_rope_fwd(want[0], want[1], None, None, cos, sin, pos)
    assert y[:, 2:4].isnan().all() and not y[:, :2].isnan().any() and not y[:, 4:].isnan().any()
    empty = lib.qk_norm_rope_bwd(q[:, :0], k[:, :0], torch.ones(64, device=DEV), None, cos, sin,
                                 q[:, :0], k[:, :0])
    assert empty[0].numel() == 0 and float(empty[2].abs().max()) == 0.0 and empty[3] is None


# ---------------------------------------------------------------------------
# linear attention
# ---------------------------------------------------------------------------

def decays(H):
    """No decay, a slow, a fast, a very fast one, no memory at all, ..."""
    return torch.tensor(([0.0, -0.01, -0.7, -9.0, -math.inf] * 4)[:H], device=DEV)


def lin_inputs(B, T, H, Dk, Dv, dtype, seed, n=None, state=True):
    g = gen(seed)
    q, k = normal(g, B, T, H, Dk, dtype=dtype), normal(g, B, T, H, Dk, dtype=dtype)
    v, do = normal(g, B, T, H, Dv, dtype=dtype), normal(g, B, T, H, Dv, dtype=dtype)
    n = B if n is None else n
    h0, dh = (normal(g, n, H, Dk, Dv) if state else None for _ in range(2))
    return q, k, v, do, h0, dh


def lin_check(lib, ins, decay, cu=None, mode="plain", scale=None):
    q, k, v, do, h0, dh = ins
    dtype, sc = q.dtype, q.shape[-1] ** -0.5 if scale is None else scale
    view = [framed(t, mode) for t in (q, k, v, do)]
    o, hT = lib.linattn_fwd(*view[:3], decay, h0, cu, scale=scale)
    dq, dk, dv, dh0 = lib.linattn_bwd(*view[:3], decay, view[3], h0, cu, dh, scale=scale)
    torch.cuda.synchronize()
    assert lib.scan_get_device_status() == lib.SCAN_OK
    a = [f64(t) for t in (q, k, v)]
    g, c = f64(decay), None if cu is None else cu.cpu()
    m = [t.abs() for t in a]
    ab = lambda t: None if t is None else f64(t).abs()  # noqa: E731
    ro, rh = ref.linattn(*a, g, f64(h0), c, sc)
    mo, mh = ref.linattn(*m, g, ab(h0), c, sc)
    rg = ref.linattn_grads(*a, g, f64(do), f64(h0), f64(dh), c, sc)
    mg = ref.linattn_grads(*m, g, ab(do), ab(h0), ab(dh), c, sc)
    # bf16: the weights within a chunk or the state as it is read, one rounding each;
    # the state: its update's operand in two parts, 2^-17 off
    T, D = q.shape[1], max(q.shape[-1], v.shape[-1])
    r = 1 if dtype == BF else 0
    terms = min(T, 256) + D
    gate(o, ro, mo, dtype=dtype, roundings=r, terms=terms, name="o")
    for got, want, mag, name in zip((dq, dk, dv), rg[:3], mg[:3], ("dq", "dk", "dv")):
        gate(got, want, mag, dtype=dtype, roundings=r, terms=terms, name=name)
    extra = 2 ** 7 if dtype == BF else 0  # 2^-17 in units of 2^-24
    gate(hT, rh, mh, dtype=F32, terms=terms + extra, name="hT")
    gate(dh0, rg[3], mg[3], dtype=F32, terms=terms + extra, name="dh0")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 2, 17, 64, 127, 128, 129, 256, 300])
def test_linattn_lengths(lib, dtype, T):
    for Dk, Dv in ((64, 64), (128, 128)):
        lin_check(lib, lin_inputs(1, T, 3, Dk, Dv, dtype, T + Dk, state=T % 2 == 0), decays(3))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Dk,Dv", [(8, 8), (8, 128), (64, 128), (128, 64), (96, 64), (72, 120), (40, 16)])
def test_linattn_head_sizes(lib, dtype, Dk, Dv):
    lin_check(lib, lin_inputs(2, 200, 2, Dk, Dv, dtype, Dk + Dv), decays(2), scale=0.3)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_linattn_decays_and_long_rows(lib, dtype):
    lin_check(lib, lin_inputs(1, 700, 5, 64, 64, dtype, 5), decays(5))
    lin_check(lib, lin_inputs(2, 1030, 2, 64, 128, dtype, 6, state=False), decays(2))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mode", ["wide", "odd"])
def test_linattn_strides(lib, dtype, mode):
    """Slices of larger tensors whose other values are NaN."""
    lin_check(lib, lin_inputs(2, 190, 2, 64, 64, dtype, 8), decays(2), mode=mode)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_linattn_broadcast_operands(lib, dtype):
    """One key head and one value head for every head: strides of zero."""
    q, k, v, do, h0, dh = lin_inputs(1, 150, 3, 64, 64, dtype, 9)
    k, v = k[:, :, :1].expand(-1, -1, 3, -1), v[:, :, :1].expand(-1, -1, 3, -1)
    lin_check(lib, (q, k, v, do, h0, dh), decays(3))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lengths", [[1], [0, 5, 0], [130, 1, 127, 0, 256, 70], [300, 1, 1, 40]])
def test_linattn_packed(lib, dtype, lengths):
    n, T = len(lengths), sum(lengths)
    for Dk, Dv in ((64, 64), (64, 128)):
        lin_check(lib, lin_inputs(1, T, 2, Dk, Dv, dtype, T + n, n=n, state=n % 2 == 0), decays(2),
                  cu=offsets(lengths))


@pytest.mark.parametrize("lengths", [[606, 644, 22, 33, 439, 88, 337, 152, 480], [1100, 1, 700]])
def test_linattn_packed_segments(lib, lengths):
    """Sequences of several segments, the first in reversed order with a ragged chunk."""
    n, T = len(lengths), sum(lengths)
    for Dk, Dv in ((64, 64), (128, 64), (64, 128)):
        lin_check(lib, lin_inputs(1, T, 2, Dk, Dv, BF, T + n, n=n, state=n % 2 == 0), decays(2), offsets(lengths))
    assert lib.scan_get_device_status() == lib.SCAN_OK


def test_linattn_many_packed_sequences(lib):
    """More (sequence, head) rows than the second axis of a grid holds, empty ones
    among them: every final state against its closed form for constant operands."""
    H, D, n = 34, 8, 2000
    lengths = torch.full((n,), 48)
    lengths[::7] = 0
    cu = torch.cat([torch.zeros(1), lengths.cumsum(0)]).to(torch.int32).to(DEV)
    T = int(lengths.sum())
    assert n * H > 65535 and T >= 32 * n  # the chunked form takes it
    g = -torch.linspace(0.01, 2.0, H, device=DEV)
    q = torch.ones(1, T, H, D, dtype=BF, device=DEV)
    o, hT = lib.linattn_fwd(q, q, q, g, None, cu, scale=1.0)
    lam = f64(g).exp()
    full = (1 - lam ** 48) / (1 - lam)
    want = torch.where(lengths[:, None] > 0, full[None], 0.0)[:, :, None, None].expand(n, H, D, D)
    gate(hT, want, want, dtype=F32, terms=48 + D + 2 ** 7, name="hT")
    ends = (cu[1:][lengths.to(DEV) > 0] - 1).long()
    got, last = f64(o[0, ends]), D * full[None, :, None].expand(len(ends), H, D)
    assert float(((got - last).abs() / last).max()) <= 3 * U16
    assert lib.scan_get_device_status() == lib.SCAN_OK


@pytest.mark.parametrize("dtype", [BF, F32])
def test_linattn_sequences_do_not_leak(lib, dtype):
    """A sequence of NaN between two others leaves their results as they are."""
    lengths = [150, 77, 200]
    cu = offsets(lengths)
    q, k, v, do, h0, dh = lin_inputs(1, sum(lengths), 2, 64, 64, dtype, 10, n=3)
    want = lib.linattn_fwd(q, k, v, decays(2), h0, cu) + lib.linattn_bwd(q, k, v, decays(2), do, h0, cu, dh)
    for t in (q, k, v, do):
        t[:, 150:227] = NAN
    got = lib.linattn_fwd(q, k, v, decays(2), h0, cu) + lib.linattn_bwd(q, k, v, decays(2), do, h0, cu, dh)
    for i, (a, b) in enumerate(zip(got, want)):
        if a.dtype == F32 and a.shape[0] == 3:  # states
            assert torch.equal(a[[0, 2]], b[[0, 2]]), i
        else:
            assert torch.equal(a[:, :150], b[:, :150]) and torch.equal(a[:, 227:], b[:, 227:]), i


def test_linattn_malformed_offsets(lib):
    q, k, v, do, _, _ = lin_inputs(1, 300, 2, 64, 64, BF, 11, n=2, state=False)
    lib.linattn_fwd(q, k, v, decays(2), None, torch.tensor([0, 400, 300], dtype=torch.int32, device=DEV))
    assert lib.scan_get_device_status() == lib.SCAN_ERR_SEQLENS
    lib.window_attn_fwd(q, k, v, 16, 0, torch.tensor([-7, 90, 20], dtype=torch.int32, device=DEV))
    assert lib.scan_get_device_status() == lib.SCAN_ERR_SEQLENS
    assert lib.scan_get_device_status() == lib.SCAN_OK


@pytest.mark.parametrize("dtype", [BF, F32])
def test_linattn_pieces_equal_the_whole(lib, dtype):
    """A row cut into pieces that hand their state on, then single tokens."""
    q, k, v, _, h0, _ = lin_inputs(2, 421, 2, 64, 128, dtype, 12)
    g = decays(2)
    whole, last = lib.linattn_fwd(q, k, v, g, h0)
    a, h = lib.linattn_fwd(q[:, :129], k[:, :129], v[:, :129], g, h0)
    b, h = lib.linattn_fwd(q[:, 129:400], k[:, 129:400], v[:, 129:400], g, h)
    steps = [lib.linattn_step(q[:, t], k[:, t], v[:, t], g, h) for t in range(400, 421)]
    got = torch.cat([a, b, torch.stack(steps, 1)], 1)
    # two results that are each within three roundings
    assert float((got - whole).double().norm() / whole.double().norm()) <= 3 * (U16 if dtype == BF else 128 * U32)
    assert float((h - last).double().norm() / last.double().norm()) <= 2 ** -15


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Dk,Dv", [(8, 8), (64, 64), (128, 128), (96, 40), (128, 64)])
def test_linattn_step(lib, dtype, Dk, Dv):
    for B, H in ((1, 1), (5, 3)):
        g = gen(B + Dk)
        q, k, v = (normal(g, B, H, d, dtype=dtype) for d in (Dk, Dk, Dv))
        state = normal(g, B + 2, H, Dk, Dv)
        slots = torch.randperm(B + 2, generator=g)[:B].to(torch.int32)
        if B > 2:
            slots[1], slots[2] = -1, B + 2  # idle
        decay = decays(H)
        before = f64(state)
        o = lib.linattn_step(q, k, v, decay, state, slots.to(DEV))
        rs, ms, ro, mo = before.clone(), before.abs(), torch.zeros(B, H, Dv).double(), torch.zeros(B, H, Dv).double()
        for b, s in enumerate(slots.tolist()):
            if 0 <= s < B + 2:
                lam = f64(decay).exp()[:, None, None]
                kv = f64(k[b])[:, :, None] * f64(v[b])[:, None, :]
                ms[s] = lam * rs[s].abs() + kv.abs()
                rs[s] = lam * rs[s] + kv
                ro[b] = (f64(q[b])[:, :, None] * rs[s]).sum(1) * Dk ** -0.5
                mo[b] = (f64(q[b]).abs()[:, :, None] * ms[s]).sum(1) * Dk ** -0.5
        gate(o, ro, mo, dtype=dtype, terms=Dk, name="o")
        gate(state, rs, ms, dtype=F32, terms=1, name="state")
    same = lib.linattn_step(q, k, v, decay, state.clone(), None)
    assert same.shape == (B, H, Dv)


def test_linattn_gradient_against_differences(lib):
    """fp32: the change of L = <dout, o> + <dhT, hT> along a random direction, by
    central differences of the forward. L is bilinear in each operand, so the
    difference quotient has no truncation error, only that of fp32 sums."""
    q, k, v, do, h0, dh = lin_inputs(1, 90, 2, 64, 64, F32, 13)
    g = decays(2)
    grads = lib.linattn_bwd(q, k, v, g, do, h0, None, dh)

    def loss(args):
        o, hT = lib.linattn_fwd(*args[:3], g, args[3])
        return float((o.double() * do.double()).sum() + (hT.double() * dh.double()).sum())

    for i in range(4):
        ins = [q, k, v, h0]
        d = normal(gen(20 + i), *ins[i].shape)
        up, down = list(ins), list(ins)
        up[i], down[i] = ins[i] + d, ins[i] - d
        num = (loss(up) - loss(down)) / 2
        exact = float((grads[i].double() * d.double()).sum())
        size = float(grads[i].double().norm() * d.double().norm())
        assert abs(num - exact) <= 1e-4 * size, (i, num, exact)


# ---------------------------------------------------------------------------
# sliding-window attention
# ---------------------------------------------------------------------------

def win_inputs(B, Tq, Tk, Hq, Hk, D, dtype, seed):
    g = gen(seed)
    q, do = normal(g, B, Tq, Hq, D, dtype=dtype), normal(g, B, Tq, Hq, D, dtype=dtype)
    k, v = normal(g, B, Tk, Hk, D, dtype=dtype), normal(g, B, Tk, Hk, D, dtype=dtype)
    return q, k, v, do


def win_check(lib, ins, W, S, cu=None, mode="plain", scale=None):
    q, k, v, do = ins
    dtype, D, sc = q.dtype, q.shape[-1], q.shape[-1] ** -0.5 if scale is None else scale
    view = [framed(t, mode) for t in (q, k, v, do)]
    o, lse = lib.window_attn_fwd(*view[:3], W, S, cu, scale=scale)
    dq, dk, dv = lib.window_attn_bwd(*view[:3], o, lse, view[3], W, S, cu, scale=scale)
    torch.cuda.synchronize()
    assert lib.scan_get_device_status() == lib.SCAN_OK
    a, c = [f64(t) for t in (q, k, v)], None if cu is None else cu.cpu()
    ro, rl = ref.window(*a, W, S, c, sc)
    mo, _ = ref.window(a[0], a[1], a[2].abs(), W, S, c, sc)
    # a score's own error: D products; it moves every weight of its row by as much
    smag = float(sc * (a[0].norm(dim=-1).max() if a[0].numel() else 0) * (a[1].norm(dim=-1).max() if a[1].numel() else 0))
    terms = min(q.shape[1] + k.shape[1], 2 * W + S) + D + 2 * D * max(1.0, smag)
    r = 1 if dtype == BF else 0
    gate(o, ro, mo, dtype=dtype, roundings=r, terms=terms, name="o")
    gate(lse, rl, torch.full_like(rl, max(1.0, smag)), dtype=F32, terms=terms, name="lse")
    (rg, mg) = ref.window_grads(*a, f64(do), W, S, c, sc)
    for got, want, mag, name in zip((dq, dk, dv), rg, mg, ("dq", "dk", "dv")):
        gate(got, want, mag, dtype=dtype, roundings=r, terms=terms, name=name)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 2, 31, 64, 127, 128, 129, 257, 400])
def test_window_lengths(lib, dtype, T):
    for D, W, S in ((64, 1 << 40, 0), (128, 100, 4)):
        win_check(lib, win_inputs(1, T, T, 2, 1, D, dtype, T + D), W, S)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W,S", [(1, 0), (1, 3), (5, 0), (64, 1), (127, 130), (128, 0), (129, 16), (200, 300),
                                 (1000, 5)])
def test_window_masks(lib, dtype, W, S):
    win_check(lib, win_inputs(1, 520, 520, 2, 2, 64, dtype, W + S), W, S)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hk,D", [(1, 1, 8), (4, 1, 64), (6, 2, 96), (5, 5, 40), (8, 1, 128), (3, 1, 120)])
def test_window_heads(lib, dtype, Hq, Hk, D):
    win_check(lib, win_inputs(2, 200, 200, Hq, Hk, D, dtype, Hq + D), 70, 4, scale=0.2)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 1), (4, 2)])
@pytest.mark.parametrize("W,S", [(16, 1), (100, 4), (129, 16), (300, 4), (150, 300)])
def test_window_first_tokens_and_gaps(lib, Hq, Hk, W, S):
    """Rows long enough that first tokens and window lie tiles apart, heads of 128
    in blocks of one and of two heads: tiles that one query tile passes over."""
    for Tq, Tk in ((900, 900), (513, 1100)):
        win_check(lib, win_inputs(1, Tq, Tk, Hq, Hk, 128, BF, W + S + Hq), W, S)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Tq,Tk", [(1, 300), (100, 300), (130, 257), (300, 100), (5, 0), (0, 5), (200, 1)])
def test_window_fewer_or_more_queries_than_keys(lib, dtype, Tq, Tk):
    """The queries are the last Tq of Tk positions; those before the first key
    see nothing and get zeros."""
    win_check(lib, win_inputs(1, Tq, Tk, 2, 1, 64, dtype, Tq + Tk), 90, 3)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mode", ["wide", "odd"])
def test_window_strides(lib, dtype, mode):
    win_check(lib, win_inputs(2, 190, 190, 2, 1, 64, dtype, 8), 60, 2, mode=mode)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lengths", [[1], [0, 5, 0], [130, 1, 127, 0, 256, 70], [300, 1, 1, 40]])
def test_window_packed(lib, dtype, lengths):
    T = sum(lengths)
    win_check(lib, win_inputs(1, T, T, 4, 2, 64, dtype, T), 100, 4, cu=offsets(lengths))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_window_sequences_do_not_leak(lib, dtype):
    lengths = [150, 77, 200]
    cu = offsets(lengths)
    q, k, v, do = win_inputs(1, sum(lengths), sum(lengths), 2, 1, 64, dtype, 10)
    def run():
        o, lse = lib.window_attn_fwd(q, k, v, 64, 4, cu)
        return (o, lse.transpose(1, 2)) + lib.window_attn_bwd(q, k, v, o, lse, do, 64, 4, cu)
    want = run()
    for t in (q, k, v, do):
        t[:, 150:227] = NAN
    got = run()
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a[:, :150], b[:, :150]) and torch.equal(a[:, 227:], b[:, 227:]), i


@pytest.mark.parametrize("dtype", [BF, F32])
def test_window_large_scores(lib, dtype):
    """Scores in the hundreds: the running maximum must carry them; one key then
    holds nearly all of a row's weight."""
    q, k, v, do = win_inputs(1, 300, 300, 1, 1, 64, dtype, 14)
    o, lse = lib.window_attn_fwd(q, k, v, 200, 4, scale=20.0)
    ro, rl = ref.window(f64(q), f64(k), f64(v), 200, 4, None, 20.0)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    # a score of up to 20 * 64 * 4 is 64 2^-24 of itself off: 2e-2
    assert float((f64(lse) - rl).abs().max()) <= 2e-2
    assert float((f64(o) - ro).norm() / ro.norm()) <= 2e-2


def test_window_gradient_against_differences(lib):
    """fp32, central differences along a random direction; the step leaves a
    truncation error of its square and a rounding error of 2^-24 / step."""
    q, k, v, do = win_inputs(1, 150, 150, 2, 1, 64, F32, 15)
    o, lse = lib.window_attn_fwd(q, k, v, 60, 3)
    grads = lib.window_attn_bwd(q, k, v, o, lse, do, 60, 3)
    eps = 2.0 ** -7
    for i in range(3):
        d = normal(gen(30 + i), *(q, k, v)[i].shape)
        vals = []
        for sgn in (1, -1):
            ins = [q, k, v]
            ins[i] = ins[i] + sgn * eps * d
            vals.append(float((lib.window_attn_fwd(*ins, 60, 3)[0].double() * do.double()).sum()))
        num = (vals[0] - vals[1]) / (2 * eps)
        exact = float((grads[i].double() * d.double()).sum())
        size = float(grads[i].double().norm() * d.double().norm())
        assert abs(num - exact) <= 1e-3 * size, (i, num, exact)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hk,D", [(1, 1, 8), (4, 1, 64), (6, 2, 96), (16, 4, 128), (20, 1, 128), (3, 1, 120)])
@pytest.mark.parametrize("W,S", [(1, 0), (16, 1), (50, 3), (300, 4), (1100, 17)])
def test_window_step(lib, dtype, Hq, Hk, D, W, S):
    """From the first token to far past the window; rows that are not filled hold NaN."""
    g = gen(D + W)
    C, G = W + S, Hq // Hk
    pos = [0, 1, W - 1, W, C - 1, C, C + 1, 3 * C + 7, -1, 5]
    B = len(pos)
    q, k, v = (normal(g, B, h, D, dtype=dtype) for h in (Hq, Hk, Hk))
    kc, vc = (normal(g, B + 1, C, Hk, D, dtype=dtype) for _ in range(2))
    slots = torch.randperm(B + 1, generator=g)[:B].to(torch.int32)
    slots[9] = B + 1  # idle, as the negative position is
    for b, (s, p) in enumerate(zip(slots.tolist(), pos)):
        if s <= B and 0 <= p < C:
            kc[s, p:], vc[s, p:] = NAN, NAN
    rk, rv = f64(kc), f64(vc)
    o = lib.window_attn_step(q, k, v, kc, vc, torch.tensor(pos, dtype=torch.int32, device=DEV), W, S, slots.to(DEV))
    for b, (s, p) in enumerate(zip(slots.tolist(), pos)):
        if s > B or p < 0:
            assert float(o[b].abs().max()) == 0.0
            continue
        at = p if p < S else S + (p - S) % W
        rk[s, at], rv[s, at] = f64(k[b]), f64(v[b])
        n = min(p + 1, C)
        kk, vv = (x[s, :n].repeat_interleave(G, 1) for x in (rk, rv))
        sc = torch.einsum("hd,nhd->hn", f64(q[b]), kk) * D ** -0.5
        w = torch.softmax(sc, -1)
        smag = max(1.0, float(f64(q[b]).norm(dim=-1).max() * kk.norm(dim=-1).max()) * D ** -0.5)
        gate(o[b], torch.einsum("hn,nhd->hd", w, vv), torch.einsum("hn,nhd->hd", w, vv.abs()), dtype=dtype,
             roundings=1 if dtype == BF else 0, terms=n + D + 2 * D * smag, name=f"o {p}")
    for got, want in ((kc, rk), (vc, rv)):
        assert torch.equal(torch.nan_to_num(f64(got), nan=9e9), torch.nan_to_num(want, nan=9e9))


@pytest.mark.parametrize("B,Hq,Hk,D", [(130, 16, 4, 128), (240, 4, 2, 64), (90, 40, 4, 64), (500, 3, 1, 72)])
def test_window_step_many_requests(lib, B, Hq, Hk, D):
    """More (request, key head) pairs than run at once: key heads share a block."""
    g = gen(B)
    W, S, G = 90, 3, Hq // Hk
    C = W + S
    q, k, v = (normal(g, B, h, D, dtype=BF) for h in (Hq, Hk, Hk))
    kc, vc = (normal(g, B, C, Hk, D, dtype=BF) for _ in range(2))
    pos = torch.randint(-1, 3 * C, (B,), generator=g)
    rk, rv = f64(kc), f64(vc)
    o = lib.window_attn_step(q, k, v, kc, vc, pos.to(torch.int32).to(DEV), W, S).cpu()
    live = pos >= 0
    at = torch.where(pos < S, pos, S + (pos - S) % W)[live]
    rk[live, at], rv[live, at] = f64(k)[live], f64(v)[live]
    kk, vv = (x.repeat_interleave(G, 2) for x in (rk, rv))
    sc = torch.einsum("bhd,bnhd->bhn", f64(q), kk) * D ** -0.5
    sc = sc.masked_fill(torch.arange(C) > pos[:, None, None], float("-inf"))
    w = torch.softmax(sc[live], -1)
    smag = max(1.0, float(f64(q).norm(dim=-1).max() * kk.norm(dim=-1).max()) * D ** -0.5)
    gate(o[live], torch.einsum("bhn,bnhd->bhd", w, vv[live]), torch.einsum("bhn,bnhd->bhd", w, vv[live].abs()),
         dtype=BF, roundings=1, terms=C + D + 2 * D * smag, name="o")
    assert float(o[~live].abs().sum()) == 0.0
    assert torch.equal(f64(kc), rk) and torch.equal(f64(vc), rv)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_window_steps_equal_the_prompt(lib, dtype):
    """Tokens one at a time through the ring give what the whole row gives."""
    B, T, W, S = 2, 90, 20, 3
    q, k, v, _ = win_inputs(B, T, T, 4, 2, 64, dtype, 16)
    whole, _ = lib.window_attn_fwd(q, k, v, W, S)
    kc = torch.full((B, W + S, 2, 64), NAN, dtype=dtype, device=DEV)
    vc = kc.clone()
    rows = [lib.window_attn_step(q[:, t], k[:, t], v[:, t], kc, vc,
                                 torch.full((B,), t, dtype=torch.int32, device=DEV), W, S) for t in range(T)]
    got = torch.stack(rows, 1)
    assert float((got - whole).double().norm() / whole.double().norm()) <= 3 * (U16 if dtype == BF else 128 * U32)


# ---------------------------------------------------------------------------
# all of them
# ---------------------------------------------------------------------------

def calls(lib, dtype):
    """Every entry point on small operands: {name: call(out, stream)}, and the
    outputs each returns."""
    g = gen(40)
    cos, sin = tables(200, 64)
    w = [normal(g, 64) for _ in range(2)]
    q, k, do = (normal(g, 1, 140, 4, 64, dtype=dtype) for _ in range(3))
    v = normal(g, 1, 140, 4, 64, dtype=dtype)
    dec = decays(4)
    h0 = normal(g, 1, 4, 64, 64)
    o, lse = lib.window_attn_fwd(q, k, v, 50, 4)
    kc, vc = normal(g, 3, 54, 4, 64, dtype=dtype), normal(g, 3, 54, 4, 64, dtype=dtype)
    state = normal(g, 3, 4, 64, 64)
    pos = torch.tensor([7, 60, 200], dtype=torch.int32, device=DEV)
    tok = [normal(g, 3, 4, 64, dtype=dtype) for _ in range(3)]
    return {
        "rope": lambda out=None, s=None: lib.qk_norm_rope_fwd(q, k, *w, cos, sin, out=out, stream=s),
        "rope_bwd": lambda out=None, s=None: lib.qk_norm_rope_bwd(q, k, *w, cos, sin, do, v, out=out, stream=s),
        "lin": lambda out=None, s=None: lib.linattn_fwd(q, k, v, dec, h0, out=out, stream=s),
        "lin_bwd": lambda out=None, s=None: lib.linattn_bwd(q, k, v, dec, do, h0, out=out, stream=s),
        "lin_step": lambda out=None, s=None: (lib.linattn_step(*tok, dec, state.clone(), out=out and out[0], stream=s),),
        "win": lambda out=None, s=None: lib.window_attn_fwd(q, k, v, 50, 4, out=out, stream=s),
        "win_bwd": lambda out=None, s=None: lib.window_attn_bwd(q, k, v, o, lse, do, 50, 4, out=out, stream=s),
        "win_step": lambda out=None, s=None: (lib.window_attn_step(*tok, kc, vc, pos, 50, 4, out=out and out[0], stream=s),),
    }


@pytest.mark.parametrize("dtype", [BF, F32])
def test_outputs_stay_in_their_bounds_and_repeat(lib, dtype):
    """Outputs given as slices of larger buffers: what lies around them is left
    alone, and the results are those of a call that allocates them, bit for bit."""
    for name, call in calls(lib, dtype).items():
        want = call()
        bufs = [torch.full((t.numel() + 512,), 77.0, dtype=t.dtype, device=DEV) for t in want]
        outs = tuple(b[256:256 + t.numel()].view(t.shape) for b, t in zip(bufs, want))
        call(outs)
        torch.cuda.synchronize()
        for b, o, t in zip(bufs, outs, want):
            assert torch.equal(o, t), name
            assert bool((b[:256] == 77).all()) and bool((b[-256:] == 77).all()), name


@pytest.mark.parametrize("dtype", [BF, F32])
def test_other_streams(lib, dtype):
    """Calls on a stream of their own, after the work that makes their inputs."""
    side = torch.cuda.Stream()
    for name, call in calls(lib, dtype).items():
        want = call()
        side.wait_stream(torch.cuda.current_stream())
        got = call(s=side)
        with torch.cuda.stream(side):
            again = call()
        side.synchronize()
        for a, b, c in zip(got, want, again):
            assert torch.equal(a, b) and torch.equal(c, b), name


def test_refusals(lib):
    q = torch.zeros(1, 8, 2, 64, device=DEV, dtype=BF)
    dec = torch.zeros(2, device=DEV)
    cos, sin = tables(16, 64)
    tok = q[:, 0]
    state = torch.zeros(1, 2, 64, 64, device=DEV)
    cache = torch.zeros(1, 12, 2, 64, device=DEV, dtype=BF)
    pos = torch.zeros(1, dtype=torch.int32, device=DEV)
    for bad, err in (
        (lambda: lib.qk_norm_rope_fwd(q.half(), q.half(), None, None, cos, sin), TypeError),
        (lambda: lib.qk_norm_rope_fwd(q, q.float(), None, None, cos, sin), TypeError),
        (lambda: lib.qk_norm_rope_fwd(q[0], q[0], None, None, cos, sin), ValueError),
        (lambda: lib.qk_norm_rope_fwd(q, q, None, None, cos, None), ValueError),
        (lambda: lib.qk_norm_rope_fwd(q, q, None, None, *tables(16, 128)), lib.ScanError),
        (lambda: lib.qk_norm_rope_fwd(q, q, None, None, *tables(16, 12)), lib.ScanError),
        (lambda: lib.qk_norm_rope_fwd(q, q, None, None, cos, sin, eps=-1.0), lib.ScanError),
        (lambda: lib.qk_norm_rope_fwd(q.transpose(2, 3), q, None, None, cos, sin), ValueError),
        (lambda: lib.qk_norm_rope_fwd(q[..., :20], q[..., :20], None, None, None, None), lib.ScanError),
        (lambda: lib.qk_norm_rope_fwd(torch.zeros(1, 8, 2, 70, device=DEV, dtype=BF)[..., 3:67], q, None, None, cos, sin), lib.ScanError),
        (lambda: lib.qk_norm_rope_fwd(q, q, None, None, cos, sin, out=(q[:, :1].expand(-1, 8, -1, -1), q)), ValueError),
        (lambda: lib.linattn_fwd(q, q, q, dec.double()), TypeError),
        (lambda: lib.linattn_fwd(q, q[:, :4], q, dec), ValueError),
        (lambda: lib.linattn_fwd(q, q, q, torch.zeros(3, device=DEV)), ValueError),
        (lambda: lib.linattn_fwd(q, q, q, dec, scale=0.0), lib.ScanError),
        (lambda: lib.linattn_fwd(q, q, q, dec, scale=float("nan")), lib.ScanError),
        (lambda: lib.linattn_fwd(q[..., :20], q[..., :20], q, dec), lib.ScanError),
        (lambda: lib.linattn_fwd(*[torch.zeros(1, 8, 2, 256, device=DEV, dtype=BF)] * 3, dec), lib.ScanError),
        (lambda: lib.linattn_fwd(q.expand(2, -1, -1, -1), q.expand(2, -1, -1, -1), q.expand(2, -1, -1, -1), dec, None, pos), ValueError),
        (lambda: lib.linattn_fwd(q, q, q, dec, state.double()), TypeError),
        (lambda: lib.linattn_bwd(q, q, q, dec, q[:, :3]), ValueError),
        (lambda: lib.linattn_step(tok, tok, tok, dec, state.expand(2, -1, -1, -1)), ValueError),
        (lambda: lib.linattn_step(tok.expand(3, -1, -1), tok.expand(3, -1, -1), tok.expand(3, -1, -1), dec, state), lib.ScanError),
        (lambda: lib.linattn_step(tok, tok, tok, dec, state[:, :1].contiguous()), ValueError),
        (lambda: lib.window_attn_fwd(q, q, q, 0), lib.ScanError),
        (lambda: lib.window_attn_fwd(q, q, q, 4, -1), lib.ScanError),
        (lambda: lib.window_attn_fwd(q[:, :, :1].expand(-1, -1, 3, -1), q, q, 4), lib.ScanError),
        (lambda: lib.window_attn_fwd(q, q[:, :4], q, 4), ValueError),
        (lambda: lib.window_attn_fwd(q, q[:, :4], q[:, :4], 4, 0, pos), (ValueError, lib.ScanError)),
        (lambda: lib.window_attn_fwd(q, q, q, 4, scale=-1.0), lib.ScanError),
        (lambda: lib.window_attn_step(tok, tok, tok, cache, cache, pos, 9, 2), ValueError),
        (lambda: lib.window_attn_step(tok, tok, tok, cache, cache.float(), pos, 10, 2), TypeError),
        (lambda: lib.window_attn_step(tok, tok, tok, cache, cache, pos.long(), 10, 2), TypeError),
        (lambda: lib.window_attn_step(tok, tok, tok, cache, cache, pos, 12, 0, scale=float("inf")), lib.ScanError),
    ):
        with pytest.raises(err):
            bad()
    torch.cuda.synchronize()
