"""GPU parity of the norms around a block and of dropout against their definitions
in 64 bits."""

import pytest
import torch

import _block_ref as ref
from _mixer_ref import U16, U32, f64, gate
from test_gpu_mixers import BF, DEV, F32, NAN, gen, normal

pytestmark = pytest.mark.gpu

TYPES = [(BF, BF), (F32, BF), (F32, F32)]


def wide(t):
    """The same values as a slice of a larger tensor that holds NaN around them."""
    big = torch.full((t.shape[0], t.shape[1] + 2, t.shape[2] + 16), NAN, dtype=t.dtype, device=t.device)
    out = big[:, 1:-1, 8:-8]
    out.copy_(t)
    return out


def check(lib, B, T, C, types, post, gated, nxt, p=0.0, alpha=1.0, eps=1e-6, strided=False, upstream=True, seed=0):
    st, dt = types
    g = gen(B + T + C + seed)
    x, y = normal(g, B, T, C, dtype=st, mul=2.0), normal(g, B, T, C, dtype=dt, mul=3.0)
    dxo, dn = normal(g, B, T, C, dtype=st), normal(g, B, T, C, dtype=dt)
    wp = normal(g, C) + 1.0 if post else None
    wn = normal(g, C) + 1.0 if nxt else None
    gt = {"none": None, "channel": normal(g, C), "row": normal(g, B, C)}[gated]
    rng = (0x123456789abcdef + seed, 3 + (seed << 33))
    keep = ref.kept((B, T, C), p, rng) if p else None
    if strided:
        x, y, dxo, dn = (wide(t) for t in (x, y, dxo, dn))
    kw = dict(alpha=alpha, eps=eps, p=p, rng=rng)
    xo, n = lib.residual_norm_fwd(x, y, wp, gt, wn, **kw)
    up = dxo if upstream or not nxt else None
    got = lib.residual_norm_bwd(xo, y, up, dn if nxt else None, wp, gt, wn, **kw)
    rx, ry = f64(x), f64(y)
    k = torch.ones(()) if keep is None else keep
    gr = None if gt is None else f64(gt)
    bx = ref.block(rx, ry, f64(wp), gr, alpha, eps, keep)
    mx = (alpha * rx).abs() + (bx - alpha * rx).abs()
    gate(xo, bx, mx, dtype=st, terms=C, name="x_out")
    assert (n is None) == (not nxt)
    sx = f64(xo)
    q = 1 / torch.sqrt((sx * sx).mean(-1, keepdim=True) + eps)
    if nxt:
        want = ref.rms(sx, f64(wn), eps)
        gate(n, want, want.abs(), dtype=dt, terms=C, name="n")
    # the gradients, at the stream as it is stored
    G = f64(dxo) if up is not None else torch.zeros_like(sx)
    Gm = G.abs()
    if nxt:
        e, xh = f64(dn) * f64(wn), sx * q
        G = G + q * (e - xh * (e * xh).mean(-1, keepdim=True))
        Gm = Gm + q * (e.abs() + xh.abs() * (e * xh).abs().mean(-1, keepdim=True))
        gate(got[4], (f64(dn) * xh).sum((0, 1)), (f64(dn) * xh).abs().sum((0, 1)), dtype=F32, terms=B * T + C, name="dw_next")
    gate(got[0], alpha * G, abs(alpha) * Gm, dtype=st, terms=C, name="dx")
    leaves = [t if t is None else t.clone().requires_grad_() for t in (ry, f64(wp), gr)]
    u = ref.block(torch.zeros_like(rx), *leaves, 0.0, eps, keep)
    have = [t for t in leaves if t is not None]
    grads = list(torch.autograd.grad((u * G).sum(), have))
    r = 1 / torch.sqrt((ry * ry).mean(-1, keepdim=True) + eps) if post else torch.ones(B, T, 1)
    gf = torch.ones(1, 1, C) if gr is None else gr.abs().view(-1, 1, C)
    f = Gm * k * gf * (f64(wp).abs() if post else 1.0)
    yh = (ry * r).abs()
    gate(got[1], grads.pop(0), r * (f + (yh * (f * yh).mean(-1, keepdim=True) if post else 0.0)), dtype=dt, terms=2 * C,
         name="dy")
    if post:
        gate(got[2], grads.pop(0), (Gm * k * gf * yh).sum((0, 1)), dtype=F32, terms=B * T + 2 * C, name="dw_post")
    if gr is not None:
        m = Gm * k * yh * (f64(wp).abs() if post else 1.0)
        gate(got[3], grads.pop(0), m.sum(1) if gated == "row" else m.sum((0, 1)), dtype=F32, terms=B * T + 2 * C, name="dgate")
    assert [t is None for t in got[2:]] == [not post, gr is None, not nxt]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("C", [8, 64, 200, 256, 264, 512, 520, 1000, 1536, 2048, 2056, 4096, 4104, 8192])
def test_widths(lib, types, C):
    check(lib, 2, 9, C, types, True, "channel", True, p=0.1, alpha=0.7)
    check(lib, 1, 1, C, types, True, "none", True)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gated", ["none", "channel", "row"])
@pytest.mark.parametrize("nxt", [True, False])
def test_parts(lib, types, post, gated, nxt):
    check(lib, 3, 37, 136, types, post, gated, nxt, p=0.3, alpha=0.9)
    check(lib, 3, 5, 1032, types, post, gated, nxt, strided=True, upstream=False)


@pytest.mark.parametrize("gated", ["channel", "row"])
@pytest.mark.parametrize("B,T", [(1, 1), (1, 3000), (700, 1), (613, 2), (5, 401), (2, 1023)])
def test_rows(lib, gated, B, T):
    """More and fewer rows, and batch rows, than blocks."""
    check(lib, B, T, 64, (F32, BF), True, gated, True, p=0.25, alpha=1.1)
    check(lib, B, T, 24, (BF, BF), False, gated, True)


def test_dropout_extremes(lib):
    """p = 1 drops everything; a p below a step of 2^-16 nothing."""
    check(lib, 2, 5, 64, (F32, BF), True, "channel", True, p=1.0)
    check(lib, 2, 5, 64, (F32, BF), True, "channel", True, p=1e-6)


def test_norm_alone(lib):
    """Without a block: the norm in front of the first one."""
    for st, dt in TYPES:
        g = gen(3)
        x, dx, dn, w = normal(g, 2, 7, 96, dtype=st), normal(g, 2, 7, 96, dtype=st), normal(g, 2, 7, 96, dtype=dt), normal(g, 96)
        same, n = lib.residual_norm_fwd(x, None, next_weight=w, dtype=dt)
        assert same is x and n.dtype == dt
        rx, rw = f64(x).requires_grad_(), f64(w).requires_grad_()
        want = ref.rms(rx, rw, 1e-6)
        gate(n, want.detach(), want.detach().abs(), dtype=dt, terms=96, name="n")
        d = lib.residual_norm_bwd(x, None, dx, dn, next_weight=w)
        ex, ew = torch.autograd.grad((want * f64(dn)).sum() + (rx * f64(dx)).sum(), (rx, rw))
        xh = (want / rw).detach().abs()
        q = 1 / torch.sqrt((f64(x) ** 2).mean(-1, keepdim=True) + 1e-6)
        e = (f64(dn) * f64(w)).abs()
        gate(d[0], ex, f64(dx).abs() + q * (e + xh * (e * xh).mean(-1, keepdim=True)), dtype=st, terms=96, name="dx")
        gate(d[4], ew, (f64(dn).abs() * xh).sum((0, 1)), dtype=F32, terms=110, name="dw")
        assert d[1] is None and d[2] is None and d[3] is None


def test_single_tokens_and_in_place(lib):
    """[B, C] operands are rows of one token; outputs may take the inputs' place."""
    g = gen(4)
    x, y, w = normal(g, 6, 512), normal(g, 6, 512, dtype=BF), normal(g, 512)
    gt = normal(g, 6, 512)
    want = lib.residual_norm_fwd(x[:, None], y[:, None], w, gt, w)
    got = lib.residual_norm_fwd(x, y, w, gt, w)
    assert all(torch.equal(a, b[:, 0]) for a, b in zip(got, want))
    dx, dn = normal(g, 6, 512), normal(g, 6, 512, dtype=BF)
    grads = lib.residual_norm_bwd(got[0], y, dx, dn, w, gt, w)
    x2, y2, dx2, dn2 = (t.clone() for t in (x, y, dx, dn))
    out = lib.residual_norm_fwd(x2, y2, w, gt, w, out=(x2, y2))
    assert out[0] is x2 and out[1] is y2 and torch.equal(x2, got[0]) and torch.equal(y2, got[1])
    lib.residual_norm_bwd(got[0], y, dx2, dn2, w, gt, w, out=(dx2, dn2) + grads[2:])
    assert torch.equal(dx2, grads[0]) and torch.equal(dn2, grads[1])


def test_no_rows(lib):
    w = torch.ones(64, device=DEV)
    for B, T in ((0, 5), (3, 0)):
        x, y = torch.empty(B, T, 64, device=DEV), torch.empty(B, T, 64, device=DEV, dtype=BF)
        assert lib.residual_norm_fwd(x, y, w, w, w)[1].shape == (B, T, 64)
        for gt in (w, torch.ones(B, 64, device=DEV)):
            d = lib.residual_norm_bwd(x, y, x, y, w, gt, w)
            assert all(float(t.abs().sum()) == 0.0 for t in d[2:])


def test_no_epsilon_and_small_rows(lib):
    """eps = 0 at rows of 1e-15, the third power of whose norms fp32 does not hold: the
    results and gradients stay finite."""
    g = gen(6)
    for C in (64, 2048):
        x, y = normal(g, 1, 3, C, mul=1e-15), normal(g, 1, 3, C, mul=1e-15)
        w = normal(g, C)
        xo, n = lib.residual_norm_fwd(x, y, w, None, w, alpha=0.0, eps=0.0)
        gate(xo, ref.rms(f64(y), f64(w), 0.0), f64(xo).abs(), dtype=F32, terms=C, name="z")
        d = lib.residual_norm_bwd(x, y, None, normal(g, 1, 3, C), w, None, w, eps=0.0)
        assert all(bool(t.isfinite().all()) for t in d if t is not None)


def test_repeatable(lib):
    g = gen(7)
    x, y, dn, w = normal(g, 4, 500, 1536), normal(g, 4, 500, 1536, dtype=BF), normal(g, 4, 500, 1536, dtype=BF), normal(g, 1536)
    first = lib.residual_norm_bwd(x, y, x, dn, w, w, w, p=0.1, rng=(1, 2))
    for _ in range(3):
        again = lib.residual_norm_bwd(x, y, x, dn, w, w, w, p=0.1, rng=(1, 2))
        assert all(torch.equal(a, b) for a, b in zip(first, again))


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (37, 1537), (2, 3, 40), (5, 1, 8, 3), (9, 4099)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout(lib, dtype, shape, p):
    x = normal(gen(len(shape)), *shape, dtype=dtype)
    rng = (0xfedcba9876543210, (1 << 40) + 5)
    keep = ref.kept(shape, p, rng)
    for call in (lib.dropout_fwd, lib.dropout_bwd):
        y = call(x, p, rng)
        gate(y, f64(x) * keep, (f64(x) * keep).abs(), dtype=dtype, terms=1, name="y")  # (the factor and the product)
        assert bool(((y == 0) == ((keep == 0).to(DEV) | (x == 0))).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_dropout_is_the_same_at_any_stride(lib, dtype):
    """The mask goes by an element's place in the shape, however it lies."""
    g = gen(2)
    for B, T, C in ((3, 5, 64), (2, 7, 33), (1, 9, 8), (4, 1, 40)):
        x = normal(g, B, T, C, dtype=dtype)
        want = lib.dropout_fwd(x, 0.4, (7, 9))
        assert torch.equal(lib.dropout_fwd(wide(x), 0.4, (7, 9)), want)
        off = torch.empty(x.numel() + 1, dtype=dtype, device=DEV)[1:].view(x.shape)
        assert lib.dropout_fwd(wide(x), 0.4, (7, 9), out=off) is off and torch.equal(off, want)
        big = torch.full((B, T, C + 5), NAN, dtype=dtype, device=DEV)
        lib.dropout_fwd(x, 0.4, (7, 9), out=big[..., 3:C + 3])
        assert torch.equal(big[..., 3:C + 3], want) and big[..., :3].isnan().all() and big[..., C + 3:].isnan().all()
        assert torch.equal(lib.dropout_fwd(x, 0.4, (7, 9), out=x), want)


def test_dropped_elements_are_zero_whatever_they_hold(lib):
    for dtype in (BF, F32):
        x = torch.full((1000,), NAN, dtype=dtype, device=DEV)
        keep = ref.kept((1000,), 0.5, (1, 1)).to(DEV)
        assert bool((lib.dropout_fwd(x, 0.5, (1, 1)).isnan() == (keep != 0)).all())
        y = lib.residual_norm_fwd(torch.zeros(1, 8, 1000, device=DEV, dtype=dtype),
                                  x.expand(1, 8, 1000).contiguous(), p=1.0, rng=(1, 1))[0]
        assert float(y.abs().max()) == 0.0


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("C", [64, 1000, 4104])
@pytest.mark.parametrize("gated", ["none", "channel", "row"])
def test_what_is_dropped_leaves_no_trace_in_the_gradients(lib, types, C, gated):
    """Infinities and NaN of the block where its dropout falls (and no norm has taken them in
    before): results and gradients are the same bits as with zeros there."""
    st, dt = types
    g = gen(C)
    x, dxo = (normal(g, 2, 9, C, dtype=st) for _ in range(2))
    y, dn = (normal(g, 2, 9, C, dtype=dt) for _ in range(2))
    wn, gt = normal(g, C), {"none": None, "channel": normal(g, C), "row": normal(g, 2, C)}[gated]
    kw = dict(p=0.3, rng=(8, 2), alpha=0.9)
    gone = (ref.kept((2, 9, C), 0.3, (8, 2)) == 0).to(DEV)
    odd = torch.tensor([NAN, float("inf"), -float("inf")], device=DEV)[torch.arange(2 * 9 * C, device=DEV) % 3].view(2, 9, C)
    results = []
    for fill in (torch.zeros_like(y), odd.to(dt)):
        z = torch.where(gone, fill, y)
        xo, n = lib.residual_norm_fwd(x, z, None, gt, wn, **kw)
        results.append((xo, n, *lib.residual_norm_bwd(xo, z, dxo, dn, None, gt, wn, **kw)))
    for a, b in zip(*results):
        assert (a is None) == (b is None)
        assert a is None or (torch.equal(a, b) and bool(a.isfinite().all()))


def test_dropout_statistics(lib):
    """Of 2^22 elements the kept ones are a binomial number, those of other calls and seeds
    independent: five standard deviations."""
    n = 1 << 22
    x = torch.ones(n, device=DEV)
    for p in (0.1, 0.5):
        masks = [lib.dropout_fwd(x, p, rng) != 0 for rng in ((1, 0), (1, 1), (2, 0), (1, 1 << 32), (1 << 32, 0))]
        sd = (p * (1 - p) / n) ** 0.5
        for i, a in enumerate(masks):
            assert abs(float(a.double().mean()) - (1 - p)) <= 5 * sd
            for b in masks[:i]:
                both = float((a & b).double().mean())
                q = (1 - p) ** 2
                assert abs(both - q) <= 5 * (q * (1 - q) / n) ** 0.5
        assert abs(float((masks[0][1:] & masks[0][:-1]).double().mean()) - (1 - p) ** 2) <= 10 * sd


def test_random_state_on_the_device(lib):
    """The same mask as of whole numbers; a captured graph draws anew as the state changes."""
    g = gen(5)
    x, y, w = normal(g, 2, 6, 64), normal(g, 2, 6, 64, dtype=BF), normal(g, 64)
    state = torch.tensor([-3, 5], dtype=torch.int64, device=DEV)
    seed = (1 << 64) - 3
    assert torch.equal(lib.dropout_fwd(x, 0.5, state), lib.dropout_fwd(x, 0.5, (seed, 5)))
    want = [lib.residual_norm_fwd(x, y, w, None, w, p=0.5, rng=(seed, c)) for c in range(5, 8)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lib.residual_norm_fwd(x, y, w, None, w, p=0.5, rng=state)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = lib.residual_norm_fwd(x, y, w, None, w, p=0.5, rng=state)
        state[1] += 1
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i])), i


def test_dropout_past_32_bits(lib):
    """Elements past 2^32 have blocks and places of their own."""
    n = (1 << 32) + 8 * 1000 + 3
    x = torch.ones(n, dtype=BF, device=DEV)
    y = lib.dropout_fwd(x, 0.5, (3, 4), out=x)
    blocks = ref.numbers(64, 3, 4)
    assert torch.equal((y[:64] != 0).cpu(), blocks >= 32768)
    # the last elements, from their own counter
    first = (n // 8) * 8
    words = _block(first // 8, 3, 4)
    assert torch.equal((y[first:] != 0).cpu(), torch.tensor(words[:n - first]) >= 32768)


def _block(block, seed, call):
    c, k = [block & 0xffffffff, block >> 32, call, 0], [seed, 0]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xffffffff, (a >> 32) ^ c[3] ^ k[1], a & 0xffffffff]
        k = [(k[0] + 0x9E3779B9) & 0xffffffff, (k[1] + 0xBB67AE85) & 0xffffffff]
    return [v for w in c for v in (w & 0xffff, w >> 16)]
