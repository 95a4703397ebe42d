"""GPU parity of attention to another sequence against its definition in 64 bits:
lengths from one up, odd sizes, shared heads, strides, padded and packed batches,
sequences without keys or queries, and values past a length that must not be used."""

import math

import pytest
import torch

import _block_ref as ref
from _mixer_ref import U16, U32, f64, gate
from test_gpu_mixers import BF, DEV, F32, NAN, framed, gen, normal, offsets

pytestmark = pytest.mark.gpu


def inputs(B, Tq, Tk, Hq, Hk, D, dtype, seed):
    g = gen(seed)
    return tuple(normal(g, B, T, H, D, dtype=dtype) for T, H in ((Tq, Hq), (Tk, Hk), (Tk, Hk), (Tq, Hq)))


def ints(*values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def check(lib, ins, lens=None, cu_q=None, cu_k=None, mode="plain", scale=None):
    q, k, v, do = ins
    dtype, (B, Tq, Hq, D), Tk = q.dtype, q.shape, k.shape[1]
    sc = D ** -0.5 if scale is None else scale
    view = [framed(t, mode) for t in (q, k, v, do)]
    seqs = ref.spans(B, Tq, Tk, lens, cu_q, cu_k)
    if lens is not None:  # what lies past a length is never used
        view = [t if t is not x else t.clone() for t, x in zip(view, ins)]
        for b, n in enumerate(lens.tolist()):
            view[1][b, n:], view[2][b, n:] = NAN, NAN
    o, lse = lib.cross_attn_fwd(*view[:3], lens, cu_q, cu_k, scale=scale)
    grads = lib.cross_attn_bwd(*view[:3], o, lse, view[3], lens, cu_q, cu_k, scale=scale)
    torch.cuda.synchronize()
    assert lib.scan_get_device_status() == lib.SCAN_OK
    a = [f64(t) for t in (q, k, v)]
    ro, rl, mo = ref.cross(*a, sc, seqs)
    # a score's own error: D products; it moves every weight of its row by as much
    top = [float(t.norm(dim=-1).max()) if t.numel() else 0.0 for t in a[:2]]
    smag = max(1.0, sc * top[0] * top[1])
    terms = Tq + Tk + D + 2 * D * smag
    r = 1 if dtype == BF else 0
    gate(o, ro, mo, dtype=dtype, roundings=r, terms=terms, name="o")
    gate(lse, rl, torch.full_like(rl, smag), dtype=F32, terms=terms, name="lse")
    want, mag = ref.cross_grads(*a, f64(do), sc, seqs)
    for got, w, m, name in zip(grads, want, mag, ("dq", "dk", "dv")):
        gate(got, w, m, dtype=dtype, roundings=r, terms=terms, name=name)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Tq,Tk", [(1, 1), (1, 300), (300, 1), (2, 127), (64, 128), (127, 129), (129, 64), (255, 257),
                                   (257, 512), (130, 700), (513, 65)])
def test_lengths(lib, dtype, Tq, Tk):
    for D in (64, 128):
        check(lib, inputs(1, Tq, Tk, 2, 1, D, dtype, Tq + Tk + D))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hk,D", [(1, 1, 8), (4, 1, 64), (6, 2, 96), (5, 5, 40), (8, 1, 128), (3, 1, 120)])
def test_heads(lib, dtype, Hq, Hk, D):
    check(lib, inputs(2, 150, 201, Hq, Hk, D, dtype, Hq + D), scale=0.2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mode", ["wide", "odd"])
def test_strides(lib, dtype, mode):
    check(lib, inputs(2, 140, 90, 4, 2, 64, dtype, 5), mode=mode)
    check(lib, inputs(2, 33, 190, 2, 2, 128, dtype, 6), lens=ints(190, 7), mode=mode)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(4, 2), (3, 1), (2, 2)])
def test_padded(lib, dtype, D, Hq, Hk):
    """Lengths at the edges of tiles, of one, of none."""
    check(lib, inputs(8, 70, 300, Hq, Hk, D, dtype, D + Hq), lens=ints(300, 0, 1, 127, 128, 129, 256, 257))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,Hq,Hk", [(64, 4, 2), (128, 3, 1), (96, 2, 2)])
def test_packed(lib, dtype, D, Hq, Hk):
    """Empty sequences on either side, single steps, tiles that end inside."""
    lq, lk = [0, 1, 130, 0, 5, 128, 300, 17], [40, 129, 0, 0, 1, 256, 3, 131]
    check(lib, inputs(1, sum(lq), sum(lk), Hq, Hk, D, dtype, D), cu_q=offsets(lq), cu_k=offsets(lk))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_short_sequences(lib, dtype):
    g = gen(9)
    lq, lk = ([int(x) for x in torch.randint(0, 12, (70,), generator=g)] for _ in range(2))
    check(lib, inputs(1, sum(lq), sum(lk), 2, 1, 64, dtype, 9), cu_q=offsets(lq), cu_k=offsets(lk))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_nothing_to_do(lib, dtype):
    """No keys at all, no queries, no heads, no batch rows."""
    for B, Tq, Tk, Hq, Hk in ((2, 5, 0, 4, 2), (2, 0, 5, 4, 2), (0, 5, 5, 4, 2), (1, 5, 5, 0, 0)):
        q, k, v, do = inputs(B, Tq, Tk, Hq, Hk, 64, dtype, 1)
        o, lse = lib.cross_attn_fwd(q, k, v)
        assert not o.numel() or float(o.abs().max()) == 0.0
        assert bool((lse == -math.inf).all()) or not o.numel() or Tk > 0
        for t in lib.cross_attn_bwd(q, k, v, o, lse, do):
            assert not t.numel() or float(t.abs().max()) == 0.0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_malformed_lengths_show(lib, dtype):
    q, k, v, do = inputs(2, 20, 30, 2, 1, 64, dtype, 2)
    want = lib.cross_attn_fwd(q, k, v, ints(30, 0))
    got = lib.cross_attn_fwd(q, k, v, ints(31, -4))
    assert lib.scan_get_device_status() == lib.SCAN_ERR_SEQLENS
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    lib.cross_attn_bwd(q, k, v, *got, do, ints(31, -4))
    assert lib.scan_get_device_status() == lib.SCAN_ERR_SEQLENS
    lib.cross_attn_fwd(q[:1], k[:1], v[:1], None, ints(0, 9, 20), ints(0, 31, 30))
    assert lib.scan_get_device_status() == lib.SCAN_ERR_SEQLENS


def test_large_scores(lib):
    """Scores of several hundred, one key far above the rest: no overflow, no NaN."""
    for dtype in (BF, F32):
        q, k, v, do = inputs(1, 140, 270, 2, 2, 64, dtype, 3)
        check(lib, ((q * 8).to(dtype), (k * 8).to(dtype), v, do), scale=0.5)


def test_results_do_not_change_from_run_to_run(lib):
    q, k, v, do = inputs(2, 700, 900, 4, 2, 128, BF, 4)
    first = lib.cross_attn_fwd(q, k, v)
    for _ in range(3):
        again = lib.cross_attn_fwd(q, k, v)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    grads = lib.cross_attn_bwd(q, k, v, *first, do)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(grads, lib.cross_attn_bwd(q, k, v, *first, do)))


def test_gradients_against_differences(lib):
    """fp32: the loss at inputs moved along a direction, both ways."""
    q, k, v, do = inputs(2, 40, 70, 2, 1, 64, F32, 8)
    lens = ints(70, 31)
    o, lse = lib.cross_attn_fwd(q, k, v, lens)
    grads = lib.cross_attn_bwd(q, k, v, o, lse, do, lens)
    g, h = gen(10), 1e-2
    for i, (x, dx) in enumerate(zip((q, k, v), grads)):
        d = normal(g, *x.shape)
        both = []
        for sign in (1, -1):
            moved = [q, k, v]
            moved[i] = x + sign * h * d
            both.append(float((lib.cross_attn_fwd(*moved, lens)[0].double() * do.double()).sum()))
        want, got = (both[0] - both[1]) / (2 * h), float((dx.double() * d.double()).sum())
        # the loss is a sum of 10^4 terms of order one (2^-24 each, over 2 h) and the third
        # derivative leaves h^2 of the gradient's own size
        size = float(dx.double().norm() * d.double().norm())
        assert abs(want - got) <= 10 * h * h * size + 1e4 * U32 / h, (i, want, got)


# ---------------------------------------------------------------------------
# single tokens
# ---------------------------------------------------------------------------

def step_check(lib, q, kc, vc, lens, slots, scale=None, **kw):
    B, Hq, D = q.shape
    N, Tk, Hk = kc.shape[:3]
    o = lib.cross_attn_step(q, kc, vc, lens, slots, scale=scale, **kw)
    at = range(B) if slots is None else slots.tolist()
    sc = D ** -0.5 if scale is None else scale
    for b, s in enumerate(at):
        n = Tk if lens is None or not 0 <= s < N else min(max(int(lens[s]), 0), Tk)
        if not 0 <= s < N or n == 0:
            assert float(o[b].abs().max()) == 0.0
            continue
        kk, vv = (f64(x[s, :n]).repeat_interleave(Hq // Hk, 1) for x in (kc, vc))
        w = torch.softmax(torch.einsum("hd,nhd->hn", f64(q[b]), kk) * sc, -1)
        smag = max(1.0, float(f64(q[b]).norm(dim=-1).max() * kk.norm(dim=-1).max()) * sc)
        gate(o[b], torch.einsum("hn,nhd->hd", w, vv), torch.einsum("hn,nhd->hd", w, vv.abs()), dtype=q.dtype,
             roundings=1 if q.dtype == BF else 0, terms=n + D + 2 * D * smag, name=f"o {b}")
    return o


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hk,D,Tk", [(1, 1, 8, 1), (4, 2, 64, 40), (16, 4, 128, 300), (12, 12, 96, 77), (20, 1, 64, 700),
                                        (34, 2, 128, 130), (3, 3, 120, 1501)])
def test_step(lib, dtype, Hq, Hk, D, Tk):
    """Lengths from none to all, caches shared by requests, idle ones; rows past a length
    hold NaN."""
    g = gen(D + Tk)
    ns = [0, 1, Tk, max(Tk - 1, 0), (Tk + 1) // 2, min(Tk, 17), Tk + 5, -3]
    N = len(ns)
    q = normal(g, N + 4, Hq, D, dtype=dtype)
    kc, vc = (normal(g, N, Tk, Hk, D, dtype=dtype) for _ in range(2))
    for s, n in enumerate(ns):
        kc[s, max(n, 0):], vc[s, max(n, 0):] = NAN, NAN
    step_check(lib, q, kc, vc, ints(*ns), ints(*torch.randperm(N, generator=g).tolist(), 2, 2, -1, N))
    kv = normal(g, 3, Tk, 2 * Hk, D, dtype=dtype)  # keys and values side by side, requests on their own caches
    step_check(lib, q[:3], kv[:, :, :Hk], kv[:, :, Hk:], None, None, scale=0.1)
    odd = framed(kv, "odd")
    step_check(lib, q[:3], odd[:, :, :Hk], odd[:, :, Hk:], None, None)


@pytest.mark.parametrize("B,Hq,Hk,D", [(130, 16, 4, 128), (240, 4, 2, 64), (90, 40, 4, 64), (500, 3, 1, 72), (70, 16, 16, 128)])
def test_step_many_requests(lib, B, Hq, Hk, D):
    g = gen(B)
    q = normal(g, B, Hq, D, dtype=BF)
    kc, vc = (normal(g, B, 93, Hk, D, dtype=BF) for _ in range(2))
    lens = torch.randint(0, 94, (B,), generator=g).to(torch.int32).to(DEV)
    step_check(lib, q, kc, vc, lens, torch.randperm(B, generator=g).to(torch.int32).to(DEV))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_steps_equal_the_whole_rows(lib, dtype):
    q, k, v, _ = inputs(3, 9, 260, 4, 2, 64, dtype, 16)
    lens = ints(260, 19, 0)
    whole, _ = lib.cross_attn_fwd(q, k, v, lens)
    got = torch.stack([lib.cross_attn_step(q[:, t], k, v, lens) for t in range(9)], 1)
    assert float((got - whole).double().norm() / whole.double().norm()) <= 3 * (U16 if dtype == BF else 128 * U32)


def test_caches_past_32_bits(lib):
    """A pool whose last cache starts past 2^32 elements."""
    N, Tk, Hk, D = 3, 20, 2, 64
    far = 1 << 32
    pool = torch.empty(2 * far + Tk * Hk * D + 8, dtype=BF, device=DEV)
    kc = pool.as_strided((N, Tk, Hk, D), (far, Hk * D, D, 1))
    g = gen(77)
    kc.copy_(normal(g, N, Tk, Hk, D, dtype=BF))
    q = normal(g, N, 4, D, dtype=BF)
    step_check(lib, q, kc, kc, ints(20, 3, 17), ints(2, 0, 1))
    check(lib, (q[:, None].contiguous(), kc, kc, normal(g, N, 1, 4, D, dtype=BF)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("place", [1, 40, 127, 128, 300])
def test_scores_that_grow(lib, D, place):
    """Keys from `place` on score some 200 above those before: the weights of what came
    before are as nothing, and the reference that they were taken from has to move, within
    a tile and between tiles, for some rows only."""
    q, k, v, do = inputs(1, 130, 400, 2, 1, D, BF, place)
    q[..., 0], k[..., 0] = 16.0, 0.0
    q[:, ::3, :, 0] = 0.0
    k[:, place:, :, 0] = 12.5
    check(lib, (q, k, v, do), scale=1.0)


def test_values_that_are_no_numbers_show(lib):
    """A score that overflows makes its own row NaN and leaves the others alone."""
    q, k, v, do = inputs(1, 200, 300, 2, 2, 64, BF, 5)
    want, _ = lib.cross_attn_fwd(q, k, v)
    q[0, 7, 1] = NAN
    got, lse = lib.cross_attn_fwd(q, k, v)
    assert bool(got[0, 7, 1].isnan().all()) and bool(lse[0, 1, 7].isnan())
    rest = torch.ones_like(got, dtype=torch.bool)
    rest[0, 7, 1] = False
    assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_step_of_more_heads_than_a_grid_has_rows(lib, dtype):
    """Requests times heads just above 65535, over a few shared caches."""
    g = gen(21)
    B, Hq, Hk, D, N, Tk = 16387, 4, 2, 64, 5, 40
    q = normal(g, B, Hq, D, dtype=dtype)
    kc, vc = (normal(g, N, Tk, Hk, D, dtype=dtype) for _ in range(2))
    lens = [40, 1, 0, 33, 17]
    slots = torch.randint(-1, N + 1, (B,), generator=g).to(torch.int32)
    o = lib.cross_attn_step(q, kc, vc, ints(*lens), slots.to(DEV))
    o, q64 = f64(o), f64(q)
    for s in range(-1, N + 1):
        at = slots == s
        if not 0 <= s < N or lens[s] == 0:
            assert float(o[at].abs().max()) == 0.0
            continue
        kk, vv = (f64(x[s, :lens[s]]).repeat_interleave(Hq // Hk, 1) for x in (kc, vc))
        w = torch.softmax(torch.einsum("bhd,nhd->bhn", q64[at], kk) * D ** -0.5, -1)
        smag = max(1.0, float(q64[at].norm(dim=-1).max() * kk.norm(dim=-1).max()) * D ** -0.5)
        gate(o[at], torch.einsum("bhn,nhd->bhd", w, vv), torch.einsum("bhn,nhd->bhd", w, vv.abs()), dtype=dtype,
             roundings=1 if dtype == BF else 0, terms=lens[s] + D + 2 * D * smag, name=f"cache {s}")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_query_heads(lib, dtype):
    """Key heads that no query head reads, and key rows that no query does: their gradients are
    sums of nothing, written."""
    for Tq, Hq in ((5, 0), (0, 0), (0, 2)):
        q, k, v, do = inputs(2, Tq, 70, Hq, 2, 64, dtype, 1)
        o, lse = lib.cross_attn_fwd(q, k, v)
        out = torch.empty_like(q), *(torch.full_like(t, NAN) for t in (k, v))
        lib.cross_attn_bwd(q, k, v, o, lse, do, out=out)
        assert all(float(t.abs().max()) == 0.0 for t in out[1:])
    assert lib.scan_get_device_status() == lib.SCAN_OK


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128])
def test_large_values(lib, dtype, D):
    """Values of up to 2^80, also where weights grow before the reference moves (scores that rise
    by four from tile to tile, so that 128 weights add up to 2^13 and more): the same bits as
    without that factor, which is exact."""
    q, k, v, _ = inputs(1, 130, 900, 2, 1, D, dtype, 12)
    v = v.clamp(-1, 1)
    q[..., 0] = 1.0
    k[0, :, :, 0] = (4.0 * (torch.arange(900, device=DEV) // 128) / D ** -0.5)[:, None].to(dtype)
    huge = (v.float() * 2.0 ** 80).to(dtype)
    o, lse = lib.cross_attn_fwd(q, k, v)
    big, same = lib.cross_attn_fwd(q, k, huge)
    assert torch.equal(big.float(), o.float() * 2.0 ** 80) and torch.equal(lse, same)
    o, big = (lib.cross_attn_step(q[:, 5], k, x) for x in (v, huge))
    assert torch.equal(big.float(), o.float() * 2.0 ** 80)
