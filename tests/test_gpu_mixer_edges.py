"""The token mixers at the edges of what their entry points accept: offsets that
name more rows than there are, an epsilon of zero, values that are not finite,
workspaces shared by calls of different sizes."""

import struct

import pytest
import torch

import _mixer_ref as ref
from _mixer_ref import f64, gate
from test_gpu_mixers import (BF, DEV, F32, calls, decays, gen, lin_inputs, normal, offsets, tables, win_check,
                             win_inputs)

pytestmark = pytest.mark.gpu


def view4(t):
    return struct.pack("Pqqq", t.data_ptr(), *t.stride()[:3])


@pytest.mark.parametrize("T,H,D,times", [(8192, 2, 64, 2), (65536, 1, 128, 4), (16384, 3, 128, 15)])
def test_linattn_overlapping_offsets_stay_in_the_workspace(lib, T, H, D, times):
    """Offsets 0, T, 0, T, ...: every second sequence holds the whole row, so that
    their segments add up to more than the workspace has room for. The status
    says so, and what lies past the workspace's reported size is left alone."""
    cu = torch.tensor([0, T] * times, dtype=torch.int32, device=DEV)
    n = 2 * times - 1
    q, k, v, do, _, _ = lin_inputs(1, T, H, D, D, BF, T + H, n=n, state=False)
    g = torch.full((H,), -0.01, device=DEV)
    size = lib.linattn_workspace_bytes(1, T, H, D, D, n)
    past = 3 * times * (T // 128) * H * D * D * 4  # every segment of four chunks that the offsets name, and more
    buf = torch.full((size + past,), 0x5a, dtype=torch.uint8, device=DEV)
    o, dq, dk, dv = (torch.empty_like(t) for t in (v, q, k, v))
    hT, dh0 = (torch.empty(n, H, D, D, device=DEV) for _ in range(2))
    raw, s = lib.lib(), torch.cuda.current_stream().cuda_stream
    for run in ("fwd", "bwd"):
        assert raw.scan_workspace_init(buf.data_ptr(), size, s) == lib.SCAN_OK
        if run == "fwd":
            st = raw.linattn_fwd(view4(q), view4(k), view4(v), g.data_ptr(), None, cu.data_ptr(), n, view4(o),
                                 hT.data_ptr(), 1, T, H, D, D, 1.0, lib.SCAN_BF16, buf.data_ptr(), size, s)
        else:
            st = raw.linattn_bwd(view4(q), view4(k), view4(v), g.data_ptr(), None, cu.data_ptr(), n, view4(do),
                                 hT.data_ptr(), view4(dq), view4(dk), view4(dv), dh0.data_ptr(), 1, T, H, D, D, 1.0,
                                 lib.SCAN_BF16, buf.data_ptr(), size, s)
        assert st == lib.SCAN_OK
        assert raw.scan_get_device_status(buf.data_ptr(), s) == lib.SCAN_ERR_SEQLENS
        assert bool((buf[size:] == 0x5a).all()), run


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,Hq,Hk,D", [(1, 3, 1, 1, 64), (2, 7, 5, 1, 96), (1, 33, 2, 6, 128), (3, 5, 4, 3, 256)])
def test_qk_norm_rope_without_epsilon(lib, dtype, B, T, Hq, Hk, D):
    """eps = 0: heads and tokens that only fill up a group of lanes have no norm,
    and add nothing to the weights' gradients of the ones that are there."""
    g = gen(D + T)
    x = [normal(g, B, T, h, D, dtype=dtype) for h in (Hq, Hk)]
    dy = [normal(g, B, T, h, D, dtype=dtype) for h in (Hq, Hk)]
    w = [normal(g, D) + 1.0 for _ in range(2)]
    cos, sin = tables(T, D)
    y = lib.qk_norm_rope_fwd(*x, *w, cos, sin, eps=0.0)
    d = lib.qk_norm_rope_bwd(*x, *w, cos, sin, *dy, eps=0.0)
    pos = torch.arange(T).expand(B, T)
    for m in range(2):
        xr, wr = f64(x[m]).requires_grad_(), f64(w[m]).requires_grad_()
        yr = ref.qk_norm_rope(xr, wr, f64(cos), f64(sin), pos, 0.0, False)
        dxr, dwr = torch.autograd.grad((yr * f64(dy[m])).sum(), (xr, wr))
        r = 1 / torch.sqrt((f64(x[m]) ** 2).mean(-1, keepdim=True))
        n = f64(x[m]) * r
        # terms: the two products of a pair; D of the norm's sum
        zmag = (n * wr.detach()).abs().amax(-1, keepdim=True)
        gate(y[m], yr.detach(), zmag.expand_as(yr), dtype=dtype, terms=D, name="y")
        gmag = 2 * f64(dy[m]).abs().amax(-1, keepdim=True) * wr.detach().abs().amax()
        mag = (r * gmag * (1 + n.abs() * n.abs().mean(-1, keepdim=True))).expand_as(dxr)
        gate(d[m], dxr, mag, dtype=dtype, terms=D, name="dx")
        dwmag = (2 * f64(dy[m]).abs().amax(-1, keepdim=True) * n.abs()).sum((0, 1, 2))
        gate(d[2 + m], dwr, dwmag, dtype=F32, terms=D, name="dw")


def test_two_threads_on_one_stream(lib):
    """Calls of growing size from two threads on one stream, whose workspace grows
    under them: each gives what it gives alone."""
    import threading
    sizes = [(1, 1000 + 700 * i, 4 + i) for i in range(8)]
    work = []
    for B, T, H in sizes:
        q, k, v, do, _, _ = lin_inputs(B, T, H, 64, 64, BF, T, state=False)
        work.append((q, k, v, torch.full((H,), -0.02, device=DEV), do))
    want = [lib.linattn_bwd(*w) for w in work]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, errors = [None] * len(work), []

    def run(which):
        try:
            for i in which:
                with torch.cuda.stream(side):
                    got[i] = lib.linattn_bwd(*work[i])
        except Exception as e:  # noqa: BLE001 - shown below
            errors.append(e)

    threads = [threading.Thread(target=run, args=(range(r, len(work), 2),)) for r in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    side.synchronize()
    assert not errors
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert lib.scan_get_device_status(stream=side) == lib.SCAN_OK


@pytest.mark.parametrize("name", ["rope", "rope_bwd", "lin", "lin_bwd", "lin_step", "win", "win_bwd", "win_step"])
def test_captured_calls(lib, name):
    """Each call in a CUDA graph: replays give what the call gives, also after a
    larger call on the same stream has replaced the workspace that they use, and
    leave the memory that is handed out since alone."""
    call = calls(lib, BF)[name]
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = call()
    for t in got:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q, k, v, do, _, _ = lin_inputs(1, 9000, 8, 128, 128, BF, 1, state=False)
        lib.linattn_bwd(q, k, v, torch.full((8,), -0.1, device=DEV), do)
        # as many small blocks as the freed workspace could have become
        since = [torch.full((1024,), 0x5a, dtype=torch.uint8, device=DEV) for _ in range(2000)]
        graph.replay()
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert all(bool((t == 0x5a).all()) for t in since)
    assert lib.scan_get_device_status(stream=side) == lib.SCAN_OK


def test_findings_of_scans_and_mixers(lib):
    """A scan and a token mixer with malformed offsets: both findings are reported."""
    bad = torch.tensor([0, 40, 30], dtype=torch.int32, device=DEV)
    assert lib.scan_get_device_status() == lib.SCAN_OK
    q = lin_inputs(1, 30, 2, 64, 64, BF, 3, state=False)[0]
    lib.window_attn_fwd(q, q, q, 8, 0, bad)
    a = torch.rand(4, 30, device=DEV)
    lib.scan_fwd(a, a, None, bad)
    assert [lib.scan_get_device_status() for _ in range(3)] == [lib.SCAN_ERR_SEQLENS] * 2 + [lib.SCAN_OK]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", [[0, 90, 20, 300], [-7, 90, 300], [0, 90, 299], [0, 301]])
def test_window_backward_reports_malformed_offsets(lib, dtype, bad):
    q, k, v, do = (normal(gen(i), 1, 300, 2, 64, dtype=dtype) for i in range(4))
    o, lse = lib.window_attn_fwd(q, k, v, 50, 2)
    assert lib.scan_get_device_status() == lib.SCAN_OK
    lib.window_attn_bwd(q, k, v, o, lse, do, 50, 2, torch.tensor(bad, dtype=torch.int32, device=DEV))
    assert [lib.scan_get_device_status() for _ in range(2)] == [lib.SCAN_ERR_SEQLENS, lib.SCAN_OK]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [7, 300, 1500])
def test_linattn_decay_of_nan_shows(lib, dtype, T):
    """A decay that is no number makes its head's outputs, states and gradients no
    numbers, whichever path the length takes, and leaves the other heads alone."""
    q, k, v, do, h0, dh = lin_inputs(1, T, 3, 64, 64, dtype, T)
    good, bad = torch.full((3,), -0.1, device=DEV), torch.tensor([-0.1, float("nan"), -0.1], device=DEV)
    want = lib.linattn_fwd(q, k, v, good, h0) + lib.linattn_bwd(q, k, v, good, do, h0, None, dh)
    got = lib.linattn_fwd(q, k, v, bad, h0) + lib.linattn_bwd(q, k, v, bad, do, h0, None, dh)
    for i, (a, b) in enumerate(zip(got, want)):
        axis = 1 if i in (1, 5) else 2  # states are [B, H, K, V]
        one, other = (t.movedim(axis, 0) for t in (a, b))
        assert torch.equal(one[[0, 2]], other[[0, 2]]), i
        if i in (3, 4):  # dk, dv: only the last step's have nothing of a later one
            assert one[1].isnan()[:, :-1].all(), i
        else:
            assert one[1].isnan().all(), i


@pytest.mark.parametrize("dtype", [BF, F32])
def test_window_scores_that_overflow_show(lib, dtype):
    """A score of +inf (finite queries and keys whose product is too large) gives NaN
    in its row's output and statistic, not the -inf of a row that sees nothing."""
    q, k, v = (normal(gen(i), 1, 100, 2, 64, dtype=dtype) for i in range(3))
    want = lib.window_attn_fwd(q, k, v, 20, 0)
    q[0, 60, 1], k[0, 60, 1] = 1e25, 1e25
    o, lse = lib.window_attn_fwd(q, k, v, 20, 0)
    assert o[0, 60, 1].isnan().all() and bool(lse[0, 1, 60].isnan())
    assert torch.equal(o[0, :60], want[0][0, :60]) and torch.equal(lse[0, :, :60], want[1][0, :, :60])
    assert torch.equal(o[0, 80:], want[0][0, 80:]) and torch.equal(lse[0, 0], want[1][0, 0])


@pytest.mark.parametrize("T", [15, 16, 31, 32])
@pytest.mark.parametrize("D,B", [(32, 30), (32, 80), (64, 80)])
def test_linattn_short_rows(lib, T, D, B):
    """Both sides of the length at which rows go by chunks, for few and many rows of
    small heads: 16 steps, or 32."""
    q, k, v, do, h0, dh = lin_inputs(B, T, 6, D, D, BF, T + B)
    keep = [0, B // 2, B - 1]
    few = lambda t: t[keep]  # noqa: E731
    g = decays(6)
    o, hT = lib.linattn_fwd(q, k, v, g, h0)
    grads = lib.linattn_bwd(q, k, v, g, do, h0, None, dh)
    args = [f64(few(t)) for t in (q, k, v)]
    mags = [t.abs() for t in args]
    ro, rh = ref.linattn(*args, f64(g), f64(few(h0)), None, D ** -0.5)
    mo, mh = ref.linattn(*mags, f64(g), f64(few(h0)).abs(), None, D ** -0.5)
    rg = ref.linattn_grads(*args, f64(g), f64(few(do)), f64(few(h0)), f64(few(dh)), None, D ** -0.5)
    mg = ref.linattn_grads(*mags, f64(g), *(f64(few(t)).abs() for t in (do, h0, dh)), None, D ** -0.5)
    # one rounding of a weight or of the state as it is read; the states by chunks: their
    # update's operand in two bf16 parts at least, 2^-17 off
    gate(few(o), ro, mo, dtype=BF, roundings=1, terms=T + D, name="o")
    gate(few(hT), rh, mh, dtype=F32, terms=T + D + 2 ** 7, name="hT")
    for got, want, mag, name in zip(grads, rg, mg, ("dq", "dk", "dv", "dh0")):
        if name == "dh0":
            gate(few(got), want, mag, dtype=F32, terms=T + D + 2 ** 7, name=name)
        else:
            gate(few(got), want, mag, dtype=BF, roundings=1, terms=T + D, name=name)


@pytest.mark.parametrize("K,V", [(64, 64), (128, 64), (64, 128), (128, 128), (96, 40)])
@pytest.mark.parametrize("T,at", [(16, 0), (16, 15), (100, 31), (128, 64), (300, 7), (300, 299), (5000, 1203)])
def test_linattn_states_are_exact_to_fp32(lib, K, V, T, at):
    """A row with one value row that is not zero: its last state is that step's product
    times a power of the decay, a sum of one term, and so is the gradient of the
    initial state for one output gradient. In units of 2^-24 of the element: two for
    each unit of the power's exponent (the rounded log of the decay and its product
    with the steps), 16 for the exponential, the weights and the three adds of the
    term's three bf16 parts, 8 a chunk for the powers that the state is multiplied
    with. A term of two parts would be up to 128 off."""
    H = 5
    g = -torch.tensor([0.0, 1e-4, 3e-3, 0.02, 0.1], device=DEV) * min(1.0, 300 / T)
    k, q = normal(gen(T), 1, T, H, K, dtype=BF), normal(gen(T + 1), 1, T, H, K, dtype=BF)
    v, do = torch.zeros(1, T, H, V, dtype=BF, device=DEV), torch.zeros(1, T, H, V, dtype=BF, device=DEV)
    v[:, at], do[:, at] = normal(gen(T + 2), 1, H, V, dtype=BF), normal(gen(T + 3), 1, H, V, dtype=BF)
    _, hT = lib.linattn_fwd(q, k, v, g, scale=0.5)
    dh0 = lib.linattn_bwd(q, k, v, g, do, scale=0.5)[3]
    for got, x, y, n, mul in ((hT, k, v, T - 1 - at, 1.0), (dh0, q, do, at + 1, 0.5)):
        power = (f64(g) * n)[:, None, None]
        want = mul * power.exp() * f64(x[0, at])[:, :, None] * f64(y[0, at])[:, None, :]
        units = 2 * power.abs() + 16 + 8 * (T // 128 + 1)
        bad = (f64(got[0]) - want).abs() > units * 2.0 ** -24 * want.abs() + 1e-37
        assert not bad.any(), (int(bad.sum()), float(((f64(got[0]) - want).abs() / want.abs().clamp(min=1e-37)).max()) * 2 ** 24)


@pytest.mark.parametrize("lengths", [[1], [130, 1, 127, 0, 256, 70], [300, 1, 1, 400], [513, 900]])
@pytest.mark.parametrize("Hq,Hk,W,S", [(1, 1, 64, 0), (4, 2, 100, 4), (3, 1, 129, 130)])
def test_window_packed_heads_of_128(lib, lengths, Hq, Hk, W, S):
    T = sum(lengths)
    win_check(lib, win_inputs(1, T, T, Hq, Hk, 128, BF, T + W), W, S, cu=offsets(lengths))


@pytest.mark.parametrize("T,W,S,lengths", [(64, 1000, 0, None), (200, 1000, 4, None), (512, 1000, 4, None), (900, 20, 4, None),
                                           (378, 138, 4, [20, 100, 60, 150, 48]), (1500, 300, 0, [500, 31, 469, 500])])
@pytest.mark.parametrize("D", [64, 96, 128])
def test_window_gradients_where_rows_see_few_keys(lib, T, W, S, lengths, D):
    """dq and dk in the 2-norm against 64 bits: the rounding of the result to bf16, and
    what a delta from the rounded output leaves, both taken from the exact values;
    a tenth more for all else, which 32 bits hold. One more rounding, of dS, would add
    as much as the first."""
    cu = None if lengths is None else offsets(lengths)
    q, k, v, do = win_inputs(1, T, T, 6, 2, D, BF, T + D)
    o, lse = lib.window_attn_fwd(q, k, v, W, S, cu)
    got = lib.window_attn_bwd(q, k, v, o, lse, do, W, S, cu)
    args, c, scale = [f64(t) for t in (q, k, v, do)], None if cu is None else cu.cpu(), D ** -0.5
    want, _ = ref.window_grads(*args, W, S, c, scale)
    ro, _ = ref.window(*args[:3], W, S, c, scale)
    # a change of delta_i by e_i changes dq_i by -e_i sum_j p_ij k_j scale, and dk alike:
    # the gradients of sum (e_i log-sum-exp_i)
    e = ((ro.to(BF).double() - ro) * args[3]).sum(-1).transpose(1, 2)  # [B, Hq, T]
    leaves = [args[0].clone().requires_grad_(), args[1].clone().requires_grad_()]
    loss = 0.0
    for _, lo, hi in ref.sequences(1, T, c):
        s = torch.einsum("ihd,jhd->hij", leaves[0][0, lo:hi], leaves[1][0, lo:hi].repeat_interleave(3, 1)) * scale
        s = s.masked_fill(~ref.visible(hi - lo, hi - lo, W, S), -torch.inf)
        loss = loss + (torch.logsumexp(s, -1) * e[0, :, lo:hi]).sum()
    moved = torch.autograd.grad(loss, leaves)
    for g, w, m, name in zip(got, want, moved, ("dq", "dk")):
        rounded = float((w.to(BF).double() - w).norm() / w.norm())
        limit = 1.1 * (rounded ** 2 + float(m.norm() / w.norm()) ** 2) ** 0.5
        err = float((f64(g) - w).norm() / w.norm())
        assert err <= limit, (name, err, limit, rounded)


@pytest.mark.parametrize("lengths", [[19], [2, 2, 3], [6, 1, 12], [128], [9, 127, 64, 1, 33]])
@pytest.mark.parametrize("Hq,Hk,D", [(2, 1, 64), (3, 3, 128)])
@pytest.mark.parametrize("W,S", [(1000, 0), (35, 16), (5, 0)])
def test_window_gradients_of_a_few_tokens(lib, lengths, Hq, Hk, D, W, S):
    """dq and dk in the 2-norm against 64 bits: rows that see one tile of keys have
    nothing but the rounding of the result to bf16 (and a tenth of it for all else)."""
    T, cu = sum(lengths), offsets(lengths)
    q, k, v, do = win_inputs(1, T, T, Hq, Hk, D, BF, T + D)
    o, lse = lib.window_attn_fwd(q, k, v, W, S, cu)
    got = lib.window_attn_bwd(q, k, v, o, lse, do, W, S, cu)
    want, _ = ref.window_grads(*[f64(t) for t in (q, k, v, do)], W, S, cu.cpu(), D ** -0.5)
    for g, w, name in zip(got, want, ("dq", "dk")):
        rounded = float((w.to(BF).double() - w).norm() / w.norm())
        err = float((f64(g) - w).norm() / w.norm())
        assert err <= 1.1 * rounded, (name, err, rounded)


def chunked(q, k, v, g, h0, scale):
    """The recurrence in 64 bits, 256 steps at a time: o, hT."""
    o, S = [], h0
    i = torch.arange(256, dtype=torch.float64, device=q.device)
    for t in range(0, q.shape[1], 256):
        a, b, c = (x[0, t:t + 256].double().transpose(0, 1) for x in (q, k, v))  # [H, n, D]
        n = a.shape[1]
        w = torch.exp(g[:, None, None] * (i[:n, None] - i[:n]).clamp(min=0)).tril()
        o.append((a @ S) * torch.exp(g[:, None] * (i[:n] + 1))[..., None] + (a @ b.transpose(1, 2) * w) @ c)
        S = S * torch.exp(g * n)[:, None, None] + (b * torch.exp(g[:, None] * (n - 1 - i[:n]))[..., None]).transpose(1, 2) @ c
    return scale * torch.cat(o, 1).transpose(0, 1)[None], S


@pytest.mark.parametrize("T", [100, 3000])
def test_linattn_recurrence_keeps_slow_decays(lib, T):
    """fp32, memories of 20 to 260 steps: outputs, gradients and states in the 2-norm of
    each head against 64 bits. An entry is rounded twice a step over a memory of 1 / (1 -
    lambda) steps: 2^-25 each (root mean square at most) that add up as their squares,
    times 4; and 2^-22 for the sums of D products. The rounding of lambda would add
    up to 2^-25 a step of the memory."""
    H, D = 12, 64
    q, k, v, do, h0, dh = lin_inputs(1, T, H, D, D, F32, T)
    g = -torch.logspace(-8, -4.3, H, base=2.0, device=DEV)
    o, hT = lib.linattn_fwd(q, k, v, g, h0, scale=0.5)
    dq, dk, dv, dh0 = lib.linattn_bwd(q, k, v, g, do, h0, None, dh, scale=0.5)
    G = g.double()
    flip = lambda t: t.flip(1)  # noqa: E731
    lam = torch.exp(G)[:, None, None]
    ro, rh = chunked(q, k, v, G, h0[0].double(), 0.5)
    rq, _ = chunked(do, v, k, G, h0[0].double().transpose(1, 2), 0.5)
    init = dh[0].double() / 0.5 / lam  # (comes in not yet decayed)
    rk, _ = chunked(flip(v), flip(do), flip(q), G, init.transpose(1, 2), 0.5)
    rv, end = chunked(flip(k), flip(q), flip(do), G, init, 0.5)
    for got, want, name in ((o, ro, "o"), (dq, rq, "dq"), (dk, flip(rk), "dk"), (dv, flip(rv), "dv"),
                            (hT[0], rh, "hT"), (dh0[0], 0.5 * lam * end, "dh0")):
        got = got.double()
        axes = (0, 1, 3) if got.dim() == 4 else (1, 2)
        err = (got - want).square().sum(axes).sqrt() / want.square().sum(axes).sqrt()
        limit = 4 * 2.0 ** -25 * (2 / (1 - torch.exp(G))).clamp(max=2 * T).sqrt() + 2.0 ** -22
        assert bool((err <= limit).all()), (name, (err / limit).tolist())


def test_linattn_recurrence_over_a_million_steps(lib):
    """What the rounding of lambda leaves out is settled on the way: the end of a row of
    more than 2^20 steps is that of its last steps alone, whose memory is 260 steps."""
    T, last = (1 << 20) + 700, 20000
    q, k, v, _, _, _ = lin_inputs(1, T, 2, 8, 8, F32, 2, state=False)
    g = -torch.logspace(-8, -6, 2, base=2.0, device=DEV)
    o, hT = lib.linattn_fwd(q, k, v, g)
    po, pT = lib.linattn_fwd(q[:, -last:], k[:, -last:], v[:, -last:], g)
    # both are within the limit of the test above of the exact value
    limit = 2 * (4 * 2.0 ** -25 * (2 * 260) ** 0.5 + 2.0 ** -22)
    assert float((hT - pT).norm() / pT.norm()) <= limit
    assert float((o[:, -600:] - po[:, -600:]).norm() / po[:, -600:].norm()) <= limit


@pytest.mark.parametrize("dtype", [BF, F32])
def test_linattn_steps_keep_slow_decays(lib, dtype):
    """1500 single tokens over memories of 20 to 260: the state that is left against 64
    bits, in the 2-norm of each head, within the limit of the recurrence over a row."""
    H, D, T = 12, 64, 1500
    q, k, v, _, h0, _ = lin_inputs(1, T, H, D, D, dtype, 4)
    g = -torch.logspace(-8, -4.3, H, base=2.0, device=DEV)
    state = h0.clone()
    for t in range(T):
        o = lib.linattn_step(q[:, t], k[:, t], v[:, t], g, state, scale=0.5)
    ro, rh = chunked(q, k, v, g.double(), h0[0].double(), 0.5)
    limit = 4 * 2.0 ** -25 * (2 / (1 - torch.exp(g.double()))).sqrt() + 2.0 ** -22
    err = (state[0].double() - rh).square().sum((1, 2)).sqrt() / rh.square().sum((1, 2)).sqrt()
    assert bool((err <= limit).all()), (err / limit).tolist()
    if dtype == F32:
        err = (o[0].double() - ro[0, -1]).norm() / ro[0, -1].norm()
        assert float(err) <= float(limit.max())
