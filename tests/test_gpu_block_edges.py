"""Attention to another sequence, the norms around a block and dropout at the edges of
what their entry points accept: outputs inside larger buffers, other streams, threads,
captured graphs, broadcast operands, refusals."""

import threading

import pytest
import torch

import _block_ref as ref
from _mixer_ref import f64, gate
from test_gpu_cross import check as cross_check
from test_gpu_cross import inputs, ints
from test_gpu_mixers import BF, DEV, F32, gen, normal, offsets

pytestmark = pytest.mark.gpu


def calls(lib, dtype):
    """Every entry point on small operands: {name: call(out, stream)}."""
    g = gen(41)
    q, k, v, do = inputs(2, 300, 210, 4, 2, 64, dtype, 3)
    lens = ints(210, 90)
    o, lse = lib.cross_attn_fwd(q, k, v, lens)
    tok, slots = normal(g, 5, 4, 64, dtype=dtype), ints(1, 0, 1, 1, 0)
    x, y, dn = normal(g, 3, 70, 136), normal(g, 3, 70, 136, dtype=dtype), normal(g, 3, 70, 136, dtype=dtype)
    w, gt = normal(g, 136), normal(g, 3, 136)
    kw = dict(p=0.2, rng=(4, 5), alpha=0.9)
    return {
        "cross": lambda out=None, s=None: lib.cross_attn_fwd(q, k, v, lens, out=out, stream=s),
        "cross_bwd": lambda out=None, s=None: lib.cross_attn_bwd(q, k, v, o, lse, do, lens, out=out, stream=s),
        "cross_step": lambda out=None, s=None: (lib.cross_attn_step(tok, k, v, lens, slots, out=out and out[0], stream=s),),
        "norm": lambda out=None, s=None: lib.residual_norm_fwd(x, y, w, gt, w, out=out, stream=s, **kw),
        "norm_bwd": lambda out=None, s=None: lib.residual_norm_bwd(x, y, x, dn, w, gt, w, out=out, stream=s, **kw),
        "dropout": lambda out=None, s=None: (lib.dropout_fwd(y, 0.3, (1, 2), out=out and out[0], stream=s),),
        "dropout_bwd": lambda out=None, s=None: (lib.dropout_bwd(y, 0.3, (1, 2), out=out and out[0], stream=s),),
    }


NAMES = ["cross", "cross_bwd", "cross_step", "norm", "norm_bwd", "dropout", "dropout_bwd"]


@pytest.mark.parametrize("dtype", [BF, F32])
def test_outputs_stay_in_their_bounds_and_repeat(lib, dtype):
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


@pytest.mark.parametrize("name", NAMES)
def test_captured_calls(lib, name):
    """Each call in a CUDA graph, replayed after a larger call on the same stream has
    replaced the workspace that it uses, many times over, and by turns with another graph of
    the same call."""
    call = calls(lib, BF)[name]
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs.append(call())
        graphs.append(graph)
    for got in outs:
        for t in got:
            t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q, k, v, do = inputs(2, 900, 1500, 4, 4, 128, BF, 4)
        o, lse = lib.cross_attn_fwd(q, k, v)
        big = lib.cross_attn_bwd(q, k, v, o, lse, do)
        for _ in range(5):
            for graph in graphs:
                graph.replay()
        again = lib.cross_attn_bwd(q, k, v, o, lse, do)
    side.synchronize()
    for got in outs:
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert all(torch.equal(a, b) for a, b in zip(big, again))
    assert lib.scan_get_device_status(stream=side) == lib.SCAN_OK


def test_two_threads_on_one_stream(lib):
    """Calls of growing size from two threads on one stream, whose workspace grows under
    them: each gives what it gives alone."""
    work = []
    for i in range(8):
        q, k, v, do = inputs(1, 200 + 150 * i, 900 - 90 * i, 4, 2, 64, BF, i)
        work.append((q, k, v, *lib.cross_attn_fwd(q, k, v), do))
    want = [lib.cross_attn_bwd(*w) for w in work]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, errors = [None] * len(work), []

    def run(which):
        try:
            for i in which:
                with torch.cuda.stream(side):
                    got[i] = lib.cross_attn_bwd(*work[i])
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


def test_two_streams_at_once(lib):
    """The same calls on two streams side by side, each with its own workspace."""
    all_calls = calls(lib, BF)
    want = {n: c() for n, c in all_calls.items()}
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for s in streams:
            got.append({n: c(s=s) for n, c in all_calls.items()})
    for s in streams:
        s.synchronize()
    for g in got:
        for n in want:
            assert all(torch.equal(a, b) for a, b in zip(g[n], want[n])), n


@pytest.mark.parametrize("dtype", [BF, F32])
def test_broadcast_operands(lib, dtype):
    """One encoder for every row of a batch, one query for every position, one row of a
    stream: operands repeated by a stride of 0."""
    g = gen(6)
    k, v = (normal(g, 1, 90, 2, 64, dtype=dtype).expand(3, -1, -1, -1) for _ in range(2))
    q, do = (normal(g, 3, 40, 4, 64, dtype=dtype) for _ in range(2))
    cross_check(lib, (q, k, v, do))
    cross_check(lib, (q[:, :1].expand(-1, 40, -1, -1), k, v, do), lens=None)
    x, y, w = normal(g, 1, 1, 64), normal(g, 2, 9, 64, dtype=dtype), normal(g, 64)
    got = lib.residual_norm_fwd(x.expand(2, 9, 64), y, w, None, w)
    want = lib.residual_norm_fwd(x.expand(2, 9, 64).contiguous(), y, w, None, w)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    one = torch.ones((), device=DEV, dtype=dtype).expand(2, 9, 64)
    with pytest.raises(ValueError, match="unit stride"):
        lib.residual_norm_bwd(want[0], y, None, one, w, None, w)


def test_many_sequences_and_heads(lib):
    """More sequences than a warp looks up at a time, and a batch of many rows."""
    g = gen(12)
    n = 150
    lq, lk = ([int(x) for x in torch.randint(0, 5, (n,), generator=g)] for _ in range(2))
    cross_check(lib, inputs(1, sum(lq), sum(lk), 4, 4, 32, BF, 1), cu_q=offsets(lq), cu_k=offsets(lk))
    cross_check(lib, inputs(70, 3, 9, 2, 1, 64, BF, 2), lens=torch.randint(0, 10, (70,), generator=g).to(torch.int32).to(DEV))


@pytest.mark.parametrize("mode", ["plain", "odd"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_walks_that_are_cut(lib, dtype, mode):
    """Few queries and many keys, whose walks are cut into pieces (or shares): padded rows of
    lengths at the pieces' ends, none and one, packed pairs with empty sequences."""
    cross_check(lib, inputs(4, 40, 900, 4, 2, 64, dtype, 1), lens=ints(900, 0, 1, 130), mode=mode)
    cross_check(lib, inputs(1, 200, 1500, 3, 1, 96, dtype, 2), cu_q=ints(0, 50, 50, 90, 200),
                cu_k=ints(0, 900, 901, 901, 1500), mode=mode)
    q, k, v, _ = inputs(1, 65, 1000, 2, 1, 128, dtype, 3)
    a, b = (lib.cross_attn_fwd(q, k, v, scale=0.1) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_few_queries_of_many_key_tiles(lib):
    """Key tiles of one or two pairs each, so that shares end within a tile's beginning."""
    for B, Tq, Tk, Hq, Hk in ((1, 5, 20000, 2, 1), (1, 200, 9000, 1, 1), (3, 1, 5000, 4, 4)):
        q, k, v, do = inputs(B, Tq, Tk, Hq, Hk, 64, BF, Tk)
        o, lse = lib.cross_attn_fwd(q, k, v)
        got = lib.cross_attn_bwd(q, k, v, o, lse, do)
        want, _ = ref.cross_grads(f64(q), f64(k), f64(v), f64(do), 64 ** -0.5, ref.spans(B, Tq, Tk))
        # in the 2-norm: an output's rounding 2^-9.2, p's or ds's the same, delta's of o's
        for a, b in zip(got, want):
            assert float((f64(a) - b).norm() / b.norm()) <= 2 ** -8
        again = lib.cross_attn_bwd(q, k, v, o, lse, do)
        assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_long_rows(lib):
    """One head, tens of thousands of keys or queries, against 64 bits on the GPU."""
    for Tq, Tk in ((130, 40000), (40000, 130)):
        q, k, v, do = inputs(1, Tq, Tk, 1, 1, 128, BF, 5)
        o, lse = lib.cross_attn_fwd(q, k, v)
        dq, dk, dv = lib.cross_attn_bwd(q, k, v, o, lse, do)
        a, b, c, d = (t[0, :, 0].double() for t in (q, k, v, do))
        s = a @ b.T * 128 ** -0.5
        p = torch.softmax(s, -1)
        dp = d @ c.T
        ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * 128 ** -0.5
        # in the 2-norm: an output's rounding 2^-9.2, those of p and ds each the same, delta's
        for got, want in ((o, p @ c), (dq, ds @ b), (dk, ds.T @ a), (dv, p.T @ d)):
            assert float((got[0, :, 0].double() - want).norm() / want.norm()) <= 2 ** -8
        assert float((lse[0, 0].double() - torch.logsumexp(s, -1)).abs().max()) <= 1e-5


def test_refusals(lib):
    q = torch.zeros(2, 8, 2, 64, device=DEV, dtype=BF)
    kv = torch.zeros(2, 12, 2, 64, device=DEV, dtype=BF)
    lens, cu = ints(12, 3), ints(0, 8)
    x, w = torch.zeros(2, 4, 64, device=DEV), torch.ones(64, device=DEV)
    y = x.to(BF)
    one = q[:1], kv[:1], kv[:1]
    for bad, err in (
        (lambda: lib.cross_attn_fwd(q.half(), kv.half(), kv.half()), TypeError),
        (lambda: lib.cross_attn_fwd(q, kv.float(), kv), TypeError),
        (lambda: lib.cross_attn_fwd(q[0], kv, kv), ValueError),
        (lambda: lib.cross_attn_fwd(q, kv, kv[:, :5]), ValueError),
        (lambda: lib.cross_attn_fwd(q, kv[:1], kv[:1]), ValueError),
        (lambda: lib.cross_attn_fwd(q, kv, kv, lens[:1]), ValueError),
        (lambda: lib.cross_attn_fwd(q, kv, kv, lens.long()), TypeError),
        (lambda: lib.cross_attn_fwd(q, kv, kv, lens.cpu()), ValueError),
        (lambda: lib.cross_attn_fwd(q[..., :20], kv[..., :20], kv[..., :20]), lib.ScanError),
        (lambda: lib.cross_attn_fwd(q[:, :, :1].expand(-1, -1, 3, -1), kv, kv), lib.ScanError),
        (lambda: lib.cross_attn_fwd(q, kv, kv, scale=0.0), lib.ScanError),
        (lambda: lib.cross_attn_fwd(*one, None, cu), ValueError),
        (lambda: lib.cross_attn_fwd(*one, ints(3), cu, cu), ValueError),
        (lambda: lib.cross_attn_fwd(*one, None, cu, ints(0, 3, 12)), ValueError),
        (lambda: lib.cross_attn_fwd(q, kv, kv, None, cu, cu), ValueError),
        (lambda: lib.cross_attn_fwd(q, kv, kv, out=(q[:, :1].expand(-1, 8, -1, -1), x)), ValueError),
        (lambda: lib.cross_attn_bwd(q, kv, kv, q, x, q), ValueError),
        (lambda: lib.cross_attn_step(q[:, 0], kv, kv[:, :4]), ValueError),
        (lambda: lib.cross_attn_step(q[:, 0], kv, kv, lens[:1]), ValueError),
        (lambda: lib.cross_attn_step(q[:, 0], kv, kv, None, lens[:1]), ValueError),
        (lambda: lib.cross_attn_step(q[:, 0].expand(2, -1, -1), kv[:1], kv[:1]), lib.ScanError),
        (lambda: lib.residual_norm_fwd(x, y[:, :3], w), ValueError),
        (lambda: lib.residual_norm_fwd(y, x, w), lib.ScanError),
        (lambda: lib.residual_norm_fwd(x.half(), y, w), TypeError),
        (lambda: lib.residual_norm_fwd(x, y.half(), w), TypeError),
        (lambda: lib.residual_norm_fwd(x, y, w[:8]), ValueError),
        (lambda: lib.residual_norm_fwd(x, y, w.to(BF)), TypeError),
        (lambda: lib.residual_norm_fwd(x, y, w, torch.ones(3, 64, device=DEV)), ValueError),
        (lambda: lib.residual_norm_fwd(x[..., :20], y[..., :20], None), lib.ScanError),
        (lambda: lib.residual_norm_fwd(x, y, w, p=0.1), ValueError),
        (lambda: lib.residual_norm_fwd(x, y, w, p=1.5, rng=(1, 2)), ValueError),
        (lambda: lib.residual_norm_fwd(x, None), lib.ScanError),
        (lambda: lib.residual_norm_fwd(x, None, next_weight=w, alpha=0.5), lib.ScanError),
        (lambda: lib.residual_norm_fwd(x, y, w, eps=-1.0), lib.ScanError),
        (lambda: lib.residual_norm_bwd(x, y, None, None, w), ValueError),
        (lambda: lib.residual_norm_bwd(x, y, x, None, w, None, w), ValueError),
        (lambda: lib.residual_norm_bwd(x, y, y, None, w), TypeError),
        (lambda: lib.dropout_fwd(x.half(), 0.1, (1, 2)), TypeError),
        (lambda: lib.dropout_fwd(x, 0.1, None), ValueError),
        (lambda: lib.dropout_fwd(x, -0.1, (1, 2)), ValueError),
        (lambda: lib.dropout_fwd(x, 0.1, torch.zeros(2, device=DEV)), TypeError),
        (lambda: lib.dropout_fwd(x, 0.1, torch.zeros(3, dtype=torch.int64, device=DEV)), ValueError),
        (lambda: lib.dropout_fwd(x.transpose(1, 2), 0.1, (1, 2)), ValueError),
        (lambda: lib.dropout_fwd(x, 0.1, (1, 2), out=x[:, :1].expand(-1, 4, -1)), ValueError),
    ):
        with pytest.raises(err):
            bad()
    torch.cuda.synchronize()


def test_dropout_in_the_norm_is_the_dropout(lib):
    """The mask inside the norms around a block is dropout_fwd's of the same numbers."""
    g = gen(8)
    x, y = normal(g, 2, 7, 72), normal(g, 2, 7, 72)
    got, _ = lib.residual_norm_fwd(x, y, p=0.4, rng=(9, 1))
    want = f64(x) + f64(lib.dropout_fwd(y, 0.4, (9, 1)))
    gate(got, want, f64(x).abs() + 2 * f64(y).abs(), dtype=F32, terms=2, name="x_out")
    assert bool(((got == x).cpu() == (ref.kept((2, 7, 72), 0.4, (9, 1)) == 0)).all())
