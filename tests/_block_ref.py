"""Plain 64-bit forms of attention to another sequence, of the norms around a block
and of dropout from a counter-based generator."""

from __future__ import annotations

import math

import torch


def spans(B, Tq, Tk, lens=None, cu_q=None, cu_k=None):
    """(batch row, queries from, to, keys from, to) of every sequence."""
    if cu_q is not None:
        q, k = cu_q.tolist(), cu_k.tolist()
        return [(0, q[i], q[i + 1], k[i], k[i + 1]) for i in range(len(q) - 1)]
    n = [Tk] * B if lens is None else lens.tolist()
    return [(b, 0, Tq, 0, n[b]) for b in range(B)]


def cross(q, k, v, scale, seqs):
    """Returns o, lse and the magnitude sum_j p |v|."""
    B, Tq, Hq, D = q.shape
    G = Hq // k.shape[2] if k.shape[2] else 1
    o, mag = torch.zeros(2, B, Tq, Hq, D, dtype=torch.float64)
    lse = torch.full((B, Hq, Tq), -math.inf, dtype=torch.float64)
    for b, qa, qe, ka, ke in seqs:
        if ke == ka:
            continue
        for h in range(Hq):
            s = (q[b, qa:qe, h] @ k[b, ka:ke, h // G].T) * scale
            p = torch.softmax(s, -1)
            o[b, qa:qe, h], mag[b, qa:qe, h] = p @ v[b, ka:ke, h // G], p @ v[b, ka:ke, h // G].abs()
            lse[b, h, qa:qe] = torch.logsumexp(s, -1)
    return o, lse, mag


def cross_grads(q, k, v, dout, scale, seqs):
    """(dq, dk, dv) from the formulas, and the magnitudes of the sums they are: of p and ds
    with their terms, and of an error of delta by one rounding of the output."""
    Hq, G = q.shape[2], q.shape[2] // k.shape[2] if k.shape[2] else 1
    dq, dk, dv, mq, mk, mv = (torch.zeros_like(x) for x in (q, k, v, q, k, v))
    for b, qa, qe, ka, ke in seqs:
        if ke == ka:
            continue
        for h in range(Hq):
            qh, kh, vh, dh = q[b, qa:qe, h], k[b, ka:ke, h // G], v[b, ka:ke, h // G], dout[b, qa:qe, h]
            p = torch.softmax((qh @ kh.T) * scale, -1)
            dp = dh @ vh.T
            delta = (p * dp).sum(-1, keepdim=True)
            ds = p * (dp - delta) * scale
            mds = p * ((dp - delta).abs() + dh.abs() @ vh.abs().amax(0)[:, None]) * scale
            dq[b, qa:qe, h], mq[b, qa:qe, h] = ds @ kh, mds @ kh.abs()
            dk[b, ka:ke, h // G] += ds.T @ qh
            mk[b, ka:ke, h // G] += mds.T @ qh.abs()
            dv[b, ka:ke, h // G] += p.T @ dh
            mv[b, ka:ke, h // G] += p.T @ dh.abs()
    return (dq, dk, dv), (mq, mk, mv)


def philox(c, k):
    """The four words of a counter of four and a key of two, after ten rounds, in Python's
    whole numbers."""
    c, k = list(c), list(k)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xffffffff, (a >> 32) ^ c[3] ^ k[1], a & 0xffffffff]
        k = [(k[0] + 0x9E3779B9) & 0xffffffff, (k[1] + 0xBB67AE85) & 0xffffffff]
    return c


def numbers(n, seed, call, first=0):
    """The generator's 16-bit numbers of n elements from block `first` on."""
    out = []
    for block in range(first, first + (n + 7) // 8):
        for w in philox((block & 0xffffffff, block >> 32, call & 0xffffffff, call >> 32),
                        (seed & 0xffffffff, seed >> 32)):
            out += [w & 0xffff, w >> 16]
    return torch.tensor(out[:n], dtype=torch.int64)


def kept(shape, p, rng):
    """0 where an element is dropped, else 1 / (1 - p) of the p that is applied."""
    limit = round(p * 65536)
    factor = 65536.0 / (65536 - limit) if limit < 65536 else 0.0
    return (numbers(math.prod(shape), *rng) >= limit).double().view(shape) * factor


def rms(x, w, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w


def block(x, y, w_post, gate, alpha, eps, keep):
    """The stream after a block (differentiable). x, y [B, T, C]."""
    z = y if w_post is None else rms(y, w_post, eps)
    if gate is not None:
        z = z * (gate[:, None] if gate.dim() == 2 else gate)
    return alpha * x + (z if keep is None else z * keep)
