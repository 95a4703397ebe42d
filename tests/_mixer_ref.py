"""Plain 64-bit forms of the token mixers (norm and rotation, linear attention
with a decay, sliding-window attention), and the error gates that the GPU tests
hold the kernels to. Each gate is a worst case: every term of a sum is rounded
at most `roundings` times to bf16 (8 significant bits: relative 2^-8 each) and the result once, or,
for fp32, accumulates in 32 bits."""

from __future__ import annotations

import math

import torch

U16 = 2.0 ** -8   # bf16's unit roundoff
U32 = 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().double().cpu()


def gate(got, ref, mag, *, dtype, roundings=0, terms=1, name=""):
    """|got - ref| <= u |ref| + (roundings u + terms-sum error) mag, element by
    element; mag is the sum of the magnitudes of the element's terms. fp32 sums
    of `terms` products in any order: (terms + 8) 2^-24 mag (8: the exponential
    or power in each term, and the scale factors)."""
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if not got.numel():
        return
    u = U16 if dtype == torch.bfloat16 else U32
    lim = u * ref.abs() + (roundings * U16 + (terms + 8) * U32) * mag + 1e-30
    same = (got == ref)  # infinities where they belong
    bad = ~((got - ref).abs() <= lim) & ~same
    assert not bad.any(), (name, int(bad.sum()), float(((got - ref).abs() / lim)[bad].max()),
                           got[bad][:4], ref[bad][:4])
    # (where the exact result cancels to nothing, as the gradient of a softmax over
    # one key does, a norm of it measures nothing)
    if roundings and got.numel() >= 4096 and ref.norm() >= 2 ** -6 * mag.expand_as(ref).norm():
        # random roundings (2^-9.2 each, root mean square) add up as their squares: three at most
        fine = torch.isfinite(ref)
        rel = float((got - ref)[fine].norm() / ref[fine].norm().clamp(min=1e-30))
        assert rel <= 1.5 * U16, (name, rel)


# ---------------------------------------------------------------------------

def qk_norm_rope(x, w, cos, sin, pos, eps, interleaved):
    """One of q or k, in 64 bits (differentiable)."""
    D = x.shape[-1]
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    z = n if w is None else n * w
    if cos is None:
        return z
    R = 2 * cos.shape[1]
    c, s = cos[pos.long()][:, :, None], sin[pos.long()][:, :, None]
    if interleaved:
        a, b = z[..., 0:R:2], z[..., 1:R:2]
        y = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = z[..., :R // 2], z[..., R // 2:R]
        y = torch.cat([a * c - b * s, a * s + b * c], -1)
    return torch.cat([y, z[..., R:D]], -1)


def sequences(B, T, cu):
    """(batch row, first step, end) of every sequence."""
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    c = cu.tolist()
    return [(0, c[i], c[i + 1]) for i in range(len(c) - 1)]


def linattn(q, k, v, g, h0, cu, scale):
    """The recurrence, step by step (differentiable). Returns o, hT."""
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    seqs = sequences(B, T, cu)
    lam = torch.exp(g)[:, None, None]
    rows = [[None] * T for _ in range(B)]
    last = []
    for i, (b, lo, hi) in enumerate(seqs):
        S = torch.zeros(H, Dk, Dv, dtype=torch.float64) if h0 is None else h0[i]
        for t in range(lo, hi):
            S = lam * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            rows[b][t] = scale * (q[b, t][:, :, None] * S).sum(1)
        last.append(S)
    zero = torch.zeros(H, Dv, dtype=torch.float64)
    o = torch.stack([torch.stack([zero if r is None else r for r in row]) if row else
                     torch.zeros(0, H, Dv, dtype=torch.float64) for row in rows])
    hT = torch.stack(last) if last else torch.zeros(0, H, Dk, Dv, dtype=torch.float64)
    return o, hT


def linattn_grads(q, k, v, g, dout, h0, dhT, cu, scale):
    """(dq, dk, dv, dh0) by differentiating the recurrence."""
    n = len(sequences(q.shape[0], q.shape[1], cu))
    h = torch.zeros(n, q.shape[2], q.shape[3], v.shape[3], dtype=torch.float64) if h0 is None else h0
    leaves = [x.clone().requires_grad_() for x in (q, k, v, h)]
    o, hT = linattn(leaves[0], leaves[1], leaves[2], g, leaves[3], cu, scale)
    loss = (o * dout).sum()
    if dhT is not None:
        loss = loss + (hT * dhT).sum()
    return torch.autograd.grad(loss, leaves)


def visible(Tq, Tk, W, S):
    i = torch.arange(Tq)[:, None] + (Tk - Tq)
    j = torch.arange(Tk)[None]
    return (j <= i) & ((i - j < W) | (j < S))


def window(q, k, v, W, S, cu, scale):
    """Returns o, lse."""
    B, Tq, Hq, D = q.shape
    Tk, Hk = k.shape[1:3]
    G = Hq // Hk if Hk else 1
    o = torch.zeros(B, Tq, Hq, D, dtype=torch.float64)
    lse = torch.full((B, Hq, Tq), -math.inf, dtype=torch.float64)
    spans = [(b, 0, Tq, 0, Tk) for b in range(B)] if cu is None else \
        [(0, a, e, a, e) for (_, a, e) in sequences(B, Tq, cu)]
    for b, qa, qe, ka, ke in spans:
        m = visible(qe - qa, ke - ka, W, S)
        some = m.any(1)
        for h in range(Hq):
            if not some.any():
                continue
            s = ((q[b, qa:qe, h] @ k[b, ka:ke, h // G].T) * scale).masked_fill(~m, -math.inf)[some]
            o[b, qa:qe, h][some] = torch.softmax(s, -1) @ v[b, ka:ke, h // G]
            lse[b, h, qa:qe][some] = torch.logsumexp(s, -1)
    return o, lse


def window_grads(q, k, v, dout, W, S, cu, scale):
    """(dq, dk, dv) and the magnitudes of the sums they are, from the formulas."""
    B, Tq, Hq, D = q.shape
    Tk, Hk = k.shape[1:3]
    G = Hq // Hk if Hk else 1
    dq, dk, dv = (torch.zeros_like(x) for x in (q, k, v))
    mq, mk, mv = (torch.zeros_like(x) for x in (q, k, v))
    spans = [(b, 0, Tq, 0, Tk) for b in range(B)] if cu is None else \
        [(0, a, e, a, e) for (_, a, e) in sequences(B, Tq, cu)]
    for b, qa, qe, ka, ke in spans:
        m = visible(qe - qa, ke - ka, W, S)
        some = m.any(1)
        for h in range(Hq):
            if not some.any():
                continue
            qh, kh, vh, dh = q[b, qa:qe, h], k[b, ka:ke, h // G], v[b, ka:ke, h // G], dout[b, qa:qe, h]
            s = ((qh @ kh.T) * scale).masked_fill(~m, -math.inf)
            p = torch.zeros_like(s)
            p[some] = torch.softmax(s[some], -1)
            dp = dh @ vh.T
            delta = (p * dp).sum(-1, keepdim=True)
            ds = p * (dp - delta) * scale
            # delta comes from the rounded output: its error is that of one rounding of o
            mds = p * ((dp - delta).abs() + dh.abs() @ vh.abs().amax(0)[:, None]) * scale
            dq[b, qa:qe, h] = ds @ kh
            mq[b, qa:qe, h] = mds @ kh.abs()
            dk[b, ka:ke, h // G] += ds.T @ qh
            mk[b, ka:ke, h // G] += mds.T @ qh.abs()
            dv[b, ka:ke, h // G] += p.T @ dh
            mv[b, ka:ke, h // G] += p.T @ dh.abs()
    return (dq, dk, dv), (mq, mk, mv)
