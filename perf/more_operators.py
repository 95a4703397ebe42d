"""Cases, plain forms and 64-bit values of what a block of a hybrid model runs around
its token mixers: attention to an encoder's states of another length, the norms
before and after a block with its gate and residual scale, and dropout from a
counter-based generator.

Sizes are the benchmark's own: 1536 and 2048 channels as 12 and 16 heads, rows of
4096 steps; encoders of some hundred to some thousand states; and odd ones between.
"""

import math
import random

import numpy
import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one decoding step of a single request over an encoder of 1500 states (latency)
        dict(name="cross_token", op="cross_step", dtype="bf16", B=1, Tk=1500, Hq=16, Hk=16, D=128),
        # one decoding step of 64 requests whose encoders have 800 to 4096 states
        dict(name="cross_tokens", op="cross_step", dtype="bf16", B=64, Tk=4096, Hq=16, Hk=4, D=128),
        # four whole rows against 1500 encoder states each
        dict(name="cross_prompt", op="cross", train=False, mode="whole", n=0, dtype="bf16", B=4, Tq=4096, Tk=1500,
             Hq=16, Hk=16, D=128),
        # an odd prompt in fp32
        dict(name="cross_prompt_f32", op="cross", train=False, mode="whole", n=0, dtype="f32", B=2, Tq=777, Tk=1031,
             Hq=12, Hk=4, D=64),
        # a training step on a padded batch: encoders of 1024 to 2048 states, forward and backward
        dict(name="cross_train", op="cross", train=True, mode="padded", n=0, dtype="bf16", B=4, Tq=4096, Tk=2048,
             Hq=16, Hk=4, D=128),
        # a training step on seven packed pairs of uneven lengths
        dict(name="cross_train_packed", op="cross", train=True, mode="packed", n=7, dtype="bf16", B=1, Tq=4001,
             Tk=5003, Hq=12, Hk=12, D=96),
        # the norms around one block for 32 single tokens (latency)
        dict(name="norm_token", op="norm", way="fwd", stream="bf16", dtype="bf16", B=32, T=1, C=2048, post=True,
             gate="channel", next=True, p=0.0),
        # a long prompt on a stream in fp32, no norm after the block
        dict(name="norm_prompt", op="norm", way="fwd", stream="f32", dtype="bf16", B=1, T=16384, C=1536, post=False,
             gate="none", next=True, p=0.0),
        # a training step, forward and backward, with dropout; the stream in fp32
        dict(name="norm_train", op="norm", way="both", stream="f32", dtype="bf16", B=8, T=4096, C=2048, post=True,
             gate="channel", next=True, p=0.1),
        # the backward on an odd batch with a gate of its own for each row, all in bf16
        dict(name="norm_train_odd", op="norm", way="bwd", stream="bf16", dtype="bf16", B=3, T=1999, C=1000, post=True,
             gate="row", next=True, p=0.0),
        # a few odd rows in fp32 (latency)
        dict(name="dropout_odd", op="dropout", dtype="f32", B=1, T=37, C=1537, p=0.3),
        # a training step's activations, forward and backward
        dict(name="dropout_train", op="dropout", dtype="bf16", B=8, T=4096, C=2048, p=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cross", "cross", "cross", "cross_step", "norm", "norm", "dropout"])
    if op == "cross_step":
        Hk = rng.choice([1, 2, 4, 12, 16])
        return dict(op=op, dtype="bf16", B=_log(rng, 1, 64), Tk=_log(rng, 1, 4096), Hk=Hk,
                    Hq=Hk * rng.choice([1, 2, 4] if Hk < 12 else [1]), D=rng.choice([64, 96, 128]))
    if op == "cross":
        f32 = rng.random() < 0.2
        train, mode = rng.random() < 0.5, rng.choice(["whole", "padded", "packed"])
        Tq, Tk = _log(rng, 1, 1024 if f32 else 4096), _log(rng, 16, 1024 if f32 else 4096)
        Hk = rng.choice([1, 2, 4, 5])
        n = rng.randint(1, 9) if mode == "packed" else 0
        return dict(op=op, train=train, mode=mode, n=n, dtype="f32" if f32 else "bf16",
                    B=1 if n else max(1, min(4, 4096 // max(Tq, Tk))), Tq=Tq, Tk=Tk, Hk=Hk,
                    Hq=Hk * rng.choice([1, 2, 3, 4]), D=rng.choice([64, 96, 128]))
    if op == "norm":
        T = _log(rng, 1, 8192)
        stream = rng.choice(["bf16", "f32"])
        return dict(op=op, way=rng.choice(["fwd", "bwd", "both"] if stream == "f32" else ["fwd", "bwd"]), stream=stream,
                    dtype=rng.choice(["bf16", "f32"]) if stream == "f32" else "bf16",
                    B=_log(rng, 1, max(1, min(32, 8192 // T))), T=T, C=8 * _log(rng, 8, 512),
                    post=rng.random() < 0.6, gate=rng.choice(["none", "channel", "row"]), next=rng.random() < 0.8,
                    p=rng.choice([0.0, 0.0, 0.1, 0.25]))
    T = _log(rng, 1, 4096)
    return dict(op=op, dtype=rng.choice(["bf16", "f32"]), B=rng.randint(1, 6), T=T, C=_log(rng, 64, 2048),
                p=rng.choice([0.05, 0.1, 0.3, 0.5]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(case, seed):
    """The lengths of a padded or packed case, or of the encoders of a step: the same ones
    for every seed, in another order. (queries, keys) of each sequence."""
    fixed = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    Tq, Tk = case.get("Tq", 1), case["Tk"]
    if case["op"] == "cross_step":  # a fifth to all of the cache; one encoder more than requests
        n = case["B"] + 1
        out = [(1, Tk if n == 2 else max(1, Tk // 5 + (Tk - Tk // 5) * i // (n - 1))) for i in range(n)]
    elif case["mode"] == "padded":  # half to all of the row
        out = [(Tq, max(1, Tk - (Tk // 2) * i // case["B"])) for i in range(case["B"])]
    else:
        n = case["n"]
        qs = sorted(fixed.randint(0, Tq) for _ in range(n - 1))
        ks = sorted(fixed.sample(range(1, Tk), n - 1))
        out = [(b - a, d - c) for a, b, c, d in zip([0] + qs, qs + [Tq], [0] + ks, ks + [Tk])]
    random.Random(seed).shuffle(out)
    return out


def _offsets(lengths):
    return torch.tensor([0] + lengths, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(DEV)


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = _dtype(case["dtype"])

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)

    op, s = case["op"], {"case": case}
    if op == "cross_step":
        B, Tk, Hq, Hk, D = (case[n] for n in ("B", "Tk", "Hq", "Hk", "D"))
        s["q"] = normal(B, Hq, D)
        s["kc"], s["vc"] = normal(B + 1, Tk, Hk, D), normal(B + 1, Tk, Hk, D)
        s["lens"] = torch.tensor([k for _, k in _lengths(case, seed)], dtype=torch.int32).to(DEV)
        s["slots"] = torch.randperm(B + 1, generator=g, device=DEV)[:B].to(torch.int32)
    elif op == "cross":
        B, Tq, Tk, Hq, Hk, D = (case[n] for n in ("B", "Tq", "Tk", "Hq", "Hk", "D"))
        s["q"] = normal(B, Tq, Hq, D)
        kv = normal(B, Tk, 2 * Hk, D)  # one projection of the encoder's states
        s["k"], s["v"] = kv[:, :, :Hk], kv[:, :, Hk:]
        s["lens"] = s["cu_q"] = s["cu_k"] = None
        if case["mode"] == "padded":
            s["lens"] = torch.tensor([k for _, k in _lengths(case, seed)], dtype=torch.int32).to(DEV)
        elif case["mode"] == "packed":
            pairs = _lengths(case, seed)
            s["cu_q"], s["cu_k"] = _offsets([q for q, _ in pairs]), _offsets([k for _, k in pairs])
        if case["train"]:
            s["do"] = normal(B, Tq, Hq, D)
    elif op == "norm":
        B, T, C = case["B"], case["T"], case["C"]
        st = _dtype(case["stream"])
        s["x"] = normal(B, T, C, dtype=st)  # before the block; of the backward: what the forward gave
        s["y"] = normal(B, T, C)
        s["w_post"] = 1 + 0.1 * normal(C, dtype=torch.float32) if case["post"] else None
        s["w_next"] = 1 + 0.1 * normal(C, dtype=torch.float32) if case["next"] else None
        s["gate"] = {"none": lambda: None, "channel": lambda: 0.5 + 0.1 * normal(C, dtype=torch.float32),
                     "row": lambda: 0.5 + 0.1 * normal(B, C, dtype=torch.float32)}[case["gate"]]()
        if case["way"] != "fwd":
            s["dx"] = normal(B, T, C, dtype=st)
            s["dn"] = normal(B, T, C) if case["next"] else None
        s["rng"] = (seed * 2654435761 % (1 << 62), seed % 1000)
    else:
        s["x"] = normal(case["B"], case["T"], case["C"])
        s["dy"] = normal(case["B"], case["T"], case["C"])
        s["rng"] = (seed * 2654435761 % (1 << 62), seed % 1000)
    return s


ALPHA = 0.9  # scale of the residual stream
EPS = 1e-6


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import associative_affine_scan_gb300 as scan
        if op == "cross_step":
            return scan.cross_attn_step(s["q"], s["kc"], s["vc"], s["lens"], s["slots"])
        if op == "cross":
            seqs = (s["lens"], s["cu_q"], s["cu_k"])
            o, lse = scan.cross_attn_fwd(s["q"], s["k"], s["v"], *seqs)
            if not case["train"]:
                return o, lse
            return o, scan.cross_attn_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], *seqs)
        if op == "norm":
            weights = (s["w_post"], s["gate"], s["w_next"])
            kw = dict(alpha=ALPHA, eps=EPS, p=case["p"], rng=s["rng"])
            if case["way"] == "bwd":
                return scan.residual_norm_bwd(s["x"], s["y"], s["dx"], s["dn"], *weights, **kw)
            x, n = scan.residual_norm_fwd(s["x"], s["y"], *weights, **kw)
            if case["way"] == "fwd":
                return x, n
            return x, n, scan.residual_norm_bwd(x, s["y"], s["dx"], s["dn"], *weights, **kw)
        y = scan.dropout_fwd(s["x"], case["p"], s["rng"])
        return y, scan.dropout_bwd(s["dy"], case["p"], s["rng"])
    return {"cross_step": _cross_step, "cross": _cross, "norm": _norm, "dropout": _dropout}[op](s)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _cross_step(s):
    case = s["case"]
    B, Hq, Hk, D = (case[n] for n in ("B", "Hq", "Hk", "D"))
    slots = s["slots"].long()
    k, v = s["kc"][slots].float(), s["vc"][slots].float()
    q = s["q"].float().view(B, Hk, Hq // Hk, D)
    p = torch.einsum("bhgd,bchd->bhgc", q, k) * D ** -0.5
    there = torch.arange(case["Tk"], device=DEV)[None] < s["lens"][slots][:, None]
    p = torch.where(there[:, None, None], p, -math.inf)
    p = (p - p.amax(-1, keepdim=True)).exp()
    p = p / p.sum(-1, keepdim=True)
    return torch.einsum("bhgc,bchd->bhgd", p, v).reshape(B, Hq, D).to(s["q"].dtype)


def _cross(s):
    case, dt = s["case"], s["q"].dtype
    B, Tq, Tk, Hq, Hk, D = (case[n] for n in ("B", "Tq", "Tk", "Hq", "Hk", "D"))
    q = s["q"].float().view(B, Tq, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4)  # [B, Hk, G, Tq, D]
    k, v = (s[n].float().permute(0, 2, 1, 3)[:, :, None] for n in ("k", "v"))
    hidden = None
    if s["lens"] is not None:
        hidden = (torch.arange(Tk, device=DEV)[None] >= s["lens"][:, None])[:, None, None, None]
    elif s["cu_q"] is not None:
        of_q, of_k = (torch.bucketize(torch.arange(T, device=DEV), s[c][1:].long(), right=True)
                      for T, c in ((Tq, "cu_q"), (Tk, "cu_k")))
        hidden = of_q[:, None] != of_k[None]
    p = (q @ k.transpose(-1, -2)).mul_(D ** -0.5)
    if hidden is not None:
        p = p.masked_fill_(hidden, -math.inf)
    m = p.amax(-1, keepdim=True)
    p = p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    p = p.div_(l)
    o = p @ v
    back = lambda x: x.permute(0, 3, 1, 2, 4).reshape(B, Tq, Hq, D).to(dt)  # noqa: E731
    if not case["train"]:
        return back(o), (m + l.log()).reshape(B, Hq, Tq)
    do = s["do"].float().view(B, Tq, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4)
    dv = (p.transpose(-1, -2) @ do).sum(2)
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(D ** -0.5)
    dq = ds @ k
    dk = (ds.transpose(-1, -2) @ q).sum(2)
    return back(o), (back(dq), dk.transpose(1, 2).to(dt), dv.transpose(1, 2).to(dt))


def _words(blocks, seed, call):
    """Philox 4x32 with 10 rounds: the four words of each block, whose counter is (block, call)
    and whose key is the seed. All in 64-bit integers: a product's upper word is put together
    from its two halves."""
    def product(a, m):
        low = a * (m & 0xffff)
        return (a * (m >> 16) + (low >> 16)) >> 16, (a * m) & 0xffffffff

    c = [blocks & 0xffffffff, blocks >> 32, torch.full_like(blocks, call & 0xffffffff),
         torch.full_like(blocks, call >> 32)]
    k0, k1 = seed & 0xffffffff, (seed >> 32) & 0xffffffff
    for _ in range(10):
        h0, l0 = product(c[0], 0xD2511F53)
        h1, l1 = product(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & 0xffffffff, (k1 + 0xBB67AE85) & 0xffffffff
    return c


def _kept(shape, p, rng):
    """What each element is multiplied by: 0, or 1 / (1 - p). Element i has bits 16 (i % 8) ..
    of block i / 8; it is dropped where they are below p, both in steps of 2^-16."""
    n = math.prod(shape)
    blocks = torch.arange((n + 7) // 8, device=DEV)
    c = _words(blocks, *rng)
    r = torch.stack([w >> h & 0xffff for w in c for h in (0, 16)], -1).flatten()[:n].view(shape)
    limit = round(p * 65536)
    return (r >= limit).float() * (65536 / (65536 - limit) if limit < 65536 else 0.0)


def _norm(s):
    case = s["case"]
    B, T, C = case["B"], case["T"], case["C"]
    st, dt = s["x"].dtype, s["y"].dtype
    gate = s["gate"]
    if gate is None:
        gate = torch.ones(C, device=DEV)
    if gate.dim() == 2:
        gate = gate[:, None]
    kept = _kept((B, T, C), case["p"], s["rng"]) if case["p"] else 1.0
    y = s["y"].float()
    r = (y.square().mean(-1, keepdim=True) + EPS).rsqrt() if case["post"] else 1.0
    yh = y * r
    z = yh * s["w_post"] if case["post"] else y
    outs = ()
    x = s["x"]
    if case["way"] != "bwd":
        x = (ALPHA * x.float() + gate * z * kept).to(st)
    xf = x.float()
    rx = (xf.square().mean(-1, keepdim=True) + EPS).rsqrt()  # of the stream as it is returned
    xh = xf * rx
    if case["way"] != "bwd":
        outs = (x, (xh * s["w_next"]).to(dt) if case["next"] else None)
        if case["way"] == "fwd":
            return outs
    g = s["dx"].float()
    dw_next = None
    if case["next"]:
        dn = s["dn"].float()
        dw_next = (dn * xh).sum((0, 1))
        e = dn * s["w_next"]
        g = g + rx * (e - xh * (e * xh).mean(-1, keepdim=True))
    dx = (ALPHA * g).to(st)
    u = g * kept
    dgate = None
    if s["gate"] is not None:
        dgate = (u * z).sum(1) if s["gate"].dim() == 2 else (u * z).sum((0, 1))
    dz = u * gate
    dw_post = None
    if case["post"]:
        dw_post = (dz * yh).sum((0, 1))
        e = dz * s["w_post"]
        dz = r * (e - yh * (e * yh).mean(-1, keepdim=True))
    grads = (dx, dz.to(dt), dw_post, dgate, dw_next)
    return grads if case["way"] == "bwd" else outs + (grads,)


def _dropout(s):
    kept = _kept(s["x"].shape, s["case"]["p"], s["rng"])
    return (s["x"].float() * kept).to(s["x"].dtype), (s["dy"].float() * kept).to(s["dy"].dtype)


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"cross_step": _exact_step, "cross": _exact_cross, "norm": _exact_norm, "dropout": _exact_dropout}[case["op"]](s)


def _exact_step(s):
    case = s["case"]
    o = torch.empty(case["B"], case["Hq"], case["D"], dtype=torch.float64, device=DEV)
    G, lens = case["Hq"] // case["Hk"], s["lens"].tolist()
    for b, slot in enumerate(s["slots"].tolist()):
        n = lens[slot]
        for h in range(case["Hk"]):
            kh, vh = s["kc"][slot, :n, h].double(), s["vc"][slot, :n, h].double()
            w = torch.softmax(s["q"][b, h * G:(h + 1) * G].double() @ kh.T / math.sqrt(case["D"]), -1)
            o[b, h * G:(h + 1) * G] = w @ vh
    return o


def _exact_cross(s):
    """Each sequence and head by itself, its gradient by differentiating that."""
    case = s["case"]
    B, Tq, Tk, Hq, Hk, D = (case[n] for n in ("B", "Tq", "Tk", "Hq", "Hk", "D"))
    train, G = case["train"], Hq // Hk
    o, dq = (torch.zeros(B, Tq, Hq, D, dtype=torch.float64, device=DEV) for _ in range(2))
    dk, dv = (torch.zeros(B, Tk, Hk, D, dtype=torch.float64, device=DEV) for _ in range(2))
    lse = torch.empty(B, Hq, Tq, dtype=torch.float64, device=DEV)
    if case["mode"] == "packed":
        cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
        rows = [(0, cq[i], cq[i + 1], ck[i], ck[i + 1]) for i in range(case["n"])]
    else:
        n = s["lens"].tolist() if s["lens"] is not None else [Tk] * B
        rows = [(b, 0, Tq, 0, n[b]) for b in range(B)]
    for b, a, e, c, f in rows:
        for h in range(Hq):
            qh, kh, vh = (x.double().requires_grad_(train) for x in
                          (s["q"][b, a:e, h], s["k"][b, c:f, h // G], s["v"][b, c:f, h // G]))
            w = qh @ kh.T / math.sqrt(D)
            oh = torch.softmax(w, -1) @ vh
            o[b, a:e, h], lse[b, h, a:e] = oh.detach(), torch.logsumexp(w.detach(), -1)
            if train:
                gq, gk, gv = torch.autograd.grad((oh * s["do"][b, a:e, h].double()).sum(), (qh, kh, vh))
                dq[b, a:e, h] = gq
                dk[b, c:f, h // G] += gk
                dv[b, c:f, h // G] += gv
    return (o, (dq, dk, dv)) if train else (o, lse)


def _draws(n, seed, call):
    """The generator's 16-bit numbers of elements 0 .. n - 1, by unsigned 64-bit products on the host."""
    u = numpy.uint64
    block = numpy.arange((n + 7) // 8, dtype=u)
    mask, half = u(0xffffffff), u(32)
    w, x = block & mask, block >> half
    y, z = numpy.full_like(block, call & 0xffffffff), numpy.full_like(block, call >> 32)
    keys = [(seed + 0x9E3779B9 * i) & 0xffffffff for i in range(10)], \
           [((seed >> 32) + 0xBB67AE85 * i) & 0xffffffff for i in range(10)]
    for a, b in zip(*keys):
        first, second = w * u(0xD2511F53), y * u(0xCD9E8D57)
        w, x, y, z = (second >> half) ^ x ^ u(a), second & mask, (first >> half) ^ z ^ u(b), first & mask
    words = numpy.stack([w, x, y, z], -1).astype("<u4")
    return torch.from_numpy(words.reshape(-1).view("<u2")[:n].astype(numpy.int32)).to(DEV)


def _survivors(shape, p, rng):
    limit = round(p * 65536)
    alive = (_draws(math.prod(shape), *rng) >= limit).view(shape)
    return alive.double() * (65536.0 / (65536 - limit) if limit < 65536 else 0.0)


def _exact_dropout(s):
    kept = _survivors(s["x"].shape, s["case"]["p"], s["rng"])
    return s["x"].double() * kept, s["dy"].double() * kept


def _exact_norm(s):
    """Row by row of the batch, the gradient by differentiating the definition (at the stream
    as it is stored between the two)."""
    case = s["case"]
    B, T, C = case["B"], case["T"], case["C"]
    kept = _survivors((B, T, C), case["p"], s["rng"]) if case["p"] else None

    def rms(v, w):
        return v / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / C + EPS) * w

    w_post, w_next, gate = (None if t is None else t.double() for t in (s["w_post"], s["w_next"], s["gate"]))
    xs, ns, dxs, dys = [], [], [], []
    sums = [None if t is None else torch.zeros_like(t) for t in (w_post, gate, w_next)]
    for b in range(B):
        leaves = [s["y"][b].double()] + [None if t is None else t for t in
                                         (w_post, gate if gate is None or gate.dim() == 1 else gate[b], w_next)]
        leaves = [t if t is None else t.detach().requires_grad_(case["way"] != "fwd") for t in leaves]
        y, wp, gt, wn = leaves
        u = y if wp is None else rms(y, wp)
        u = u if gt is None else gt * u
        u = u if kept is None else u * kept[b]
        x = s["x"][b].double()
        if case["way"] != "bwd":
            x = ALPHA * x + u.detach()
            xs.append(x)
        # the stream is stored in its own type
        x = x.to(_dtype(case["stream"])).double() if case["way"] != "bwd" and case["stream"] == "bf16" else x
        x = x.detach().requires_grad_(case["way"] != "fwd")
        n = None if wn is None else rms(x, wn)
        if n is not None:
            ns.append(n.detach())
        if case["way"] == "fwd":
            continue
        total = s["dx"][b].double()
        if n is not None:
            gx, gw = torch.autograd.grad((n * s["dn"][b].double()).sum(), (x, wn))
            total = total + gx
            sums[2] += gw
        dxs.append(ALPHA * total)
        asked = [t for t in (y, wp, gt) if t is not None]
        got = list(torch.autograd.grad((u * total).sum(), asked))
        dys.append(got.pop(0))
        if wp is not None:
            sums[0] += got.pop(0)
        if gt is not None and gate.dim() == 1:
            sums[1] += got.pop(0)
        elif gt is not None:
            sums[1][b] = got.pop(0)
    outs = () if case["way"] == "bwd" else (torch.stack(xs), torch.stack(ns) if ns else None)
    if case["way"] == "fwd":
        return outs
    grads = (torch.stack(dxs), torch.stack(dys), sums[0], sums[1], sums[2])
    return grads if case["way"] == "bwd" else outs + (grads,)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op == "cross_step":
        keys = [k for _, k in _lengths(case, 0)]
        keys = sum(keys) * case["B"] / len(keys)  # of the encoders that requests have, in the mean
        D, Hq, Hk = case["D"], case["Hq"], case["Hk"]
        return {"bytes": (keys * 2 * Hk + case["B"] * 2 * Hq) * D * e, "flops": keys * 4 * Hq * D}
    if op == "cross":
        B, Tq, Tk, Hq, Hk, D = (case[n] for n in ("B", "Tq", "Tk", "Hq", "Hk", "D"))
        seqs = [(Tq, Tk)] * B if case["mode"] == "whole" else _lengths(case, 0)
        pairs, keys = sum(a * b for a, b in seqs), sum(b for _, b in seqs)
        q, k = B * Tq * Hq * D * e, keys * Hk * D * e
        if case["train"]:  # q, do, k, v in; o, dq, dk, dv out
            return {"bytes": 4 * q + 2 * k + 2 * B * Tk * Hk * D * e, "flops": 14 * pairs * Hq * D}
        return {"bytes": 2 * q + 2 * k + B * Tq * Hq * 4, "flops": 4 * pairs * Hq * D}
    n = case["B"] * case["T"] * case["C"]
    if op == "norm":
        x = 2 if case["stream"] == "bf16" else 4
        fwd = 2 * x + e + (e if case["next"] else 0)
        # the forward's operands and results once each: its y and stream serve the backward as well
        bwd = 2 * x + e + (e if case["next"] else 0) + (x + e if case["way"] == "bwd" else 0)
        return {"bytes": n * {"fwd": fwd, "bwd": bwd, "both": fwd + bwd}[case["way"]],
                "flops": n * {"fwd": 12, "bwd": 30, "both": 42}[case["way"]]}
    return {"bytes": n * 4 * e, "flops": n * 4}
