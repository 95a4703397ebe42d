"""Cases, plain forms and 64-bit values of the token mixers around the scans: the
norm and rotation of queries and keys, linear attention with a decay for each
head, and attention with a sliding window and first tokens that stay visible.

Sizes are the benchmark's own: 1536 and 2048 channels as 12 and 16 heads of 128,
rows of 4096 steps, packed sequences of 512 to 8192 steps; and odd ones between.
"""

import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one decoding step of 32 requests: queries and keys of one token each (latency)
        dict(name="rope_token", op="rope", train=False, dtype="bf16", B=32, T=1, Hq=16, Hk=4, D=128,
             R=128, pairs=False),
        # a prompt of odd length in fp32, half of each head rotated, neighbouring pairs
        dict(name="rope_prompt_f32", op="rope", train=False, dtype="f32", B=3, T=1999, Hq=12, Hk=12,
             D=96, R=48, pairs=True),
        # the norm and rotation of a training step, forward and backward
        dict(name="rope_train", op="rope", train=True, dtype="bf16", B=8, T=4096, Hq=16, Hk=4, D=128,
             R=128, pairs=False),
        # one decoding step of 64 requests in a pool of states
        dict(name="linear_token", op="linear_step", dtype="bf16", B=64, H=16, Dk=128, Dv=128),
        # a long prompt of one request; the state goes on to decoding
        dict(name="linear_prompt", op="linear", train=False, packed=0, dtype="bf16", B=1, T=16384, H=16,
             Dk=128, Dv=128, state=False),
        # six prompts of odd lengths packed in one row
        dict(name="linear_packed", op="linear", train=False, packed=6, dtype="bf16", B=1, T=9001, H=12,
             Dk=64, Dv=128, state=False),
        # a training step, forward and backward
        dict(name="linear_train", op="linear", train=True, packed=0, dtype="bf16", B=4, T=4096, H=16,
             Dk=128, Dv=128, state=False),
        # a piece of a longer text in training: an odd length, odd heads, a state coming in
        dict(name="linear_train_odd", op="linear", train=True, packed=0, dtype="bf16", B=2, T=1537, H=5,
             Dk=96, Dv=64, state=True),
        # a long prompt of one request through a window of 2048
        dict(name="window_prompt", op="window", train=False, packed=0, dtype="bf16", B=1, T=16384, Hq=16,
             Hk=4, D=128, W=2048, S=4),
        # a training step, forward and backward
        dict(name="window_train", op="window", train=True, packed=0, dtype="bf16", B=2, T=4096, Hq=16,
             Hk=4, D=128, W=1024, S=4),
        # one decoding step of a single request (latency)
        dict(name="window_token", op="window_step", dtype="bf16", B=1, Hq=16, Hk=4, D=128, W=2048, S=4),
        # one decoding step of 64 requests at different lengths, most of them past the window
        dict(name="window_tokens", op="window_step", dtype="bf16", B=64, Hq=16, Hk=4, D=128, W=4096, S=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "linear_step", "linear", "linear", "window", "window", "window_step"])
    if op == "rope":
        D = rng.choice([64, 96, 128])
        Hk = rng.choice([1, 2, 4, 12])
        T = _log(rng, 1, 4096)
        return dict(op=op, train=rng.random() < 0.5, dtype=rng.choice(["bf16", "f32"]),
                    B=_log(rng, 1, max(1, min(64, 24576 // T))), T=T, Hq=Hk * rng.choice([1, 2, 4] if Hk < 12 else [1]),
                    Hk=Hk, D=D, R=rng.choice([D, D // 2]), pairs=rng.random() < 0.3)
    if op == "linear_step":
        return dict(op=op, dtype="bf16", B=_log(rng, 1, 64), H=rng.choice([5, 8, 12, 16]),
                    Dk=rng.choice([64, 96, 128]), Dv=rng.choice([64, 128]))
    if op == "linear":
        T = _log(rng, 17, 8192)
        packed = rng.choice([0, 0, rng.randint(2, 9)])
        return dict(op=op, train=rng.random() < 0.5, packed=packed, dtype="bf16",
                    B=1 if packed else max(1, min(4, 8192 // T)), T=T, H=rng.choice([5, 8, 12, 16]),
                    Dk=rng.choice([64, 96, 128]), Dv=rng.choice([64, 128]), state=rng.random() < 0.5)
    Hk = rng.choice([1, 2, 4, 5])
    Hq = Hk * rng.choice([1, 2, 3, 4])
    if op == "window":
        train = rng.random() < 0.5
        T = _log(rng, 17, 4096 if train else 8192)
        packed = rng.choice([0, 0, rng.randint(2, 9)])
        return dict(op=op, train=train, packed=packed, dtype="bf16", B=1 if packed else max(1, min(2, 4096 // T)),
                    T=T, Hq=Hq, Hk=Hk, D=rng.choice([64, 96, 128]), W=_log(rng, 16, 2048), S=rng.choice([0, 1, 4, 16]))
    return dict(op=op, dtype="bf16", B=_log(rng, 1, 48), Hq=Hq, Hk=Hk, D=rng.choice([64, 96, 128]),
                W=_log(rng, 64, 4096), S=rng.choice([0, 1, 4, 16]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _cu(case, seed):
    """Offsets of case["packed"] sequences of uneven lengths that fill T steps."""
    if not case["packed"]:
        return None
    g = torch.Generator().manual_seed(seed)
    cuts = torch.randint(0, case["T"] + 1, (case["packed"] - 1,), generator=g).sort().values
    return torch.cat([torch.zeros(1), cuts, torch.full((1,), case["T"])]).to(torch.int32).to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dt)

    op, s = case["op"], {"case": case}
    if op == "rope":
        B, T, Hq, Hk, D, R = (case[n] for n in ("B", "T", "Hq", "Hk", "D", "R"))
        qkv = normal(B, T, Hq + 2 * Hk, D)  # the fused projection's output
        s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
        s["wq"], s["wk"] = (1 + 0.1 * torch.randn(D, generator=g, device=DEV) for _ in range(2))
        P = max(8192, T)
        freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
        angle = torch.arange(P, dtype=torch.float64)[:, None] * freq
        s["cos"], s["sin"] = (f(angle).float().to(DEV) for f in (torch.cos, torch.sin))
        start = torch.randint(0, P - T + 1, (B, 1), generator=g, device=DEV)
        s["pos"] = (start + torch.arange(T, device=DEV)).to(torch.int32)
        if case["train"]:
            s["dq"], s["dk"] = normal(B, T, Hq, D), normal(B, T, Hk, D)
    elif op == "linear_step":
        B, H, Dk, Dv = (case[n] for n in ("B", "H", "Dk", "Dv"))
        s["q"], s["k"], s["v"] = normal(B, H, Dk), normal(B, H, Dk), normal(B, H, Dv)
        s["state"] = 4 * torch.randn(B + 3, H, Dk, Dv, generator=g, device=DEV)
        s["slots"] = torch.randperm(B + 3, generator=g, device=DEV)[:B].to(torch.int32)
        s["decay"] = _decay(H)
    elif op == "linear":
        B, T, H, Dk, Dv = (case[n] for n in ("B", "T", "H", "Dk", "Dv"))
        s["q"], s["k"] = normal(B, T, H, Dk), normal(B, T, H, Dk)
        s["v"] = normal(B, T, H, Dv + 8)[..., :Dv]  # a slice of a wider projection
        s["decay"] = _decay(H)
        s["cu"] = _cu(case, seed)
        n = case["packed"] or B
        s["h0"] = torch.randn(n, H, Dk, Dv, generator=g, device=DEV) if case["state"] else None
        if case["train"]:
            s["do"] = normal(B, T, H, Dv)
    elif op == "window":
        B, T, Hq, Hk, D = (case[n] for n in ("B", "T", "Hq", "Hk", "D"))
        s["q"], s["k"] = normal(B, T, Hq, D), normal(B, T, Hk, D)
        s["v"] = normal(B, T, 2 * Hk, D)[:, :, Hk:]
        s["cu"] = _cu(case, seed)
        if case["train"]:
            s["do"] = normal(B, T, Hq, D)
    else:
        B, Hq, Hk, D, W, S = (case[n] for n in ("B", "Hq", "Hk", "D", "W", "S"))
        s["q"], s["k"], s["v"] = normal(B, Hq, D), normal(B, Hk, D), normal(B, Hk, D)
        s["kc"], s["vc"] = normal(B + 1, S + W, Hk, D), normal(B + 1, S + W, Hk, D)
        s["slots"] = torch.randperm(B + 1, generator=g, device=DEV)[:B].to(torch.int32)
        s["pos"] = torch.randint(W // 2 if B > 1 else 2 * W, 4 * W, (B,), generator=g, device=DEV).to(torch.int32)
    return s


def _decay(H):
    """log(lambda) of each head: half-lives from one step to a few hundred."""
    return -(2.0 ** (-8.0 * (torch.arange(H, dtype=torch.float32, device=DEV) + 1) / H))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import associative_affine_scan_gb300 as scan
        if op == "rope":
            args = (s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"])
            y = scan.qk_norm_rope_fwd(*args, s["pos"], interleaved=case["pairs"])
            if not case["train"]:
                return y
            return y, scan.qk_norm_rope_bwd(*args, s["dq"], s["dk"], s["pos"], interleaved=case["pairs"])
        if op == "linear_step":
            o = scan.linattn_step(s["q"], s["k"], s["v"], s["decay"], s["state"], s["slots"])
            return o, s["state"]
        if op == "linear":
            args = (s["q"], s["k"], s["v"], s["decay"])
            y = scan.linattn_fwd(*args, s["h0"], s["cu"], need_state=not case["train"])
            if not case["train"]:
                return y
            return y[0], scan.linattn_bwd(*args, s["do"], s["h0"], s["cu"], need_dh0=case["state"])
        if op == "window":
            o, lse = scan.window_attn_fwd(s["q"], s["k"], s["v"], case["W"], case["S"], s["cu"])
            if not case["train"]:
                return o, lse
            return o, scan.window_attn_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], case["W"], case["S"], s["cu"])
        o = scan.window_attn_step(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["pos"], case["W"], case["S"], s["slots"])
        return o, s["kc"], s["vc"]
    return {"rope": _rope, "linear_step": _linear_step, "linear": _linear, "window": _window,
            "window_step": _window_step}[op](s)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _split(x, R, pairs):
    """The two members of each rotated pair, and the part that is not rotated."""
    if pairs:
        return x[..., 0:R:2], x[..., 1:R:2], x[..., R:]
    return x[..., :R // 2], x[..., R // 2:R], x[..., R:]


def _join(a, b, rest, pairs):
    rot = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([rot, rest], -1)


def _turn(x, cos, sin, R, pairs):
    a, b, rest = _split(x, R, pairs)
    return _join(a * cos - b * sin, a * sin + b * cos, rest, pairs)


def _rope(s):
    case, eps = s["case"], 1e-6
    R, pairs, dt = case["R"], case["pairs"], s["q"].dtype
    pos = s["pos"].long()
    cos, sin = s["cos"][pos][:, :, None], s["sin"][pos][:, :, None]

    def forward(x, w):
        x = x.float()
        r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
        return _turn(x * r * w, cos, sin, R, pairs).to(dt)

    def backward(x, w, dy):
        x = x.float()
        r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
        n = x * r
        dz = _turn(dy.float(), cos, -sin, R, pairs)
        g = dz * w
        dx = r * (g - n * (g * n).mean(-1, keepdim=True))
        return dx.to(dt), (dz * n).sum((0, 1, 2))

    y = forward(s["q"], s["wq"]), forward(s["k"], s["wk"])
    if not case["train"]:
        return y
    dq, dwq = backward(s["q"], s["wq"], s["dq"])
    dk, dwk = backward(s["k"], s["wk"], s["dk"])
    return y, (dq, dk, dwq, dwk)


def _linear_step(s):
    slots = s["slots"].long()
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    h = s["state"][slots] * s["decay"].exp()[None, :, None, None] + k[..., :, None] * v[..., None, :]
    s["state"][slots] = h
    o = (q[..., :, None] * h).sum(-2) * q.shape[-1] ** -0.5
    return o.to(s["q"].dtype), s["state"]


def _places(cu, B, T):
    """Of each step: its sequence, its place in it, and how many steps follow there; of each sequence: its length."""
    t = torch.arange(T, device=DEV)
    if cu is None:
        return torch.zeros_like(t), t, T - 1 - t, torch.full((B,), T, device=DEV)
    seq = torch.bucketize(t, cu[1:].long(), right=True)
    return seq, t - cu.long()[seq], cu.long()[seq + 1] - 1 - t, (cu[1:] - cu[:-1]).long()


def _linear(s):
    case, dt = s["case"], s["q"].dtype
    B, T = case["B"], case["T"]
    q, k, v = (s[n].float().transpose(1, 2) for n in ("q", "k", "v"))  # [B, H, T, D]
    scale, g = q.shape[-1] ** -0.5, s["decay"]
    seq, place, after, length = _places(s["cu"], B, T)
    d = place[:, None] - place[None, :]
    seen = (d >= 0) & (seq[:, None] == seq[None, :])
    D = torch.where(seen, torch.exp(g[:, None, None] * d.clamp(min=0)), 0.0)  # [H, T, T]
    before = torch.exp(g[:, None] * (place + 1))  # what is left of h0 at each step
    to_end = torch.exp(g[:, None] * after)  # what is left of each step at its sequence's end
    # packed: which step is whose, [n, T]
    whose = (seq[None] == torch.arange(len(length), device=DEV)[:, None]).float()

    def from_state(x, h):  # x_t times the state of its sequence
        if s["cu"] is None:
            return x @ h
        return torch.einsum("nt,htk,nhkv->htv", whose, x[0], h)[None]

    def to_state(x, y, w):  # the sum of w_t x_t y_t^T over each sequence
        x = x * w[..., None]
        if s["cu"] is None:
            return x.transpose(-1, -2) @ y
        return torch.einsum("nt,htk,htv->nhkv", whose, x[0], y[0])

    a = (q @ k.transpose(-1, -2)) * D
    o = a @ v
    if s["h0"] is not None:
        o = o + from_state(q, s["h0"]) * before[..., None]
    o = (o * scale).transpose(1, 2).to(dt)
    if not case["train"]:
        h = to_state(k, v, to_end)
        if s["h0"] is not None:
            h = h + s["h0"] * torch.exp(g[None, :] * length[:, None])[..., None, None]
        return o, h
    do = s["do"].float().transpose(1, 2) * scale
    dv = a.transpose(-1, -2) @ do
    b = (do @ v.transpose(-1, -2)) * D
    dq, dk = b @ k, b.transpose(-1, -2) @ q
    dh0 = None
    if s["h0"] is not None:
        dq = dq + from_state(do, s["h0"].transpose(-1, -2)) * before[..., None]
        dh0 = to_state(q, do, before)
    return o, tuple(x.transpose(1, 2).to(dt) for x in (dq, dk, dv)) + (dh0,)


def _window(s):
    case, dt = s["case"], s["q"].dtype
    B, T, Hq, Hk, D = (case[n] for n in ("B", "T", "Hq", "Hk", "D"))
    q = s["q"].float().view(B, T, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4)  # [B, Hk, G, T, D]
    k, v = (s[n].float().permute(0, 2, 1, 3)[:, :, None] for n in ("k", "v"))
    seq, place, _, _ = _places(s["cu"], B, T)
    d = place[:, None] - place[None, :]
    hidden = (d < 0) | ((d >= case["W"]) & (place[None, :] >= case["S"])) | (seq[:, None] != seq[None, :])
    p = (q @ k.transpose(-1, -2)).mul_(D ** -0.5).masked_fill_(hidden, -math.inf)
    m = p.amax(-1, keepdim=True)
    p = p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    p = p.div_(l)
    o = p @ v
    back = lambda x: x.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D).to(dt)  # noqa: E731
    if not case["train"]:
        return back(o), (m + l.log()).reshape(B, Hq, T)
    do = s["do"].float().view(B, T, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4)
    dv = (p.transpose(-1, -2) @ do).sum(2)
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(D ** -0.5)
    dq = ds @ k
    dk = (ds.transpose(-1, -2) @ q).sum(2)
    return back(o), (back(dq), dk.transpose(1, 2).to(dt), dv.transpose(1, 2).to(dt))


def _window_step(s):
    case = s["case"]
    B, Hq, Hk, D, W, S = (case[n] for n in ("B", "Hq", "Hk", "D", "W", "S"))
    pos, slots = s["pos"].long(), s["slots"].long()
    at = torch.where(pos < S, pos, S + (pos - S) % W)
    s["kc"][slots, at], s["vc"][slots, at] = s["k"], s["v"]
    k, v = s["kc"][slots].float(), s["vc"][slots].float()
    q = s["q"].float().view(B, Hk, Hq // Hk, D)
    p = torch.einsum("bhgd,bchd->bhgc", q, k) * D ** -0.5
    filled = torch.arange(S + W, device=DEV)[None] <= pos[:, None]
    p = torch.where(filled[:, None, None], p, -math.inf)
    p = (p - p.amax(-1, keepdim=True)).exp()
    o = torch.einsum("bhgc,bchd->bhgd", p, v) / p.sum(-1, keepdim=True)
    return o.reshape(B, Hq, D).to(s["q"].dtype), s["kc"], s["vc"]


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _exact_rope(s)
    if op == "linear_step":
        o = torch.empty(case["B"], case["H"], case["Dv"], dtype=torch.float64, device=DEV)
        h = s["state"].double()
        lam = s["decay"].double().exp()
        for b, slot in enumerate(s["slots"].tolist()):
            h[slot] = lam[:, None, None] * h[slot] + torch.einsum("hk,hv->hkv", s["k"][b].double(), s["v"][b].double())
            o[b] = torch.einsum("hk,hkv->hv", s["q"][b].double(), h[slot]) / math.sqrt(case["Dk"])
        return o, h
    if op == "linear":
        return _exact_linear(s)
    if op == "window":
        return _exact_window(s)
    o = torch.empty(case["B"], case["Hq"], case["D"], dtype=torch.float64, device=DEV)
    kc, vc = s["kc"].double(), s["vc"].double()
    W, S, G = case["W"], case["S"], case["Hq"] // case["Hk"]
    for b, (slot, p) in enumerate(zip(s["slots"].tolist(), s["pos"].tolist())):
        at = p if p < S else S + (p - S) % W
        kc[slot, at], vc[slot, at] = s["k"][b].double(), s["v"][b].double()
        n = min(p + 1, S + W)
        for h in range(case["Hq"]):
            w = torch.softmax(kc[slot, :n, h // G] @ s["q"][b, h].double() / math.sqrt(case["D"]), 0)
            o[b, h] = w @ vc[slot, :n, h // G]
    return o, kc, vc


def _exact_rope(s):
    case = s["case"]
    R, B, T = case["R"], case["B"], case["T"]
    angle = s["pos"].long().reshape(-1)
    turn = torch.complex(s["cos"].double()[angle], s["sin"].double()[angle])[:, None]
    outs, grads = [], []
    for x, w, dy in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        H, D = x.shape[2:]
        x = x.double().reshape(B * T, H, D).requires_grad_()
        w = w.double().requires_grad_()
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + 1e-6) * w
        z = y[..., :R].reshape(B * T, H, R // 2, 2) if case["pairs"] else y[..., :R].reshape(B * T, H, 2, R // 2).transpose(-1, -2)
        z = torch.view_as_real(torch.complex(z[..., 0], z[..., 1]) * turn)
        z = z if case["pairs"] else z.transpose(-1, -2)
        y = torch.cat([z.reshape(B * T, H, R), y[..., R:]], -1).reshape(B, T, H, D)
        outs.append(y.detach())
        if dy is not None:
            dx, dw = torch.autograd.grad((y * dy.double()).sum(), (x, w))
            grads.append((dx.reshape(B, T, H, D), dw))
    if not case["train"]:
        return tuple(outs)
    return tuple(outs), (grads[0][0], grads[1][0], grads[0][1], grads[1][1])


def _exact_linear(s):
    """The recurrence a block of steps at a time, its gradient by differentiating that."""
    case = s["case"]
    train = case["train"]
    q, k, v = (s[n].double().requires_grad_(train) for n in ("q", "k", "v"))
    g = s["decay"].double()[:, None]
    n = case["packed"] or case["B"]
    H, Dk, Dv = case["H"], case["Dk"], case["Dv"]
    h0 = s["h0"].double() if s["h0"] is not None else torch.zeros(n, H, Dk, Dv, dtype=torch.float64, device=DEV)
    h0.requires_grad_(train)
    rows = [(b, 0, case["T"]) for b in range(n)] if not case["packed"] else \
        [(0, a, e) for a, e in zip(s["cu"].tolist()[:-1], s["cu"].tolist()[1:])]
    outs, last = [], []
    for i, (b, a, e) in enumerate(rows):
        h = h0[i]
        for t in range(a, e, 256):
            u = min(e, t + 256)
            j = torch.arange(u - t, device=DEV)
            qc, kc, vc = (x[b, t:u].transpose(0, 1) for x in (q, k, v))
            w = torch.tril(torch.exp(g[..., None] * (j[:, None] - j[None, :]).clamp(min=0)))
            outs.append((((qc @ kc.mT) * w) @ vc + torch.exp(g * (j + 1))[..., None] * (qc @ h)) / math.sqrt(Dk))
            h = torch.exp(g * (u - t))[..., None] * h + (kc * torch.exp(g * (u - t - 1 - j))[..., None]).mT @ vc
        last.append(h)
    o = torch.cat(outs, 1).transpose(0, 1).reshape(case["B"], case["T"], H, Dv)
    if not train:
        return o, torch.stack(last)
    grads = torch.autograd.grad((o * s["do"].double()).sum(), (q, k, v, h0))
    return o.detach(), grads[:3] + (grads[3] if s["h0"] is not None else None,)


def _exact_window(s):
    """Softmax of each block of queries over the keys that it can see, its gradient by differentiating that."""
    case = s["case"]
    train, W, S, G = case["train"], case["W"], case["S"], case["Hq"] // case["Hk"]
    B, T, Hq, D = case["B"], case["T"], case["Hq"], case["D"]
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    dq, dk, dv = (torch.zeros_like(x) for x in (q, k, v))
    o = torch.empty(B, T, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, Hq, T, dtype=torch.float64, device=DEV)
    rows = [(b, 0, T) for b in range(B)] if not case["packed"] else \
        [(0, a, e) for a, e in zip(s["cu"].tolist()[:-1], s["cu"].tolist()[1:])]
    for b, a, e in rows:
        for t in range(a, e, 1024):
            u = min(e, t + 1024)
            lo = max(a, t - W + 1)
            near = torch.arange(lo, u, device=DEV)
            first = torch.arange(a, min(a + S, lo), device=DEV)
            keys = torch.cat([first, near])
            i = torch.arange(t, u, device=DEV)[:, None]
            hidden = (keys[None] > i) | ((i - keys[None] >= W) & (keys[None] - a >= S))
            for h in range(Hq):
                qb, kb, vb = (x.detach().requires_grad_(train) for x in (q[b, t:u, h], k[b, keys, h // G], v[b, keys, h // G]))
                w = (qb @ kb.T / math.sqrt(D)).masked_fill(hidden, -math.inf)
                ob = torch.softmax(w, -1) @ vb
                o[b, t:u, h], lse[b, h, t:u] = ob.detach(), torch.logsumexp(w.detach(), -1)
                if train:
                    gq, gk, gv = torch.autograd.grad((ob * s["do"][b, t:u, h].double()).sum(), (qb, kb, vb))
                    dq[b, t:u, h] = gq
                    dk[b, :, h // G].index_add_(0, keys, gk)
                    dv[b, :, h // G].index_add_(0, keys, gv)
    return (o, (dq, dk, dv)) if train else (o, lse)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _pairs(T, W, S):
    """Pairs of a query and a key that it sees, for one head and sequence of T steps."""
    near = T * (T + 1) // 2 if T <= W else W * (W + 1) // 2 + (T - W) * W
    # query i sees min(S, i + 1 - W) first keys beyond its window
    n = max(0, T - W)
    far = n * (n + 1) // 2 if n <= S else S * (S + 1) // 2 + (n - S) * S
    return near + far


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op == "rope":
        n = case["B"] * case["T"] * (case["Hq"] + case["Hk"])
        rows = n * case["D"] * e
        tables = min(8192, case["B"] * case["T"]) * case["R"] * 4
        if case["train"]:
            return {"bytes": 4 * rows + tables, "flops": n * case["D"] * 25}
        return {"bytes": 2 * rows + tables, "flops": n * case["D"] * 8}
    if op == "linear_step":
        n = case["B"] * case["H"]
        return {"bytes": n * (8 * case["Dk"] * case["Dv"] + e * 2 * (case["Dk"] + case["Dv"])),
                "flops": 5 * n * case["Dk"] * case["Dv"]}
    if op == "linear":
        n, Dk, Dv = case["B"] * case["T"] * case["H"], case["Dk"], case["Dv"]
        states = (case["packed"] or case["B"]) * case["H"] * Dk * Dv * 4
        if case["train"]:  # q, k, v, do in; o, dq, dk, dv out; two reads and an update of the state each way
            return {"bytes": n * 4 * (Dk + Dv) * e + (2 * states if case["state"] else 0), "flops": 12 * n * Dk * Dv}
        return {"bytes": n * 2 * (Dk + Dv) * e + states * (2 if case["state"] else 1), "flops": 4 * n * Dk * Dv}
    D = case["D"]
    if op == "window":
        T = case["T"]
        if case["packed"]:  # as of sequences of one length
            pairs = case["packed"] * _pairs(max(1, T // case["packed"]), case["W"], case["S"])
        else:
            pairs = case["B"] * _pairs(T, case["W"], case["S"])
        n = case["B"] * T
        if case["train"]:
            return {"bytes": n * D * e * 4 * (case["Hq"] + case["Hk"]), "flops": 14 * pairs * D * case["Hq"]}
        return {"bytes": n * D * e * 2 * (case["Hq"] + case["Hk"]) + n * 4 * case["Hq"], "flops": 4 * pairs * D * case["Hq"]}
    # positions are drawn evenly from W / 2 (or past the window) to 4 W
    kept = (case["S"] + case["W"]) * (1.0 if case["B"] == 1 else 0.96)
    return {"bytes": case["B"] * (kept * 2 * case["Hk"] + 2 * (case["Hq"] + case["Hk"])) * D * e,
            "flops": case["B"] * kept * 4 * case["Hq"] * D}
