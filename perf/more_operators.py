"""Workloads of the state-space layer's operators, and their plain forms.

Three operators and their gradients, as a layer built on a selective state
space runs them on a prompt, in training and token by token:

  causal convolution     y[t] = act(bias + sum over j of weight[j] x[t - K + 1 + j]),
                         a channel at a time ("conv"), its gradient
                         ("conv_train") and one token of many requests ("conv_step")
  selective scan         h[t] = exp(dt a) h[t-1] + dt x[t] b[t],  y[t] = c[t] . h[t] + skip x[t],
                         with dt = softplus(delta + bias) a channel and token, gated
                         by z ("scan"), its gradient ("scan_train") and one token
                         of many requests ("scan_step")
  group norm             of channels that lie last, with an activation: of
                         each token ("norm", s = 1) or over a whole sequence,
                         and its gradient ("norm_train")

With ``own`` false, ``run`` computes them from elementary torch operations;
with ``own`` true it calls this repository's package.
"""

import math

import torch

own = False

if torch.cuda.is_available():
    DEV = torch.device("cuda", 0)
else:
    DEV = torch.device("cpu")
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # one request's next token in a small model: latency alone
        dict(name="scan step one request", op="scan_step", b=1, pool=1, d=1536, n=16, g=1, type="bf16", gate=True),
        # the next token of a full serving batch, states in a pool, a few rows idle
        dict(name="scan step full batch", op="scan_step", b=128, pool=144, d=4096, n=16, g=1, type="bf16", gate=True),
        # a long document after a cached prefix: one sequence
        dict(name="scan prompt long", op="scan", b=1, t=8192, d=4096, n=16, g=1, type="bf16", gate=True,
             initial=True, ragged=False),
        # a padded batch in full precision, odd sizes, two groups of input and readout rows
        dict(name="scan prompt f32 odd", op="scan", b=5, t=777, d=330, n=12, g=2, type="f32", gate=False,
             initial=True, ragged=True),
        # a training step of an ordinary layer
        dict(name="scan train bf16", op="scan_train", b=4, t=2048, d=2048, n=16, g=1, type="bf16", gate=True,
             initial=False, ragged=False),
        # full-precision gradients: odd sizes, a state carried in and a gradient of the last one
        dict(name="scan train f32 odd", op="scan_train", b=3, t=333, d=210, n=10, g=3, type="f32", gate=False,
             initial=True, ragged=True),
        # the convolution before the scan, over a padded batch of prompts
        dict(name="conv prompts", op="conv", b=8, t=2048, d=4096, k=4, type="bf16", act=True, initial=False,
             ragged=True),
        # the same for one token of a full serving batch
        dict(name="conv step full batch", op="conv_step", b=128, pool=144, d=4096, k=4, type="bf16", act=True),
        # its gradient in full precision, odd sizes, a state carried in
        dict(name="conv train f32 odd", op="conv_train", b=3, t=1111, d=1050, k=3, type="f32", act=True,
             initial=True, ragged=True),
        # every token's heads normed on their own, as what leaves a linear-attention layer is
        dict(name="norm heads of tokens", op="norm", n=16384, s=1, c=2048, g=16, type="bf16", act=True),
        # a training step of a norm over whole sequences
        dict(name="norm sequences train", op="norm_train", n=8, s=4096, c=512, g=32, type="bf16", act=True),
        # full-precision gradients of odd groups, token by token
        dict(name="norm train f32 odd", op="norm_train", n=2000, s=1, c=370, g=5, type="f32", act=False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_train", "scan_step", "conv", "conv_train", "conv_step", "norm", "norm_train"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_train"):
        g = rng.choice([1, 2, 4, 5, 8, 16, 32])
        c = g * _spread(rng, 2, 4096 // g)
        s = rng.choice([1, _spread(rng, 2, 4096)])
        most = 16384 * 2048 // (1 if op == "norm" else 2) // (1 if kind == "bf16" else 2)
        n = max(1, min(_spread(rng, 1, 16384 if s == 1 else 16), most // (s * c)))
        return dict(op=op, n=n, s=s, c=c, g=g, type=kind, act=rng.random() < 0.5)
    g = rng.choice([1, 1, 2, 4])
    d = g * _spread(rng, 32, 4096 // g)
    if rng.random() < 0.6:
        d = max(64 * g, d // (64 * g) * 64 * g)
    if op.startswith("conv"):
        k = rng.choice([2, 3, 4, 4])
        act = rng.random() < 0.7
        if op == "conv_step":
            b = _spread(rng, 1, 128)
            return dict(op=op, b=b, pool=b + rng.randint(0, 16), d=d, k=k, type=kind, act=act)
        t = _spread(rng, 1, 8192)
        b = max(1, min(_spread(rng, 1, 16), 8 * 2048 * 2048 // (t * d)))
        return dict(op=op, b=b, t=t, d=d, k=k, type=kind, act=act, initial=rng.random() < 0.5,
                    ragged=rng.random() < 0.4)
    n = rng.choice([16, 16, 16, rng.randint(1, 16), 32])
    gate = rng.random() < 0.6
    if op == "scan_step":
        b = _spread(rng, 1, 128)
        return dict(op=op, b=b, pool=b + rng.randint(0, 16), d=d, n=min(n, 16), g=g, type=kind, gate=gate)
    most = (8192 * 4096 if op == "scan" else 4 * 2048 * 1024) * 16 // max(n, 16)
    t = min(_spread(rng, 1, 8192), most // d)
    b = max(1, min(_spread(rng, 1, 8), most // (t * d)))
    return dict(op=op, b=b, t=t, d=d, n=n, g=g, type=kind, gate=gate, initial=rng.random() < 0.5,
                ragged=rng.random() < 0.4)


# ---------------------------------------------------------------- inputs

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _uniform(gen, *shape):
    return torch.rand(shape, generator=gen, device=DEV, dtype=torch.float32)


def _slots(gen, b, pool):
    slots = torch.randperm(pool, generator=gen, device=DEV)[:b].to(torch.int32)
    if b >= 8:  # rows of the batch that hold no request
        slots[torch.randperm(b, generator=gen, device=DEV)[:b // 16 + 1]] = -1
    return slots


def _lengths(gen, c):
    if not c["ragged"]:
        return None
    lengths = torch.randint(0, c["t"] + 1, (c["b"],), generator=gen, device=DEV, dtype=torch.int32)
    lengths[0] = c["t"]
    return lengths


def _prepare_norm(c, gen, ty):
    shape = (c["n"], c["c"]) if c["s"] == 1 else (c["n"], c["s"], c["c"])
    s = {"case": c, "x": (_normal(gen, *shape) * (0.5 + _uniform(gen, c["c"])) + 0.5 * _normal(gen, c["c"])).to(ty)}
    s["w"], s["bias"] = 1 + 0.2 * _normal(gen, c["c"]), 0.2 * _normal(gen, c["c"])
    if c["op"] == "norm_train":
        s["go"] = _normal(gen, *shape).to(ty)
    return s


def _prepare_conv(c, gen, ty):
    b, d, k = c["b"], c["d"], c["k"]
    t = c.get("t", 1)
    # the inputs are one half of a projection's output, the gate the other
    s = {"case": c, "x": _normal(gen, b, t, 2 * d).to(ty)[..., :d]}
    s["w"], s["bias"] = (2 * _uniform(gen, d, k) - 1) * k ** -0.5, (2 * _uniform(gen, d) - 1) * k ** -0.5
    if c["op"] == "conv_step":
        s["x"] = s["x"][:, 0]
        s["state"] = _normal(gen, c["pool"], k - 1, d).to(ty)
        s["slots"] = _slots(gen, b, c["pool"])
        return s
    s["initial"] = _normal(gen, b, k - 1, d).to(ty) if c["initial"] else None
    s["lengths"] = _lengths(gen, c)
    if c["op"] == "conv_train":
        s["go"] = _normal(gen, b, t, d).to(ty)
        s["gs"] = _normal(gen, b, k - 1, d).to(ty) if c["initial"] else None
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    c, ty = case, TYPES[case["type"]]
    if c["op"].startswith("norm"):
        return _prepare_norm(c, gen, ty)
    if c["op"].startswith("conv"):
        return _prepare_conv(c, gen, ty)
    b, d, n, g = c["b"], c["d"], c["n"], c["g"]
    t = c.get("t", 1)
    s = {"case": c}
    # what leaves the convolution; the gate is half of a projection's output
    x = _normal(gen, b, t, d)
    s["x"] = (x * torch.sigmoid(x)).to(ty)
    s["z"] = _normal(gen, b, t, 2 * d).to(ty)[..., d:] if c["gate"] else None
    # rows of input and readout are slices of one projection, a narrow piece of delta's in front of them
    bc = _normal(gen, b, t, d // 16 + 1 + 2 * g * n).to(ty)[..., d // 16 + 1:]
    s["b"], s["c"] = bc[..., :g * n].view(b, t, g, n), bc[..., g * n:].view(b, t, g, n)
    # steps of 1e-3 to 1e-1 as softplus(bias) sets them, moved by the token; rates of 1 to n
    s["delta"] = (0.5 * _normal(gen, b, t, d)).to(ty)
    dt = torch.exp(_uniform(gen, d) * math.log(100.0) + math.log(1e-3))
    s["dbias"] = dt + torch.log(-torch.expm1(-dt))
    s["a"] = -torch.arange(1, n + 1, device=DEV, dtype=torch.float32) * (0.5 + _uniform(gen, d, n))
    s["skip"] = 1 + 0.1 * _normal(gen, d)
    if c["op"] == "scan_step":
        for name in ("x", "z", "b", "c", "delta"):
            if s[name] is not None:
                s[name] = s[name][:, 0]
        s["state"] = _normal(gen, c["pool"], d, n)
        s["slots"] = _slots(gen, b, c["pool"])
        return s
    s["initial"] = _normal(gen, b, d, n) if c["initial"] else None
    s["lengths"] = _lengths(gen, c)
    if c["op"] == "scan_train":
        s["go"] = _normal(gen, b, t, d).to(ty)
        s["gs"] = _normal(gen, b, d, n) if c["initial"] else None
    return s


# ---------------------------------------------------------------- the plain forms

def _silu(u):
    return u * torch.sigmoid(u)


def _silu_slope(u):
    p = torch.sigmoid(u)
    return p * (1 + u * (1 - p))


def _live(s, t):
    b = s["x"].shape[0]
    if s["lengths"] is None:
        return torch.ones(b, t, dtype=torch.bool, device=DEV)
    return torch.arange(t, device=DEV)[None, :] < s["lengths"][:, None]


def _window(s):
    """The inputs in 32 bits with the K - 1 before them in front, [B, K - 1 + T, D], and which tokens there are."""
    b, t, d = s["x"].shape
    k = s["w"].shape[1]
    live = _live(s, t)
    x = torch.where(live[..., None], s["x"].float(), 0.0)
    front = x.new_zeros(b, k - 1, d) if s["initial"] is None else s["initial"].float()
    return torch.cat([front, x], 1), live


def _last_inputs(s, seen):
    """Where the last K - 1 inputs of each row stand in the window, [B, K - 1, D]."""
    b, t, d = s["x"].shape
    k = s["w"].shape[1]
    n = torch.full((b,), t, device=DEV) if s["lengths"] is None else s["lengths"].long()
    return (n[:, None] + torch.arange(k - 1, device=DEV))[..., None].expand(b, k - 1, d)


def _plain_conv(s):
    c, t = s["case"], s["x"].shape[1]
    k, ty = c["k"], s["x"].dtype
    x, live = _window(s)
    u = s["bias"].expand(s["x"].shape).float()
    for j in range(k):
        u = u + s["w"][:, j] * x[:, j:j + t]
    y = _silu(u) if c["act"] else u
    return torch.where(live[..., None], y, 0.0).to(ty), x.gather(1, _last_inputs(s, x)).to(ty)


def _plain_conv_train(s):
    c, t = s["case"], s["x"].shape[1]
    k, ty = c["k"], s["x"].dtype
    x, live = _window(s)
    u = s["bias"].expand(s["x"].shape).float()
    for j in range(k):
        u = u + s["w"][:, j] * x[:, j:j + t]
    gu = s["go"].float() * _silu_slope(u) if c["act"] else s["go"].float()
    gu = torch.where(live[..., None], gu, 0.0)
    gx = torch.zeros_like(x)
    for j in range(k):
        gx[:, j:j + t] += s["w"][:, j] * gu
    if s["gs"] is not None:
        gx.scatter_add_(1, _last_inputs(s, x), s["gs"].float())
    gw = torch.stack([(gu * x[:, j:j + t]).sum((0, 1)) for j in range(k)], 1)
    got = [torch.where(live[..., None], gx[:, k - 1:], 0.0).to(ty), gw, gu.sum((0, 1))]
    return got + [gx[:, :k - 1].to(ty)] if s["initial"] is not None else got


def _plain_conv_step(s):
    c = s["case"]
    used = (s["slots"] >= 0) & (s["slots"] < c["pool"])
    at = torch.where(used, s["slots"], 0).long()
    x = torch.cat([s["state"][at].float(), s["x"].float()[:, None]], 1)
    u = (s["w"].t() * x).sum(1) + s["bias"]
    y = _silu(u) if c["act"] else u
    s["state"][at[used]] = x[used, 1:].to(s["state"].dtype)
    return torch.where(used[:, None], y, 0.0).to(s["x"].dtype), s["state"]


def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(v.clamp_max(20.0))))


def _recurrence(a, b):
    """h[t] = a[t] h[t-1] + b[t] along dim 1, from zero: spans of twice the length joined until one is left."""
    span = 1
    while span < b.shape[1]:
        b = torch.cat([b[:, :span], a[:, span:] * b[:, :-span] + b[:, span:]], 1)
        a = torch.cat([a[:, :span], a[:, span:] * a[:, :-span]], 1)
        span *= 2
    return b


def _rows(x, d):
    """[B, T, G, N] in 32 bits, each group's row given to its channels, [B, T, D, N]."""
    return x.float().repeat_interleave(d // x.shape[2], dim=2)


def _states(s):
    """The steps dt, decays, states before and after each token, and which tokens there are."""
    b, t, d = s["x"].shape
    live = _live(s, t)
    v = s["delta"].float() + s["dbias"]
    dt = torch.where(live[..., None], _softplus(v), 0.0)
    x = torch.where(live[..., None], s["x"].float(), 0.0)
    decay = torch.exp(dt[..., None] * s["a"])
    rows = torch.where(live[..., None, None], _rows(s["b"], d), 0.0)
    source = (dt * x)[..., None] * rows
    start = source.new_zeros(b, d, s["a"].shape[1]) if s["initial"] is None else s["initial"]
    source[:, 0] += decay[:, 0] * start
    h = _recurrence(decay, source)
    return v, dt, x, decay, rows, h, start, live


def _plain_scan(s):
    d = s["x"].shape[-1]
    v, dt, x, decay, rows, h, start, live = _states(s)
    del decay, rows
    y = (torch.where(live[..., None, None], _rows(s["c"], d), 0.0) * h).sum(-1) + s["skip"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return torch.where(live[..., None], y, 0.0).to(s["x"].dtype), h[:, -1].contiguous()


def _grouped(x, g):
    """The sum over the channels of each group, [B, T, D, N] to [B, T, G, N]."""
    b, t, d, n = x.shape
    return x.view(b, t, g, d // g, n).sum(3)


def _plain_scan_train(s):
    c, d, ty = s["case"], s["x"].shape[-1], s["x"].dtype
    v, dt, x, decay, rows, h, start, live = _states(s)
    readout = torch.where(live[..., None, None], _rows(s["c"], d), 0.0)
    gy = torch.where(live[..., None], s["go"].float(), 0.0)
    gz = None
    if s["z"] is not None:
        z = torch.where(live[..., None], s["z"].float(), 0.0)
        y = (readout * h).sum(-1) + s["skip"] * x
        gz = gy * y * _silu_slope(z)
        gy = gy * _silu(z)
    # the adjoint of the state after each token, last to first
    into = readout * gy[..., None]
    if s["gs"] is not None:
        into[:, -1] += s["gs"]
    later = torch.cat([torch.ones_like(decay[:, :1]), decay[:, 1:].flip(1)], 1)
    adj = _recurrence(later, into.flip(1)).flip(1)
    del into, later
    gc = _grouped(gy[..., None] * h, c["g"]).to(ty)
    gb = _grouped((dt * x)[..., None] * adj, c["g"]).to(ty)
    before = torch.cat([start[:, None], h[:, :-1]], 1)
    carried = adj * decay * before
    g_initial = decay[:, 0] * adj[:, 0]
    sourced = (adj * rows).sum(-1)
    gdt = (carried * s["a"]).sum(-1) + x * sourced
    gdelta = torch.where(live[..., None], gdt * torch.sigmoid(v), 0.0)
    gx = torch.where(live[..., None], dt * sourced + s["skip"] * gy, 0.0)
    got = [gx.to(ty), gdelta.to(ty), (dt[..., None] * carried).sum((0, 1)), gb, gc, (gy * x).sum((0, 1)),
           gdelta.sum((0, 1))]
    if gz is not None:
        got.append(gz.to(ty))
    return got + [g_initial] if s["initial"] is not None else got


def _plain_scan_step(s):
    c, d = s["case"], s["x"].shape[-1]
    used = (s["slots"] >= 0) & (s["slots"] < c["pool"])
    at = torch.where(used, s["slots"], 0).long()
    x, dt = s["x"].float(), _softplus(s["delta"].float() + s["dbias"])
    b, r = (_rows(s[name][:, None], d)[:, 0] for name in ("b", "c"))
    new = torch.exp(dt[..., None] * s["a"]) * s["state"][at] + (dt * x)[..., None] * b
    y = (new * r).sum(-1) + s["skip"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["state"][at[used]] = new[used]
    return torch.where(used[:, None], y, 0.0).to(s["x"].dtype), s["state"]


def _normed(s):
    c = s["case"]
    x = s["x"].float().view(c["n"], c["s"], c["g"], c["c"] // c["g"])
    off = x - x.mean((1, 3), keepdim=True)
    r = torch.rsqrt((off * off).mean((1, 3), keepdim=True) + EPS)
    n = off * r
    w, bias = (s[name].view(c["g"], -1) for name in ("w", "bias"))
    return n, r, w, n * w + bias


def _plain_norm(s):
    n, r, w, u = _normed(s)
    return (_silu(u) if s["case"]["act"] else u).to(s["x"].dtype).view(s["x"].shape)


def _plain_norm_train(s):
    c = s["case"]
    n, r, w, u = _normed(s)
    gu = s["go"].float().view(n.shape)
    if c["act"]:
        gu = gu * _silu_slope(u)
    gn = gu * w
    gx = r * (gn - gn.mean((1, 3), keepdim=True) - n * (gn * n).mean((1, 3), keepdim=True))
    return gx.to(s["x"].dtype).view(s["x"].shape), (gu * n).sum((0, 1)).view(-1), gu.sum((0, 1)).view(-1)


# ---------------------------------------------------------------- the calls

def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"conv": _plain_conv, "conv_train": _plain_conv_train, "conv_step": _plain_conv_step,
                "scan": _plain_scan, "scan_train": _plain_scan_train, "scan_step": _plain_scan_step,
                "norm": _plain_norm, "norm_train": _plain_norm_train}[op](s)
    import scan_primitives_amd as sx
    act = "silu" if c.get("act") else None
    if op == "conv":
        return sx.causal_conv(s["x"], s["w"], bias=s["bias"], initial=s["initial"], lengths=s["lengths"],
                              activation=act, return_state=True)
    if op == "conv_train":
        got = sx.causal_conv_backward(s["x"], s["w"], s["go"], bias=s["bias"], initial=s["initial"],
                                      lengths=s["lengths"], activation=act, grad_state=s["gs"])
        return list(got) if s["initial"] is not None else list(got[:3])
    if op == "conv_step":
        y = sx.causal_conv_step(s["x"], s["w"], s["state"], bias=s["bias"], slots=s["slots"], activation=act)
        return y, s["state"]
    if op == "scan":
        return sx.selective_scan(s["x"], s["delta"], s["a"], s["b"], s["c"], skip=s["skip"], z=s["z"],
                                 delta_bias=s["dbias"], initial=s["initial"], lengths=s["lengths"], return_state=True)
    if op == "scan_train":
        gx, gdelta, ga, gb, gc, gskip, gz, gdbias, gi = sx.selective_scan_backward(
            s["x"], s["delta"], s["a"], s["b"], s["c"], s["go"], skip=s["skip"], z=s["z"], delta_bias=s["dbias"],
            initial=s["initial"], lengths=s["lengths"], grad_state=s["gs"])
        return [gx, gdelta, ga, gb, gc, gskip, gdbias] + ([gz] if s["z"] is not None else []) + (
            [gi] if s["initial"] is not None else [])
    if op == "scan_step":
        y = sx.selective_scan_step(s["x"], s["delta"], s["a"], s["b"], s["c"], s["state"], slots=s["slots"],
                                   skip=s["skip"], z=s["z"], delta_bias=s["dbias"])
        return y, s["state"]
    if op == "norm":
        return sx.group_norm(s["x"], c["g"], weight=s["w"], bias=s["bias"], eps=EPS, activation=act)
    return list(sx.group_norm_backward(s["x"], c["g"], s["go"], weight=s["w"], bias=s["bias"], eps=EPS,
                                       activation=act))


def work(case):
    c = case
    e = 2 if c["type"] == "bf16" else 4
    op = c["op"]
    if op in ("norm", "norm_train"):
        numel = c["n"] * c["s"] * c["c"]
        act = 6 if c["act"] else 0
        if op == "norm":
            return {"bytes": 2 * e * numel + 8 * c["c"], "flops": (7 + act) * numel}
        return {"bytes": 3 * e * numel + 16 * c["c"], "flops": (17 + 2 * act) * numel}
    b, d = c["b"], c["d"]
    t = c.get("t", 1)
    live = b * t
    if op.endswith("_step"):
        live = b - (b // 16 + 1 if b >= 8 else 0)
    elif c["ragged"]:
        live = b * t * (0.5 + 0.5 / b)  # lengths are spread evenly, the first is whole
    if op.startswith("conv"):
        k = c["k"]
        weights, act = 4 * d * (k + 1), 6 if c["act"] else 0
        state = e * b * (k - 1) * d
        if op == "conv_step":
            return {"bytes": e * live * d * (1 + 2 * (k - 1)) + e * b * d + weights + 4 * b,
                    "flops": (2 * k + act) * live * d}
        if op == "conv":
            return {"bytes": e * d * (live + b * t) + weights + state * (2 if c["initial"] else 1),
                    "flops": (2 * k + act) * live * d}
        return {"bytes": e * d * (2 * live + b * t) + 2 * weights + (3 * state if c["initial"] else 0),
                "flops": (6 * k + 2 * act) * live * d}
    n, g = c["n"], c["g"]
    weights = 4 * d * (n + 2)
    rows = 2 * e * g * n
    state = 4 * d * n
    wide = 3 if c["gate"] else 2  # x, delta and the gate
    if op == "scan_step":
        return {"bytes": live * (2 * state + e * d * wide + rows) + e * b * d + weights + 4 * b,
                "flops": live * d * (7 * n + 20)}
    if op == "scan":
        return {"bytes": live * (e * d * wide + rows) + e * b * t * d + weights
                + b * state * (2 if c["initial"] else 1), "flops": live * d * (7 * n + 20)}
    return {"bytes": live * (e * d * (wide + 1) + rows) + b * t * (e * d * wide + rows) + 2 * weights
            + (3 * b * state if c["initial"] else 0), "flops": live * d * (21 * n + 40)}


# ---------------------------------------------------------------- the definitions in 64 bits

def _taps(x, w):
    """Products with each tap as a convolution over [B, D, K - 1 + T]: one row a channel."""
    d, k = w.shape
    return sum(w[None, :, j, None] * x[:, :, j:x.shape[2] - (k - 1 - j)] for j in range(k))


def _exact_conv(s):
    """One row after the other, with only the tokens that it has."""
    c = s["case"]
    b, t, d = s["x"].shape
    k, f64 = c["k"], torch.float64
    train = c["op"] == "conv_train"
    w, bias = s["w"].double(), s["bias"].double()
    y = torch.zeros(b, t, d, dtype=f64, device=DEV)
    last = torch.zeros(b, k - 1, d, dtype=f64, device=DEV)
    gx, gi, gw, gb = torch.zeros_like(y), torch.zeros_like(last), torch.zeros_like(w), torch.zeros_like(bias)
    for i in range(b):
        n = t if s["lengths"] is None else int(s["lengths"][i])
        front = torch.zeros(k - 1, d, dtype=f64, device=DEV) if s["initial"] is None else s["initial"][i].double()
        x = torch.cat([front, s["x"][i, :n].double()]).t().contiguous()
        if train:
            x.requires_grad_()
        wi, bi = w.clone().requires_grad_(train), bias.clone().requires_grad_(train)
        u = _taps(x[None], wi)[0] + bi[:, None] if n > 0 else x[:, :0]
        out = u / (1 + torch.exp(-u)) if c["act"] else u
        if not train:
            y[i, :n], last[i] = out.t(), x[:, n:].t()
            continue
        loss = (out * s["go"][i, :n].double().t()).sum() + 0 * (x.sum() + wi.sum() + bi.sum())
        if s["gs"] is not None:
            loss = loss + (x[:, n:] * s["gs"][i].double().t()).sum()
        dx, dw, db = torch.autograd.grad(loss, (x, wi, bi))
        gx[i, :n], gi[i] = dx[:, k - 1:].t(), dx[:, :k - 1].t()
        gw += dw
        gb += db
    if not train:
        return y, last
    return [gx, gw, gb, gi] if s["initial"] is not None else [gx, gw, gb]


def _exact_conv_step(s):
    c = s["case"]
    state = s["state"].double().clone()
    y = torch.zeros(c["b"], c["d"], dtype=torch.float64, device=DEV)
    for i, slot in enumerate(s["slots"].tolist()):
        if not 0 <= slot < c["pool"]:
            continue
        x = torch.cat([state[slot], s["x"][i:i + 1].double()])
        u = torch.einsum("dk,kd->d", s["w"].double(), x) + s["bias"].double()
        y[i] = u / (1 + torch.exp(-u)) if c["act"] else u
        state[slot] = x[1:]
    return y, state


def _wide_rows(x, d):
    """A token's rows [B, G, N] in 64 bits, [B, D, N]."""
    return x.double().repeat_interleave(d // x.shape[1], dim=1)


def _steps(v):
    return torch.clamp_min(v, 0) + torch.log1p(torch.exp(-v.abs()))


def _exact_scan(s):
    """Token after token."""
    c = s["case"]
    b, t, d = s["x"].shape
    n, g, f64 = c["n"], c["g"], torch.float64
    a = s["a"].double()
    lengths = torch.full((b,), t, device=DEV) if s["lengths"] is None else s["lengths"]
    h = torch.zeros(b, d, n, dtype=f64, device=DEV) if s["initial"] is None else s["initial"].double()
    train = c["op"] == "scan_train"
    y = torch.zeros(b, t, d, dtype=f64, device=DEV)
    kept = torch.empty(t + 1, b, d, n, dtype=f64, device=DEV) if train else None
    for i in range(t):
        if train:
            kept[i] = h
        on = (i < lengths)[:, None]
        dt = _steps(s["delta"][:, i].double() + s["dbias"].double())
        x = s["x"][:, i].double()
        new = torch.exp(dt[..., None] * a) * h + (dt * x)[..., None] * _wide_rows(s["b"][:, i], d)
        h = torch.where(on[..., None], new, h)
        y[:, i] = torch.where(on, (h * _wide_rows(s["c"][:, i], d)).sum(-1) + s["skip"].double() * x, 0.0)
    if not train:
        if s["z"] is not None:
            z = s["z"].double()
            y = torch.where((torch.arange(t, device=DEV)[None] < lengths[:, None])[..., None], y * z / (1 + torch.exp(-z)),
                            0.0)
        return y, h
    kept[t] = h
    gx, gdelta, gz = (torch.zeros_like(y) for _ in range(3))
    ga, gskip, gdbias = torch.zeros_like(a), torch.zeros(d, dtype=f64, device=DEV), torch.zeros(d, dtype=f64, device=DEV)
    gb, gc = (torch.zeros(b, t, g, n, dtype=f64, device=DEV) for _ in range(2))
    adj = torch.zeros_like(h) if s["gs"] is None else s["gs"].double()
    for i in range(t - 1, -1, -1):
        on = (i < lengths)[:, None]
        v = s["delta"][:, i].double() + s["dbias"].double()
        dt, x = _steps(v), s["x"][:, i].double()
        gy = torch.where(on, s["go"][:, i].double(), 0.0)
        if s["z"] is not None:
            z = s["z"][:, i].double()
            p = 1 / (1 + torch.exp(-z))
            gz[:, i] = gy * y[:, i] * (p + z * p * (1 - p))
            gy = gy * z * p
        here = adj + gy[..., None] * _wide_rows(s["c"][:, i], d)
        gc[:, i] = (gy[..., None] * kept[i + 1]).view(b, g, d // g, n).sum(2)
        gb[:, i] = torch.where(on[..., None], ((dt * x)[..., None] * here).view(b, g, d // g, n).sum(2), 0.0)
        back = torch.exp(dt[..., None] * a) * here
        turned = torch.where(on[..., None], back * kept[i], 0.0)
        ga += (dt[..., None] * turned).sum(0)
        by_source = (here * _wide_rows(s["b"][:, i], d)).sum(-1)
        gd = torch.where(on, ((turned * a).sum(-1) + x * by_source) / (1 + torch.exp(-v)), 0.0)
        gdelta[:, i] = gd
        gdbias += gd.sum(0)
        gx[:, i] = torch.where(on, dt * by_source + s["skip"].double() * gy, 0.0)
        gskip += (gy * x).sum(0)
        adj = torch.where(on[..., None], back, adj)
    got = [gx, gdelta, ga, gb, gc, gskip, gdbias] + ([gz] if s["z"] is not None else [])
    return got + [adj] if s["initial"] is not None else got


def _exact_scan_step(s):
    """One request after the other."""
    c, d = s["case"], s["x"].shape[-1]
    state = s["state"].double().clone()
    y = torch.zeros(c["b"], d, dtype=torch.float64, device=DEV)
    for i, slot in enumerate(s["slots"].tolist()):
        if not 0 <= slot < c["pool"]:
            continue
        x = s["x"][i].double()
        dt = _steps(s["delta"][i].double() + s["dbias"].double())
        b, r = (_wide_rows(s[name][i:i + 1], d)[0] for name in ("b", "c"))
        state[slot] = state[slot] * torch.exp(dt[:, None] * s["a"].double()) + torch.einsum("d,dn->dn", dt * x, b)
        y[i] = torch.einsum("dn,dn->d", state[slot], r) + s["skip"].double() * x
        if s["z"] is not None:
            z = s["z"][i].double()
            y[i] *= z / (1 + torch.exp(-z))
    return y, state


def _exact_norm(s):
    """Means by sums over a group's elements; the gradient as that of the variance's root, in parts."""
    c = s["case"]
    m = c["s"] * (c["c"] // c["g"])
    x = s["x"].double().view(c["n"], c["s"], c["g"], -1).transpose(1, 2).reshape(c["n"], c["g"], m)
    mean = x.sum(-1, keepdim=True) / m
    root = torch.sqrt(((x - mean) ** 2).sum(-1, keepdim=True) / m + EPS)

    def spread(v):  # a channel's value to [1, G, S Cg]
        return v.double().view(1, c["g"], 1, -1).expand(1, c["g"], c["s"], -1).reshape(1, c["g"], m)

    def back(v):
        return v.view(c["n"], c["g"], c["s"], -1).transpose(1, 2).reshape(s["x"].shape)

    n = (x - mean) / root
    u = n * spread(s["w"]) + spread(s["bias"])
    if c["op"] == "norm":
        return back(u / (1 + torch.exp(-u)) if c["act"] else u)
    go = s["go"].double().view(c["n"], c["s"], c["g"], -1).transpose(1, 2).reshape(c["n"], c["g"], m)
    if c["act"]:
        p = 1 / (1 + torch.exp(-u))
        go = go * (p + u * p * (1 - p))
    per = go * spread(s["w"])
    g_root = -(per * (x - mean)).sum(-1, keepdim=True) / root ** 2
    gx = per / root + g_root * (x - mean) / (m * root)
    gx = gx - gx.sum(-1, keepdim=True) / m

    def channels(v):
        return v.view(c["n"], c["g"], c["s"], -1).sum((0, 2)).reshape(-1)

    return back(gx), channels(go * n), channels(go)


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "conv_train": _exact_conv, "conv_step": _exact_conv_step, "scan": _exact_scan,
            "scan_train": _exact_scan, "scan_step": _exact_scan_step, "norm": _exact_norm,
            "norm_train": _exact_norm}[case["op"]](s)
