"""Workloads of the linear-attention operators, and their plain forms.

Two operators and their gradients, as a decoder with linear attention runs
them on a prompt, in training and token by token:

  decay attention        S[t] = exp(g[t]) S[t-1] + k[t] v[t]^T,  o[t] = scale S[t]^T q[t]
                         over a prompt ("prompt"), its gradient ("train") and
                         one token of many requests ("step")
  head norm + rotation   a root-mean-square norm of each head of q and k and
                         the position rotation ("rotate"), and its gradient
                         ("rotate_train")

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
CHUNK = 64


def listed():
    return [
        # one request's next token in a small model: latency alone
        dict(name="step one request", op="step", b=1, pool=1, h=4, hq=4, hv=4, dk=64, dv=64, type="bf16"),
        # the next token of a full serving batch, states in a pool, a few rows idle
        dict(name="step full batch", op="step", b=64, pool=80, h=16, hq=16, hv=16, dk=128, dv=128, type="bf16"),
        # a short question: less than one tile of tokens
        dict(name="prompt short", op="prompt", b=1, t=37, h=4, hq=4, hv=4, dk=64, dv=64, type="bf16", decay="head",
             initial=False, ragged=False),
        # a long document after a cached prefix: one sequence, few heads
        dict(name="prompt long", op="prompt", b=1, t=8192, h=16, hq=16, hv=16, dk=128, dv=128, type="bf16",
             decay="token", initial=True, ragged=False),
        # a padded batch of prompts; one query and key head serves all value heads, documents reset the state
        dict(name="prompt ragged shared", op="prompt", b=8, t=2048, h=16, hq=1, hv=16, dk=64, dv=64, type="bf16",
             decay="reset", initial=False, ragged=True),
        # full precision, odd head sizes
        dict(name="prompt f32 odd", op="prompt", b=2, t=777, h=6, hq=6, hv=3, dk=40, dv=72, type="f32",
             decay="token", initial=True, ragged=False),
        # a training step of an ordinary layer
        dict(name="train bf16", op="train", b=4, t=4096, h=8, hq=8, hv=8, dk=128, dv=128, type="bf16", decay="token",
             initial=False, ragged=False),
        # full-precision gradients: shared heads, per-head decay, a state carried in and a gradient of the last one
        dict(name="train f32 odd", op="train", b=2, t=333, h=6, hq=2, hv=6, dk=48, dv=80, type="f32", decay="head",
             initial=True, ragged=True),
        # one token's queries and keys, far into a document
        dict(name="rotate one token", op="rotate", b=1, t=1, hq=32, hk=8, d=128, rot=128, type="bf16", pairs="half",
             first=1000003),
        # the queries and keys of a batch of prompts
        dict(name="rotate prompts", op="rotate", b=4, t=4096, hq=16, hk=16, d=128, rot=128, type="bf16", pairs="half",
             first=0),
        # a training step of shared key heads
        dict(name="rotate train", op="rotate_train", b=2, t=2048, hq=16, hk=4, d=128, rot=128, type="bf16",
             pairs="half", first=0),
        # odd sizes in full precision, half of each head turned, neighbouring pairs
        dict(name="rotate train f32 odd", op="rotate_train", b=3, t=333, hq=6, hk=2, d=80, rot=40, type="f32",
             pairs="neighbours", first=131072),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "prompt", "prompt", "train", "rotate", "rotate_train"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op in ("rotate", "rotate_train"):
        d = 2 * rng.randint(8, 128)
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 2, 3, 4])
        most = 4 * 4096 * 32 * 128 // (2 if op == "rotate_train" or kind == "f32" else 1)
        t = _spread(rng, 1, 4096)
        b = max(1, min(_spread(rng, 1, 16), most // (t * (hq + hk) * d)))
        return dict(op=op, b=b, t=t, hq=hq, hk=hk, d=d, rot=2 * rng.randint(1, d // 2), type=kind,
                    pairs=rng.choice(["half", "neighbours"]), first=_spread(rng, 1, 1 << 20))
    h = rng.choice([2, 4, 6, 8, 12, 16])
    hq, hv = rng.choice([h, h, h // 2, 1]), rng.choice([h, h, h // 2])
    dk, dv = rng.randint(16, 128), rng.randint(16, 128)
    if rng.random() < 0.5:
        dk, dv = max(16, dk // 16 * 16), max(16, dv // 16 * 16)
    if op == "step":
        b = _spread(rng, 1, 64)
        return dict(op=op, b=b, pool=b + rng.randint(0, 16), h=h, hq=hq, hv=hv, dk=dk, dv=dv, type=kind)
    t = _spread(rng, 1, 4096)
    most = 4 * 4096 * 8 if op == "prompt" else 2 * 4096 * 8
    b = max(1, min(_spread(rng, 1, 8), most // (t * h)))
    return dict(op=op, b=b, t=min(t, most // h), h=h, hq=hq, hv=hv, dk=dk, dv=dv, type=kind,
                decay=rng.choice(["head", "token", "reset"]), initial=rng.random() < 0.5, ragged=rng.random() < 0.4)


# ---------------------------------------------------------------- inputs

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    c, ty = case, TYPES[case["type"]]
    s = {"case": case}
    if c["op"] in ("rotate", "rotate_train"):
        b, t, hq, hk, d = c["b"], c["t"], c["hq"], c["hk"], c["d"]
        # queries and keys are two slices of one projection's output, values behind them
        qkv = (_normal(gen, b, t, (hq + 2 * hk) * d) * 2.5).to(ty)
        s["q"] = qkv[..., :hq * d].view(b, t, hq, d)
        s["k"] = qkv[..., hq * d:(hq + hk) * d].view(b, t, hk, d)
        s["qw"], s["kw"] = 1 + 0.2 * _normal(gen, d), 1 + 0.2 * _normal(gen, d)
        starts = torch.randint(0, 64, (b, 1), generator=gen, device=DEV)
        s["positions"] = c["first"] + starts + torch.arange(t, device=DEV)[None, :]
        i = torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64)
        s["turns"] = 10000.0 ** (-2.0 * i / c["rot"]) / (2 * math.pi)
        if c["op"] == "rotate_train":
            s["gq"], s["gk"] = _normal(gen, b, t, hq, d).to(ty), _normal(gen, b, t, hk, d).to(ty)
        return s
    b, h, hq, hv, dk, dv = c["b"], c["h"], c["hq"], c["hv"], c["dk"], c["dv"]
    t = c.get("t", 1)
    # queries and keys as a norm leaves them; values beside them in one buffer
    s["q"] = _normal(gen, b, t, hq, dk).to(ty)
    kv = _normal(gen, b, t, hq * dk + hv * dv).to(ty)
    s["k"] = kv[..., :hq * dk].view(b, t, hq, dk)
    s["v"] = kv[..., hq * dk:].view(b, t, hv, dv)
    s["scale"] = dk ** -0.5
    per_head = torch.log1p(-torch.exp2(-2.0 - 6.0 * torch.rand(h, generator=gen, device=DEV)))
    if c["op"] == "step":
        s["q"], s["k"], s["v"] = s["q"][:, 0], s["k"][:, 0], s["v"][:, 0]
        s["g"] = per_head * (0.25 + 1.5 * torch.rand(b, h, generator=gen, device=DEV))
        s["state"] = _normal(gen, c["pool"], h, dk, dv)
        slots = torch.randperm(c["pool"], generator=gen, device=DEV)[:b].to(torch.int32)
        if b >= 8:  # rows of the batch that hold no request
            slots[torch.randperm(b, generator=gen, device=DEV)[:b // 16 + 1]] = -1
        s["slots"] = slots
        return s
    if c["decay"] == "head":
        s["g"] = per_head
    else:
        s["g"] = per_head * (0.25 + 1.5 * torch.rand(b, t, h, generator=gen, device=DEV))
        if c["decay"] == "reset":  # a document begins: nothing of the one before is left
            begins = torch.rand(b, t, generator=gen, device=DEV) < 1 / 256
            s["g"] = torch.where(begins[..., None], torch.full_like(s["g"], -math.inf), s["g"])
    s["initial"] = _normal(gen, b, h, dk, dv) if c["initial"] else None
    s["lengths"] = None
    if c["ragged"]:
        s["lengths"] = torch.randint(0, t + 1, (b,), generator=gen, device=DEV, dtype=torch.int32)
        s["lengths"][0] = t
    if c["op"] == "train":
        s["go"] = _normal(gen, b, t, h, dv).to(ty)
        s["gs"] = _normal(gen, b, h, dk, dv) if c["initial"] else None
    return s


# ---------------------------------------------------------------- the plain forms

def _heads(x, h):
    """[B, T, Hx, D] to [B, H, T, D] in 32 bits, each head given to the heads that share it."""
    b, t, hx, d = x.shape
    x = x.to(torch.float32).permute(0, 2, 1, 3)
    return x[:, :, None].expand(b, hx, h // hx, t, d).reshape(b, h, t, d)


def _shared(x, hx):
    """The sum over the heads that share one, [B, H, T, D] to [B, T, Hx, D]."""
    b, h, t, d = x.shape
    return x.view(b, hx, h // hx, t, d).sum(2).permute(0, 2, 1, 3)


def _chunks(x, n):
    """[B, H, T, ...] to [B, H, n, CHUNK, ...], zeros behind the last token."""
    b, h, t = x.shape[:3]
    pad = x.new_zeros((b, h, n * CHUNK - t) + tuple(x.shape[3:]))
    return torch.cat([x, pad], 2).view(b, h, n, CHUNK, *x.shape[3:])


def _laid_out(s):
    """Chunked q, k, v, the running log decay within a chunk (64 bits), and which tokens there are."""
    h, t = s["g"].shape[-1], s["q"].shape[1]
    n = (t + CHUNK - 1) // CHUNK
    b = s["q"].shape[0]
    live = torch.ones(b, t, dtype=torch.bool, device=DEV)
    if s["lengths"] is not None:
        live = torch.arange(t, device=DEV)[None, :] < s["lengths"][:, None]
    q, k, v = (torch.where(live[:, None, :, None], _heads(s[x], h), 0.0) for x in "qkv")
    g = s["g"].to(torch.float64).clamp_min(-800.0).expand(b, t, h)  # exp(-800) is nothing in 32 bits
    g = torch.where(live[:, None, :], g.permute(0, 2, 1), 0.0)
    return _chunks(q, n), _chunks(k, n), _chunks(v, n), _chunks(g, n).cumsum(-1), live


def _decays(run):
    """exp of the log decay from each source to each row of a chunk, row to end, start to row, and the whole."""
    diff = run[..., :, None] - run[..., None, :]
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    inside = torch.where(lower, diff, -math.inf).exp().float()
    return inside, (run[..., -1:] - run).exp().float()[..., None], run.exp().float()[..., None]


def _between(run):
    """exp of the log decay from the end of chunk j to the start of chunk i, i > j; and from the start of all."""
    total = run[..., -1]
    ends = total.cumsum(-1)
    starts = ends - total
    n = total.shape[-1]
    later = torch.ones(n, n, dtype=torch.bool, device=DEV).tril(-1)
    return torch.where(later, starts[..., :, None] - ends[..., None, :], -math.inf).exp().float(), starts, ends


def _states(k, v, to_end, between, starts, initial):
    """The state at the start of every chunk."""
    own_part = torch.matmul((k * to_end).transpose(-1, -2).contiguous(), v)
    b, h, n, dk, dv = own_part.shape
    states = torch.matmul(between, own_part.view(b, h, n, dk * dv)).view(b, h, n, dk, dv)
    if initial is not None:
        states = states + starts.exp().float()[..., None, None] * initial[:, :, None]
    return states, own_part


def _plain_prompt(s):
    q, k, v, run, live = _laid_out(s)
    inside, to_end, from_start = _decays(run)
    between, starts, _ = _between(run)
    states, own_part = _states(k, v, to_end, between, starts, s["initial"])
    a = torch.matmul(q, k.transpose(-1, -2).contiguous()) * inside
    o = torch.matmul(a, v) + torch.matmul(q * from_start, states)
    last = states[:, :, -1] * run[:, :, -1, -1].exp().float()[..., None, None] + own_part[:, :, -1]
    b, h, n = o.shape[:3]
    o = (o * s["scale"]).reshape(b, h, n * CHUNK, -1)[:, :, :s["q"].shape[1]]
    return o.permute(0, 2, 1, 3).to(s["q"].dtype), last


def _plain_train(s):
    q, k, v, run, live = _laid_out(s)
    b, h, n = q.shape[:3]
    t, hq, hv = s["q"].shape[1], s["q"].shape[2], s["v"].shape[2]
    scale, ty = s["scale"], s["q"].dtype
    go = _chunks(torch.where(live[:, None, :, None], _heads(s["go"], h), 0.0), n) * scale
    inside, to_end, from_start = _decays(run)
    between, starts, ends = _between(run)
    states, _ = _states(k, v, to_end, between, starts, s["initial"])
    # the adjoint of the state at the end of every chunk
    dk, dv = q.shape[-1], v.shape[-1]
    part = torch.matmul((q * from_start).transpose(-1, -2).contiguous(), go)
    adj = torch.matmul(between.transpose(-1, -2).contiguous(), part.view(b, h, n, dk * dv)).view(b, h, n, dk, dv)
    if s["gs"] is not None:
        adj = adj + (ends[..., -1:] - ends).exp().float()[..., None, None] * s["gs"][:, :, None]
    whole = run[..., -1].exp().float()
    g_initial = whole[:, :, 0, None, None] * adj[:, :, 0] + part[:, :, 0]
    a = torch.matmul(q, k.transpose(-1, -2).contiguous()) * inside
    da = torch.matmul(go, v.transpose(-1, -2).contiguous()) * inside
    q_far = from_start * torch.matmul(go, states.transpose(-1, -2).contiguous())
    k_far = to_end * torch.matmul(v, adj.transpose(-1, -2).contiguous())
    gq = torch.matmul(da, k) + q_far
    gk = torch.matmul(da.transpose(-1, -2).contiguous(), q) + k_far
    gv = torch.matmul(a.transpose(-1, -2).contiguous(), go) + to_end * torch.matmul(k, adj)
    # what a token's decay carries: every source before it with every row from it on
    pairs = torch.matmul(q, k.transpose(-1, -2).contiguous()) * da
    before = (pairs.cumsum(-1) - pairs).tril()  # [row, token]: sources before the token
    far_rows = (q * q_far).sum(-1)
    far_sources = (k * k_far).sum(-1)
    gg = before.sum(-2) + far_rows.flip(-1).cumsum(-1).flip(-1) + far_sources.cumsum(-1) - far_sources
    gg = gg + (whole * (adj * states).sum((-1, -2)))[..., None]

    def out(x, hx):
        return _shared(x.reshape(b, h, n * CHUNK, -1)[:, :, :t], hx).to(ty)

    gg = gg.reshape(b, h, n * CHUNK)[:, :, :t].permute(0, 2, 1)
    gg = torch.where(live[..., None], gg, 0.0)
    if s["g"].dim() == 1:
        gg = gg.sum((0, 1))
    got = [out(gq, hq), out(gk, hq), out(gv, hv), gg]
    return got + [g_initial] if s["initial"] is not None else got


def _plain_step(s):
    c = s["case"]
    h = c["h"]
    used = (s["slots"] >= 0) & (s["slots"] < c["pool"])
    at = torch.where(used, s["slots"], 0).long()
    q, k, v = (_heads(s[x][:, None], h)[:, :, 0] for x in "qkv")
    old = s["state"][at]
    new = s["g"].exp()[..., None, None] * old + k[..., :, None] * v[..., None, :]
    o = (q[..., :, None] * new).sum(-2) * s["scale"]
    s["state"][at[used]] = new[used]
    return torch.where(used[:, None, None], o, 0.0).to(s["q"].dtype), s["state"]


def _angles(s):
    turn = s["positions"].double()[..., None] * s["turns"]
    turn = (turn - torch.floor(turn)) * (2 * math.pi)
    return turn.cos().float()[:, :, None], turn.sin().float()[:, :, None]


def _turned(u, cos, sin, rot, pairs):
    """The first `rot` components turned in pairs, the others left."""
    head, rest = u[..., :rot], u[..., rot:]
    if pairs == "half":
        x, y = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat([x * cos - y * sin, x * sin + y * cos], -1)
    else:
        x, y = head[..., 0::2], head[..., 1::2]
        head = torch.stack([x * cos - y * sin, x * sin + y * cos], -1).flatten(-2)
    return torch.cat([head, rest], -1)


EPS = 1e-6


def _plain_rotate(s):
    c = s["case"]
    cos, sin = _angles(s)

    def one(x, w):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        return _turned(x * r * w, cos, sin, c["rot"], c["pairs"])

    return one(s["q"], s["qw"]).to(s["q"].dtype), one(s["k"], s["kw"]).to(s["k"].dtype)


def _plain_rotate_train(s):
    c = s["case"]
    cos, sin = _angles(s)

    def one(x, w, gy):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        n = x * r
        gu = _turned(gy.float(), cos, -sin, c["rot"], c["pairs"])
        gn = gu * w
        gx = r * (gn - n * (gn * n).mean(-1, keepdim=True))
        return gx.to(s["q"].dtype), (gu * n).sum((0, 1, 2))

    gq, gqw = one(s["q"], s["qw"], s["gq"])
    gk, gkw = one(s["k"], s["kw"], s["gk"])
    return gq, gk, gqw, gkw


# ---------------------------------------------------------------- the calls

def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import scan_primitives_amd as sx
        if op == "prompt":
            return sx.decay_attention(s["q"], s["k"], s["v"], s["g"], initial=s["initial"], lengths=s["lengths"],
                                      scale=s["scale"], return_state=True)
        if op == "train":
            got = sx.decay_attention_backward(s["q"], s["k"], s["v"], s["g"], s["go"], initial=s["initial"],
                                              lengths=s["lengths"], scale=s["scale"], grad_state=s["gs"])
            return list(got) if s["initial"] is not None else list(got[:4])
        if op == "step":
            o = sx.decay_attention_step(s["q"], s["k"], s["v"], s["g"], s["state"], slots=s["slots"],
                                        scale=s["scale"])
            return o, s["state"]
        near = c["pairs"] == "neighbours"
        if op == "rotate":
            return sx.head_norm_rotate(s["q"], s["k"], s["positions"], s["turns"], q_weight=s["qw"],
                                       k_weight=s["kw"], eps=EPS, neighbours=near)
        return sx.head_norm_rotate_backward(s["q"], s["k"], s["positions"], s["turns"], s["gq"], s["gk"],
                                            q_weight=s["qw"], k_weight=s["kw"], eps=EPS, neighbours=near)
    return {"prompt": _plain_prompt, "train": _plain_train, "step": _plain_step, "rotate": _plain_rotate,
            "rotate_train": _plain_rotate_train}[op](s)


def work(case):
    c = case
    e = 2 if c["type"] == "bf16" else 4
    if c["op"] in ("rotate", "rotate_train"):
        rows = c["b"] * c["t"] * (c["hq"] + c["hk"])
        n = rows * c["d"]
        passes, flops = (2, 8) if c["op"] == "rotate" else (3, 18)
        weights = 4 * c["d"] * (2 if c["op"] == "rotate" else 4)
        return {"bytes": passes * e * n + 8 * c["b"] * c["t"] + 4 * c["rot"] + weights, "flops": flops * n}
    b, h, hq, hv, dk, dv = c["b"], c["h"], c["hq"], c["hv"], c["dk"], c["dv"]
    t = c.get("t", 1)
    state = 4 * b * h * dk * dv
    qkv = e * b * t * (2 * hq * dk + hv * dv)
    out = e * b * t * h * dv
    mults = b * t * h * dk * dv
    if c["op"] == "step":
        idle = (b // 16 + 1) / b if b >= 8 else 0.0
        return {"bytes": (1 - idle) * (2 * state + qkv) + out + 4 * b * (h + 1), "flops": (1 - idle) * 5 * mults}
    g = 4 * h * (1 if c["decay"] == "head" else b * t)
    part = 0.5 + 0.5 / b if c["ragged"] else 1.0  # lengths are spread evenly, the first is whole
    lengths = 4 * b if c["ragged"] else 0
    if c["op"] == "prompt":
        return {"bytes": part * (qkv + g) + out + (state if c["initial"] else 0) + state + lengths,
                "flops": part * 4 * mults}
    return {"bytes": part * (qkv + out + g) + qkv + g + (3 * state if c["initial"] else 0) + lengths,
            "flops": part * 10 * mults}


# ---------------------------------------------------------------- the definitions in 64 bits

def _wide(s, name, b, h):
    """Head h of batch row b of s[name], [T, D] in 64 bits."""
    x, heads = s[name], s["g"].shape[-1]
    return x[b, :, h // (heads // x.shape[2])].double()


def _exact_attention(s):
    """The recurrence unrolled: o = scale ((q k^T) * decay) v over all pairs of tokens, head by head, with the
    gradients of that matrix form."""
    c = s["case"]
    b, t, h = c["b"], c["t"], c["h"]
    dev, f64 = s["q"].device, torch.float64
    train = c["op"] == "train"
    hq, hv = s["q"].shape[2], s["v"].shape[2]
    o = torch.zeros(b, t, h, c["dv"], dtype=f64, device=dev)
    last = torch.zeros(b, h, c["dk"], c["dv"], dtype=f64, device=dev)
    gq, gk = (torch.zeros(b, t, hq, c["dk"], dtype=f64, device=dev) for _ in range(2))
    gv = torch.zeros(b, t, hv, c["dv"], dtype=f64, device=dev)
    gg = torch.zeros(b, t, h, dtype=f64, device=dev)
    g0 = torch.zeros_like(last)
    for i in range(b):
        n = t if s["lengths"] is None else int(s["lengths"][i])
        for j in range(h):
            jq, jv = j // (h // hq), j // (h // hv)
            start = s["initial"][i, j].double() if s["initial"] is not None else torch.zeros_like(last[i, j])
            end = s["gs"][i, j].double() if train and s["gs"] is not None else torch.zeros_like(start)
            if n == 0:
                last[i, j], g0[i, j] = start, end
                continue
            q, k, v = (_wide(s, x, i, j)[:n] for x in "qkv")
            g = (s["g"][j].expand(n) if s["g"].dim() == 1 else s["g"][i, :n, j]).double().clamp_min(-2000.0)
            cum = torch.cumsum(g, 0)
            mask = torch.full((n, n), -math.inf, dtype=f64, device=dev).triu(1)
            d = torch.exp(cum[:, None] - cum[None, :] + mask)
            del mask
            first, tail = torch.exp(cum)[:, None], torch.exp(cum[-1] - cum)[:, None]
            score = (q @ k.T) * d
            if not train:
                o[i, :n, j] = s["scale"] * (score @ v + first * (q @ start))
                last[i, j] = first[-1] * start + k.T @ (tail * v)
                continue
            go = s["scale"] * s["go"][i, :n, j].double()
            dscore = (go @ v.T) * d
            del d
            from_init, to_end = first * (go @ start.T), tail * (v @ end.T)
            gq[i, :n, jq] += dscore @ k + from_init
            gk[i, :n, jq] += dscore.T @ q + to_end
            gv[i, :n, jv] += score.T @ go + tail * (k @ end)
            g0[i, j] = q.T @ (first * go) + first[-1] * end
            # a decay carries what rows from it on get, less what they get from sources from it on
            rows = (q * (dscore @ k + from_init)).sum(-1)
            sources = (k * (dscore.T @ q + to_end)).sum(-1)
            out_end = (k * to_end).sum() + first[-1, 0] * (start * end).sum()
            back = (rows - sources).flip(0).cumsum(0).flip(0) + out_end
            gg[i, :n, j] = torch.where(g <= -1000.0, 0.0, back)
    if not train:
        return o, last
    got = [gq, gk, gv, gg.sum((0, 1)) if s["g"].dim() == 1 else gg]
    return got + [g0] if s["initial"] is not None else got


def _exact_step(s):
    """One request and head after the other."""
    c = s["case"]
    state = s["state"].double().clone()
    o = torch.zeros(c["b"], c["h"], c["dv"], dtype=torch.float64, device=state.device)
    per_q, per_v = c["h"] // c["hq"], c["h"] // c["hv"]
    for i, slot in enumerate(s["slots"].tolist()):
        if not 0 <= slot < c["pool"]:
            continue
        for j in range(c["h"]):
            k, v = s["k"][i, j // per_q].double(), s["v"][i, j // per_v].double()
            state[slot, j] = state[slot, j] * torch.exp(s["g"][i, j].double()) + torch.outer(k, v)
            o[i, j] = s["scale"] * torch.mv(state[slot, j].T, s["q"][i, j // per_q].double())
    return o, state


def _exact_rotate(s):
    """Pairs as complex numbers; the gradient by the product rule on them."""
    c = s["case"]
    rot, train = c["rot"], c["op"] == "rotate_train"
    angle = 2 * math.pi * torch.frac(s["positions"].double()[..., None] * s["turns"])[:, :, None]
    unit = torch.complex(torch.cos(angle), torch.sin(angle))

    def turn(x, by):
        head = x[..., :rot]
        if c["pairs"] == "half":
            z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * by
            head = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * by
            head = torch.view_as_real(z).reshape(head.shape)
        return torch.cat([head, x[..., rot:]], -1)

    out, weights = [], []
    for name in "qk":
        x, w = s[name].double(), s[name + "w"].double()
        norm = torch.sqrt(x.square().sum(-1, keepdim=True) / c["d"] + EPS)
        if not train:
            out.append(turn(w * x / norm, unit))
            continue
        back = turn(s["g" + name].double(), unit.conj())
        weights.append((back * x / norm).flatten(0, 2).sum(0))
        along = (back * w * x).sum(-1, keepdim=True) / c["d"]
        out.append(back * w / norm - x * along / norm ** 3)
    return out + weights if train else tuple(out)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "step":
        return _exact_step(s)
    if case["op"] in ("rotate", "rotate_train"):
        return _exact_rotate(s)
    return _exact_attention(s)
