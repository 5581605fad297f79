"""Plain CPU oracle for the operators of a layer on a selective state space.

TEST INFRASTRUCTURE, NOT PRODUCT CODE; shares no code with the HIP library.

Each operator is its definition in float64, the scan and the convolution token
after token. ``size=True`` runs the same sums over absolute values: what a
result's terms add up to before they cancel, which is the scale of its
rounding errors.
"""

import numpy as np


def _f64(x):
    return None if x is None else np.asarray(x, np.float64)


def _sigmoid(u):
    return 1.0 / (1.0 + np.exp(-u))


def silu(u):
    return u * _sigmoid(u)


def silu_slope(u, size=False):
    """A sum of two terms that cancel near u = -1.28."""
    p = _sigmoid(u)
    return p + (np.abs(u) if size else u) * p * (1.0 - p)


def _lengths(lengths, b, t):
    return np.full(b, t) if lengths is None else np.clip(np.asarray(lengths), 0, t)


# ---------------------------------------------------------------- causal convolution

def _conv_inputs(x, weight, initial, lengths):
    """[B, K - 1 + T, D]: the inputs behind those before the first; zeros where a token does not exist."""
    x, w = _f64(x), _f64(weight)
    b, t, d = x.shape
    n = _lengths(lengths, b, t)
    x = np.where((np.arange(t)[None, :] < n[:, None])[..., None], x, 0.0)
    front = np.zeros((b, w.shape[1] - 1, d)) if initial is None else _f64(initial)
    return np.concatenate([front, x], 1), n


def _conv_u(x, w, bias, t):
    u = np.zeros((x.shape[0], t, x.shape[2])) if bias is None else np.broadcast_to(bias, (x.shape[0], t, x.shape[2]))
    for j in range(w.shape[1]):
        u = u + w[:, j] * x[:, j:j + t]
    return u


def causal_conv(x, weight, bias=None, initial=None, lengths=None, activation=None, size=False):
    """(out, the last K - 1 inputs)."""
    w, bias, t = _f64(weight), _f64(bias), np.shape(x)[1]
    full, n = _conv_inputs(x, w, initial, lengths)
    k = w.shape[1]
    last = np.stack([full[i, n[i]:n[i] + k - 1] for i in range(len(n))]) if len(n) else full[:, :k - 1]
    if size:
        # |silu'| is below 1.1, and |silu(u)| below |u|
        full, w, bias = np.abs(full), np.abs(w), None if bias is None else np.abs(bias)
    out = _conv_u(full, w, bias, t)
    if activation == "silu" and not size:
        out = silu(out)
    live = (np.arange(t)[None, :] < n[:, None])[..., None]
    return np.where(live, out, 0.0), last


def causal_conv_vjp(x, weight, grad_out, bias=None, initial=None, lengths=None, activation=None, grad_state=None,
                    size=False):
    """Gradients (x, weight, bias, initial) of sum(grad_out * out) + sum(grad_state * last inputs)."""
    w, bias, go = _f64(weight), _f64(bias), _f64(grad_out)
    b, t, d = np.shape(x)
    full, n = _conv_inputs(x, w, initial, lengths)
    k = w.shape[1]
    live = (np.arange(t)[None, :] < n[:, None])[..., None]
    gu = np.where(live, go, 0.0)
    if activation == "silu":
        u = _conv_u(full, w, bias, t)
        if size:
            # the slope (up to 1.1) and its own error: its change (up to 0.5) times u's size
            reach = _conv_u(np.abs(full), np.abs(w), None if bias is None else np.abs(bias), t)
            gu = np.abs(gu) * (1.1 + 0.5 * reach)
        else:
            gu = gu * silu_slope(u)
    if size:
        full, w, gu = np.abs(full), np.abs(w), np.abs(gu)
    gx, gw = np.zeros(full.shape), np.zeros(w.shape)
    for j in range(k):
        gx[:, j:j + t] += w[:, j] * gu
        gw[:, j] = (gu * full[:, j:j + t]).sum((0, 1))
    if grad_state is not None:
        for i in range(b):
            gx[i, n[i]:n[i] + k - 1] += np.abs(_f64(grad_state)[i]) if size else _f64(grad_state)[i]
    return np.where(live, gx[:, k - 1:], 0.0), gw, gu.sum((0, 1)), gx[:, :k - 1]


def causal_conv_step(x, weight, state, bias=None, slots=None, activation=None):
    """(out, every state after it). A row whose slot lies outside the pool is idle."""
    x, w, state = _f64(x), _f64(weight), np.array(state, np.float64)
    out = np.zeros(x.shape)
    for i in range(x.shape[0]):
        s = i if slots is None else int(slots[i])
        if not 0 <= s < state.shape[0]:
            continue
        seen = np.concatenate([state[s], x[i:i + 1]])
        u = (w.T * seen).sum(0) + (0.0 if bias is None else _f64(bias))
        out[i] = silu(u) if activation == "silu" else u
        state[s] = seen[1:]
    return out, state


# ---------------------------------------------------------------- selective scan

def _setup(x, delta, a, b, c, skip, z, delta_bias, softplus, lengths):
    x, delta, a, b, c, skip, z, delta_bias = (_f64(v) for v in (x, delta, a, b, c, skip, z, delta_bias))
    rows, t, d = x.shape
    per = d // b.shape[2]
    live = np.arange(t)[None, :] < _lengths(lengths, rows, t)[:, None]
    # what does not exist is not read, whatever it holds
    x, delta = (np.where(live[..., None], v, 0.0) for v in (x, delta))
    b, c = (np.where(live[..., None, None], np.repeat(v, per, axis=2), 0.0) for v in (b, c))
    z = None if z is None else np.where(live[..., None], z, 0.0)
    v = delta + (0.0 if delta_bias is None else delta_bias)
    dt = np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v))) if softplus else v
    dt = np.where(live[..., None], dt, 0.0)
    return x, dt, v, a, b, c, np.zeros(d) if skip is None else skip, z, live


def _states(x, dt, a, b, h):
    """Every state, the one before the first token in front."""
    states = [h]
    for t in range(x.shape[1]):
        states.append(np.exp(dt[:, t, :, None] * a) * states[-1] + (dt[:, t] * x[:, t])[..., None] * b[:, t])
    return states


def selective_scan(x, delta, a, b, c, skip=None, z=None, delta_bias=None, softplus=True, initial=None, lengths=None,
                   size=False):
    """(out, last state)."""
    x, dt, _, a, b, c, skip, z, live = _setup(x, delta, a, b, c, skip, z, delta_bias, softplus, lengths)
    h = np.zeros((x.shape[0],) + a.shape) if initial is None else _f64(initial)
    if size:
        x, b, c, skip, h = np.abs(x), np.abs(b), np.abs(c), np.abs(skip), np.abs(h)
        states = _states(x * np.sign(dt), dt, a, b, h)
    else:
        states = _states(x, dt, a, b, h)
    y = np.stack([(states[t + 1] * c[:, t]).sum(-1) for t in range(x.shape[1])], 1) if x.shape[1] else np.zeros(x.shape)
    y = y + skip * x
    if z is not None:
        y = y * (np.abs(silu(z)) if size else silu(z))
    return np.where(live[..., None], y, 0.0), states[-1]


def selective_scan_vjp(x, delta, a, b, c, grad_out, skip=None, z=None, delta_bias=None, softplus=True, initial=None,
                       lengths=None, grad_state=None, size=False):
    """Gradients (x, delta, a, b, c, skip, z, delta_bias, initial) of sum(grad_out * out) + sum(grad_state * last
    state), the adjoint of the state carried from the last token to the first."""
    groups = np.shape(b)[2]
    x, dt, v, a, b, c, skip, z, live = _setup(x, delta, a, b, c, skip, z, delta_bias, softplus, lengths)
    rows, t_all, d = x.shape
    h = np.zeros((rows,) + a.shape) if initial is None else _f64(initial)
    adj = np.zeros(h.shape) if grad_state is None else _f64(grad_state)
    go = np.where(live[..., None], _f64(grad_out), 0.0)
    rate = a
    if size:
        x, b, c, skip, h, adj, go, rate = (np.abs(u) for u in (x, b, c, skip, h, adj, go, a))
        dt_abs = np.abs(dt)
    else:
        dt_abs = dt
    states = [h]
    for t in range(t_all):
        states.append(np.exp(dt[:, t, :, None] * a) * states[-1] + (dt_abs[:, t] * x[:, t])[..., None] * b[:, t])
    y = np.stack([(states[t + 1] * c[:, t]).sum(-1) for t in range(t_all)], 1) if t_all else np.zeros(x.shape)
    y = y + skip * x
    gz = None
    gy = go
    if z is not None:
        gz = go * y * silu_slope(z, size)
        gy = go * (np.abs(silu(z)) if size else silu(z))
    gx, gdt, ga = np.zeros(x.shape), np.zeros(x.shape), np.zeros(a.shape)
    gb, gc = np.zeros(b.shape), np.zeros(c.shape)
    for t in range(t_all - 1, -1, -1):
        lam = adj + gy[:, t, :, None] * c[:, t]
        gc[:, t] = gy[:, t, :, None] * states[t + 1]
        gb[:, t] = (dt_abs[:, t] * x[:, t])[..., None] * lam
        adj = np.exp(dt[:, t, :, None] * a) * lam
        turned = adj * states[t]
        ga += (dt_abs[:, t, :, None] * turned).sum(0)
        by = (lam * b[:, t]).sum(-1)
        gx[:, t] = dt_abs[:, t] * by + skip * gy[:, t]
        gdt[:, t] = (rate * turned).sum(-1) + x[:, t] * by
    gdelta = gdt * (_sigmoid(v) if softplus else 1.0)
    gdelta, gx = (np.where(live[..., None], u, 0.0) for u in (gdelta, gx))
    group = lambda u: np.where(live[..., None, None], u.reshape(rows, t_all, groups, d // groups, -1).sum(3), 0.0)  # noqa: E731
    return gx, gdelta, ga, group(gb), group(gc), (gy * x).sum((0, 1)), gz, gdelta.sum((0, 1)), adj


def selective_scan_step(x, delta, a, b, c, state, slots=None, skip=None, z=None, delta_bias=None, softplus=True,
                        size=False):
    """(out, every state after it). A row whose slot lies outside the pool is idle."""
    state, out = np.array(state, np.float64), np.zeros(np.shape(x))
    if size:
        state = np.abs(state)
    one = lambda u, i: None if u is None else np.asarray(u)[i:i + 1, None]  # noqa: E731
    for i in range(np.shape(x)[0]):
        s = i if slots is None else int(slots[i])
        if not 0 <= s < state.shape[0]:
            continue
        o, h = selective_scan(one(x, i), one(delta, i), a, one(b, i), one(c, i), skip, one(z, i), delta_bias, softplus,
                              initial=state[s:s + 1], size=size)
        out[i], state[s] = o[0, 0], h[0]
    return out, state


# ---------------------------------------------------------------- group norm

def _norm(x, groups, weight, bias, eps):
    x = _f64(x)
    c = x.shape[-1]
    v = x.reshape(x.shape[0], -1, groups, c // groups)
    mean = v.mean((1, 3), keepdims=True)
    root = np.sqrt(((v - mean) ** 2).mean((1, 3), keepdims=True) + eps)
    w = np.ones(c) if weight is None else _f64(weight)
    b = np.zeros(c) if bias is None else _f64(bias)
    return v, mean, root, w.reshape(groups, -1), b.reshape(groups, -1)


def group_norm(x, groups, weight=None, bias=None, eps=1e-5, activation=None):
    v, mean, root, w, b = _norm(x, groups, weight, bias, eps)
    u = (v - mean) / root * w + b
    return (silu(u) if activation == "silu" else u).reshape(np.shape(x))


def group_norm_vjp(x, groups, grad_out, weight=None, bias=None, eps=1e-5, activation=None):
    """Gradients (x, weight, bias) of sum(grad_out * out), and what each one's terms add up to in absolute value."""
    v, mean, root, w, b = _norm(x, groups, weight, bias, eps)
    n = (v - mean) / root
    u = n * w + b
    gu = _f64(grad_out).reshape(v.shape)
    if activation == "silu":
        gu = gu * silu_slope(u)
    gn = gu * w
    gx = (gn - gn.mean((1, 3), keepdims=True) - n * (gn * n).mean((1, 3), keepdims=True)) / root
    size = (np.abs(gn) + np.abs(gn).mean((1, 3), keepdims=True)
            + np.abs(n) * np.abs(gn * n).mean((1, 3), keepdims=True)) / root
    flat = lambda q: q.sum((0, 1)).reshape(-1)  # noqa: E731
    return ((gx.reshape(np.shape(x)), flat(gu * n), flat(gu)),
            (size.reshape(np.shape(x)), flat(np.abs(gu * n)), flat(np.abs(gu))))
