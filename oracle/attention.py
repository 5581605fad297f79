"""Plain CPU oracle for the linear-attention operators.

TEST INFRASTRUCTURE, NOT PRODUCT CODE; shares no code with the HIP library.

Each operator is its definition as a serial loop over tokens in float64: no
chunks, no matrix form, no running totals of decays. ``size=True`` runs the
same sums over absolute values: what a result's terms add up to before they
cancel, which is the scale of its rounding errors.
"""

import numpy as np


def _heads(x, h):
    """[B, T, Hx, D] to [B, T, H, D], each head given to the heads that share it."""
    return np.repeat(np.asarray(x, np.float64), h // x.shape[2], axis=2)


def _shared(x, hx):
    b, t, h, d = x.shape
    return x.reshape(b, t, hx, h // hx, d).sum(3)


def _setup(q, k, v, g, initial, lengths, size):
    g = np.asarray(g, np.float64)
    h, (b, t) = g.shape[-1], q.shape[:2]
    q, k, v = (_heads(x, h) for x in (q, k, v))
    live = np.arange(t)[None, :] < (np.full(b, t) if lengths is None else np.asarray(lengths))[:, None]
    # what does not exist is not read: whatever it holds
    q, k, v = (np.where(live[:, :, None, None], x, 0.0) for x in (q, k, v))
    a = np.where(live[:, :, None], np.exp(np.broadcast_to(g, (b, t, h))), 1.0)
    s0 = np.zeros((b, h, q.shape[-1], v.shape[-1])) if initial is None else np.asarray(initial, np.float64)
    if size:
        q, k, v, s0 = np.abs(q), np.abs(k), np.abs(v), np.abs(s0)
    return q, k, v, a, s0, live


def _states(k, v, a, s0):
    """Every state, [T + 1] of [B, H, dk, dv], the one before the first token in front."""
    states = [s0]
    for t in range(k.shape[1]):
        kept = np.where(a[:, t, :, None, None] == 0.0, 0.0, a[:, t, :, None, None] * states[-1])
        states.append(kept + k[:, t, :, :, None] * v[:, t, :, None, :])
    return states


def decay_attention(q, k, v, g, initial=None, lengths=None, scale=1.0, size=False):
    """``S[t] = exp(g[t]) S[t-1] + k[t] v[t]^T``, ``out[t] = scale S[t]^T q[t]``: (out, last state)."""
    q, k, v, a, s, live = _setup(q, k, v, g, initial, lengths, size)
    states = _states(k, v, a, s)
    out = np.zeros(v.shape)
    for t in range(q.shape[1]):
        out[:, t] = abs(scale) * np.einsum("bhkv,bhk->bhv", states[t + 1], q[:, t]) if size else \
            scale * np.einsum("bhkv,bhk->bhv", states[t + 1], q[:, t])
    return np.where(live[:, :, None, None], out, 0.0), states[-1]


def decay_attention_vjp(q, k, v, g, grad_out, initial=None, lengths=None, scale=1.0, grad_state=None, size=False):
    """Gradients (q, k, v, g, initial) of sum(grad_out * out) + sum(grad_state * last state), the adjoint of
    the state carried from the last token to the first."""
    shapes = [x.shape for x in (q, k, v)]
    g = np.asarray(g, np.float64)
    q, k, v, a, s0, live = _setup(q, k, v, g, initial, lengths, size)
    b, t_all, h = a.shape
    go = np.where(live[:, :, None, None], np.asarray(grad_out, np.float64), 0.0) * scale
    adj = np.zeros(s0.shape) if grad_state is None else np.asarray(grad_state, np.float64)
    if size:
        go, adj = np.abs(go), np.abs(adj)
    states = _states(k, v, a, s0)
    gq, gk, gv, gg = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape), np.zeros(a.shape)
    for t in range(t_all - 1, -1, -1):
        adj = adj + q[:, t, :, :, None] * go[:, t, :, None, :]
        gq[:, t] = np.einsum("bhkv,bhv->bhk", states[t + 1], go[:, t])
        gk[:, t] = np.einsum("bhkv,bhv->bhk", adj, v[:, t])
        gv[:, t] = np.einsum("bhkv,bhk->bhv", adj, k[:, t])
        gg[:, t] = a[:, t] * (adj * states[t]).sum((-1, -2))
        adj = a[:, t, :, None, None] * adj
    gg = np.where(live[:, :, None], gg, 0.0)
    if g.ndim == 1:
        gg = gg.sum((0, 1))
    return tuple(_shared(x, s[2]) for x, s in zip((gq, gk, gv), shapes)) + (gg, adj)


def decay_attention_step(q, k, v, g, state, slots=None, scale=1.0, size=False):
    """One token of each row: (out, every state after it). A row whose slot lies outside the pool is idle."""
    state = np.array(state, np.float64)
    if size:
        state = np.abs(state)
    pool, h = state.shape[:2]
    b = q.shape[0]
    q, k, v = (_heads(x[:, None], h)[:, 0] for x in (q, k, v))
    if size:
        q, k, v, scale = np.abs(q), np.abs(k), np.abs(v), abs(scale)
    g = np.broadcast_to(np.asarray(g, np.float64), (b, h))
    out = np.zeros((b, h, v.shape[-1]))
    for i in range(b):
        s = i if slots is None else int(slots[i])
        if not 0 <= s < pool:
            continue
        state[s] = np.exp(g[i])[:, None, None] * state[s] + k[i][:, :, None] * v[i][:, None, :]
        out[i] = scale * np.einsum("hkv,hk->hv", state[s], q[i])
    return out, state


def _turn(x, cos, sin, rot, neighbours, size=False):
    y = x.copy()
    i = np.arange(rot // 2)
    first, second = (2 * i, 2 * i + 1) if neighbours else (i, i + rot // 2)
    a, b = x[..., first], x[..., second]
    if size:
        y[..., first] = y[..., second] = np.abs(a) + np.abs(b)
        return np.abs(y)
    y[..., first], y[..., second] = a * cos - b * sin, a * sin + b * cos
    return y


def _angles(positions, turns):
    turn = np.asarray(positions, np.float64)[:, :, None, None] * np.asarray(turns, np.float64)
    turn = 2.0 * np.pi * (turn - np.rint(turn))
    return np.cos(turn), np.sin(turn)


def head_norm_rotate(x, positions, turns, weight=None, eps=1e-6, neighbours=False, size=False):
    """The norm of each row of x [B, T, heads, d] and the rotation of its first 2 len(turns) components."""
    x = np.asarray(x, np.float64)
    cos, sin = _angles(positions, turns)
    u = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if weight is None else np.asarray(weight, np.float64))
    return _turn(u, cos, sin, 2 * len(turns), neighbours, size)


def head_norm_rotate_vjp(x, positions, turns, grad_out, weight=None, eps=1e-6, neighbours=False, size=False):
    """Gradients (x, weight) of sum(grad_out * head_norm_rotate(x))."""
    x, gy = np.asarray(x, np.float64), np.asarray(grad_out, np.float64)
    w = np.ones(x.shape[-1]) if weight is None else np.asarray(weight, np.float64)
    cos, sin = _angles(positions, turns)
    norm = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    gu = _turn(gy, cos, -sin, 2 * len(turns), neighbours, size)
    if size:
        x, w = np.abs(x), np.abs(w)
        return gu * w / norm + x * (gu * w * x).mean(-1, keepdims=True) / norm ** 3, (gu * x / norm).sum((0, 1, 2))
    # d(x / norm) = dx / norm - x (x . dx) / (d norm^3)
    gx = gu * w / norm - x * (gu * w * x).mean(-1, keepdims=True) / norm ** 3
    return gx, (gu * x / norm).sum((0, 1, 2))
