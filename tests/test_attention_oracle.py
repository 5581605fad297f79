"""Pins for the oracle of the linear-attention operators: closed forms, the matrix form, differences."""

import numpy as np
import pytest

from oracle import attention as oa


def _case(seed, b=2, t=7, h=4, hq=2, hv=4, dk=3, dv=5, per_head=False):
    r = np.random.default_rng(seed)
    g = -r.random(h if per_head else (b, t, h))
    return (r.standard_normal((b, t, hq, dk)), r.standard_normal((b, t, hq, dk)), r.standard_normal((b, t, hv, dv)), g,
            r.standard_normal((b, h, dk, dv)))


@pytest.mark.parametrize("per_head", [False, True])
def test_decay_attention_is_the_masked_matrix_form(per_head):
    q, k, v, g, s0 = _case(1, per_head=per_head)
    out, last = oa.decay_attention(q, k, v, g, s0, scale=0.5)
    b, t, h = 2, 7, 4
    gf = np.broadcast_to(g, (b, t, h))
    for i in range(b):
        for j in range(h):
            c = np.cumsum(gf[i, :, j])
            d = np.tril(np.exp(c[:, None] - c[None, :]))
            qq, kk, vv = q[i, :, j // 2], k[i, :, j // 2], v[i, :, j]
            want = 0.5 * ((qq @ kk.T * d) @ vv + np.exp(c)[:, None] * (qq @ s0[i, j]))
            np.testing.assert_allclose(out[i, :, j], want, rtol=1e-12, atol=1e-12)
            np.testing.assert_allclose(last[i, j], np.exp(c[-1]) * s0[i, j] + kk.T @ (np.exp(c[-1] - c)[:, None] * vv),
                                       rtol=1e-12, atol=1e-12)


def test_no_decay_and_one_query_sums_the_values():
    v = np.arange(12.0).reshape(1, 4, 1, 3)
    one = np.ones((1, 4, 1, 1))
    out, last = oa.decay_attention(one, one, v, np.zeros(1))
    np.testing.assert_array_equal(out, np.cumsum(v, 1))
    out, _ = oa.decay_attention(one, one, v, np.full(1, -np.inf))
    np.testing.assert_array_equal(out, v)


def test_tokens_past_the_length_change_nothing():
    q, k, v, g, s0 = _case(2)
    lengths = np.array([4, 0])
    out, last = oa.decay_attention(q, k, v, g, s0, lengths)
    short, last4 = oa.decay_attention(q[:, :4], k[:, :4], v[:, :4], g[:, :4], s0)
    np.testing.assert_array_equal(out[0, :4], short[0])
    np.testing.assert_array_equal(last[0], last4[0])
    np.testing.assert_array_equal(last[1], s0[1])
    assert not out[0, 4:].any() and not out[1].any()


def test_steps_in_turn_are_the_prompt():
    q, k, v, g, s0 = _case(3)
    out, last = oa.decay_attention(q, k, v, g, s0, scale=0.3)
    state = s0
    for t in range(q.shape[1]):
        o, state = oa.decay_attention_step(q[:, t], k[:, t], v[:, t], g[:, t], state, scale=0.3)
        np.testing.assert_allclose(o, out[:, t], rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(state, last, rtol=1e-12, atol=1e-13)


def test_the_step_leaves_other_states_alone():
    q, k, v, g, _ = _case(4, b=3)
    state = np.random.default_rng(5).standard_normal((4, 4, 3, 5))
    out, after = oa.decay_attention_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], state, slots=[2, -1, 9])
    assert not out[1:].any() and out[0].any()
    np.testing.assert_array_equal(after[[0, 1, 3]], state[[0, 1, 3]])


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("lengths", [None, [5, 7], [0, 3]])
def test_decay_attention_vjp_matches_differences(per_head, lengths):
    q, k, v, g, s0 = _case(6, per_head=per_head)
    r = np.random.default_rng(7)
    go, gs = r.standard_normal((2, 7, 4, 5)), r.standard_normal(s0.shape)

    def loss(*x):
        out, last = oa.decay_attention(*x, lengths=lengths, scale=0.7)
        return (go * out).sum() + (gs * last).sum()

    args = [q, k, v, g, s0]
    got = oa.decay_attention_vjp(q, k, v, g, go, s0, lengths, 0.7, gs)
    for i, x in enumerate(args):
        d = r.standard_normal(x.shape)
        e = 1e-5
        up, down = (loss(*[y + s * e * d if j == i else y for j, y in enumerate(args)]) for s in (1, -1))
        assert got[i].shape == x.shape
        np.testing.assert_allclose((got[i] * d).sum(), (up - down) / (2 * e), rtol=1e-7, atol=1e-7)


def test_rotation_keeps_the_norm_and_turns_by_the_difference():
    r = np.random.default_rng(8)
    turns = np.array([0.1, 0.01, 0.001])
    for near in (False, True):
        x, y = r.standard_normal((1, 1, 1, 8)), r.standard_normal((1, 1, 1, 8))
        at = lambda z, p: oa.head_norm_rotate(z, np.array([[p]]), turns, neighbours=near)[0, 0, 0]  # noqa: E731
        np.testing.assert_allclose((at(x, 5) ** 2).mean(), 1.0, rtol=1e-5)
        np.testing.assert_allclose(at(x, 3) @ at(y, 10), at(x, 103) @ at(y, 110), rtol=1e-9, atol=1e-12)
        np.testing.assert_array_equal(at(x, 9)[6:], at(x, 0)[6:])


def test_rotation_of_one_pair_is_a_turn():
    x = np.array([[[[1.0, 0.0]]]])
    got = oa.head_norm_rotate(x, np.array([[1]]), np.array([0.25]), eps=0.0)
    np.testing.assert_allclose(got[0, 0, 0], [0.0, np.sqrt(2.0)], atol=1e-15)


@pytest.mark.parametrize("near", [False, True])
def test_head_norm_rotate_vjp_matches_differences(near):
    r = np.random.default_rng(9)
    x, w, gy = r.standard_normal((2, 3, 2, 7)), r.standard_normal(7), r.standard_normal((2, 3, 2, 7))
    pos, turns = r.integers(0, 99, (2, 3)), np.array([0.13, 0.07])
    loss = lambda a, c: (gy * oa.head_norm_rotate(a, pos, turns, c, neighbours=near)).sum()  # noqa: E731
    gx, gw = oa.head_norm_rotate_vjp(x, pos, turns, gy, w, neighbours=near)
    e, dx, dw = 1e-6, r.standard_normal(x.shape), r.standard_normal(7)
    np.testing.assert_allclose((gx * dx).sum(), (loss(x + e * dx, w) - loss(x - e * dx, w)) / (2 * e), rtol=1e-6)
    np.testing.assert_allclose((gw * dw).sum(), (loss(x, w + e * dw) - loss(x, w - e * dw)) / (2 * e), rtol=1e-6)
