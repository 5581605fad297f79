"""Pins for the oracle of the state-space operators: closed forms, other forms of the sums, differences."""

import numpy as np
import pytest

from oracle import state_space as os_


def _scan_case(seed, b=2, t=6, d=6, g=2, n=3, gate=True):
    r = np.random.default_rng(seed)
    return dict(x=r.standard_normal((b, t, d)), delta=r.standard_normal((b, t, d)), a=-r.random((d, n)) - 0.1,
                b=r.standard_normal((b, t, g, n)), c=r.standard_normal((b, t, g, n)), skip=r.standard_normal(d),
                z=r.standard_normal((b, t, d)) if gate else None, delta_bias=r.standard_normal(d),
                initial=r.standard_normal((b, d, n)))


@pytest.mark.parametrize("softplus", [True, False])
def test_the_scan_is_the_sum_over_pairs_of_tokens(softplus):
    s = _scan_case(1, gate=False)
    out, last = os_.selective_scan(softplus=softplus, **s)
    v = s["delta"] + s["delta_bias"]
    dt = np.log1p(np.exp(v)) if softplus else v
    for i in range(2):
        for d in range(6):
            run = np.cumsum(dt[i, :, d])
            row, read = s["b"][i, :, d // 3], s["c"][i, :, d // 3]
            decay = np.exp((run[:, None] - run[None, :])[..., None] * s["a"][d]) * np.tril(np.ones((6, 6)))[..., None]
            source = (dt[i, :, d] * s["x"][i, :, d])[:, None] * row
            h = (decay * source[None]).sum(1) + np.exp(run[:, None] * s["a"][d]) * s["initial"][i, d]
            np.testing.assert_allclose(out[i, :, d], (read * h).sum(-1) + s["skip"][d] * s["x"][i, :, d], rtol=1e-11)
            np.testing.assert_allclose(last[i, d], h[-1], rtol=1e-11)


def test_a_step_of_one_without_decay_counts():
    one = np.ones((1, 4, 1))
    out, last = os_.selective_scan(one, one, np.zeros((1, 1)), one[..., None], one[..., None], softplus=False)
    np.testing.assert_array_equal(out[0, :, 0], [1, 2, 3, 4])
    assert last[0, 0, 0] == 4


def test_tokens_past_the_length_change_nothing():
    s = _scan_case(2)
    lengths = np.array([4, 0])
    out, last = os_.selective_scan(lengths=lengths, **s)
    cut = {k: (v[:, :4] if k in ("x", "delta", "b", "c", "z") else v) for k, v in s.items()}
    short, last4 = os_.selective_scan(**cut)
    np.testing.assert_array_equal(out[0, :4], short[0])
    np.testing.assert_array_equal(last[0], last4[0])
    np.testing.assert_array_equal(last[1], s["initial"][1])
    assert not out[0, 4:].any() and not out[1].any()


def _differences(f, args, names, grads, weight):
    r = np.random.default_rng(9)
    for name, g in zip(names, grads):
        if args.get(name) is None:
            continue
        step = r.standard_normal(args[name].shape)
        e = 1e-6
        up, down = (weight(f(**{**args, name: args[name] + k * e * step})) for k in (1, -1))
        np.testing.assert_allclose((up - down) / (2 * e), (g * step).sum(), rtol=2e-7, atol=1e-7, err_msg=name)


@pytest.mark.parametrize("gate,softplus,lengths", [(True, True, None), (False, True, [6, 2]), (True, False, [0, 5])])
def test_the_scans_gradient_is_that_of_differences(gate, softplus, lengths):
    s = _scan_case(3, gate=gate)
    r = np.random.default_rng(4)
    go, gs = r.standard_normal(s["x"].shape), r.standard_normal(s["initial"].shape)
    grads = os_.selective_scan_vjp(grad_out=go, grad_state=gs, softplus=softplus, lengths=lengths, **s)
    _differences(lambda **k: os_.selective_scan(softplus=softplus, lengths=lengths, **k), s,
                 ("x", "delta", "a", "b", "c", "skip", "z", "delta_bias", "initial"), grads,
                 lambda o: (go * o[0]).sum() + (gs * o[1]).sum())


def test_the_scans_step_is_its_prompt():
    s = _scan_case(5)
    out, last = os_.selective_scan(**s)
    state, per_row = s["initial"], ("x", "delta", "b", "c", "z")
    for t in range(6):
        o, state = os_.selective_scan_step(**{k: (v[:, t] if k in per_row else v) for k, v in s.items() if k != "initial"},
                                           state=state)
        np.testing.assert_allclose(o, out[:, t], rtol=1e-12)
    np.testing.assert_allclose(state, last, rtol=1e-12)


@pytest.mark.parametrize("k", [1, 2, 4])
@pytest.mark.parametrize("activation", [None, "silu"])
def test_the_convolution_is_numpys_and_its_gradient_that_of_differences(k, activation):
    r = np.random.default_rng(6)
    s = dict(x=r.standard_normal((2, 7, 3)), weight=r.standard_normal((3, k)), bias=r.standard_normal(3),
             initial=r.standard_normal((2, k - 1, 3)))
    out, last = os_.causal_conv(activation=activation, **s)
    for i in range(2):
        for d in range(3):
            full = np.concatenate([s["initial"][i, :, d], s["x"][i, :, d]])
            u = np.convolve(full, s["weight"][d, ::-1], "valid") + s["bias"][d]
            np.testing.assert_allclose(out[i, :, d], u / (1 + np.exp(-u)) if activation else u, rtol=1e-12)
            np.testing.assert_array_equal(last[i, :, d], full[7:])
    go, gs = r.standard_normal((2, 7, 3)), r.standard_normal((2, k - 1, 3))
    for lengths in (None, [7, 1], [0, 3]):
        grads = os_.causal_conv_vjp(grad_out=go, grad_state=gs, activation=activation, lengths=lengths, **s)
        _differences(lambda **a: os_.causal_conv(activation=activation, lengths=lengths, **a), s,
                     ("x", "weight", "bias", "initial"), grads, lambda o: (go * o[0]).sum() + (gs * o[1]).sum())
    state = s["initial"]
    for t in range(7):
        o, state = os_.causal_conv_step(s["x"][:, t], s["weight"], state, s["bias"], activation=activation)
        np.testing.assert_allclose(o, out[:, t], rtol=1e-12)


@pytest.mark.parametrize("activation", [None, "silu"])
@pytest.mark.parametrize("shape", [(3, 8), (2, 5, 6), (2, 2, 3, 4)])
def test_the_norm_has_no_mean_and_its_gradient_is_that_of_differences(shape, activation):
    r = np.random.default_rng(7)
    s = dict(x=r.standard_normal(shape), weight=r.standard_normal(shape[-1]), bias=r.standard_normal(shape[-1]))
    n = os_.group_norm(s["x"], 2, eps=0.0).reshape(shape[0], -1, 2, shape[-1] // 2)
    np.testing.assert_allclose(n.mean((1, 3)), 0, atol=1e-12)
    np.testing.assert_allclose((n * n).mean((1, 3)), 1, rtol=1e-12)
    go = r.standard_normal(shape)
    grads, _ = os_.group_norm_vjp(groups=2, grad_out=go, activation=activation, **s)
    _differences(lambda **a: os_.group_norm(groups=2, activation=activation, **a), s, ("x", "weight", "bias"), grads,
                 lambda o: (go * o).sum())
