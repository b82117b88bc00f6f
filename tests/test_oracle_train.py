"""The oracle of the training operators against differences and against its own definitions (CPU)."""
import numpy as np
import pytest

from oracle import train as T


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_gradients_match_central_differences(kind):
    """Step h = 1e-5 in float64: truncation below 1e-9 and cancellation below 1e-10 of values of order 1."""
    rng = np.random.default_rng(3)
    h = 1e-5
    a, wg, wu = rng.standard_normal((3, 4)), rng.standard_normal((5, 4)), rng.standard_normal((5, 4))
    dh = rng.standard_normal((3, 5))
    _, gate, up = T.gated(a, wg, wu, kind)
    loss = lambda a_, g_, u_: float((T.gated(a_, g_, u_, kind)[0] * dh).sum())
    for k, grad in enumerate(T.gated_backward(dh, gate, up, a, wg, wu, kind)):
        args = [a, wg, wu]
        for i in np.ndindex(args[k].shape):
            hi, lo = [t.copy() for t in args], [t.copy() for t in args]
            hi[k][i] += h
            lo[k][i] -= h
            assert abs((loss(*hi) - loss(*lo)) / (2 * h) - grad[i]) < 1e-7
    x, w, b, dy = rng.standard_normal((6, 8)), rng.standard_normal(8), rng.standard_normal(8), rng.standard_normal((6, 8))
    f = lambda x_, w_, b_: float((T.group_norm(x_, w_, b_, 2, 3, 1e-3, kind)[0] * dy).sum())
    _, mean, rstd = T.group_norm(x, w, b, 2, 3, 1e-3, kind)
    for k, grad in enumerate(T.group_norm_backward(dy, x, mean, rstd, w, b, 2, 3, kind)):
        args = [x, w, b]
        for i in np.ndindex(args[k].shape):
            hi, lo = [t.copy() for t in args], [t.copy() for t in args]
            hi[k][i] += h
            lo[k][i] -= h
            assert abs((f(*hi) - f(*lo)) / (2 * h) - grad[i]) < 1e-7


@pytest.mark.parametrize("top,power", [(127, 2), (255, 4)])
def test_codes_are_the_nearest_in_the_companded_scale(top, power):
    rng = np.random.default_rng(top)
    x = rng.standard_normal(1000) * 10.0 ** rng.uniform(-6, 0, 1000)
    if power == 4:
        x = x * x
    codes, scale = T.encode(x, top, power)
    assert np.abs(codes).max() == top and (np.sign(codes[codes != 0]) == np.sign(x[codes != 0])).all()
    # coded again, the values keep their codes (the scale is the block's largest value either way)
    again, scale2 = T.encode(T.decode(codes, scale, top, power), top, power)
    assert np.array_equal(codes, again)
    assert np.abs(scale2 / scale - 1).max() < 2 ** -22
    if power == 4:
        assert (codes[x > 0] >= 1).all()
    # the error is at most half the step between neighbouring codes of the root
    root = lambda v: (np.abs(v) / np.repeat(scale, T.BLOCK)[:v.size]) ** (1.0 / power) * top
    far = np.abs(root(x) - np.abs(codes))
    assert far[np.abs(codes) > 1].max() <= 0.5 + 1e-4


def test_code_blocks_with_zeros_and_values_that_are_not_finite():
    x = np.zeros(600)
    x[300] = np.inf
    x[599] = -2.0
    codes, scale = T.encode(x, 127, 2)
    assert scale[0] == 0 and np.isnan(scale[1]) and scale[2] == 2.0
    assert (codes[:599] == 0).all() and codes[599] == -127
    assert np.isnan(T.decode(codes, scale, 127, 2)[256:512]).all()


@pytest.mark.parametrize("kind", ["none", "relu", "silu", "gelu"])
def test_activations_keep_nan(kind):
    z = np.array([-1.0, np.nan, 0.0, 2.0])
    assert np.array_equal(np.isnan(T.act(z, kind)), np.isnan(z))
    assert np.isfinite(T.act_slope(z, kind)[[0, 2, 3]]).all()
    if kind == "relu":
        assert T.act(z, kind)[[0, 2, 3]].tolist() == [0.0, 0.0, 2.0] and T.act_slope(z, kind).tolist() == [0.0, 1.0, 0.0, 1.0]
