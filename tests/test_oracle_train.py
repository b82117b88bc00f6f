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


@pytest.mark.parametrize("post,pre", [("none", "rms"), ("rms", "layer"), ("layer", "none"), ("layer", "rms")])
def test_residual_norm_gradients_match_central_differences(post, pre):
    """Step and bound as above; two rows share a gate row, and both results enter the loss."""
    rng = np.random.default_rng(11)
    h_step, shape = 1e-5, (4, 6)
    x, h, gate = rng.standard_normal(shape), rng.standard_normal(shape), rng.standard_normal((2, 6))
    vectors = [1 + 0.3 * rng.standard_normal(6) for _ in range(4)]
    dy, du = rng.standard_normal(shape), rng.standard_normal(shape) if pre != "none" else None

    def loss(x_, h_, gate_, *v):
        y, u, _, _ = T.residual_norm(x_, h_, gate_, 2, post, pre, v, 0.8, 1.3, 1e-3)
        return float((y * dy).sum() + (0.0 if du is None else (u * du).sum()))
    y, _, ps, qs = T.residual_norm(x, h, gate, 2, post, pre, vectors, 0.8, 1.3, 1e-3)
    dx, dh, dgate, grads = T.residual_norm_backward(dy, du, y, h, gate, 2, post, pre, vectors, ps, qs, 0.8, 1.3)
    args = [x, h, gate] + vectors
    for k, grad in enumerate([dx, dh, dgate] + grads):
        if grad is None:
            continue
        for i in np.ndindex(args[k].shape):
            hi, lo = [t.copy() for t in args], [t.copy() for t in args]
            hi[k][i] += h_step
            lo[k][i] -= h_step
            assert abs((loss(*hi) - loss(*lo)) / (2 * h_step) - grad[i]) < 1e-7


@pytest.mark.parametrize("pre", ["rms", "layer"])
def test_gradients_without_a_block_match_central_differences(pre):
    """The stream reaches the norm as it is there, so skip scales neither u nor the gradient; step and bound as above."""
    rng = np.random.default_rng(14)
    h_step, x = 1e-5, rng.standard_normal((4, 6))
    w, b = 1 + 0.3 * rng.standard_normal(6), rng.standard_normal(6)
    dy, du = rng.standard_normal((4, 6)), rng.standard_normal((4, 6))

    def forward(x_, skip):
        return T.residual_norm(x_, None, None, 1, "none", pre, (None, None, w, b), skip, 1.3, 1e-3)
    for skip in (1.0, 0.5, 0.0, -2.0):
        y, _, _, qs = forward(x, skip)
        dx = T.residual_norm_backward(dy, du, y, None, None, 1, "none", pre, (None, None, w, b), None, qs, skip, 1.3)[0]
        for i in np.ndindex(x.shape):
            hi, lo = x.copy(), x.copy()
            hi[i] += h_step
            lo[i] -= h_step
            loss = [float((y * dy).sum() + (u * du).sum()) for y, u, _, _ in (forward(hi, skip), forward(lo, skip))]
            assert abs((loss[0] - loss[1]) / (2 * h_step) - dx[i]) < 1e-7


def test_residual_norm_is_the_composition_of_its_parts():
    rng = np.random.default_rng(12)
    x, h, gate = rng.standard_normal((6, 8)), 3 + rng.standard_normal((6, 8)), rng.standard_normal((3, 8))
    w, b = rng.standard_normal(8), rng.standard_normal(8)
    y, u, ps, qs = T.residual_norm(x, h, gate, 2, "layer", "layer", (w, b, w, b), 1.0, 0.5, 1e-6)
    z = T.group_norm(h, w, b, 1, 1, 1e-6, "none")[0]
    assert np.allclose(y, x + 0.5 * np.repeat(gate, 2, 0) * z, atol=1e-12)
    assert np.allclose(u, T.group_norm(y, w, b, 1, 1, 1e-6, "none")[0], atol=1e-12)
    r = T.residual_norm(x, None, None, 1, "none", "rms", (None, None, None, None), 1.0, 1.0, 0.0)[1]
    assert np.allclose((r ** 2).mean(1), 1.0)


@pytest.mark.parametrize("shape", [(5, 5), (3, 9), (9, 3), (1, 4), (4, 1)])
def test_newton_schulz_is_the_iteration_of_its_products(shape):
    rng = np.random.default_rng(13)
    g = rng.standard_normal(shape)
    steps = [(3.4445, -4.7750, 2.0315)] * 4 + [(15 / 8, -10 / 8, 3 / 8)]
    x = g / (np.sqrt((g ** 2).sum()) + 1e-7)
    for a, b, c in steps:
        s = x @ x.T
        x = a * x + (b * s + c * s @ s) @ x
    assert np.allclose(T.newton_schulz(g, steps, 1e-7), x, atol=1e-12)
    assert np.allclose(T.newton_schulz(g.T, steps, 1e-7), x.T, atol=1e-12)
    assert not T.newton_schulz(0 * g, steps, 0.0).any()
    # twenty steps of Newton's own cubic make the nearest matrix with orthonormal rows or columns
    q = T.newton_schulz(g, [(1.5, -0.5, 0.0)] * 40, 0.0)
    gram = q @ q.T if shape[0] <= shape[1] else q.T @ q
    assert np.allclose(gram, np.eye(min(shape)), atol=1e-9)


def test_muon_step_by_hand():
    """One value: its own singular value, 1 after scaling, so O = a + b + c = 0.701 with the sign of u."""
    k = [(3.4445, -4.7750, 2.0315)]
    p, m = T.muon([[2.0]], [[0.5]], [[-1.0]], 0.1, 0.9, True, 0.01, 3.0, 2.0, k, 0.0)
    assert np.allclose(m, 0.1)                   # 0.9 * -1 + 2 * 0.5
    assert np.allclose(p, 2.0 * 0.999 - 0.1 * 3.0 * 0.701)          # u = 1 + 0.9 * 0.1 > 0
    p, m = T.muon([[2.0]], [[0.5]], [[-1.0]], 0.1, 0.9, False, 0.0, 1.0, 1.0, k, 0.0)
    assert np.allclose(m, -0.4) and np.allclose(p, 2.0 + 0.1 * 0.701)
