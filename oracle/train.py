"""Float64 oracle of the training operators: AdamW with float32 or 8-bit moments, group norm with an
activation, the norms around a block with its gate and residual stream, and the gated projection, each with
its gradients, and Newton-Schulz products with the step that applies them.  Written from the formulas; shares no
code with the GPU path."""
import math

import numpy as np

BLOCK = 256


# ---------------------------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------------------------

def adam_moments(m, v, g, beta1, beta2):
    m, v, g = (np.asarray(t, np.float64) for t in (m, v, g))
    return beta1 * m + (1.0 - beta1) * g, beta2 * v + (1.0 - beta2) * (g * g)


def adam_param(p, m, v, lr, beta1, beta2, eps, weight_decay, step):
    m_hat, v_hat = m / (1.0 - beta1 ** step), v / (1.0 - beta2 ** step)
    return np.asarray(p, np.float64) * (1.0 - lr * weight_decay) - lr * m_hat / (np.sqrt(v_hat) + eps)


def decode(codes, scale, top, power):
    """The values of 8-bit codes: scale * sign(c) * (|c| / top)^power, blocks of 256."""
    c = np.asarray(codes, np.float64)
    s = np.repeat(np.asarray(scale, np.float64), BLOCK)[:c.size]
    return s * np.sign(c) * (np.abs(c) / top) ** power


def encode(x, top, power):
    """Codes (int) and float32 scales of x by block; the nearest code is found by comparing the value
    with the half-way points of the scale of codes (a value on one, to within 2^-40, is not over it)."""
    x = np.asarray(x, np.float64)
    codes = np.zeros(x.size, np.int64)
    scale = np.zeros(-(-x.size // BLOCK), np.float32)
    edges = ((np.arange(top) + 0.5) / top) ** power * (1 + 2.0 ** -40)
    for b in range(scale.size):
        v = x[b * BLOCK:(b + 1) * BLOCK]
        with np.errstate(over="ignore"):
            finite = np.isfinite(v.astype(np.float32)).all()
        if not finite:
            scale[b] = np.nan
            continue
        largest = np.abs(v).max()
        scale[b] = np.float32(largest)
        if scale[b] > 0:
            c = np.searchsorted(edges, np.abs(v) / largest, side="right")
            if power == 4:
                c = np.where(v > 0, np.maximum(c, 1), c)
            codes[b * BLOCK:(b + 1) * BLOCK] = np.where(v < 0, -c, c)
        elif power == 4:
            codes[b * BLOCK:(b + 1) * BLOCK] = v > 0
    return codes, scale


# ---------------------------------------------------------------------------------------------
# activations
# ---------------------------------------------------------------------------------------------

_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(z, kind):
    if kind == "relu":
        return np.where(z <= 0, 0.0, z)          # NaN stays NaN
    if kind == "silu":
        return z / (1.0 + np.exp(-z))
    if kind == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    return z


def act_slope(z, kind):
    if kind == "relu":
        return np.where(z <= 0, 0.0, 1.0)
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s + z * s * (1.0 - s)
    if kind == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return np.ones_like(z)


# ---------------------------------------------------------------------------------------------
# group norm, channels last: x [samples * positions, c]
# ---------------------------------------------------------------------------------------------

def group_norm(x, w, b, groups, positions, eps, kind):
    """(y, mean, rstd); statistics per sample and group of c / groups neighbouring channels."""
    x = np.asarray(x, np.float64)
    c = x.shape[1]
    xg = x.reshape(-1, positions, groups, c // groups)
    mean = xg.mean((1, 3))
    rstd = 1.0 / np.sqrt(((xg - mean[:, None, :, None]) ** 2).mean((1, 3)) + eps)
    z = ((xg - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(x.shape)
    z = z * (1.0 if w is None else w) + (0.0 if b is None else b)
    return act(z, kind), mean, rstd


def group_norm_backward(dy, x, mean, rstd, w, b, groups, positions, kind):
    """(dx, dw, db) for given statistics."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    mean, rstd = np.asarray(mean, np.float64), np.asarray(rstd, np.float64)
    c = x.shape[1]
    shape = (-1, positions, groups, c // groups)
    xhat = ((x.reshape(shape) - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(x.shape)
    wv = np.ones(c) if w is None else np.asarray(w, np.float64)
    dz = dy * act_slope(xhat * wv + (0.0 if b is None else b), kind)
    q = (dz * wv).reshape(shape)
    xh = xhat.reshape(shape)
    dx = rstd[:, None, :, None] * (q - q.mean((1, 3), keepdims=True) - xh * (q * xh).mean((1, 3), keepdims=True))
    return dx.reshape(x.shape), (dz * xhat).sum(0), dz.sum(0)


# ---------------------------------------------------------------------------------------------
# the norms around a block: rows [rows, c], a gate row for `positions` of them
# ---------------------------------------------------------------------------------------------

def row_norm(v, kind, w, b, eps):
    """(result, statistics [rows, 2]) of every row's norm: "none", "rms" or "layer"."""
    v = np.asarray(v, np.float64)
    mean = v.mean(1, keepdims=True) if kind == "layer" else np.zeros((v.shape[0], 1))
    rstd = np.ones_like(mean) if kind == "none" else 1.0 / np.sqrt(((v - mean) ** 2).mean(1, keepdims=True) + eps)
    return (v - mean) * rstd * (1.0 if w is None else w) + (0.0 if b is None else b), np.concatenate([mean, rstd], 1)


def row_norm_backward(dz, v, kind, stats, w):
    """(dv, dw, db) for given statistics."""
    dz, v, stats = (np.asarray(t, np.float64) for t in (dz, v, stats))
    xhat = (v - stats[:, :1]) * stats[:, 1:]
    q = dz * (1.0 if w is None else np.asarray(w, np.float64))
    dv = q.copy()
    if kind != "none":
        dv -= xhat * (q * xhat).mean(1, keepdims=True)
    if kind == "layer":
        dv -= q.mean(1, keepdims=True)
    return dv * stats[:, 1:], (dz * xhat).sum(0), dz.sum(0)


def residual_norm(x, h, gate, positions, post, pre, vectors, skip, branch, eps):
    """(y, u, post statistics, pre statistics); vectors: post weight and bias, pre weight and bias; h may be None."""
    y, post_stats = np.asarray(x, np.float64), None
    if h is not None:
        z, post_stats = row_norm(h, post, vectors[0], vectors[1], eps)
        g = 1.0 if gate is None else np.repeat(np.asarray(gate, np.float64), positions, 0)
        y = skip * y + branch * (g * z)
    u, pre_stats = row_norm(y, pre, vectors[2], vectors[3], eps)
    return y, u, post_stats, pre_stats


def residual_norm_backward(dy, du, y, h, gate, positions, post, pre, vectors, post_stats, pre_stats, skip, branch):
    """(dx, dh, dgate, [post weight's and bias's, pre weight's and bias's gradients]) for given statistics."""
    t = np.zeros(np.shape(y)) if dy is None else np.asarray(dy, np.float64)
    grads = [None] * 4
    if pre != "none":
        dv, grads[2], grads[3] = row_norm_backward(du, y, pre, pre_stats, vectors[2])
        t = t + dv
    if h is None:                                # u is the norm of x itself: skip has no part
        return t, None, None, grads
    g = np.ones((t.shape[0] // positions, t.shape[1])) if gate is None else np.asarray(gate, np.float64)
    h = np.asarray(h, np.float64)
    z = (h - post_stats[:, :1]) * post_stats[:, 1:] * (1.0 if vectors[0] is None else vectors[0])
    z = z + (0.0 if vectors[1] is None else vectors[1])
    dgate = (branch * t * z).reshape(-1, positions, t.shape[1]).sum(1)
    dh, grads[0], grads[1] = row_norm_backward(branch * t * np.repeat(g, positions, 0), h, post, post_stats, vectors[0])
    return skip * t, dh, dgate, grads


# ---------------------------------------------------------------------------------------------
# gated projection
# ---------------------------------------------------------------------------------------------

def gated(a, wg, wu, kind):
    a, wg, wu = (np.asarray(t, np.float64) for t in (a, wg, wu))
    gate, up = a @ wg.T, a @ wu.T
    return act(gate, kind) * up, gate, up


def gated_backward(dh, gate, up, a, wg, wu, kind):
    dh, gate, up, a, wg, wu = (np.asarray(t, np.float64) for t in (dh, gate, up, a, wg, wu))
    dg, du = dh * up * act_slope(gate, kind), dh * act(gate, kind)
    return dg @ wg + du @ wu, dg.T @ a, du.T @ a


# ---------------------------------------------------------------------------------------------
# Newton-Schulz products and the step that applies them
# ---------------------------------------------------------------------------------------------

def newton_schulz(x, coefficients, eps):
    """X = x / (|x| + eps), whose singular values s go through a s + b s^3 + c s^5 for each (a, b, c)."""
    x = np.asarray(x, np.float64)
    size = np.sqrt((x * x).sum()) + eps
    if size == 0.0:
        return np.zeros_like(x)
    u, s, vt = np.linalg.svd(x / size, full_matrices=False)
    for a, b, c in coefficients:
        s = a * s + b * s ** 3 + c * s ** 5
    return (u * s) @ vt


def muon(p, g, m, lr, beta, nesterov, weight_decay, scale, grad_scale, coefficients, eps):
    """(new parameter, new momentum)."""
    p, g, m = (np.asarray(t, np.float64) for t in (p, g, m))
    g = grad_scale * g
    m = beta * m + g
    o = newton_schulz(g + beta * m if nesterov else m, coefficients, eps)
    return p * (1.0 - lr * weight_decay) - lr * scale * o, m
