"""Float64 oracle of the training operators: AdamW with float32 or 8-bit moments, group norm with an
activation, and the gated projection, each with its gradients.  Written from the formulas; shares no
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
