"""Rotary positions with a root-mean-square norm, and their gradients, in float64: each pair is a complex number that is
multiplied by factor e^(i p f)."""
import numpy as np


def pairs(rot, interleaved):
    """Channels (a, b) of the pairs."""
    c = np.arange(rot // 2)
    return (2 * c, 2 * c + 1) if interleaved else (c, c + rot // 2)


def turn(x, pos, freq, interleaved=False, factor=1.0):
    """Rows x [N, H, D] turned by their positions pos [N]; freq [rot / 2] radians per position."""
    x, freq = np.asarray(x, np.float64), np.asarray(freq, np.float64)
    a, b = pairs(2 * freq.size, interleaved)
    angle = np.asarray(pos, np.float64)[:, None, None] * freq
    z = (x[..., a] + 1j * x[..., b]) * (factor * np.exp(1j * angle))
    y = x.copy()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def norm(x, w, eps):
    x = np.asarray(x, np.float64)
    return x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * np.asarray(w, np.float64)


def forward(x, pos, freq, interleaved=False, factor=1.0, w=None, eps=0.0):
    return turn(x if w is None else norm(x, w, eps), pos, freq, interleaved, factor)


def backward(dy, pos, freq, interleaved=False, factor=1.0, x=None, w=None, eps=0.0):
    """(dx, dw): a turn's transpose turns back; dw None without a norm."""
    g = turn(dy, -np.asarray(pos, np.float64), freq, interleaved, factor)
    if w is None:
        return g, None
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    n, gw = x * r, g * w
    return r * (gw - n * np.mean(gw * n, -1, keepdims=True)), (g * n).sum((0, 1))
