"""fp64 definition of the per-head norm with position rotation, and its gradient (numpy)."""
import numpy as np


def _pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _turn(y, cos, sin, interleaved):
    a, b = _pairs(2 * cos.shape[-1], interleaved)
    out = y.copy()
    out[..., a] = y[..., a] * cos - y[..., b] * sin
    out[..., b] = y[..., b] * cos + y[..., a] * sin
    return out


def forward(x, w, cos, sin, eps, interleaved):
    """x [..., d]; w [d]; cos, sin broadcastable to [..., rot / 2]."""
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return _turn(x * r * w, cos, sin, interleaved)


def backward(g, x, w, cos, sin, eps, interleaved):
    """(dx [..., d], dw [d], and the sums of magnitudes behind each, for error bounds)."""
    x, g = np.asarray(x, np.float64), np.asarray(g, np.float64)
    d = x.shape[-1]
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = _turn(g, cos, -sin, interleaved)
    h = g * w
    dx = r * h - x * r ** 3 * (h * x).mean(-1, keepdims=True)
    size = r * np.abs(h).max(-1, keepdims=True) + np.abs(x) * r ** 3 * np.abs(h * x).mean(-1, keepdims=True)
    t = (g * x * r).reshape(-1, d)
    return dx, t.sum(0), size, np.abs(t).sum(0)
