"""Oracle for the RMS norm of query and key heads with the rotation by position.

TEST INFRASTRUCTURE ONLY.  Plain fp64 numpy.  For a head row x of D elements
at position p:

    y = gamma x / sqrt(mean(x^2) + eps),   theta_t = <freq_t, p>,
    (o1, o2) = (y1 cos - y2 sin, y1 sin + y2 cos)

for the rotated pairs t = (t, t + R) or (2t, 2t + 1); other elements pass.
The VJP is the chain rule written out: the cotangent rotated back, then
through the norm; theta_bar = o1 g2 - o2 g1.

Pins (tests/test_oracle_attention.py): rotations keep norms and make scores
depend on position differences only; a pair by hand; both layouts through a
permutation; the VJP against the complex step.
"""

from __future__ import annotations

import numpy as np


def pairs(R, interleaved):
    t = np.arange(R)
    return (2 * t, 2 * t + 1) if interleaved else (t, t + R)


def fwd(x, gamma, pos, freq, eps, interleaved=False):
    """x [N, H, D], gamma [D], pos [N, 3], freq [R, 3]; complex inputs allowed."""
    y = gamma * x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    a, b = pairs(len(freq), interleaved)
    th = (pos @ freq.T)[:, None, :]
    o = y.copy()
    o[..., a] = y[..., a] * np.cos(th) - y[..., b] * np.sin(th)
    o[..., b] = y[..., a] * np.sin(th) + y[..., b] * np.cos(th)
    return o


def vjp(x, gamma, pos, freq, eps, g, interleaved=False):
    """(x_bar, gamma_bar, pos_bar)"""
    D = x.shape[-1]
    s2 = (x * x).mean(-1, keepdims=True) + eps
    u = x / np.sqrt(s2)
    a, b = pairs(len(freq), interleaved)
    th = (pos @ freq.T)[:, None, :]
    o = fwd(x, gamma, pos, freq, eps, interleaved)
    th_bar = o[..., a] * g[..., b] - o[..., b] * g[..., a]
    gy = g.copy()
    gy[..., a] = g[..., a] * np.cos(th) + g[..., b] * np.sin(th)
    gy[..., b] = g[..., b] * np.cos(th) - g[..., a] * np.sin(th)
    gg = gamma * gy
    x_bar = gg / np.sqrt(s2) - x * (gg * x).sum(-1, keepdims=True) / (D * s2 ** 1.5)
    return x_bar, (gy * u).sum((0, 1)), th_bar.sum(1) @ freq
