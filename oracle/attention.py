"""Oracle for attention among the rows of each segment and its VJP.

TEST INFRASTRUCTURE ONLY.  Plain fp64 numpy, one segment and head at a time:

    u = scale Q K^T,  t = cap tanh(u / cap),  s = t - slope |p_i - p_j|,
    out = softmax(s) V,  lse = log sum exp(s)  over the visible keys:
    all of the segment's, or when causal j < prefix or j <= i + (Lk - Lq).

A row without a visible key has out = 0, lse = -inf and adds nothing.

Pins (tests/test_oracle_attention.py): rows by hand, uniform scores, segments
one by one, shared heads by repetition, the causal rule counted, the
single-query form as a row of the causal one, the VJP against the complex step
(distances and tanh are analytic away from coincidences).
"""

from __future__ import annotations

import numpy as np


def visible(lq, lk, causal=False, prefix=0):
    i, j = np.arange(lq)[:, None], np.arange(lk)[None, :]
    if not causal:
        return np.ones((lq, lk), bool)
    return (j < prefix) | (j <= i + (lk - lq))


def _scores(q, k, scale, cap, slope, pq, pk):
    u = scale * (q @ k.T)
    th = np.tanh(u / cap) if cap else None
    t = cap * th if cap else u
    if slope is None:
        return t, th, None, None
    diff = pq[:, None, :] - pk[None, :, :]
    r2 = (diff * diff).sum(-1)
    r = np.where(r2 == 0, 0, np.sqrt(np.where(r2 == 0, 1, r2)))
    return t - slope * r, th, r, diff


def _softmax(s, see):
    """(P, lse) over the visible entries; zero rows where there are none."""
    P = np.zeros_like(s)
    lse = np.full(len(s), -np.inf, dtype=s.dtype)
    for i in np.nonzero(see.any(1))[0]:
        m = s[i, see[i]].real.max()
        e = np.exp(s[i, see[i]] - m)
        P[i, see[i]] = e / e.sum()
        lse[i] = m + np.log(e.sum())
    return P, lse


def _blocks(off_q, off_k, hq, hk):
    for s in range(len(off_q) - 1):
        for h in range(hq):
            yield s, h, h // (hq // hk), slice(off_q[s], off_q[s + 1]), slice(off_k[s], off_k[s + 1])


def fwd(q, k, v, off_q, off_k, scale, cap=0.0, slope=None, pos_q=None, pos_k=None, causal=False, prefix=None):
    """q [Nq, Hq, D], k, v [Nk, Hk, D]; returns out [Nq, Hq, D], lse [Nq, Hq]."""
    hq, hk = q.shape[1], k.shape[1]
    dt = np.result_type(q, k, v, *(x for x in (slope, pos_q, pos_k) if x is not None))
    out = np.zeros(q.shape, dt)
    lse = np.full(q.shape[:2], -np.inf, dt)
    for s, h, g, a, b in _blocks(off_q, off_k, hq, hk):
        see = visible(a.stop - a.start, b.stop - b.start, causal, 0 if prefix is None else prefix[s])
        sc = _scores(q[a, h], k[b, g], scale, cap, None if slope is None else slope[h],
                     None if slope is None else pos_q[a], None if slope is None else pos_k[b])[0]
        P, l = _softmax(sc, see)
        out[a, h] = P @ v[b, g]
        lse[a, h] = l
    return out, lse


def vjp(q, k, v, off_q, off_k, scale, g_out, cap=0.0, slope=None, pos_q=None, pos_k=None, causal=False, prefix=None):
    """dict of q, k, v and, with a bias, slope, pos_q, pos_k gradients."""
    hq, hk = q.shape[1], k.shape[1]
    r = {"q": np.zeros(q.shape), "k": np.zeros(k.shape), "v": np.zeros(v.shape)}
    if slope is not None:
        r.update(slope=np.zeros(hq), pos_q=np.zeros(pos_q.shape), pos_k=np.zeros(pos_k.shape))
    for s, h, g, a, b in _blocks(off_q, off_k, hq, hk):
        see = visible(a.stop - a.start, b.stop - b.start, causal, 0 if prefix is None else prefix[s])
        sc, th, dist, diff = _scores(q[a, h], k[b, g], scale, cap, None if slope is None else slope[h],
                                     None if slope is None else pos_q[a], None if slope is None else pos_k[b])
        P, _ = _softmax(sc, see)
        r["v"][b, g] += P.T @ g_out[a, h]
        dP = g_out[a, h] @ v[b, g].T
        dS = P * (dP - (P * dP).sum(1, keepdims=True))
        if slope is not None:
            r["slope"][h] -= (dS * dist).sum()
            w = np.where(dist > 0, -slope[h] * dS / np.where(dist > 0, dist, 1), 0)[..., None] * diff
            r["pos_q"][a] += w.sum(1)
            r["pos_k"][b] -= w.sum(0)
        if cap:
            dS = dS * (1 - th * th)
        r["q"][a, h] += scale * dS @ k[b, g]
        r["k"][b, g] += scale * dS.T @ q[a, h]
    return r
