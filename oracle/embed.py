"""Oracle for the scaled embedding lookup and its gradient.

TEST INFRASTRUCTURE ONLY.  Plain fp64 numpy.

    out[n] = scale table[ids[n]],   table_bar[r] = scale sum_{n: ids[n] = r} g[n],

ids outside the table are padding: a zero row, no gradient.

Pins (tests/test_oracle_attention.py): one-hot products, padding rows, the
adjoint identity <g, out(table)> = <table_bar(g), table>.
"""

from __future__ import annotations

import numpy as np


def embed_fwd(table, ids, scale):
    ids = np.asarray(ids)
    real = (ids >= 0) & (ids < table.shape[0])
    return np.where(real[:, None], scale * table[np.where(real, ids, 0)], 0.0)


def embed_vjp(n_rows, ids, g, scale):
    out = np.zeros((n_rows, g.shape[1]))
    for n, i in enumerate(np.asarray(ids)):
        if 0 <= i < n_rows:
            out[i] += scale * g[n]
    return out
