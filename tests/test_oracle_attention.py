"""Pins of the embedding, query/key norm and attention oracles."""
import numpy as np
import pytest

from oracle import attention as att, embed, qk_rope


def rng(seed):
    return np.random.default_rng(seed)


# -------------------------------------------------------------- embedding --

def test_embed_is_a_one_hot_product():
    r = rng(0)
    table, ids, g = r.standard_normal((7, 5)), np.array([3, 0, 3, 6, -1, 7, 2]), r.standard_normal((7, 5))
    hot = (ids[:, None] == np.arange(7)).astype(float)   # padding rows are zero
    assert np.allclose(embed.embed_fwd(table, ids, 2.5), 2.5 * hot @ table, rtol=0, atol=1e-15)
    assert np.allclose(embed.embed_vjp(7, ids, g, 2.5), 2.5 * hot.T @ g, rtol=0, atol=1e-14)


# ------------------------------------------------------- query/key rotation --

def test_rope_pair_by_hand():
    x = np.array([[[3.0, 4.0]]])
    o = qk_rope.fwd(x, np.array([1.0, 2.0]), np.array([[0.5, 0.0, 0.0]]), np.array([[np.pi, 7.0, 9.0]]), 0.0)
    y = np.array([3.0, 8.0]) / np.sqrt(12.5)       # quarter turn
    assert np.allclose(o[0, 0], [-y[1], y[0]], atol=1e-15)


def test_rope_scores_depend_on_differences_only():
    r = rng(1)
    x, z = r.standard_normal((2, 1, 1, 8))
    freq, g = r.standard_normal((4, 3)), np.ones(8)
    p, q, shift = r.standard_normal((3, 1, 3))
    dot = lambda a, b: (qk_rope.fwd(x, g, a, freq, 1e-3) * qk_rope.fwd(z, g, b, freq, 1e-3)).sum()
    assert abs(dot(p, q) - dot(p + shift, q + shift)) < 1e-12
    assert abs(dot(p, q) - dot(p, q + shift)) > 1e-3
    n = lambda a: np.linalg.norm(qk_rope.fwd(x, g, a, freq, 1e-3))
    assert abs(n(p) - n(q)) < 1e-13


def test_rope_layouts_agree_through_a_permutation():
    r = rng(2)
    x, gamma, pos, freq = r.standard_normal((3, 2, 10)), r.standard_normal(10), r.standard_normal((3, 3)), r.standard_normal((4, 3))
    perm = np.empty(10, int)                      # half layout position of each interleaved element
    perm[0:8:2], perm[1:8:2], perm[8:] = np.arange(4), np.arange(4) + 4, [8, 9]
    half = qk_rope.fwd(x, gamma, pos, freq, 0.1)
    inter = qk_rope.fwd(x[..., perm], gamma[perm], pos, freq, 0.1, interleaved=True)
    assert np.allclose(inter, half[..., perm], atol=1e-14)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_vjp_against_complex_step(interleaved):
    r = rng(3)
    x, gamma, pos, freq = r.standard_normal((2, 3, 8)), r.standard_normal(8), r.standard_normal((2, 3)), r.standard_normal((3, 3))
    g = r.standard_normal(x.shape)
    grads = qk_rope.vjp(x, gamma, pos, freq, 0.05, g, interleaved)
    args = [x, gamma, pos]
    for which, grad in enumerate(grads):
        for idx in np.ndindex(*args[which].shape):
            c = [a.astype(complex) for a in args]
            c[which][idx] += 1e-20j
            d = (g * qk_rope.fwd(*c, freq, 0.05, interleaved)).sum().imag / 1e-20
            assert abs(d - grad[idx]) < 1e-12 * max(1.0, np.abs(grad).max())


# -------------------------------------------------------------- attention --

def test_two_keys_by_hand():
    q, k, v = np.array([[[2.0]]]), np.array([[[1.0]], [[3.0]]]), np.array([[[10.0]], [[20.0]]])
    out, lse = att.fwd(q, k, v, [0, 1], [0, 2], 0.5, slope=np.array([0.25]), pos_q=np.zeros((1, 3)),
                       pos_k=np.array([[0, 0, 4.0], [0, 3.0, 4.0]]))
    s = np.array([1.0 - 1.0, 3.0 - 1.25])
    assert np.allclose(lse, np.log(np.exp(s).sum())) and np.allclose(out, np.exp(s) @ [10, 20] / np.exp(s).sum())
    out, lse = att.fwd(q, k, v, [0, 1], [0, 2], 0.5, cap=2.0)
    s = 2 * np.tanh(np.array([0.5, 1.5]))
    assert np.allclose(out, np.exp(s) @ [10, 20] / np.exp(s).sum())


def test_causal_rule():
    assert att.visible(3, 5, True).tolist() == [[True] * 3 + [False] * 2, [True] * 4 + [False], [True] * 5]
    assert att.visible(3, 2, True).tolist() == [[False, False], [True, False], [True, True]]   # an empty row
    assert att.visible(3, 3, True, 2).tolist() == [[True, True, False], [True, True, False], [True] * 3]


def inputs(seed, hq=4, hk=2, D=8, lens_q=(3, 0, 5), lens_k=(4, 2, 3)):
    r = rng(seed)
    oq, ok = np.cumsum((0,) + lens_q), np.cumsum((0,) + lens_k)
    q, k, v = r.standard_normal((oq[-1], hq, D)), r.standard_normal((ok[-1], hk, D)), r.standard_normal((ok[-1], hk, D))
    return r, oq, ok, q, k, v, r.random(hq), r.standard_normal((oq[-1], 3)), r.standard_normal((ok[-1], 3))


def test_segments_shared_heads_and_empty_rows():
    r, oq, ok, q, k, v, slope, pq, pk = inputs(4)
    kw = dict(cap=3.0, causal=True, prefix=[1, 0, 0])
    out, lse = att.fwd(q, k, v, oq, ok, 0.4, slope=slope, pos_q=pq, pos_k=pk, **kw)
    # repeated key heads, one segment alone
    o2, _ = att.fwd(q[3:], k[6:].repeat(2, 1), v[6:].repeat(2, 1), [0, 5], [0, 3], 0.4, slope=slope, pos_q=pq[3:],
                    pos_k=pk[6:], cap=3.0, causal=True, prefix=[0])
    assert np.allclose(out[3:], o2)
    # five queries over three keys: the first two see nothing
    assert (out[3:5] == 0).all() and np.isneginf(lse[3:5]).all() and np.isfinite(lse[5:]).all()
    # the last query alone is the last row of the batch
    o3, _ = att.fwd(q[7:], k[6:], v[6:], [0, 1], [0, 3], 0.4, slope=slope, pos_q=pq[7:], pos_k=pk[6:], cap=3.0, causal=True)
    assert np.allclose(out[7:], o3)


@pytest.mark.parametrize("cap,bias,causal", [(0.0, False, False), (2.0, True, False), (0.0, True, True), (1.5, False, True)])
def test_attention_vjp_against_complex_step(cap, bias, causal):
    r, oq, ok, q, k, v, slope, pq, pk = inputs(5, D=4)
    g = r.standard_normal(q.shape)
    names = ["q", "k", "v"] + (["slope", "pos_q", "pos_k"] if bias else [])
    args = dict(q=q, k=k, v=v)
    if bias:
        args.update(slope=slope, pos_q=pq, pos_k=pk)
    kw = dict(cap=cap, causal=causal, prefix=[2, 0, 1] if causal else None)
    grads = att.vjp(off_q=oq, off_k=ok, scale=0.6, g_out=g, **args, **kw)
    for n in names:
        for idx in np.ndindex(*args[n].shape):
            c = dict(args)
            c[n] = args[n].astype(complex)
            c[n][idx] += 1e-20j
            d = (g * att.fwd(off_q=oq, off_k=ok, scale=0.6, **c, **kw)[0]).sum().imag / 1e-20
            assert abs(d - grads[n][idx]) < 1e-12 * max(1.0, np.abs(grads[n]).max()), (n, idx)
