"""GPU parity of attention among the rows of segments against the oracle.

Tolerances are first-order bounds, element by element, from the magnitudes of
each sum (``bounds``): u = 2^-24 per fp32 rounding, n u for a sum of n terms in
any order, half a step of bfloat16 (2^-8) where the kernels round matrix
operands (probabilities, score gradients) and outputs."""
import numpy as np
import pytest

from oracle import attention as att

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F = lambda t: t.double().cpu().numpy()
TYPES = ["f32", "bf16"]


class Case:
    """One problem on the GPU.  ``tail`` rows behind the last segment hold NaN
    and must stay untouched in every output."""

    def __init__(self, dtype, lens_q, lens_k=None, hq=2, hk=1, D=32, cap=0.0, bias=False, causal=False, prefix=None,
                 self_pos=None, strided=False, tail=0, seed=0, scale=None, spread=3.0, segments=True):
        from cartesian_tensor_product_amd import flashcart as fc
        self.fc = fc
        rng = np.random.default_rng(seed)
        self.dt = dt = torch.float32 if dtype == "f32" else torch.bfloat16
        own_keys = lens_k is None
        lens_k = lens_q if own_keys else lens_k
        self.oq, self.ok = np.cumsum([0] + list(lens_q)), np.cumsum([0] + list(lens_k))
        self.rows_q, self.rows_k = int(self.oq[-1]), int(self.ok[-1])
        nq, nk = self.rows_q + tail, self.rows_k + tail

        def t(n, rows, *s):
            a = torch.from_numpy(rng.standard_normal((n,) + s)).float()
            a[rows:] = float("nan")
            return a

        if strided:   # parts of one projection
            a = t(nq, self.rows_q, (hq + 2 * hk) * D).to(dt).cuda()
            self.q = a[:, :hq * D].view(nq, hq, D)
            self.k = a[:, hq * D:(hq + hk) * D].view(nq, hk, D)
            self.v = a[:, (hq + hk) * D:].view(nq, hk, D)
        else:
            self.q = t(nq, self.rows_q, hq, D).to(dt).cuda()
            self.k, self.v = t(nk, self.rows_k, hk, D).to(dt).cuda(), t(nk, self.rows_k, hk, D).to(dt).cuda()
        self.g = t(nq, self.rows_q, hq, D).to(dt).cuda()
        self.cap, self.causal, self.prefix, self.hq, self.hk, self.D = cap, causal, prefix, hq, hk, D
        self.scale = float(np.float32(1 / np.sqrt(D) if scale is None else scale))
        self.slope = self.pos_q = self.pos_k = None
        self.self_pos = own_keys if self_pos is None else self_pos
        if bias:
            self.slope = torch.from_numpy(0.2 + rng.random(hq)).float().cuda()
            self.pos_q = spread * t(nq, self.rows_q, 3).cuda()
            self.pos_k = None if self.self_pos else spread * t(nk, self.rows_k, 3).cuda()
        seg_k = None if own_keys else self.ok
        self.seg = fc.Segments(self.oq, seg_k, prefix) if segments else None
        self.d = fc.attn_desc(nq, nk, len(lens_q), hq, hk, D, self.scale, cap, fc.FC_F32 if dtype == "f32" else fc.FC_BF16,
                              fc.FC_ATTN_CAUSAL if causal else 0)

    def inputs(self):
        return self.d, self.seg, self.q, self.k, self.v, self.slope, self.pos_q, self.pos_k

    def fwd(self):
        out = torch.full(self.g.shape, float("nan"), dtype=self.dt, device="cuda")
        lse = torch.full(self.g.shape[:2], float("nan"), device="cuda")
        self.fc.fc_attention_fwd(*self.inputs(), out, lse, self.fc.workspace(self.fc.fc_attention_workspace_bytes(self.d, 0)))
        return out, lse

    def names(self):
        n = ["q", "k", "v"]
        if self.slope is not None:
            n += ["slope", "pos_q"] + ([] if self.pos_k is None else ["pos_k"])
        return n

    def vjp(self, out, lse, want=None):
        """dict of gradients, those in ``want`` (all by default)."""
        like = {"q": self.g, "k": self.k, "v": self.v, "slope": self.slope, "pos_q": self.pos_q, "pos_k": self.pos_k}
        want = self.names() if want is None else want
        r = {n: torch.full(like[n].shape, float("nan"), dtype=like[n].dtype, device="cuda") for n in want}
        self.fc.fc_attention_vjp(*self.inputs(), out, lse, self.g, *(r.get(n) for n in like),
                                 self.fc.workspace(self.fc.fc_attention_workspace_bytes(self.d, 1)))
        return r

    # -------------------------------------------------------------- oracle --

    def arrays(self):
        nq, nk = self.rows_q, self.rows_k
        bias = {}
        if self.slope is not None:
            pq = F(self.pos_q)[:nq]
            bias = dict(slope=F(self.slope), pos_q=pq, pos_k=pq if self.pos_k is None else F(self.pos_k)[:nk])
        return F(self.q)[:nq], F(self.k)[:nk], F(self.v)[:nk], F(self.g)[:nq], bias

    def bounds(self, want_out, want_lse):
        """First-order bounds of every output's error."""
        q, k, v, g, bias = self.arrays()
        rho = 2.0 ** -8 if self.dt == torch.bfloat16 else 0.0
        half = max(rho, U)
        G = self.hq // self.hk
        b = {"out": np.zeros(q.shape), "lse": np.zeros(q.shape[:2]), "q": np.zeros(q.shape), "k": np.zeros(k.shape),
             "v": np.zeros(v.shape), "slope": np.zeros(self.hq), "pos_q": np.zeros((len(q), 3)), "pos_k": np.zeros((len(k), 3))}
        for s, h, kh, A, B in att._blocks(self.oq, self.ok, self.hq, self.hk):
            lq, lk = A.stop - A.start, B.stop - B.start
            if lq == 0 or lk == 0:
                continue
            see = att.visible(lq, lk, self.causal, 0 if self.prefix is None else self.prefix[s])
            sl = bias["slope"][h] if bias else None
            sc, th, r, diff = att._scores(q[A, h], k[B, kh], self.scale, self.cap, sl, *((bias["pos_q"][A], bias["pos_k"][B]) if bias else (None, None)))
            P, lse = att._softmax(sc, see)
            lse = np.where(np.isfinite(lse), lse, 0)[:, None]
            size = self.scale * np.abs(q[A, h]) @ np.abs(k[B, kh]).T
            es = U * ((self.D + 4) * size + 5 * self.cap + 8 * (np.abs(sc) + (2 * sl * r if bias else 0)) + 4)
            es = np.where(see, es, 0)
            el = es.max(1, keepdims=True) + (lk + 8) * U + 4 * U * np.abs(lse)
            eP = es + el
            b["lse"][A, h] = el[:, 0]
            b["out"][A, h] = (P * (eP + rho + (lk + 2) * U)) @ np.abs(v[B, kh]) + half * np.abs(want_out[A, h])
            dP = g[A, h] @ v[B, kh].T
            edP = (self.D + 2) * U * np.abs(g[A, h]) @ np.abs(v[B, kh]).T
            delta = (P * dP).sum(1, keepdims=True)
            # delta: from the scores, also of rows that see few keys, or from out
            scores = (P * (np.abs(dP) * (eP + (lk + 2) * U) + edP)).sum(1, keepdims=True)
            out = (np.abs(g[A, h]) * (b["out"][A, h] + (self.D + 2) * U * np.abs(want_out[A, h]))).sum(1, keepdims=True)
            ed = scores if rho and bias else np.where(see.sum(1, keepdims=True) <= 32, scores, out)
            dS = P * (dP - delta)
            edS = np.abs(dS) * (eP + 4 * U) + P * (edP + ed)
            n = lq * lk
            if bias:
                b["slope"][h] += ((edS + np.abs(dS) * (n + 8) * U) * r).sum()
                w = sl * (edS + np.abs(dS) * (max(lq, lk) * self.hq + 8) * U)
                unit = np.abs(diff) / np.where(r > 0, r, 1)[..., None]
                b["pos_q"][A] += (w[..., None] * unit).sum(1)
                b["pos_k"][B] += (w[..., None] * unit).sum(0)
            edS = edS + 16 * U * np.abs(dS)
            b["q"][A, h] += self.scale * (edS + (rho + (lk + 2) * U) * np.abs(dS)) @ np.abs(k[B, kh])
            b["k"][B, kh] += self.scale * (edS + (rho + (lq * G + 2) * U) * np.abs(dS)).T @ np.abs(q[A, h])
            b["v"][B, kh] += (P * (eP + rho + (lq * G + 2) * U)).T @ np.abs(g[A, h])
        return b, half

    def check(self, back=True):
        q, k, v, g, bias = self.arrays()
        kw = dict(cap=float(np.float32(self.cap)), causal=self.causal, prefix=self.prefix, **bias)
        out, lse = self.fwd()
        grads = self.vjp(out, lse) if back else {}
        torch.cuda.synchronize()
        want_out, want_lse = att.fwd(q, k, v, self.oq, self.ok, self.scale, **kw)
        bound, half = self.bounds(want_out, want_lse)
        nq = self.rows_q
        assert torch.isnan(out[nq:]).all() and torch.isnan(lse[nq:]).all(), "rows behind the segments were written"
        self.close("out", F(out)[:nq], want_out, bound["out"])
        empty = np.isneginf(want_lse)
        got = F(lse)[:nq]
        assert np.isneginf(got[empty]).all() and (F(out)[:nq][empty] == 0).all()
        self.close("lse", got[~empty], want_lse[~empty], bound["lse"][~empty])
        if not back:
            return
        want = att.vjp(q, k, v, self.oq, self.ok, self.scale, g, **kw)
        if bias and self.pos_k is None:
            want["pos_q"] = want["pos_q"] + want["pos_k"]
            bound["pos_q"] = bound["pos_q"] + bound["pos_k"]
        for n in self.names():
            rows = len(want[n])
            if n != "slope":
                assert torch.isnan(grads[n][rows:]).all(), f"{n}: rows behind the segments were written"
            step = half if n in "qkv" else 2 * U
            self.close(n, F(grads[n])[:rows], want[n], bound[n] + step * np.abs(want[n]))

    @staticmethod
    def close(name, got, want, tol):
        err = np.abs(got - want)
        bad = ~(err <= tol + 1e-30)
        assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off, worst {err[bad].max():.3e} for a bound {tol[bad][err[bad].argmax()]:.3e}"


RAGGED = (1, 0, 31, 32, 33, 70, 2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [8, 16, 24, 32, 40, 64, 72, 96, 128])
def test_head_dims(dtype, D):
    Case(dtype, RAGGED, hq=2, hk=1, D=D, bias=True, seed=D).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (4, 1), (6, 2), (8, 8), (5, 1)])
def test_head_layouts(dtype, hq, hk):
    Case(dtype, (40, 9, 129), hq=hq, hk=hk, D=16, bias=True, cap=5.0, seed=hq).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cap", [0.0, 2.0])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("causal", [False, True])
def test_options(dtype, cap, bias, causal):
    """Lengths around the tile sizes, more queries than keys (empty rows when
    causal) and fewer, segments without queries or without keys."""
    Case(dtype, (5, 64, 0, 33, 130, 7), (9, 63, 4, 65, 40, 0), hq=4, hk=2, D=32, cap=cap, bias=bias, causal=causal,
         seed=1).check()


@pytest.mark.parametrize("dtype", TYPES)
def test_causal_prefix(dtype):
    Case(dtype, (70, 1, 150, 40), (70, 30, 100, 60), hq=2, hk=1, D=64, causal=True, prefix=[33, 30, 0, 7], bias=True,
         seed=2).check()


@pytest.mark.parametrize("dtype", TYPES)
def test_long_segments(dtype):
    Case(dtype, (700, 389), hq=2, hk=2, D=32, bias=True, seed=3).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bias", [False, True])
def test_single_queries_over_many_keys(dtype, bias):
    """The walk over keys is split and joined."""
    Case(dtype, (1, 1, 3), (2500, 1, 1200), hq=4, hk=2, D=64, bias=bias, cap=3.0, seed=4).check()


@pytest.mark.parametrize("dtype", TYPES)
def test_few_keys_under_many_queries(dtype):
    """The walk over queries is split and joined."""
    Case(dtype, (2000, 900), (2, 5), hq=4, hk=2, D=32, bias=True, seed=5).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens_q,lens_k", [((40, 700, 0, 300, 1, 500, 33), None), ((300, 0, 500, 129, 129), (5, 60, 200, 0, 900))])
def test_segments_of_different_lengths(dtype, causal, lens_q, lens_k):
    """More blocks than run at once: the long segments are started first."""
    Case(dtype, lens_q, lens_k, hq=16, hk=16, D=16, causal=causal, bias=not causal).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("lens_q,lens_k,causal", [((1, 1), None, True), ((5, 0, 1, 70), (1, 1, 1, 1), False), ((300,), (1,), False)])
def test_rows_of_one_key(dtype, cap, bias, lens_q, lens_k, causal):
    """Their probability is 1 whatever the score: no score gradient, not a rounding's rest."""
    c = Case(dtype, lens_q, lens_k, hq=4, hk=2, D=48, cap=cap, bias=bias, causal=causal)
    grads = c.vjp(*c.fwd())
    for name, x in grads.items():
        assert name == "v" or not x.any(), name
    c.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens", [(2,), (2, 3, 9, 32), (33, 40)])
def test_causal_rows_of_few_keys(dtype, lens):
    """Differences dP - delta far below dP."""
    Case(dtype, lens, hq=4, hk=1, D=128, causal=True, cap=20.0).check()
    Case(dtype, lens, hq=2, hk=2, D=64, causal=True, scale=1.0).check()


@pytest.mark.parametrize("dtype", TYPES)
def test_single_causal_query_is_the_last_row(dtype):
    """The form for one new row: its output is that of the whole batch."""
    whole = Case(dtype, (300,), hq=4, hk=2, D=64, causal=True, bias=True, seed=6)
    out, lse = whole.fwd()
    one = Case(dtype, (1,), (300,), hq=4, hk=2, D=64, causal=True, bias=True, seed=6)
    one.q, one.k, one.v, one.slope = whole.q[-1:].clone(), whole.k, whole.v, whole.slope
    one.pos_q, one.pos_k = whole.pos_q[-1:].clone(), whole.pos_q
    o1, l1 = one.fwd()
    step = 2.0 ** -7 if dtype == "bf16" else 400 * U
    assert (o1[0] - out[-1]).abs().max() <= step * out.abs().max() and (l1[0] - lse[-1]).abs().max() <= 400 * U * 10


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_behind_the_segments(dtype):
    """NaN rows behind the last segment are not read and not written, with
    split and whole walks."""
    Case(dtype, (20, 45), hq=2, hk=1, D=32, bias=True, tail=13, seed=7).check()
    Case(dtype, (2,), (1500,), hq=2, hk=1, D=32, bias=True, tail=5, seed=8).check()
    Case(dtype, (1500,), (2,), hq=2, hk=1, D=32, bias=True, tail=5, seed=9).check()


@pytest.mark.parametrize("dtype", TYPES)
def test_parts_of_a_projection(dtype):
    Case(dtype, (50, 3, 81), hq=4, hk=2, D=64, strided=True, bias=True, seed=10).check()


@pytest.mark.parametrize("dtype", TYPES)
def test_one_segment_without_offsets(dtype):
    Case(dtype, (77,), hq=2, hk=2, D=32, bias=True, segments=False, seed=11).check()


def test_many_segments():
    """More segments than a wave looks at per step, many of them empty."""
    rng = np.random.default_rng(12)
    lens = tuple(int(x) for x in rng.integers(0, 7, 5000))
    Case("f32", lens, hq=1, hk=1, D=8, bias=True, seed=12).check()


def test_coincident_points():
    """Distance 0 has gradient 0 (every atom with itself, and doubled atoms)."""
    c = Case("f32", (40,), hq=2, hk=1, D=16, bias=True, seed=13)
    c.pos_q[20:] = c.pos_q[:20]
    c.check()


@pytest.mark.parametrize("dtype", TYPES)
def test_large_scores(dtype):
    """Sharp rows (one key takes all) and scores far below the first ones."""
    Case(dtype, (150,), (300,), hq=2, hk=1, D=32, scale=6.0, seed=14).check()
    Case(dtype, (150,), (300,), hq=2, hk=1, D=32, bias=True, spread=200.0, seed=15).check()


def test_no_rows():
    for lq, lk in (((0,), (5,)), ((5,), (0,)), ((0, 0), (0, 0))):
        Case("f32", lq, lk, hq=2, hk=1, D=16, bias=True, seed=16).check()


def test_gradients_against_differences():
    """Central differences of <g, out> along random directions; the forward's
    fp32 noise is about 1e-6 of its size, the step keeps it below 1e-2."""
    c = Case("f32", (30, 41), hq=2, hk=1, D=16, cap=4.0, bias=True, causal=True, seed=17)
    grads = c.vjp(*c.fwd())
    leaves = {"q": c.q, "k": c.k, "v": c.v, "slope": c.slope, "pos_q": c.pos_q}
    for n, t in leaves.items():
        rnd = torch.randn(t.shape, generator=torch.Generator().manual_seed(3)).cuda()
        keep, h, vals = t.clone(), 1e-2, []
        for sgn in (1, -1):
            t.copy_(keep + sgn * h * rnd)
            vals.append((c.fwd()[0].double() * c.g.double()).sum().item())
        t.copy_(keep)
        want = (vals[0] - vals[1]) / (2 * h)
        size = (grads[n].double().abs() * rnd.double().abs()).sum().item()
        assert abs((grads[n].double() * rnd.double()).sum().item() - want) <= 1e-2 * size, n


@pytest.mark.parametrize("dtype", TYPES)
def test_single_gradients_agree_with_all(dtype):
    c = Case(dtype, (60, 35), hq=4, hk=2, D=32, bias=True, self_pos=False, seed=18)
    out, lse = c.fwd()
    full = c.vjp(out, lse)
    for n in c.names():
        got = c.vjp(out, lse, want=[n])[n]
        if dtype == "bf16" and n in "qk":   # delta then comes from out: test_options without a bias
            continue
        assert torch.equal(got, full[n]), n


@pytest.mark.parametrize("lens_q,lens_k", [((100, 200), None), ((3,), (4000,))])
def test_bitwise_reproducible(lens_q, lens_k):
    c = Case("bf16", lens_q, lens_k, hq=4, hk=2, D=64, bias=True, seed=19)
    a, b = c.fwd(), c.fwd()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    ga, gb = c.vjp(*a), c.vjp(*b)
    assert all(torch.equal(ga[n], gb[n]) for n in ga)


def test_two_streams_at_once():
    """Two calls that overlap, a workspace each."""
    cs = [Case("bf16", (500, 300), hq=4, hk=2, D=64, bias=True, seed=20),
          Case("f32", (4,), (3000,), hq=4, hk=2, D=32, bias=True, seed=21)]
    alone = [(c.fwd(), c.vjp(*c.fwd())) for c in cs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cs], []
    for c, s in zip(cs, streams):
        with torch.cuda.stream(s):
            f = c.fwd()
            got.append((f, c.vjp(*f)))
    torch.cuda.synchronize()
    for (f0, g0), (f1, g1) in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(f0, f1)) and all(torch.equal(g0[n], g1[n]) for n in g0)


@pytest.mark.parametrize("lens_q,lens_k", [((100, 200), None), ((2, 1), (1500, 900))])
def test_captured(lens_q, lens_k):
    """Forward and VJP in a graph, replayed on new values with eager calls in
    between."""
    c = Case("f32", lens_q, lens_k, hq=2, hk=1, D=32, bias=True, seed=22)
    fc = c.fc
    ws = [fc.workspace(fc.fc_attention_workspace_bytes(c.d, op)) for op in (0, 1)]
    out, lse = torch.empty_like(c.g), torch.empty(c.g.shape[:2], device="cuda")
    like = {"q": c.g, "k": c.k, "v": c.v, "slope": c.slope, "pos_q": c.pos_q, "pos_k": c.pos_k}
    r = {n: None if t is None else torch.empty_like(t) for n, t in like.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fc.fc_attention_fwd(*c.inputs(), out, lse, ws[0])
        fc.fc_attention_vjp(*c.inputs(), out, lse, c.g, *r.values(), ws[1])
    for i in range(3):
        c.q.mul_(1.1)
        c.pos_q.add_(0.1 * i)
        graph.replay()
        torch.cuda.synchronize()
        o, l = c.fwd()
        eager = c.vjp(o, l)
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(lse, l)
        assert all(torch.equal(r[n], eager[n]) for n in eager)


def test_offsets_past_two_gib():
    """Keys and values of 2.6 GB each: the last segment lies behind 2^31
    bytes."""
    from cartesian_tensor_product_amd import flashcart as fc
    hk, D, nk = 8, 128, 640000
    k = torch.zeros(nk, hk, D, device="cuda", dtype=torch.bfloat16).repeat(1, 2, 1)[:, :hk]   # rows 2 hk D apart
    assert k.stride(0) * nk * 2 > 2 ** 31
    tail = torch.randn(70, hk, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    k[-70:] = tail
    q = torch.randn(3, hk, D, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    d = fc.attn_desc(3, nk, 2, hk, hk, D, 0.1, 0.0, fc.FC_BF16)
    out, lse = torch.empty_like(q), torch.empty(3, hk, device="cuda")
    fc.fc_attention_fwd(d, fc.Segments([0, 0, 3], [0, nk - 70, nk]), q, k, k, None, None, None, out, lse,
                        fc.workspace(fc.fc_attention_workspace_bytes(d, 0)))
    d2 = fc.attn_desc(3, 70, 1, hk, hk, D, 0.1, 0.0, fc.FC_BF16)
    o2, l2 = torch.empty_like(q), torch.empty(3, hk, device="cuda")
    fc.fc_attention_fwd(d2, None, q, tail, tail, None, None, None, o2, l2, fc.workspace(fc.fc_attention_workspace_bytes(d2, 0)))
    assert torch.allclose(lse, l2, atol=1e-5) and (out.float() - o2.float()).abs().max() <= 2.0 ** -7 * o2.float().abs().max()
