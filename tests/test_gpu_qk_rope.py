"""GPU parity of the query/key norm with rotation against the oracle.

Tolerances (u = 2^-24, first order, any order of summation): the norm is an
fp32 sum of D squares, a root and two products, cosine and sine are within 2u,
so an output element is within (D/2 + 16) u of (|y1| + |y2|) of its pair, plus
half a step of its type; the VJP adds a second sum of D products; parameter
and position gradients add the length of their sums."""
import numpy as np
import pytest

from oracle import qk_rope

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F = lambda t: t.double().cpu().numpy()


class Case:
    def __init__(self, dtype, N, hq, hk, D, R, interleaved=False, seed=0, eps=1e-5, strided=False, gammas=True,
                 far=0.0):
        from cartesian_tensor_product_amd import flashcart as fc
        self.fc, self.inter, self.eps = fc, interleaved, eps
        self.shape = (N, hq, hk, D, R)
        rng = np.random.default_rng(seed)
        self.dt = dt = torch.float32 if dtype == "f32" else torch.bfloat16
        t = lambda *s: torch.from_numpy(rng.standard_normal(s)).float()
        if strided:   # parts of one projection
            a = t(N, (hq + 2 * hk) * D).to(dt).cuda()
            self.q, self.k = a[:, :hq * D].view(N, hq, D), a[:, hq * D:(hq + hk) * D].view(N, hk, D)
        else:
            self.q, self.k = t(N, hq, D).to(dt).cuda(), t(N, hk, D).to(dt).cuda()
        self.gq, self.gk = ((1 + 0.2 * t(D)).cuda(), (1 + 0.2 * t(D)).cuda()) if gammas else (None, None)
        self.pos, self.freq = (5 * t(N, 3) + far).cuda(), t(R, 3).cuda()
        self.g_q, self.g_k = t(N, hq, D).to(dt).cuda(), t(N, hk, D).to(dt).cuda()
        self.d = fc.qk_rope_desc(N, hq, hk, D, R, eps, fc.FC_F32 if dtype == "f32" else fc.FC_BF16,
                                 fc.FC_ROPE_INTERLEAVED if interleaved else 0)

    def inputs(self):
        return self.d, self.q, self.k, self.gq, self.gk, self.pos, self.freq

    def fwd(self):
        qo, ko = torch.empty_like(self.g_q), torch.empty_like(self.g_k)
        self.fc.fc_qk_norm_rope_fwd(*self.inputs(), qo, ko)
        return qo, ko

    def vjp(self, want="qkabp"):
        new = lambda c, t: torch.full_like(t, float("nan")) if c in want else None
        D = self.shape[3]
        z = torch.zeros(D, device="cuda")
        outs = (new("q", self.g_q), new("k", self.g_k), new("a", z), new("b", z), new("p", self.pos))
        self.fc.fc_qk_norm_rope_vjp(*self.inputs(), self.g_q, self.g_k, *outs,
                                    self.fc.workspace(self.fc.fc_qk_norm_rope_workspace_bytes(self.d)))
        return outs

    def check(self):
        N, hq, hk, D, R = self.shape
        outs, grads = self.fwd(), self.vjp()
        torch.cuda.synchronize()
        half = torch.finfo(self.dt).eps / 2
        pos, freq, eps = F(self.pos), F(self.freq), float(np.float32(self.eps))
        a, b = qk_rope.pairs(R, self.inter)
        mate = np.arange(D)
        mate[a], mate[b] = b, a
        pos_want, pos_size = np.zeros((N, 3)), np.zeros((N, 3))
        for x, gam, o, g, xb, gb in ((self.q, self.gq, outs[0], self.g_q, grads[0], grads[2]),
                                     (self.k, self.gk, outs[1], self.g_k, grads[1], grads[3])):
            if x.shape[1] == 0:
                continue
            x, g, gam = F(x), F(g), np.ones(D) if gam is None else F(gam)
            want = qk_rope.fwd(x, gam, pos, freq, eps, self.inter)
            r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
            y = np.abs(gam * x) * r
            pair = y + y[..., mate]
            assert (np.abs(F(o) - want) <= (D / 2 + 16) * U * pair + half * np.abs(want)).all()
            wx, wg, wp = qk_rope.vjp(x, gam, pos, freq, eps, g, self.inter)
            gp = np.abs(g) + np.abs(g)[..., mate]          # bound of the cotangent rotated back
            gg = np.abs(gam) * gp
            size = r * (gg + np.abs(x) * r * r * (gg * np.abs(x)).sum(-1, keepdims=True) / D)
            assert (np.abs(F(xb) - wx) <= (2 * D + 40) * U * size + half * np.abs(wx)).all()
            size = (gp * np.abs(x) * r).sum((0, 1))
            assert (np.abs(F(gb) - wg) <= (N * x.shape[1] + D + 40) * U * size).all()
            pos_want += wp
            th = ((gp * pair)[..., a]).sum(1) * 2
            pos_size += th @ np.abs(freq)
        assert (np.abs(F(grads[4]) - pos_want) <= ((hq + hk) * R + D + 40) * U * pos_size).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N,hq,hk,D,R", [(1, 1, 1, 2, 1), (5, 4, 2, 16, 8), (37, 3, 1, 24, 12), (9, 4, 4, 32, 5),
                                         (130, 8, 2, 64, 32), (3, 2, 1, 6, 3), (21, 5, 2, 80, 40), (40, 16, 4, 128, 48),
                                         (11, 2, 2, 128, 64), (4, 1, 0, 32, 16), (6, 2, 1, 48, 0)])
def test_shapes(dtype, interleaved, N, hq, hk, D, R):
    Case(dtype, N, hq, hk, D, R, interleaved, seed=N + D).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_nodes(dtype):
    """More nodes than one turn of the VJP's grid."""
    Case(dtype, 70000 if dtype == "f32" else 30011, 2, 1, 32, 16, seed=1).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,R", [(64, 32), (20, 7)])
def test_parts_of_a_projection(dtype, D, R):
    Case(dtype, 50, 4, 2, D, R, seed=2, strided=True).check()


def test_without_gamma_and_large_eps():
    Case("f32", 12, 2, 2, 32, 16, seed=3, gammas=False, eps=0.5).check()


def test_far_positions():
    """Angles of 1e5 and more radians keep their digits."""
    Case("f32", 40, 2, 1, 32, 16, seed=4, far=30000.0).check()


def test_no_rotation():
    c = Case("f32", 8, 2, 1, 16, 8, seed=5)
    want = c.fwd()
    c.freq.zero_()
    zero = c.fwd()
    c.pos = c.freq = None
    none = c.fwd()
    assert all(torch.equal(a, b) for a, b in zip(zero, none)) and not torch.equal(want[0], none[0])


def test_single_outputs_agree_with_all():
    c = Case("bf16", 33, 4, 2, 64, 32, seed=6)
    full = c.vjp()
    for i, w in enumerate("qkabp"):
        got = c.vjp(want=w)
        assert torch.equal(got[i], full[i]) and all(g is None for j, g in enumerate(got) if j != i)


def test_zero_rows_and_no_nodes():
    c = Case("f32", 7, 2, 1, 16, 8, seed=7)
    c.q.zero_()
    assert (c.fwd()[0] == 0).all() and all(torch.isfinite(t).all() for t in c.vjp())
    c = Case("f32", 0, 2, 1, 16, 8, seed=8)
    c.fwd()
    assert (c.vjp()[2] == 0).all()


def test_bitwise_reproducible_and_captured():
    c = Case("bf16", 3000, 8, 2, 64, 32, seed=9)
    a, b = c.vjp(), c.vjp()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    ws = c.fc.workspace(c.fc.fc_qk_norm_rope_workspace_bytes(c.d))
    outs = [torch.empty_like(t) for t in a]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.fc.fc_qk_norm_rope_vjp(*c.inputs(), c.g_q, c.g_k, *outs, ws)
    for i in range(3):
        c.pos.add_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, c.vjp()))
        torch.cuda.synchronize()
