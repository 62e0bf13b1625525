"""The path from species to attention and back, as a program runs it: embedding,
one linear map to queries, keys and values, norm and rotation, attention, and
the VJPs in reverse, against the oracles chained in fp64.  The parity bar is
that of the other GPU tests (1e-4 of each output's largest value)."""
import numpy as np
import pytest

from oracle import attention as att, embed, qk_rope
from tests.gpu_common import assert_close

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LENS, ROWS, C, HQ, HK, D, R = (40, 1, 65, 0, 22), 11, 48, 4, 2, 16, 6
F = lambda t: t.double().cpu().numpy()


class Path:
    def __init__(self, seed=0, device="cuda"):
        from cartesian_tensor_product_amd import flashcart as fc
        self.fc = fc
        rng = np.random.default_rng(seed)
        t = lambda *s: torch.from_numpy(rng.standard_normal(s)).float().to(device)
        n = self.n = sum(LENS)
        self.ids = torch.from_numpy(rng.integers(0, ROWS, n).astype(np.int32)).to(device)
        self.table, self.W = t(ROWS, C), t(C, (HQ + 2 * HK) * D) / np.sqrt(C)
        self.gq, self.gk, self.slope = 1 + 0.1 * t(D), 1 + 0.1 * t(D), 0.3 + 0.1 * t(HQ)
        self.pos, self.freq, self.g = 3 * t(n, 3), 0.3 * t(R, 3), t(n, HQ, D)
        self.offsets = np.cumsum((0,) + LENS)
        self.seg = fc.Segments(self.offsets, device=device)
        self.de = fc.embed_desc(n, ROWS, C, 0.5)
        self.dr = fc.qk_rope_desc(n, HQ, HK, D, R, 1e-5)
        self.da = fc.attn_desc(n, n, len(LENS), HQ, HK, D, 0.25, 8.0)
        new = lambda *s: torch.empty(s, device=device)
        self.h, self.qkv = new(n, C), new(n, (HQ + 2 * HK) * D)
        self.q, self.k, self.v = self.parts(self.qkv)
        self.qn, self.kn, self.out, self.lse = new(n, HQ, D), new(n, HK, D), new(n, HQ, D), new(n, HQ)
        self.gqn, self.gkn, self.gv = new(n, HQ, D), new(n, HK, D), new(n, HK, D)
        self.gq_raw, self.gk_raw = new(n, HQ, D), new(n, HK, D)
        self.g_slope, self.gp1, self.gp2 = new(HQ), new(n, 3), new(n, 3)
        self.g_gq, self.g_gk, self.g_table = new(D), new(D), new(ROWS, C)
        self.ws = [fc.workspace(b, device) for b in (fc.fc_embed_workspace_bytes(self.de),
                                                     fc.fc_qk_norm_rope_workspace_bytes(self.dr),
                                                     fc.fc_attention_workspace_bytes(self.da, 0),
                                                     fc.fc_attention_workspace_bytes(self.da, 1))]

    def parts(self, qkv):
        n = qkv.shape[0]
        return (qkv[:, :HQ * D].reshape(n, HQ, D), qkv[:, HQ * D:(HQ + HK) * D].reshape(n, HK, D),
                qkv[:, (HQ + HK) * D:].reshape(n, HK, D))

    def step(self):
        fc = self.fc
        fc.fc_embed_fwd(self.de, self.table, self.ids, self.h)
        torch.mm(self.h, self.W, out=self.qkv)
        rope = (self.dr, self.q, self.k, self.gq, self.gk, self.pos, self.freq)
        fc.fc_qk_norm_rope_fwd(*rope, self.qn, self.kn)
        attn = (self.da, self.seg, self.qn, self.kn, self.v, self.slope, self.pos, None)
        fc.fc_attention_fwd(*attn, self.out, self.lse, self.ws[2])
        fc.fc_attention_vjp(*attn, self.out, self.lse, self.g, self.gqn, self.gkn, self.gv, self.g_slope, self.gp1, None,
                            self.ws[3])
        fc.fc_qk_norm_rope_vjp(*rope, self.gqn, self.gkn, self.gq_raw, self.gk_raw, self.g_gq, self.g_gk, self.gp2,
                               self.ws[1])
        g_qkv = torch.cat([t.flatten(1) for t in (self.gq_raw, self.gk_raw, self.gv)], 1)
        g_W, g_h = self.h.t() @ g_qkv, (g_qkv @ self.W.t()).contiguous()
        fc.fc_embed_vjp(self.de, self.ids, g_h, self.g_table, self.ws[0])
        return {"out": self.out, "table": self.g_table, "W": g_W, "gamma_q": self.g_gq, "gamma_k": self.g_gk,
                "slope": self.g_slope, "pos": self.gp1 + self.gp2}

    def oracle(self):
        ids, table, W, gq, gk, sl, pos, freq, g = (F(t) if t.is_floating_point() else t.cpu().numpy() for t in (
            self.ids, self.table, self.W, self.gq, self.gk, self.slope, self.pos, self.freq, self.g))
        eps = float(np.float32(1e-5))
        h = embed.embed_fwd(table, ids, 0.5)
        q, k, v = self.parts(h @ W)
        qn, kn = qk_rope.fwd(q, gq, pos, freq, eps), qk_rope.fwd(k, gk, pos, freq, eps)
        kw = dict(off_q=self.offsets, off_k=self.offsets, scale=0.25, cap=8.0, slope=sl, pos_q=pos, pos_k=pos)
        out, _ = att.fwd(qn, kn, v, **kw)
        a = att.vjp(qn, kn, v, g_out=g, **kw)
        xq, g_gq, p1 = qk_rope.vjp(q, gq, pos, freq, eps, a["q"])
        xk, g_gk, p2 = qk_rope.vjp(k, gk, pos, freq, eps, a["k"])
        g_qkv = np.concatenate([t.reshape(self.n, -1) for t in (xq, xk, a["v"])], 1)
        return {"out": out, "table": embed.embed_vjp(ROWS, ids, g_qkv @ W.T, 0.5), "W": h.T @ g_qkv, "gamma_q": g_gq,
                "gamma_k": g_gk, "slope": a["slope"], "pos": a["pos_q"] + a["pos_k"] + p1 + p2}


def test_path_against_the_oracles():
    p = Path()
    got = p.step()
    torch.cuda.synchronize()
    for n, want in p.oracle().items():
        assert_close(n, got[n].cpu().numpy(), want)


def test_forces_do_not_depend_on_the_frame():
    """A common shift of all positions changes no output beyond fp32 rounding
    of the positions: the position gradients of each structure sum to zero."""
    p = Path(1)
    f = p.step()["pos"].double()
    for a, b in zip(p.offsets, p.offsets[1:]):
        assert f[a:b].sum(0).abs().max() <= 1e-4 * f.abs().max() if b > a else True


def test_path_in_a_graph():
    """The library's calls of one step captured (the linear maps stay outside,
    their results are this test's inputs), replayed on new positions."""
    p = Path(2)
    p.step()
    torch.cuda.synchronize()
    fc = p.fc
    rope = (p.dr, p.q, p.k, p.gq, p.gk, p.pos, p.freq)
    attn = (p.da, p.seg, p.qn, p.kn, p.v, p.slope, p.pos, None)

    def calls():
        fc.fc_embed_fwd(p.de, p.table, p.ids, p.h)
        fc.fc_qk_norm_rope_fwd(*rope, p.qn, p.kn)
        fc.fc_attention_fwd(*attn, p.out, p.lse, p.ws[2])
        fc.fc_attention_vjp(*attn, p.out, p.lse, p.g, p.gqn, p.gkn, p.gv, p.g_slope, p.gp1, None, p.ws[3])
        fc.fc_qk_norm_rope_vjp(*rope, p.gqn, p.gkn, p.gq_raw, p.gk_raw, p.g_gq, p.g_gk, p.gp2, p.ws[1])
        fc.fc_embed_vjp(p.de, p.ids, p.h, p.g_table, p.ws[0])
        return [p.out, p.lse, p.gq_raw, p.gk_raw, p.gv, p.g_slope, p.gp1, p.gp2, p.g_gq, p.g_gk, p.g_table]

    outputs = calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(3):
        p.pos.mul_(1.05)
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in outputs]
        eager = calls()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, eager))


def test_embedding_feeds_a_message_block():
    """h0 of a message block from species: the energy is the one that the
    gathered rows give."""
    from cartesian_tensor_product_amd import flashcart as fc, inputs
    N, Cb, l = 60, 32, 1
    spec = inputs.edge_conv_inputs(1, N, 12, 8.0, Cb, 1, 2, 4)
    cd = fc.conv_desc(N, len(spec["sender"]), Cb, 0, l, l, 5.0)
    ld = fc.ladder_desc(N, Cb, l, l, 0, 2, fc.FC_LADDER_PATH_REDUCED)
    graph = fc.DeviceGraph(spec["rowptr"], spec["sender"], N)
    gen = torch.Generator().manual_seed(0)
    w = (0.1 * torch.randn(fc.fc_message_block_weight_floats(cd, ld), generator=gen)).cuda()
    pos, table = torch.from_numpy(spec["pos"]).cuda(), torch.randn(4, Cb, generator=gen).cuda()
    ids = torch.randint(0, 4, (N,), generator=gen).int().cuda()
    h0 = torch.empty(N, Cb, device="cuda")
    fc.fc_embed_fwd(fc.embed_desc(N, 4, Cb, 1.0), table, ids, h0)
    ws = fc.workspace(fc.fc_message_block_workspace_bytes(cd, ld))
    energies = []
    for h in (h0, table[ids.long()]):
        e = torch.empty(1, dtype=torch.float64, device="cuda")
        fc.fc_message_block_energy_forces(cd, graph, pos, None, h.view(N, 1, Cb).contiguous(), ld, w, 0.3, 1e-5, e, None,
                                          None, ws)
        torch.cuda.synchronize()
        energies.append(e.item())
    assert energies[0] == energies[1] and np.isfinite(energies[0]) and energies[0] != 0
