"""GPU parity of the embedding lookup and its gradient against the oracle.

Tolerances: the lookup is one fp32 product, rounded once to the output type
(half a step); a gradient entry is an fp32 sum of n terms, off by at most
(n + 1) 2^-24 of the sum of their magnitudes in any order."""
import numpy as np
import pytest

from oracle import embed

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = ["f32", "bf16"]


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def case(dtype, N, R, C, seed, ids=None, scale=1.7, pad=0):
    """(desc, table, ids, g) on the GPU; ``pad`` elements in front of each
    array shift it off its natural alignment."""
    from cartesian_tensor_product_amd import flashcart as fc
    rng = np.random.default_rng(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    if ids is None:   # skewed, with padding on both sides of the table
        ids = np.minimum((R + 2) ** rng.random(N), R + 1).astype(np.int64) - 1
        ids[rng.random(N) < 0.05] = -5
    t = lambda *s: torch.cat([torch.zeros(pad), torch.from_numpy(rng.standard_normal(s)).float().flatten()]).to(dt)
    up = lambda a, *s: a.cuda()[pad:].view(*s)
    table, g = up(t(R, C), R, C), up(t(N, C), N, C)
    d = fc.embed_desc(N, R, C, scale, fc.FC_F32 if dtype == "f32" else fc.FC_BF16)
    return fc, d, table, torch.from_numpy(np.asarray(ids, np.int32)).cuda(), g


def run_fwd(fc, d, table, ids):
    out = torch.full((d.n_tokens, d.channels), float("nan"), dtype=table.dtype, device="cuda")
    fc.fc_embed_fwd(d, table, ids, out)
    return out


def run_vjp(fc, d, ids, g):
    grad = torch.full((d.n_rows, d.channels), float("nan"), device="cuda")
    fc.fc_embed_vjp(d, ids, g, grad, fc.workspace(fc.fc_embed_workspace_bytes(d)))
    return grad


def check(fc, d, table, ids, g):
    out, grad = run_fwd(fc, d, table, ids), run_vjp(fc, d, ids, g)
    torch.cuda.synchronize()
    f = lambda t: t.double().cpu().numpy()
    scale = float(np.float32(d.scale))
    want = embed.embed_fwd(f(table), ids.cpu().numpy(), scale)
    tol = (half_step(table.dtype) + 2 * U) * np.abs(want)
    assert (np.abs(f(out) - want) <= tol).all()
    host = ids.cpu().numpy()
    want = embed.embed_vjp(d.n_rows, host, f(g), scale)
    size = embed.embed_vjp(d.n_rows, host, np.abs(f(g)), scale)
    n = np.bincount(host[(host >= 0) & (host < d.n_rows)], minlength=d.n_rows)[:, None]
    err = np.abs(f(grad) - want)
    assert (err <= (n + 1) * U * size).all(), (err - (n + 1) * U * size).max()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,R,C", [(1, 1, 1), (1, 95, 128), (33, 7, 8), (257, 255, 5), (1000, 256, 128),
                                   (2049, 300, 100), (5000, 70000, 24), (4096, 3, 1024), (300, 5, 2056),
                                   (4095, 60000, 5), (4096, 255, 2), (4097, 256, 12), (9000, 300, 6),
                                   (5000, 128, 100), (5000, 129, 100), (3000, 64, 320), (2500, 2, 1), (5000, 255, 72)])
def test_sizes(dtype, N, R, C):
    check(*case(dtype, N, R, C, N + R + C))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ids", ["one", "sorted", "reversed", "padding", "last"])
@pytest.mark.parametrize("N,R", [(3001, 40), (3001, 300), (9001, 300)])
def test_orders_of_ids(dtype, N, R, ids):
    """One row for every token (a run over many chunks), sorted and reversed
    ids, nothing but padding, the last row alone."""
    i = {"one": np.full(N, 17), "sorted": np.arange(N) * R // N, "reversed": R - 1 - np.arange(N) * R // N,
         "padding": np.where(np.arange(N) % 2, -1, R), "last": np.full(N, R - 1)}[ids]
    check(*case(dtype, N, R, 36, 3, ids=i))


@pytest.mark.parametrize("R", [9, 300])
def test_long_runs_and_many_chunks(R):
    """More tokens than one pass of chunks: a row of tens of thousands."""
    rng = np.random.default_rng(9)
    ids = np.where(rng.random(70000) < 0.5, 2, rng.integers(0, R, 70000))
    check(*case("f32", 70000, R, 16, 4, ids=ids))


@pytest.mark.parametrize("dtype", TYPES)
def test_unaligned_arrays(dtype):
    check(*case(dtype, 130, 20, 64, 5, pad=1))


def test_no_tokens():
    fc, d, table, ids, g = case("f32", 0, 6, 12, 1, ids=np.zeros(0))
    assert run_fwd(fc, d, table, ids).numel() == 0
    assert (run_vjp(fc, d, ids, g) == 0).all()


def test_offsets_past_two_gib():
    """300 000 rows x 2048 channels (2.4 GB): the last rows in and out."""
    from cartesian_tensor_product_amd import flashcart as fc
    R, C = 300000, 2048
    table = torch.empty(R, C, device="cuda")
    table[-2:] = torch.arange(2 * C, device="cuda").view(2, C).float()
    ids = torch.tensor([R - 1, R - 2, R - 1], dtype=torch.int32, device="cuda")
    d = fc.embed_desc(3, R, C, 1.0)
    out = run_fwd(fc, d, table, ids)
    assert torch.equal(out, table[ids.long()])
    grad = run_vjp(fc, d, ids, out)
    assert torch.equal(grad[-1], 2 * table[-1]) and torch.equal(grad[-2], table[-2]) and not grad[:-2].any()


def test_bitwise_reproducible_and_captured():
    """Two calls agree bit for bit; a captured call replays on new ids."""
    fc, d, table, ids, g = case("bf16", 20000, 500, 64, 6)
    first = run_vjp(fc, d, ids, g)
    assert torch.equal(first, run_vjp(fc, d, ids, g))
    ws = fc.workspace(fc.fc_embed_workspace_bytes(d))
    out, grad = torch.empty_like(g), torch.empty(d.n_rows, d.channels, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fc.fc_embed_fwd(d, table, ids, out)
        fc.fc_embed_vjp(d, ids, g, grad, ws)
    for seed in range(3):
        ids.copy_(torch.randint(-1, 501, ids.shape, generator=torch.Generator().manual_seed(seed)).int())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, run_fwd(fc, d, table, ids))
        assert torch.equal(grad, run_vjp(fc, d, ids, g))
        torch.cuda.synchronize()
