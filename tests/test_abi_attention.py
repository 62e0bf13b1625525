"""Host-side checks of the embedding, query/key norm and attention calls (no
GPU needed): refusals of descriptors, arrays and segment offsets."""
import os

import pytest

from cartesian_tensor_product_amd import flashcart as fc

pytestmark = pytest.mark.skipif(not os.path.exists(fc.LIB_PATH), reason="libflashcart.so not built")


def raises(status, f, *args, **kw):
    with pytest.raises(fc.FlashCartError) as ei:
        f(*args, **kw)
    assert ei.value.status == status, ei.value


@pytest.mark.parametrize("bad,status", [
    (dict(n_tokens=-1), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(n_rows=0), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(channels=0), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(n_rows=2 ** 31 - 1), fc.FC_ERR_UNSUPPORTED),
    (dict(n_rows=2 ** 28 + 1), fc.FC_ERR_UNSUPPORTED),    # more threads than a launch may have
    (dict(n_tokens=2 ** 30 + 1), fc.FC_ERR_UNSUPPORTED),
    (dict(channels=2 ** 21 + 1), fc.FC_ERR_UNSUPPORTED),
    (dict(scale=float("nan")), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(dtype=2), fc.FC_ERR_UNSUPPORTED),
    (dict(), fc.FC_ERR_INVALID_ARGUMENT),                 # NULL arrays
])
def test_embed_refusals(bad, status):
    d = fc.embed_desc(**{**dict(n_tokens=4, n_rows=3, channels=8), **bad})
    assert (fc.fc_embed_workspace_bytes(d) == 0) == bool(bad)
    raises(status, fc.fc_embed_fwd, d, None, None, None, stream=0)
    raises(status, fc.fc_embed_vjp, d, None, None, None, None, stream=0)


@pytest.mark.parametrize("bad,status", [
    (dict(n_nodes=-1), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(heads_q=0), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(heads_k=-1), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(head_dim=7), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(head_dim=130), fc.FC_ERR_UNSUPPORTED),
    (dict(n_freq=9), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(n_freq=-1), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(eps=0.0), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(eps=float("inf")), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(flags=2), fc.FC_ERR_UNSUPPORTED),
    (dict(dtype=-1), fc.FC_ERR_UNSUPPORTED),
    (dict(heads_q=2000), fc.FC_ERR_UNSUPPORTED),
    (dict(n_nodes=2 ** 25 + 1), fc.FC_ERR_UNSUPPORTED),
    (dict(), fc.FC_ERR_INVALID_ARGUMENT),                 # NULL arrays
])
def test_qk_norm_rope_refusals(bad, status):
    d = fc.qk_rope_desc(**{**dict(n_nodes=4, heads_q=2, heads_k=1, head_dim=16, n_freq=8, eps=1e-5), **bad})
    assert (fc.fc_qk_norm_rope_workspace_bytes(d) == 0) == bool(bad)
    raises(status, fc.fc_qk_norm_rope_fwd, d, *[None] * 8, stream=0)
    raises(status, fc.fc_qk_norm_rope_vjp, d, *[None] * 14, stream=0)


@pytest.mark.parametrize("bad,status", [
    (dict(n_query=-1), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(n_key=-1), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(n_segments=0), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(heads_q=3), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(heads_k=0), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(heads_q=512), fc.FC_ERR_UNSUPPORTED),
    (dict(head_dim=0), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(head_dim=12), fc.FC_ERR_UNSUPPORTED),
    (dict(head_dim=136), fc.FC_ERR_UNSUPPORTED),
    (dict(scale=0.0), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(scale=float("inf")), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(cap=-1.0), fc.FC_ERR_INVALID_ARGUMENT),
    (dict(flags=4), fc.FC_ERR_UNSUPPORTED),
    (dict(dtype=3), fc.FC_ERR_UNSUPPORTED),
    (dict(n_query=2 ** 30, n_key=2 ** 30), fc.FC_ERR_UNSUPPORTED),
    (dict(n_query=2 ** 28, n_key=2 ** 29), fc.FC_ERR_UNSUPPORTED),
    (dict(), fc.FC_ERR_INVALID_ARGUMENT),                 # NULL arrays
])
def test_attention_refusals(bad, status):
    d = fc.attn_desc(**{**dict(n_query=4, n_key=4, n_segments=1, heads_q=4, heads_k=2, head_dim=16, scale=0.25), **bad})
    assert (fc.fc_attention_workspace_bytes(d, 1) == 0) == bool(bad)
    assert fc.fc_attention_workspace_bytes(d, 2) == 0
    raises(status, fc.fc_attention_fwd, d, None, *[None] * 9, stream=0)
    raises(status, fc.fc_attention_vjp, d, None, *[None] * 16, stream=0)


def test_attention_array_refusals():
    """Combinations of arrays, strides and alignments, on made-up addresses
    (every call fails before anything is launched)."""
    L = fc.lib()
    d = fc.attn_desc(4, 4, 1, 4, 2, 16, 0.25)
    ok = dict(seg=None, q=4096, k=8192, v=12288, slope=None, pos_q=None, pos_k=None, out=16384, lse=20480, ws=0)

    def fwd(d=d, **kw):
        a = {**ok, **kw}
        st = L.fc_attention_fwd(d, a["seg"], a["q"], a["k"], a["v"], a["slope"], a["pos_q"], a["pos_k"], a["out"],
                                a["lse"], None, a["ws"], None)
        return st, L.fc_last_error_message()

    bad = fc.FC_ERR_INVALID_ARGUMENT
    assert fwd(q=None)[0] == bad and fwd(out=None)[0] == bad and fwd(lse=None)[0] == bad
    assert fwd(q=4100)[0] == bad and fwd(v=8)[0] == bad and fwd(out=16388)[0] == bad and fwd(lse=2)[0] == bad
    assert fwd(slope=64)[0] == bad and fwd(pos_q=64)[0] == bad
    other = fc.attn_desc(4, 5, 1, 4, 2, 16, 0.25)
    st, msg = fwd(other, slope=64, pos_q=64)
    assert st == bad and b"pos_k may be NULL only" in msg
    st, msg = fwd(other, seg=fc.SegmentPtrs(64, None, None))
    assert st == bad and b"shared offsets" in msg
    assert fwd(seg=fc.SegmentPtrs(None, 64, None))[0] == bad
    st, msg = fwd(seg=fc.SegmentPtrs(64, 64, 64))
    assert st == bad and b"prefix" in msg
    st, msg = fwd(fc.attn_desc(4, 4, 2, 4, 2, 16, 0.25))
    assert st == bad and b"offsets" in msg
    for f, v in (("q_stride", 60), ("q_stride", 66), ("k_stride", 16), ("v_stride", 33)):
        e = fc.AttnDesc.from_buffer_copy(d)
        setattr(e, f, v)
        assert fwd(e)[0] == bad, (f, v)
    # few queries over many keys need a workspace
    long = fc.attn_desc(1, 5000, 1, 4, 2, 16, 0.25)
    assert fc.fc_attention_workspace_bytes(long, 0) > 0
    st, msg = fwd(long)
    assert st == fc.FC_ERR_WORKSPACE
    vjp = lambda *g: L.fc_attention_vjp(d, None, 4096, 8192, 12288, None, None, None, 16384, 20480, 24576, *g, None, 0, None)
    assert vjp(*[None] * 6) == bad                       # nothing wanted
    assert vjp(28672, None, None, 64, None, None) == bad  # slope gradient without slope
    assert vjp(28680, None, None, None, None, None) == bad
    assert vjp(28672, None, None, None, None, None) == fc.FC_ERR_WORKSPACE


def test_segments_checked_before_upload():
    good = fc.Segments([0, 3, 3, 7], prefix=[1, 0, 4], device="cpu")
    assert (good.n_segments, good.n_query, good.n_key) == (3, 7, 7)
    for kw in (dict(offsets_q=[1, 3]), dict(offsets_q=[0, 3, 2]), dict(offsets_q=[0]), dict(offsets_q=[0, -1]),
               dict(offsets_q=[0, 3], offsets_k=[0, 1, 2]), dict(offsets_q=[0, 3], prefix=[4]),
               dict(offsets_q=[0, 3], prefix=[-1]), dict(offsets_q=[0, 3], prefix=[1, 1]),
               dict(offsets_q=[0, 2 ** 31])):
        raises(fc.FC_ERR_INVALID_ARGUMENT, fc.Segments, device="cpu", **kw)
    raises(fc.FC_ERR_INVALID_ARGUMENT, fc.fc_segments_validate, 2, 6, [0, 3, 7])


def test_bindings_check_tensors():
    """Shapes, types and places are checked before any pointer is taken."""
    torch = pytest.importorskip("torch")
    d = fc.embed_desc(4, 3, 8)
    with pytest.raises(ValueError, match="must live on the GPU"):
        fc.fc_embed_fwd(d, torch.zeros(3, 8), None, None, stream=0)
    with pytest.raises(TypeError):
        fc.fc_embed_fwd(d, [1.0], None, None, stream=0)
