"""Thin Python binding of libflashcart.so (ctypes).

Every function has the name of the C entry point it wraps and only marshals
arguments: torch tensors become device pointers, the stream defaults to
torch's current stream, and a non-OK status raises ``FlashCartError``.  All
computation happens in the library's HIP kernels; there is no fallback.
"""

from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libflashcart.so")

FC_OK, FC_ERR_INVALID_ARGUMENT, FC_ERR_UNSUPPORTED, FC_ERR_WORKSPACE, FC_ERR_HIP = range(5)
FC_LADDER_FULL, FC_LADDER_PATH_REDUCED = 0, 1
FC_CONV_ALL_PARITIES = 1   # descriptor flag: every triangle-allowed path (odd J too)
FC_CONV_SUM_PATHS = 2      # descriptor flag: outputs of the paths of each rank summed
FC_CONV_MLP_MATERIALIZE = 4  # descriptor flag: radial-network calls store w [E][P][C] instead of fusing it
FC_CONV_MLP_FUSE = 8         # descriptor flag: radial-network calls form w in the convolution's lanes
FC_F32, FC_BF16 = 0, 1     # element types of the embedding, query/key norm and attention calls
FC_ROPE_INTERLEAVED = 1    # descriptor flag: rotated pairs are neighbours (2t, 2t + 1)
FC_ATTN_CAUSAL = 1         # descriptor flag: a query sees the prefix and the keys up to its own place


class FlashCartError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_status_name(status)}: {msg}")
        self.status = status


class ConvDesc(ctypes.Structure):
    _fields_ = [("n_nodes", ctypes.c_int32), ("n_edges", ctypes.c_int32), ("channels", ctypes.c_int32),
                ("l_in", ctypes.c_int32), ("l_edge", ctypes.c_int32), ("l_out", ctypes.c_int32),
                ("n_basis", ctypes.c_int32), ("r_cut", ctypes.c_float), ("flags", ctypes.c_uint32)]


class Graph(ctypes.Structure):
    _fields_ = [("rowptr", ctypes.c_void_p), ("sender", ctypes.c_void_p), ("receiver", ctypes.c_void_p),
                ("t_rowptr", ctypes.c_void_p), ("t_edge", ctypes.c_void_p)]


class LadderDesc(ctypes.Structure):
    _fields_ = [("n_nodes", ctypes.c_int32), ("channels", ctypes.c_int32), ("l_a", ctypes.c_int32),
                ("l_prod", ctypes.c_int32), ("l_out", ctypes.c_int32), ("order", ctypes.c_int32),
                ("variant", ctypes.c_int32)]


class NormDesc(ctypes.Structure):
    _fields_ = [("n_nodes", ctypes.c_int32), ("channels", ctypes.c_int32), ("l_max", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class EmbedDesc(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int32), ("n_rows", ctypes.c_int32), ("channels", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class QkRopeDesc(ctypes.Structure):
    _fields_ = [("n_nodes", ctypes.c_int32), ("heads_q", ctypes.c_int32), ("heads_k", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("n_freq", ctypes.c_int32), ("q_stride", ctypes.c_int32),
                ("k_stride", ctypes.c_int32), ("dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("flags", ctypes.c_uint32)]


class AttnDesc(ctypes.Structure):
    _fields_ = [("n_query", ctypes.c_int32), ("n_key", ctypes.c_int32), ("n_segments", ctypes.c_int32),
                ("heads_q", ctypes.c_int32), ("heads_k", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("q_stride", ctypes.c_int32), ("k_stride", ctypes.c_int32), ("v_stride", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("cap", ctypes.c_float),
                ("flags", ctypes.c_uint32)]


class SegmentPtrs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("prefix", ctypes.c_void_p)]


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int32
_SZ = ctypes.c_size_t
_PD = ctypes.POINTER(ConvDesc)
_PL = ctypes.POINTER(LadderDesc)
_PG = ctypes.POINTER(Graph)
_PN = ctypes.POINTER(NormDesc)
_PE = ctypes.POINTER(EmbedDesc)
_PQ = ctypes.POINTER(QkRopeDesc)
_PA = ctypes.POINTER(AttnDesc)
_PS = ctypes.POINTER(SegmentPtrs)
_PI = ctypes.POINTER(ctypes.c_int32)
_PSZ = ctypes.POINTER(ctypes.c_size_t)

_SIGS = {
    "fc_status_string": (ctypes.c_char_p, [_I]),
    "fc_last_error_message": (ctypes.c_char_p, []),
    "fc_abi_version": (_I, []),
    "fc_conv_layout": (_I, [_PD, _PI, _PI, _PI]),
    "fc_conv_path": (_I, [_PD, _I, _PI, _PI, _PI]),
    "fc_graph_transpose_workspace_bytes": (_SZ, [_I]),
    "fc_graph_transpose": (_I, [_I, _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "fc_graph_validate": (_I, [_I, _I, _PI, _PI]),
    "fc_edge_conv_workspace_bytes": (_SZ, [_PD, _I]),
    "fc_edge_conv_fwd": (_I, [_PD, _PG, _P, _P, _P, _P, _P, _P]),
    "fc_edge_conv_vjp": (_I, [_PD, _PG, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "fc_edge_conv_vjp_noalloc": (_I, [_PD, _PG, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "fc_edge_conv_vjp_vjp": (_I, [_PD, _PG, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "fc_edge_conv_fwd_w": (_I, [_PD, _PG, _P, _P, _P, _P, _P, _P]),
    "fc_edge_conv_vjp_w": (_I, [_PD, _PG, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "fc_edge_conv_vjp_vjp_w": (_I, [_PD, _PG, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "fc_ladder_layout": (_I, [_PL, _PSZ, _PSZ]),
    "fc_ladder_workspace_bytes": (_SZ, [_PL, _I]),
    "fc_ladder_weight_block": (_I, [_PL, _I, _PSZ, _PI, _PI, _PI]),
    "fc_node_ladder_fwd": (_I, [_PL, _P, _P, _P, _P, _P, _SZ, _P]),
    "fc_node_ladder_vjp": (_I, [_PL, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "fc_node_ladder_vjp_vjp": (_I, [_PL, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "fc_radial_mlp_weight_floats": (_SZ, [_PD]),
    "fc_edge_conv_mlp_workspace_bytes": (_SZ, [_PD, _I]),
    "fc_radial_mlp": (_I, [_PD, _PG, _P, _P, _P, _P, _P, _SZ, _P]),
    "fc_edge_conv_mlp_fwd": (_I, [_PD, _PG, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "fc_edge_conv_mlp_vjp": (_I, [_PD, _PG, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "fc_rms_norm_fwd": (_I, [_PN, _P, _P, _P, _P, _P]),
    "fc_rms_norm_workspace_bytes": (_SZ, [_PN]),
    "fc_rms_norm_vjp": (_I, [_PN, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "fc_embed_fwd": (_I, [_PE, _P, _P, _P, _P]),
    "fc_embed_workspace_bytes": (_SZ, [_PE]),
    "fc_embed_vjp": (_I, [_PE, _P, _P, _P, _P, _SZ, _P]),
    "fc_qk_norm_rope_fwd": (_I, [_PQ, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "fc_qk_norm_rope_workspace_bytes": (_SZ, [_PQ]),
    "fc_qk_norm_rope_vjp": (_I, [_PQ, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "fc_segments_validate": (_I, [_I, _I, _PI]),
    "fc_attention_workspace_bytes": (_SZ, [_PA, _I]),
    "fc_attention_fwd": (_I, [_PA, _PS, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "fc_attention_vjp": (_I, [_PA, _PS, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "fc_message_block_weight_floats": (_SZ, [_PD, _PL]),
    "fc_message_block_workspace_bytes": (_SZ, [_PD, _PL]),
    "fc_message_block_energy_forces": (_I, [_PD, _PG, _P, _P, _P, _PL, _P, ctypes.c_float, ctypes.c_float, _P, _P,
                                            _P, _P, _SZ, _P]),
    "fc_block_workspace_bytes": (_SZ, [_PD, _PL]),
    "fc_block_energy_forces": (_I, [_PD, _PG, _P, _P, _P, _P, _PL, _P, ctypes.c_float, _P, _P, _P, _P, _SZ, _P]),
}


def lib() -> ctypes.CDLL:
    """Loads libflashcart.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(python -m cartesian_tensor_product_amd.build)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _status_name(s: int) -> str:
    try:
        return lib().fc_status_string(s).decode()
    except Exception:  # pragma: no cover - only when the library is absent
        return str(s)


def _check(status: int) -> None:
    if status != FC_OK:
        raise FlashCartError(status, lib().fc_last_error_message().decode())


def _ptr(t, dtype=None):
    if t is None:
        return None
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("tensor must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"expected dtype {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _f32(t):
    import torch
    return _ptr(t, torch.float32)


def _i32(t):
    import torch
    return _ptr(t, torch.int32)


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(getattr(stream, "cuda_stream", stream))


def conv_desc(n_nodes, n_edges, channels, l_in, l_edge, l_out, r_cut, n_basis=8, flags=0) -> ConvDesc:
    return ConvDesc(n_nodes, n_edges, channels, l_in, l_edge, l_out, n_basis, r_cut, flags)


def norm_desc(n_nodes, channels, l_max, eps) -> NormDesc:
    return NormDesc(n_nodes, channels, l_max, eps)


def ladder_desc(n_nodes, channels, l_a, l_prod, l_out, order, variant) -> LadderDesc:
    return LadderDesc(n_nodes, channels, l_a, l_prod, l_out, order, variant)


# ------------------------------------------------------------------ layout --

def fc_abi_version() -> int:
    return lib().fc_abi_version()


def fc_conv_layout(d: ConvDesc):
    p, i, o = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(lib().fc_conv_layout(ctypes.byref(d), ctypes.byref(p), ctypes.byref(i), ctypes.byref(o)))
    return p.value, i.value, o.value


def fc_conv_path(d: ConvDesc, i: int):
    a, b, c = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(lib().fc_conv_path(ctypes.byref(d), i, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)))
    return a.value, b.value, c.value


def fc_graph_validate(n_nodes: int, n_edges: int, rowptr, sender) -> None:
    """Host arrays (numpy int32)."""
    import numpy as np
    rp = np.ascontiguousarray(rowptr, dtype=np.int32)
    sd = np.ascontiguousarray(sender, dtype=np.int32)
    _check(lib().fc_graph_validate(n_nodes, n_edges, rp.ctypes.data_as(_PI), sd.ctypes.data_as(_PI)))


def fc_edge_conv_workspace_bytes(d: ConvDesc, op: int) -> int:
    return lib().fc_edge_conv_workspace_bytes(ctypes.byref(d), op)


def fc_ladder_layout(d: LadderDesc):
    w, s = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().fc_ladder_layout(ctypes.byref(d), ctypes.byref(w), ctypes.byref(s)))
    return w.value, s.value


def fc_ladder_workspace_bytes(d: LadderDesc, op: int) -> int:
    return lib().fc_ladder_workspace_bytes(ctypes.byref(d), op)


def fc_ladder_weight_block(d: LadderDesc, i: int):
    """(offset, rows, cols, kind) of block i of the flat weight buffer."""
    off, r, c, k = ctypes.c_size_t(), ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(lib().fc_ladder_weight_block(ctypes.byref(d), i, ctypes.byref(off), ctypes.byref(r), ctypes.byref(c),
                                        ctypes.byref(k)))
    return off.value, r.value, c.value, k.value


def ladder_weight_blocks(d: LadderDesc):
    out, i = [], 0
    while True:
        try:
            out.append(fc_ladder_weight_block(d, i))
        except FlashCartError:
            return out
        i += 1


# ------------------------------------------------------------------- graph --

def fc_graph_transpose(n_nodes, n_edges, rowptr, sender, receiver, t_rowptr, t_edge, workspace, stream=None):
    _check(lib().fc_graph_transpose(n_nodes, n_edges, _i32(rowptr), _i32(sender), _i32(receiver),
                                    _i32(t_rowptr), _i32(t_edge), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream)))


class DeviceGraph:
    """Receiver-sorted CSR plus its sender-sorted transpose, on the GPU.

    Holds the int32 device tensors and the ``Graph`` struct passed to the
    convolution calls.  The transpose is built by ``fc_graph_transpose``.
    """

    def __init__(self, rowptr, sender, n_nodes: int, device="cuda", stream=None):
        import numpy as np
        import torch
        # the device calls do not check graph contents: validate the host
        # copy (an out-of-range sender would make the transpose write out of
        # bounds)
        h_rowptr = np.ascontiguousarray(torch.as_tensor(rowptr).cpu().numpy(), dtype=np.int32)
        h_sender = np.ascontiguousarray(torch.as_tensor(sender).cpu().numpy(), dtype=np.int32)
        if h_rowptr.shape != (n_nodes + 1,):
            raise FlashCartError(FC_ERR_INVALID_ARGUMENT,
                                 f"rowptr has {h_rowptr.size} entries, expected n_nodes + 1 = {n_nodes + 1}")
        fc_graph_validate(n_nodes, int(h_sender.size), h_rowptr, h_sender)
        self.n_nodes = n_nodes
        self.rowptr = torch.as_tensor(rowptr, dtype=torch.int32, device=device).contiguous()
        self.sender = torch.as_tensor(sender, dtype=torch.int32, device=device).contiguous()
        self.n_edges = int(self.sender.numel())
        E = max(self.n_edges, 1)
        self.receiver = torch.empty(E, dtype=torch.int32, device=device)
        self.t_rowptr = torch.empty(n_nodes + 1, dtype=torch.int32, device=device)
        self.t_edge = torch.empty(E, dtype=torch.int32, device=device)
        nbytes = lib().fc_graph_transpose_workspace_bytes(n_nodes)
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
        sender_t = self.sender if self.n_edges else torch.zeros(1, dtype=torch.int32, device=device)
        fc_graph_transpose(n_nodes, self.n_edges, self.rowptr, sender_t, self.receiver, self.t_rowptr,
                           self.t_edge, ws, stream)
        self._ws = ws
        self.struct = Graph(self.rowptr.data_ptr(), sender_t.data_ptr(), self.receiver.data_ptr(),
                            self.t_rowptr.data_ptr(), self.t_edge.data_ptr())
        self._sender_t = sender_t


# ---------------------------------------------------------- edge convolution --

def fc_edge_conv_fwd(d: ConvDesc, graph: DeviceGraph, pos, shift, x, radial_w, z, stream=None):
    _check(lib().fc_edge_conv_fwd(ctypes.byref(d), ctypes.byref(graph.struct), _f32(pos), _f32(shift), _f32(x),
                                  _f32(radial_w), _f32(z), _stream(stream)))


def fc_edge_conv_vjp(d: ConvDesc, graph: DeviceGraph, pos, shift, x, radial_w, g_z, x_grad, pos_grad,
                     radial_w_grad, workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fc_edge_conv_vjp(ctypes.byref(d), ctypes.byref(graph.struct), _f32(pos), _f32(shift), _f32(x),
                                  _f32(radial_w), _f32(g_z), _f32(x_grad), _f32(pos_grad), _f32(radial_w_grad),
                                  _ptr(workspace), nbytes, _stream(stream)))


def fc_edge_conv_vjp_noalloc(d: ConvDesc, graph: DeviceGraph, pos, shift, x, radial_w, g_z, x_grad, pos_grad,
                             radial_w_grad, stream=None):
    """fc_edge_conv_vjp with the library's own per-GPU scratch (no workspace)."""
    _check(lib().fc_edge_conv_vjp_noalloc(ctypes.byref(d), ctypes.byref(graph.struct), _f32(pos), _f32(shift),
                                          _f32(x), _f32(radial_w), _f32(g_z), _f32(x_grad), _f32(pos_grad),
                                          _f32(radial_w_grad), _stream(stream)))


def fc_edge_conv_fwd_w(d: ConvDesc, graph: DeviceGraph, pos, shift, x, w, z, stream=None):
    _check(lib().fc_edge_conv_fwd_w(ctypes.byref(d), ctypes.byref(graph.struct), _f32(pos), _f32(shift), _f32(x),
                                    _f32(w), _f32(z), _stream(stream)))


def fc_edge_conv_vjp_w(d: ConvDesc, graph: DeviceGraph, pos, shift, x, w, g_z, x_grad, pos_grad, w_grad,
                       workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fc_edge_conv_vjp_w(ctypes.byref(d), ctypes.byref(graph.struct), _f32(pos), _f32(shift), _f32(x),
                                    _f32(w), _f32(g_z), _f32(x_grad), _f32(pos_grad), _f32(w_grad), _ptr(workspace),
                                    nbytes, _stream(stream)))


def fc_edge_conv_vjp_vjp(d: ConvDesc, graph: DeviceGraph, pos, shift, x, radial_w, g_z, v_x, v_pos, v_radial_w,
                         g_hat, x_hat, pos_hat, radial_w_hat, workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fc_edge_conv_vjp_vjp(ctypes.byref(d), ctypes.byref(graph.struct), _f32(pos), _f32(shift),
                                      _f32(x), _f32(radial_w), _f32(g_z), _f32(v_x), _f32(v_pos),
                                      _f32(v_radial_w), _f32(g_hat), _f32(x_hat), _f32(pos_hat),
                                      _f32(radial_w_hat), _ptr(workspace), nbytes, _stream(stream)))


def fc_edge_conv_vjp_vjp_w(d: ConvDesc, graph: DeviceGraph, pos, shift, x, w, g_z, v_x, v_pos, v_w,
                           g_hat, x_hat, pos_hat, w_hat, workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fc_edge_conv_vjp_vjp_w(ctypes.byref(d), ctypes.byref(graph.struct), _f32(pos), _f32(shift),
                                        _f32(x), _f32(w), _f32(g_z), _f32(v_x), _f32(v_pos), _f32(v_w),
                                        _f32(g_hat), _f32(x_hat), _f32(pos_hat), _f32(w_hat), _ptr(workspace),
                                        nbytes, _stream(stream)))


# ------------------------------------------------------------------ ladder --

def fc_node_ladder_fwd(d: LadderDesc, A, weights, z, saved, workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fc_node_ladder_fwd(ctypes.byref(d), _f32(A), _f32(weights), _f32(z), _f32(saved),
                                    _ptr(workspace), nbytes, _stream(stream)))


def fc_node_ladder_vjp(d: LadderDesc, A, weights, saved, g_z, A_grad, weights_grad, workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fc_node_ladder_vjp(ctypes.byref(d), _f32(A), _f32(weights), _f32(saved), _f32(g_z),
                                    _f32(A_grad), _f32(weights_grad), _ptr(workspace), nbytes, _stream(stream)))


# ------------------------------------------------------------------ radial --

def fc_radial_mlp_weight_floats(d: ConvDesc) -> int:
    return lib().fc_radial_mlp_weight_floats(ctypes.byref(d))


def fc_edge_conv_mlp_workspace_bytes(d: ConvDesc, op: int) -> int:
    return lib().fc_edge_conv_mlp_workspace_bytes(ctypes.byref(d), op)


def fc_radial_mlp(d: ConvDesc, graph: DeviceGraph, pos, shift, mlp_w, w, workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fc_radial_mlp(ctypes.byref(d), ctypes.byref(graph.struct), _f32(pos), _f32(shift), _f32(mlp_w),
                               _f32(w), _ptr(workspace), nbytes, _stream(stream)))


def fc_edge_conv_mlp_fwd(d: ConvDesc, graph: DeviceGraph, pos, shift, x, mlp_w, z, workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fc_edge_conv_mlp_fwd(ctypes.byref(d), ctypes.byref(graph.struct), _f32(pos), _f32(shift), _f32(x),
                                      _f32(mlp_w), _f32(z), _ptr(workspace), nbytes, _stream(stream)))


def fc_edge_conv_mlp_vjp(d: ConvDesc, graph: DeviceGraph, pos, shift, x, mlp_w, g_z, x_grad, pos_grad, mlp_w_grad,
                         workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fc_edge_conv_mlp_vjp(ctypes.byref(d), ctypes.byref(graph.struct), _f32(pos), _f32(shift), _f32(x),
                                      _f32(mlp_w), _f32(g_z), _f32(x_grad), _f32(pos_grad), _f32(mlp_w_grad),
                                      _ptr(workspace), nbytes, _stream(stream)))


# -------------------------------------------------------------------- norm --

def fc_rms_norm_fwd(d: NormDesc, x, gamma, y, inv_scale, stream=None):
    _check(lib().fc_rms_norm_fwd(ctypes.byref(d), _f32(x), _f32(gamma), _f32(y), _f32(inv_scale),
                                 _stream(stream)))


def fc_rms_norm_workspace_bytes(d: NormDesc) -> int:
    return lib().fc_rms_norm_workspace_bytes(ctypes.byref(d))


def fc_rms_norm_vjp(d: NormDesc, x, gamma, inv_scale, g_y, x_grad, gamma_grad, workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fc_rms_norm_vjp(ctypes.byref(d), _f32(x), _f32(gamma), _f32(inv_scale), _f32(g_y), _f32(x_grad),
                                 _f32(gamma_grad), _ptr(workspace), nbytes, _stream(stream)))


def fc_node_ladder_vjp_vjp(d: LadderDesc, A, weights, saved, g_z, v_A, v_weights, g_hat, A_hat, weights_hat,
                           workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fc_node_ladder_vjp_vjp(ctypes.byref(d), _f32(A), _f32(weights), _f32(saved), _f32(g_z), _f32(v_A),
                                        _f32(v_weights), _f32(g_hat), _f32(A_hat), _f32(weights_hat),
                                        _ptr(workspace), nbytes, _stream(stream)))


# ------------------------------------------------------------------- block --

def fc_block_workspace_bytes(conv: ConvDesc, lad: LadderDesc) -> int:
    return lib().fc_block_workspace_bytes(ctypes.byref(conv), ctypes.byref(lad))


def fc_block_energy_forces(conv: ConvDesc, graph: DeviceGraph, pos, shift, x, radial_w, lad: LadderDesc, ladder_w,
                           conv_scale: float, energy, e_atom, forces, workspace, stream=None):
    import torch
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fc_block_energy_forces(ctypes.byref(conv), ctypes.byref(graph.struct), _f32(pos), _f32(shift),
                                        _f32(x), _f32(radial_w), ctypes.byref(lad), _f32(ladder_w),
                                        ctypes.c_float(conv_scale), _ptr(energy, torch.float64), _f32(e_atom),
                                        _f32(forces), _ptr(workspace), nbytes, _stream(stream)))


def workspace(nbytes: int, device="cuda"):
    import torch
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def fc_message_block_weight_floats(conv: ConvDesc, lad: LadderDesc) -> int:
    return lib().fc_message_block_weight_floats(ctypes.byref(conv), ctypes.byref(lad))


def fc_message_block_workspace_bytes(conv: ConvDesc, lad: LadderDesc) -> int:
    return lib().fc_message_block_workspace_bytes(ctypes.byref(conv), ctypes.byref(lad))


def fc_message_block_energy_forces(conv: ConvDesc, graph: DeviceGraph, pos, shift, h0, lad: LadderDesc, weights,
                                   conv_scale: float, eps: float, energy, e_atom, forces, workspace, stream=None):
    import torch
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fc_message_block_energy_forces(ctypes.byref(conv), ctypes.byref(graph.struct), _f32(pos),
                                                _f32(shift), _f32(h0), ctypes.byref(lad), _f32(weights),
                                                ctypes.c_float(conv_scale), ctypes.c_float(eps),
                                                _ptr(energy, torch.float64), _f32(e_atom), _f32(forces),
                                                _ptr(workspace), nbytes, _stream(stream)))


# ------------------------------------------- embedding, queries/keys, attention --
#
# These calls check dtype, shape and device of every tensor against the
# descriptor, and run on the tensors' device (its current stream by default).

def embed_desc(n_tokens, n_rows, channels, scale=1.0, dtype=FC_F32) -> EmbedDesc:
    return EmbedDesc(n_tokens, n_rows, channels, dtype, scale)


def qk_rope_desc(n_nodes, heads_q, heads_k, head_dim, n_freq, eps, dtype=FC_F32, flags=0) -> QkRopeDesc:
    """Row strides of q and k are taken from the tensors of each call."""
    return QkRopeDesc(n_nodes, heads_q, heads_k, head_dim, n_freq, 0, 0, dtype, eps, flags)


def attn_desc(n_query, n_key, n_segments, heads_q, heads_k, head_dim, scale, cap=0.0, dtype=FC_F32,
              flags=0) -> AttnDesc:
    """Row strides of q, k and v are taken from the tensors of each call."""
    return AttnDesc(n_query, n_key, n_segments, heads_q, heads_k, head_dim, 0, 0, 0, dtype, scale, cap, flags)


def _bad(msg: str):
    return FlashCartError(FC_ERR_INVALID_ARGUMENT, msg)


def _place(t, name: str) -> int:
    """Index of the GPU that a call runs on: that of its leading tensor (-1
    without one; the library then refuses the call)."""
    import torch
    if t is None:
        return -1
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: tensor must live on the GPU")
    return dev


def _refuse(t, dtype, shape, dev, name):
    _place(t, name)
    if t.get_device() != dev:
        raise ValueError(f"{name}: tensor on cuda:{t.get_device()}, the others on cuda:{dev}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: expected dtype {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise _bad(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: tensor must be contiguous")


def _arr(t, dtype, shape, dev, name):
    """Pointer of a contiguous tensor of this dtype and shape on GPU dev (None
    passes).  Few attribute reads: small calls are bound by the host."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.get_device() == dev and (shape is None or t.shape == shape) and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, dtype, shape, dev, name)


def _rows(t, dtype, shape, dev, name):
    """(pointer, row stride in elements; 0 for packed rows) of [rows][heads][dim]."""
    if t is None or not hasattr(t, "is_contiguous") or t.is_contiguous():
        return _arr(t, dtype, shape, dev, name), 0
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _refuse(t, dtype, shape, dev, name)
    if (shape[2] > 1 and t.stride(2) != 1) or (shape[1] > 1 and t.stride(1) != shape[2]):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    stride = t.stride(0)
    if stride < shape[1] * shape[2]:
        raise _bad(f"{name}: rows overlap (stride {stride})")
    return t.data_ptr(), stride


def _elem(dtype: int):
    import torch
    return torch.bfloat16 if dtype == FC_BF16 else torch.float32


def _run(f, dev: int, stream, *args):
    """f(*args, stream) with GPU dev current; the stream defaults to its
    current one."""
    import torch
    if dev < 0:
        return _check(f(*args, None))
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)   # current_stream(dev).cuda_stream without the object
    else:
        stream = getattr(stream, "cuda_stream", stream)
    if dev == torch.cuda.current_device():
        _check(f(*args, stream))
    else:
        with torch.cuda.device(dev):
            _check(f(*args, stream))


def _ws(workspace, dev):
    import torch
    return (None, 0) if workspace is None else (_arr(workspace, torch.uint8, None, dev, "workspace"), workspace.numel())


def fc_embed_fwd(d: EmbedDesc, table, ids, out, stream=None):
    import torch
    dev, elem, n, c = _place(table, "table"), _elem(d.dtype), d.n_tokens, d.channels
    _run(lib().fc_embed_fwd, dev, stream, d, _arr(table, elem, (d.n_rows, c), dev, "table"),
         _arr(ids, torch.int32, (n,), dev, "ids"), _arr(out, elem, (n, c), dev, "out"))


def fc_embed_workspace_bytes(d: EmbedDesc) -> int:
    return lib().fc_embed_workspace_bytes(d)


def fc_embed_vjp(d: EmbedDesc, ids, g_out, table_grad, workspace, stream=None):
    import torch
    dev, n, c = _place(table_grad, "table_grad"), d.n_tokens, d.channels
    _run(lib().fc_embed_vjp, dev, stream, d, _arr(ids, torch.int32, (n,), dev, "ids"),
         _arr(g_out, _elem(d.dtype), (n, c), dev, "g_out"),
         _arr(table_grad, torch.float32, (d.n_rows, c), dev, "table_grad"), *_ws(workspace, dev))


def _qk_inputs(d: QkRopeDesc, elem, dev, q, k, gamma_q, gamma_k, pos, freq):
    import torch
    n, dim, f32 = d.n_nodes, d.head_dim, torch.float32
    pq, sq = _rows(q, elem, (n, d.heads_q, dim), dev, "q")
    pk, sk = _rows(k, elem, (n, d.heads_k, dim), dev, "k")
    if sq or sk:
        d = QkRopeDesc.from_buffer_copy(d)
        d.q_stride, d.k_stride = sq, sk
    return (d, pq, pk, _arr(gamma_q, f32, (dim,), dev, "gamma_q"), _arr(gamma_k, f32, (dim,), dev, "gamma_k"),
            _arr(pos, f32, (n, 3), dev, "pos"), _arr(freq, f32, (d.n_freq, 3), dev, "freq"))


def fc_qk_norm_rope_fwd(d: QkRopeDesc, q, k, gamma_q, gamma_k, pos, freq, q_out, k_out, stream=None):
    dev, elem = _place(q, "q"), _elem(d.dtype)
    n, dim = d.n_nodes, d.head_dim
    _run(lib().fc_qk_norm_rope_fwd, dev, stream, *_qk_inputs(d, elem, dev, q, k, gamma_q, gamma_k, pos, freq),
         _arr(q_out, elem, (n, d.heads_q, dim), dev, "q_out"), _arr(k_out, elem, (n, d.heads_k, dim), dev, "k_out"))


def fc_qk_norm_rope_workspace_bytes(d: QkRopeDesc) -> int:
    return lib().fc_qk_norm_rope_workspace_bytes(d)


def fc_qk_norm_rope_vjp(d: QkRopeDesc, q, k, gamma_q, gamma_k, pos, freq, g_q, g_k, q_grad, k_grad, gamma_q_grad,
                        gamma_k_grad, pos_grad, workspace, stream=None):
    import torch
    dev, elem, f32 = _place(q, "q"), _elem(d.dtype), torch.float32
    n, dim = d.n_nodes, d.head_dim
    sq, sk = (n, d.heads_q, dim), (n, d.heads_k, dim)
    _run(lib().fc_qk_norm_rope_vjp, dev, stream, *_qk_inputs(d, elem, dev, q, k, gamma_q, gamma_k, pos, freq),
         _arr(g_q, elem, sq, dev, "g_q"), _arr(g_k, elem, sk, dev, "g_k"), _arr(q_grad, elem, sq, dev, "q_grad"),
         _arr(k_grad, elem, sk, dev, "k_grad"), _arr(gamma_q_grad, f32, (dim,), dev, "gamma_q_grad"),
         _arr(gamma_k_grad, f32, (dim,), dev, "gamma_k_grad"), _arr(pos_grad, f32, (n, 3), dev, "pos_grad"),
         *_ws(workspace, dev))


def fc_segments_validate(n_segments: int, n_rows: int, offsets) -> None:
    """Host array (numpy int32)."""
    import numpy as np
    o = np.ascontiguousarray(offsets, dtype=np.int32)
    if o.shape != (n_segments + 1,):
        raise _bad(f"{o.size} offsets for {n_segments} segments")
    _check(lib().fc_segments_validate(n_segments, n_rows, o.ctypes.data_as(_PI)))


class Segments:
    """Segment offsets (structures of a batch, documents) on the GPU.

    ``offsets_q`` [S+1] gives the first query row of each segment,
    ``offsets_k`` the first key row (None: the same rows), ``prefix`` [S] the
    number of leading keys that every query sees under ``FC_ATTN_CAUSAL``.
    The host copies are checked before they are uploaded.
    """

    def __init__(self, offsets_q, offsets_k=None, prefix=None, device="cuda"):
        import numpy as np
        import torch
        host = lambda a: np.asarray(torch.as_tensor(a).cpu().numpy(), dtype=np.int64)
        q = host(offsets_q)
        k = q if offsets_k is None else host(offsets_k)
        if q.ndim != 1 or q.size < 2 or k.shape != q.shape:
            raise _bad("offsets need one entry per segment and the end, the same number for queries and keys")
        self.n_segments = int(q.size) - 1
        self.n_query, self.n_key = int(q[-1]), int(k[-1])
        for o in (q, k):
            if o.min() < 0 or o.max() > 2 ** 31 - 1:
                raise _bad("offsets out of range")
            fc_segments_validate(self.n_segments, int(o[-1]), o)
        up = lambda a: torch.as_tensor(a.astype(np.int32), device=device)
        self.q, self.k = up(q), None if offsets_k is None else up(k)
        self.prefix = None
        if prefix is not None:
            p = host(prefix)
            if p.shape != (self.n_segments,) or (p < 0).any() or (p > np.diff(k)).any():
                raise _bad("prefix needs one length per segment, within its keys")
            self.prefix = up(p)
        ptr = lambda t: None if t is None else t.data_ptr()
        self.struct = SegmentPtrs(ptr(self.q), ptr(self.k), ptr(self.prefix))


def _attn_inputs(d: AttnDesc, elem, dev, seg, q, k, v, slope, pos_q, pos_k):
    import torch
    f32 = torch.float32
    nq, nk, hq, hk, dim = d.n_query, d.n_key, d.heads_q, d.heads_k, d.head_dim
    if seg is not None:
        if seg.n_segments != d.n_segments:
            raise _bad(f"{seg.n_segments} segments, the descriptor has {d.n_segments}")
        if seg.n_query > nq or seg.n_key > nk:
            raise _bad(f"segments end at rows {seg.n_query}, {seg.n_key}, beyond the descriptor's {nq}, {nk}")
        if seg.q.get_device() != dev:
            raise ValueError(f"segments: offsets on another device than cuda:{dev}")
        seg = seg.struct
    pq, sq = _rows(q, elem, (nq, hq, dim), dev, "q")
    pk, sk = _rows(k, elem, (nk, hk, dim), dev, "k")
    pv, sv = _rows(v, elem, (nk, hk, dim), dev, "v")
    if sq or sk or sv:
        d = AttnDesc.from_buffer_copy(d)
        d.q_stride, d.k_stride, d.v_stride = sq, sk, sv
    return (d, seg, pq, pk, pv, _arr(slope, f32, (hq,), dev, "slope"), _arr(pos_q, f32, (nq, 3), dev, "pos_q"),
            _arr(pos_k, f32, (nk, 3), dev, "pos_k"))


def fc_attention_workspace_bytes(d: AttnDesc, op: int) -> int:
    return lib().fc_attention_workspace_bytes(d, op)


def fc_attention_fwd(d: AttnDesc, seg, q, k, v, slope, pos_q, pos_k, out, lse, workspace, stream=None):
    """``seg`` is a ``Segments`` or None (one segment of all rows)."""
    import torch
    dev, elem = _place(q, "q"), _elem(d.dtype)
    _run(lib().fc_attention_fwd, dev, stream, *_attn_inputs(d, elem, dev, seg, q, k, v, slope, pos_q, pos_k),
         _arr(out, elem, (d.n_query, d.heads_q, d.head_dim), dev, "out"),
         _arr(lse, torch.float32, (d.n_query, d.heads_q), dev, "lse"), *_ws(workspace, dev))


def fc_attention_vjp(d: AttnDesc, seg, q, k, v, slope, pos_q, pos_k, out, lse, g_out, q_grad, k_grad, v_grad,
                     slope_grad, pos_q_grad, pos_k_grad, workspace, stream=None):
    import torch
    dev, elem, f32 = _place(q, "q"), _elem(d.dtype), torch.float32
    qs, ks = (d.n_query, d.heads_q, d.head_dim), (d.n_key, d.heads_k, d.head_dim)
    _run(lib().fc_attention_vjp, dev, stream, *_attn_inputs(d, elem, dev, seg, q, k, v, slope, pos_q, pos_k),
         _arr(out, elem, qs, dev, "out"), _arr(lse, f32, (d.n_query, d.heads_q), dev, "lse"),
         _arr(g_out, elem, qs, dev, "g_out"), _arr(q_grad, elem, qs, dev, "q_grad"), _arr(k_grad, elem, ks, dev, "k_grad"),
         _arr(v_grad, elem, ks, dev, "v_grad"), _arr(slope_grad, f32, (d.heads_q,), dev, "slope_grad"),
         _arr(pos_q_grad, f32, (d.n_query, 3), dev, "pos_q_grad"), _arr(pos_k_grad, f32, (d.n_key, 3), dev, "pos_k_grad"),
         *_ws(workspace, dev))
