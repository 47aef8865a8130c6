"""Thin Python binding of the spec-tree C ABI (include/spec_tree.h).

Argument marshalling only: every step of the hot path runs in the CUDA
kernels of libspec_tree.so.  PyTorch supplies device memory and streams.
Importing this module without the built library raises, so a missing native
build can never fall back to anything else.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
import struct
import threading
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libspec_tree.so")

BF16, F32, F16 = 0, 1, 2   # F16: key-value cache, queries and attention outputs only
BUILDER_TOPR, BUILDER_SMART = 0, 1
PROBE_FIRST, PROBE_LAST = 0, 1
ROOT, DET, PROBE, FILL = 0, 1, 2, 3
OK, E_PARAM, E_LAYOUT, E_CUDA = 0, -1, -3, -4
S_NONFINITE_DRAFT, S_NONFINITE_TARGET, S_RESIDUAL_EMPTY = 1, 2, 4
S_OVERFLOW, S_TIMEOUT, S_ROWS, S_LAYERS = 8, 16, 32, 64
S_PAGES, S_NODES = 128, 256
MAX_SUPPORT = 1024
SUPPORT_DENSE = 0x40000000   # |S| = V for any vocabulary
DENSE_MAX_K = 64
STATIC_MAX_TREES = 64
DEFAULT_SUPPORT = 128

EXPORTS = ("spec_tree_rows_needed", "spec_tree_check_params", "spec_tree_select_expand", "spec_tree_rank",
           "spec_tree_build", "spec_tree_verify", "spec_tree_layer_state_bytes", "spec_tree_layer_rows",
           "spec_tree_layer", "spec_tree_finish", "spec_tree_layer_static", "spec_tree_smart_fit",
           "spec_tree_wait_selftest", "spec_tree_verify_dense", "spec_tree_kv_append", "spec_tree_attend",
           "spec_tree_attend_workspace_bytes", "spec_tree_kv_commit", "spec_tree_strerror")


class SpecTreeError(RuntimeError):
    pass


class c_params(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int32), ("m", ctypes.c_int32), ("W", ctypes.c_int32), ("depth", ctypes.c_int32),
                ("R", ctypes.c_int32), ("support", ctypes.c_int32), ("temperature", ctypes.c_float),
                ("builder", ctypes.c_int32), ("lam", ctypes.c_float), ("beta", ctypes.c_float),
                ("gamma", ctypes.c_float), ("delta", ctypes.c_float), ("rho", ctypes.c_float),
                ("eta", ctypes.c_float), ("alpha", ctypes.c_float), ("verify_order", ctypes.c_int32)]


class c_tree(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "node_token", "node_parent", "node_depth", "node_kind", "node_slot", "node_exp_row", "node_score",
        "n_nodes", "sup_id", "sup_q", "sup_qT", "sup_z", "sup_zT", "probe_pos")] + [
        ("n_rows", ctypes.c_int32), ("max_nodes", ctypes.c_int32), ("sup_stride", ctypes.c_int32),
        ("sched", ctypes.c_void_p)]


class c_kv(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "page_table", "seq_len")] + [
        (n, ctypes.c_int64) for n in ("layer_stride", "page_stride", "token_stride", "head_stride")] + [
        (n, ctypes.c_int32) for n in ("dtype", "n_layers", "n_pages", "page_size", "n_kv_heads", "head_dim",
                                      "max_pages", "table_stride")]


class c_heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p)] + [(n, ctypes.c_int64) for n in ("tree_stride", "node_stride",
                                                                            "head_stride")]


class c_nodes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("parent", "depth", "n_nodes")] + [
        (n, ctypes.c_int32) for n in ("stride", "begin", "count")]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -c \"import __graft_entry__ as g; g.build()\"`")
    lib = ctypes.CDLL(LIB_PATH)
    P, T, vp, i32, i64 = ctypes.POINTER(c_params), ctypes.POINTER(c_tree), ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    lib.spec_tree_rows_needed.argtypes = [P]
    lib.spec_tree_check_params.argtypes = [P, i32]
    lib.spec_tree_select_expand.argtypes = [P, i32, i32, i32, vp, i64, vp, T, vp, vp]
    lib.spec_tree_rank.argtypes = [P, i32, i32, T, vp, vp]
    lib.spec_tree_build.argtypes = [P, i32, i32, i32, vp, i64, vp, T, vp, vp]
    lib.spec_tree_verify.argtypes = [P, i32, i32, i32, vp, i64, T, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.spec_tree_verify_dense.argtypes = [P, i32, i32, i32, vp, i64, vp, i64, T, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.spec_tree_layer_state_bytes.argtypes = []
    lib.spec_tree_layer_state_bytes.restype = ctypes.c_size_t
    lib.spec_tree_layer_rows.argtypes = [P, i32]
    lib.spec_tree_layer.argtypes = [P, i32, i32, i32, i32, vp, i64, vp, T, vp, vp, vp, vp, vp]
    lib.spec_tree_finish.argtypes = [P, i32, i32, T, vp, vp, vp]
    lib.spec_tree_layer_static.argtypes = [P, i32, i32, i32, i32, vp, i64, vp, T, vp, vp, vp, vp]
    dp = ctypes.POINTER(ctypes.c_double)
    lib.spec_tree_smart_fit.argtypes = [i32, dp, dp, dp, ctypes.c_double, dp, P, dp, dp]
    lib.spec_tree_wait_selftest.argtypes = [ctypes.c_uint32, vp, vp, vp]
    # structures by address: these calls are made once per layer of a model, and their arguments are packed
    lib.spec_tree_kv_append.argtypes = [i32, vp, i32, vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, vp, vp,
                                        ctypes.c_float, vp, vp]
    lib.spec_tree_attend.argtypes = [i32, vp, i32, vp, i32, vp, vp, ctypes.c_float, vp, ctypes.c_size_t, vp, vp]
    lib.spec_tree_attend_workspace_bytes.argtypes = [i32] * 5
    lib.spec_tree_attend_workspace_bytes.restype = ctypes.c_size_t
    lib.spec_tree_kv_commit.argtypes = [i32, vp, vp, vp, i32, vp, vp, vp]
    lib.spec_tree_strerror.argtypes = [i32]
    lib.spec_tree_strerror.restype = ctypes.c_char_p
    for name in EXPORTS:
        if name not in ("spec_tree_strerror", "spec_tree_layer_state_bytes", "spec_tree_attend_workspace_bytes"):
            getattr(lib, name).restype = ctypes.c_int
    return lib


_lib = _load()


@dataclasses.dataclass
class Params:
    K: int
    m: int
    W: int
    depth: int
    R: int
    temperature: float = 1.0
    support: int = 128
    builder: int = BUILDER_TOPR
    lam: float = 0.02
    beta: float = 0.0
    gamma: float = 0.5
    delta: float = 0.01
    rho: float = 1.3
    eta: float = 0.0
    alpha: float = 1.0
    verify_order: int = PROBE_FIRST

    def c(self) -> c_params:
        return c_params(self.K, self.m, self.W, self.depth, self.R, self.support, self.temperature, self.builder,
                        self.lam, self.beta, self.gamma, self.delta, self.rho, self.eta, self.alpha,
                        self.verify_order)

    @staticmethod
    def from_workload(wl) -> "Params":
        return Params(K=wl.K, m=wl.m, W=wl.W, depth=wl.depth, R=wl.R, temperature=wl.temperature,
                      support=wl.support, builder=BUILDER_SMART if wl.builder == "smart" else BUILDER_TOPR,
                      lam=wl.lam, beta=wl.beta, gamma=wl.gamma, delta=wl.delta, rho=wl.rho, eta=wl.eta,
                      alpha=wl.alpha, verify_order=PROBE_LAST if wl.verify_order == "rrsw" else PROBE_FIRST)


def _cp(params) -> c_params:
    """Params or an already marshalled c_params (callers in a loop can marshal once)."""
    return params if isinstance(params, c_params) else params.c()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:  # the handle of the current stream, without the Stream object around it (2.9 us a call)
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()))
    return ctypes.c_void_p(stream.cuda_stream)


def _check(rc: int):
    if rc:
        raise SpecTreeError(f"spec_tree error {rc}: {_lib.spec_tree_strerror(rc).decode()}")


class TreeBuffers:
    """Device buffers of a batch of trees (the spec_tree_t of the C ABI)."""

    def __init__(self, params: Params, B: int, n_rows: Optional[int] = None, device="cuda", V: Optional[int] = None):
        i32, f32 = torch.int32, torch.float32
        self.B = B
        self.n_rows = n_rows if n_rows is not None else rows_needed(params)
        self.max_nodes = params.R + 1
        # support arrays hold |S| = min(support, V) ranks per row, at least 128 wide; a dense
        # support of a vocabulary above MAX_SUPPORT tokens keeps K ranks and the probe
        if params.support == SUPPORT_DENSE:
            self.sup_stride = MAX_SUPPORT if V is None or V <= MAX_SUPPORT else max(DEFAULT_SUPPORT, params.K + 1)
        else:
            self.sup_stride = max(DEFAULT_SUPPORT, params.support or DEFAULT_SUPPORT)
        mk = lambda shape, dt: torch.empty(shape, dtype=dt, device=device)  # noqa: E731
        n = (B, self.max_nodes)
        self.node_token, self.node_parent, self.node_depth = mk(n, i32), mk(n, i32), mk(n, i32)
        self.node_kind, self.node_slot, self.node_exp_row = mk(n, i32), mk(n, i32), mk(n, i32)
        self.node_score = mk(n, f32)
        self.n_nodes = mk((B,), i32)
        r = (B, self.n_rows)
        self.sup_id = mk(r + (self.sup_stride,), i32)
        self.sup_q = mk(r + (self.sup_stride,), f32)
        self.sup_qT = mk(r + (self.sup_stride,), f32)
        self.sup_z, self.sup_zT, self.probe_pos = mk(r, f32), mk(r, f32), mk(r, i32)
        # row counter of the support selection (zero; every call leaves it zero) and the latest
        # call's cut key, a threshold hint for the next call's first rows
        self.sched = torch.zeros((3,), dtype=i32, device=device)

    def c(self) -> c_tree:
        if getattr(self, "_c", None) is None:
            t = c_tree()
            for name, _ in c_tree._fields_[:14]:
                setattr(t, name, getattr(self, name).data_ptr())
            t.n_rows, t.max_nodes, t.sup_stride = self.n_rows, self.max_nodes, self.sup_stride
            t.sched = self.sched.data_ptr()
            self._c = t
        return self._c


def _dtype_code(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return BF16
    if x.dtype == torch.float32:
        return F32
    raise SpecTreeError(f"unsupported logits dtype {x.dtype}")


def _row_stride(x: torch.Tensor, rows_per_tree: int) -> int:
    if x.dim() != 3 or x.stride(2) != 1 or x.stride(1) != x.stride(0) // rows_per_tree or \
            x.stride(0) != rows_per_tree * x.stride(1) or x.shape[1] != rows_per_tree:
        raise SpecTreeError("logits must be [B][rows][row_stride] with contiguous rows")
    return x.stride(1)


def rows_needed(params: Params) -> int:
    return _lib.spec_tree_rows_needed(ctypes.byref(_cp(params)))


def spec_tree_check_params(params: Params, V: int) -> int:
    return _lib.spec_tree_check_params(ctypes.byref(_cp(params)), V)


def spec_tree_select_expand(params: Params, V: int, draft: torch.Tensor, u_probe: torch.Tensor, tree: TreeBuffers,
                            status: torch.Tensor, stream=None):
    _check(_lib.spec_tree_select_expand(ctypes.byref(_cp(params)), tree.B, V, _dtype_code(draft), _ptr(draft),
                                        _row_stride(draft, tree.n_rows), _ptr(u_probe), ctypes.byref(tree.c()),
                                        _ptr(status), _stream(stream)))


def spec_tree_rank(params: Params, V: int, tree: TreeBuffers, status: torch.Tensor, stream=None):
    _check(_lib.spec_tree_rank(ctypes.byref(_cp(params)), tree.B, V, ctypes.byref(tree.c()), _ptr(status),
                               _stream(stream)))


def spec_tree_build(params: Params, V: int, draft: torch.Tensor, u_probe: torch.Tensor, tree: TreeBuffers,
                    status: torch.Tensor, stream=None):
    _check(_lib.spec_tree_build(ctypes.byref(_cp(params)), tree.B, V, _dtype_code(draft), _ptr(draft),
                                _row_stride(draft, tree.n_rows), _ptr(u_probe), ctypes.byref(tree.c()),
                                _ptr(status), _stream(stream)))


def spec_tree_verify(params: Params, V: int, target: torch.Tensor, tree: TreeBuffers, u_verify: torch.Tensor,
                     u_bonus: torch.Tensor, accept_len: torch.Tensor, out_tok: torch.Tensor,
                     out_node: torch.Tensor, margins: Optional[torch.Tensor], status: torch.Tensor, stream=None):
    _check(_lib.spec_tree_verify(ctypes.byref(_cp(params)), tree.B, V, _dtype_code(target), _ptr(target),
                                 _row_stride(target, tree.max_nodes), ctypes.byref(tree.c()), _ptr(u_verify),
                                 _ptr(u_bonus), _ptr(accept_len), _ptr(out_tok), _ptr(out_node), _ptr(margins),
                                 _ptr(status), _stream(stream)))


def spec_tree_verify_dense(params: Params, V: int, target: torch.Tensor, draft: torch.Tensor, tree: TreeBuffers,
                           u_verify: torch.Tensor, u_bonus: torch.Tensor, accept_len: torch.Tensor,
                           out_tok: torch.Tensor, out_node: torch.Tensor, margins: Optional[torch.Tensor],
                           status: torch.Tensor, stream=None):
    """spec_tree_verify for trees built on the dense support of a vocabulary above MAX_SUPPORT tokens: it
    reads the node's draft row (the tensor the tree was built from) for the tail law."""
    _check(_lib.spec_tree_verify_dense(ctypes.byref(_cp(params)), tree.B, V, _dtype_code(target), _ptr(target),
                                       _row_stride(target, tree.max_nodes), _ptr(draft),
                                       _row_stride(draft, tree.n_rows), ctypes.byref(tree.c()), _ptr(u_verify),
                                       _ptr(u_bonus), _ptr(accept_len), _ptr(out_tok), _ptr(out_node),
                                       _ptr(margins), _ptr(status), _stream(stream)))


def is_dense(params: Params, V: int) -> bool:
    """The dense support of a vocabulary too large for the support arrays (verify with spec_tree_verify_dense)."""
    return params.support == SUPPORT_DENSE and V > MAX_SUPPORT


def spec_tree_layer_state_bytes() -> int:
    return _lib.spec_tree_layer_state_bytes()


def spec_tree_layer_rows(params: Params, layer: int) -> int:
    return _lib.spec_tree_layer_rows(ctypes.byref(_cp(params)), layer)


class LayerState:
    """Caller-owned per-tree state of the layer-by-layer builder, and the frontier it names."""

    def __init__(self, params: Params, B: int, device="cuda"):
        self.B = B
        self.state = torch.empty((B, spec_tree_layer_state_bytes()), dtype=torch.uint8, device=device)
        self.frontier_token = torch.empty((B, params.W), dtype=torch.int32, device=device)
        self.frontier_parent = torch.empty((B, params.W), dtype=torch.int32, device=device)


def spec_tree_layer(params: Params, V: int, layer: int, layer_draft: torch.Tensor, u_probe: torch.Tensor,
                    tree: TreeBuffers, state: LayerState, status: torch.Tensor, stream=None):
    rows = spec_tree_layer_rows(params, layer)
    _check(_lib.spec_tree_layer(ctypes.byref(_cp(params)), tree.B, V, layer, _dtype_code(layer_draft),
                                _ptr(layer_draft), _row_stride(layer_draft, rows), _ptr(u_probe),
                                ctypes.byref(tree.c()), _ptr(state.state), _ptr(state.frontier_token),
                                _ptr(state.frontier_parent), _ptr(status), _stream(stream)))


def spec_tree_finish(params: Params, V: int, tree: TreeBuffers, state: LayerState, status: torch.Tensor,
                     stream=None):
    _check(_lib.spec_tree_finish(ctypes.byref(_cp(params)), tree.B, V, ctypes.byref(tree.c()), _ptr(state.state),
                                 _ptr(status), _stream(stream)))


def spec_tree_layer_static(params: Params, V: int, layer: int, layer_draft: torch.Tensor, u_probe: torch.Tensor,
                           tree: TreeBuffers, frontier_token: Optional[torch.Tensor],
                           frontier_parent: Optional[torch.Tensor], status: torch.Tensor, stream=None):
    """spec_tree_layer with the builder's state inside the library (no state buffer to allocate); the
    last layer's call also writes the node arrays.  At most STATIC_MAX_TREES trees; builds must not
    overlap on the GPU."""
    rows = spec_tree_layer_rows(params, layer)
    _check(_lib.spec_tree_layer_static(ctypes.byref(_cp(params)), tree.B, V, layer, _dtype_code(layer_draft),
                                       _ptr(layer_draft), _row_stride(layer_draft, rows), _ptr(u_probe),
                                       ctypes.byref(tree.c()), _ptr(frontier_token), _ptr(frontier_parent),
                                       _ptr(status), _stream(stream)))


@dataclasses.dataclass
class CostFit:
    lam: float
    gamma: float
    delta: float
    rho: float
    rms_draft: float
    rms_verify: float

    def apply(self, params: Params) -> Params:
        """params with the fitted SMART cost coefficients (beta = eta = 0)."""
        return dataclasses.replace(params, lam=self.lam, beta=0.0, gamma=self.gamma, delta=self.delta,
                                   rho=self.rho, eta=0.0)


def spec_tree_smart_fit(sizes, t_draft, t_verify, t_base: float, weights=None) -> CostFit:
    """Fit the SMART cost model to profiled step times (host only, no GPU)."""
    def arr(x):
        a = (ctypes.c_double * len(x))(*[float(v) for v in x])
        return ctypes.cast(a, ctypes.POINTER(ctypes.c_double)), a

    n = len(sizes)
    if len(t_draft) != n or len(t_verify) != n or (weights is not None and len(weights) != n):
        raise SpecTreeError("sizes, timings and weights must have the same length")
    (pn, _an), (pd, _ad), (pv, _av) = arr(sizes), arr(t_draft), arr(t_verify)
    pw, _aw = arr(weights) if weights is not None else (None, None)
    coef = (ctypes.c_double * 4)()
    rms = (ctypes.c_double * 2)()
    _check(_lib.spec_tree_smart_fit(n, pn, pd, pv, float(t_base), pw, None,
                                    ctypes.cast(coef, ctypes.POINTER(ctypes.c_double)),
                                    ctypes.cast(rms, ctypes.POINTER(ctypes.c_double))))
    return CostFit(lam=coef[0], gamma=coef[1], delta=coef[2], rho=coef[3], rms_draft=rms[0], rms_verify=rms[1])


class VerifyOutputs:
    def __init__(self, params: Params, B: int, device="cuda"):
        self.accept_len = torch.empty((B,), dtype=torch.int32, device=device)
        self.out_tok = torch.empty((B, params.depth + 1), dtype=torch.int32, device=device)
        self.out_node = torch.empty((B, params.depth + 1), dtype=torch.int32, device=device)
        self.margins = torch.zeros((2,), dtype=torch.int32, device=device)


def spec_tree_wait_selftest(polls: int, status: torch.Tensor, result: torch.Tensor, stream=None):
    """Let one CTA-scope and one cluster-scope bounded wait run out (`polls` polls each) on a barrier
    nothing arrives on; result (4 x int32 on the device) = gave up / polls made, per CTA."""
    _check(_lib.spec_tree_wait_selftest(polls, _ptr(status), _ptr(result), _stream(stream)))


# --------------------------------------------------- the model's side of a step ---

_HALF = {torch.bfloat16: BF16, torch.float16: F16}
_I32, _U32 = torch.int32, torch.uint32
_current_device = getattr(torch._C, "_cuda_getDevice", None)  # looked up once: calls are made once per layer
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _ready(device: int, status: torch.Tensor, stream) -> int:
    """The stream's handle, if `status` and the cache (of that device) are where a kernel can reach them."""
    kind = status.dtype
    if (kind is not _I32 and kind is not _U32) or status.numel() < 1 or status.get_device() != device:
        raise SpecTreeError("status must be an int32 tensor on the cache's device")
    if device < 0 or _current_device() != device:
        raise SpecTreeError("the cache must be on the current GPU")
    if stream is None:
        return _raw_stream(device)
    if stream.device.index != device:
        raise SpecTreeError("the stream must be of the cache's device")
    return stream.cuda_stream


class KVCache:
    """A paged key-value cache (the spec_tree_kv_t of the C ABI).

    k, v: [layers][pages][page_size][kv heads][head_dim], bf16 or f16, any strides with contiguous
    head_dim (a [layers][pages][heads][page_size][head_dim] pool is passed transposed);
    page_table: int32 [B][max_pages], a row for each sequence (contiguous, none over another);
    seq_len: int32 [B], committed tokens.  All are on one device, as is whatever a call takes with them; a call
    wants it to be the current GPU.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, seq_len: torch.Tensor):
        if k.dim() != 5 or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride():
            raise SpecTreeError("k and v must be alike, [layers][pages][page_size][kv heads][head_dim]")
        if k.dtype not in _HALF:
            raise SpecTreeError(f"unsupported cache dtype {k.dtype}")
        if k.stride(4) != 1:
            raise SpecTreeError("head_dim must be contiguous")
        if page_table.dim() != 2 or page_table.dtype != torch.int32 or page_table.stride(1) != 1:
            raise SpecTreeError("page_table must be int32 [B][max_pages] with contiguous rows")
        rows, width = page_table.shape
        table_stride = page_table.stride(0) if rows > 1 else width  # the stride of a single row means nothing
        if not width <= table_stride < 1 << 31:
            raise SpecTreeError("rows of page_table overlap (an expanded table is to be copied) or lie too far apart")
        device = k.get_device()
        if v.get_device() != device or page_table.get_device() != device:
            raise SpecTreeError("k, v and page_table must be on one device")
        self.k, self.v, self.page_table, self.B, self.device = k, v, page_table, rows, device
        layers, pages, size, heads, dim = k.shape
        c = c_kv(k.data_ptr(), v.data_ptr(), page_table.data_ptr(), None, k.stride(0), k.stride(1), k.stride(2),
                 k.stride(3), _HALF[k.dtype], layers, pages, size, heads, dim, width, table_stride)
        self._c, self.at = c, ctypes.addressof(c)
        self.shape = (self.B, heads, dim, k.dtype, device)
        self.set_lengths(seq_len)

    def set_lengths(self, seq_len: torch.Tensor):
        """Committed tokens from now on, e.g. the new_len of spec_tree_kv_commit."""
        self._c.seq_len = _int_rows("seq_len", seq_len, (self.B,), self.device)
        self.seq_len = seq_len

    def c(self) -> c_kv:
        return self._c


@dataclasses.dataclass
class NodeArrays:
    """Node arrays of a batch of trees where no TreeBuffers holds them (a drafter's frontiers, a chain with
    n_nodes alone): int32 node_parent, node_depth [B][nodes] and n_nodes [B], each or None."""
    node_parent: Optional[torch.Tensor] = None
    node_depth: Optional[torch.Tensor] = None
    n_nodes: Optional[torch.Tensor] = None


def _int_rows(name: str, t: torch.Tensor, shape, device: int) -> int:
    """Address of a contiguous int32 tensor of that shape and device."""
    if t.dtype is not _I32 or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        raise SpecTreeError(f"{name} must be contiguous int32 {list(shape)} on the cache's device")
    return t.data_ptr()


class _Packed(threading.local):
    """One call's spec_tree_nodes_t and up to four spec_tree_heads_t, packed into memory of the thread's own
    (the entry points read them before they return)."""
    NODES, HEADS2, HEADS4 = struct.Struct("@3P3i"), struct.Struct("@P3qP3q"), struct.Struct("@P3qP3qP3qP3q")

    def __init__(self):
        self.buf = ctypes.create_string_buffer(64 + self.HEADS4.size)
        self.nodes_at = ctypes.addressof(self.buf)
        self.heads_at = tuple(self.nodes_at + 64 + i * (self.HEADS4.size // 4) for i in range(4))

    def nodes(self, tree, B: int, begin: int, count: int, device: int) -> int:
        """A TreeBuffers, a NodeArrays or None (a chain of which every node exists)."""
        if tree is None:
            self.NODES.pack_into(self.buf, 0, 0, 0, 0, 0, begin, count)
            return self.nodes_at
        parent, depth, n = tree.node_parent, tree.node_depth, tree.n_nodes
        at, stride = 0, 0
        if parent is not None:
            stride = parent.shape[-1]
            at = _int_rows("node_parent", parent, (B, stride), device)
        elif depth is not None:
            raise SpecTreeError("node_depth without node_parent")
        self.NODES.pack_into(self.buf, 0, at,
                             0 if depth is None else _int_rows("node_depth", depth, (B, stride), device),
                             0 if n is None else _int_rows("n_nodes", n, (B,), device), stride, begin, count)
        return self.nodes_at

    def heads2(self, a, b):
        """Two tensors' _vectors; their addresses in the buffer."""
        self.HEADS2.pack_into(self.buf, 64, *a, *b)
        return self.heads_at

    def heads4(self, a, b, c, d):
        self.HEADS4.pack_into(self.buf, 64, *a, *b, *c, *d)
        return self.heads_at


def _vectors(name: str, x: torch.Tensor, dtype, shape, device: int):
    """Address and strides of x; refuses what is not [B][nodes][heads][head_dim] of that shape, dtype and device
    with contiguous head_dim."""
    if x.dtype is dtype and x.shape == shape and x.get_device() == device:
        tree, node, head, element = x.stride()
        if element == 1:
            return x.data_ptr(), tree, node, head
    raise SpecTreeError(f"{name} must be {list(shape)} of {dtype}, head_dim contiguous, on the cache's device")


_packed = _Packed()


def _count(q: torch.Tensor):
    if q.dim() != 4:
        raise SpecTreeError("q must be [B][nodes][heads][head_dim]")
    return q.shape[1], q.shape[2]


def rope_table(rows: int, rot_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """Cosines and sines of positions 0 .. rows - 1, [rows][rot_dim] float32: row t holds cos(t f_j), then
    sin(t f_j), f_j = base^(-2 j / rot_dim); the angles are taken in float64."""
    half = rot_dim // 2
    f = base ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
    a = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def spec_tree_kv_append(cache: KVCache, layer: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                        q_out: torch.Tensor, rope: Optional[torch.Tensor], status: torch.Tensor, tree=None,
                        node_begin: int = 0, q_weight: Optional[torch.Tensor] = None,
                        k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False,
                        stream=None):
    """Nodes node_begin .. node_begin + q.shape[1] - 1 of every tree: head norms (with weights), rotation
    (with a rope table [rows][rot_dim]), keys and values into the cache, queries to q_out."""
    (n, hq), (B, hkv, dim, dtype, device), pack = _count(q), cache.shape, _packed
    rows = rot = rope_at = 0
    if rope is not None:
        if rope.dim() != 2 or rope.dtype is not torch.float32 or not rope.is_contiguous() or rope.get_device() != device:
            raise SpecTreeError("rope must be contiguous float32 [rows][rot_dim] on the cache's device")
        rows, rot = rope.shape
        rope_at = rope.data_ptr()
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and (w.dtype is not dtype or w.shape != (dim,) or not w.is_contiguous()
                              or w.get_device() != device):
            raise SpecTreeError(f"{name} must be [head_dim] of the cache's dtype on its device")
    qs, ks = (B, n, hq, dim), (B, n, hkv, dim)
    q_at, k_at, v_at, out_at = pack.heads4(_vectors("q", q, dtype, qs, device), _vectors("k", k, dtype, ks, device),
                                           _vectors("v", v, dtype, ks, device), _vectors("q_out", q_out, dtype, qs, device))
    nodes_at = pack.nodes(tree, B, node_begin, n, device)
    stream = _ready(device, status, stream)
    _check(_lib.spec_tree_kv_append(B, cache.at, layer, nodes_at, hq, q_at, k_at, v_at, out_at, rope_at, rows, rot,
                                    interleaved, None if q_weight is None else q_weight.data_ptr(),
                                    None if k_weight is None else k_weight.data_ptr(), eps, status.data_ptr(), stream))


class AttendWorkspace:
    """Workspace of spec_tree_attend for calls of up to B trees and `count` nodes (one call at a time)."""

    def __init__(self, B: int, count: int, n_q_heads: int, n_kv_heads: int, head_dim: int, device="cuda"):
        with torch.cuda.device(device):
            n = _lib.spec_tree_attend_workspace_bytes(B, count, n_q_heads, n_kv_heads, head_dim)
        if n == 0:
            raise SpecTreeError("spec_tree_attend takes no such heads or nodes")
        self.data = torch.zeros(n, dtype=torch.uint8, device=device)
        self.at, self.bytes, self.device = self.data.data_ptr(), n, self.data.get_device()


def spec_tree_attend(cache: KVCache, layer: int, q: torch.Tensor, out: torch.Tensor, workspace: AttendWorkspace,
                     status: torch.Tensor, tree=None, node_begin: int = 0, scale: Optional[float] = None,
                     stream=None):
    """Nodes node_begin .. node_begin + q.shape[1] - 1 of every tree attend to the committed tokens, their
    ancestors and themselves; scale defaults to head_dim ** -0.5."""
    (n, hq), (B, _, dim, dtype, device), pack = _count(q), cache.shape, _packed
    qs = (B, n, hq, dim)
    q_at, out_at, _, _ = pack.heads2(_vectors("q", q, dtype, qs, device), _vectors("out", out, dtype, qs, device))
    nodes_at = pack.nodes(tree, B, node_begin, n, device)
    stream = _ready(device, status, stream)
    if workspace.device != device:
        raise SpecTreeError("the workspace must be on the cache's device")
    _check(_lib.spec_tree_attend(B, cache.at, layer, nodes_at, hq, q_at, out_at, dim ** -0.5 if scale is None else scale,
                                 workspace.at, workspace.bytes, status.data_ptr(), stream))


def spec_tree_kv_commit(cache: KVCache, accept_len: torch.Tensor, out_node: torch.Tensor, new_len: torch.Tensor,
                        status: torch.Tensor, stream=None):
    """Move the accepted path (spec_tree_verify's accept_len and out_node) behind the committed tokens in
    every layer; new_len [B] receives the new committed lengths (then cache.set_lengths(new_len))."""
    B, device = (cache.B,), cache.device
    if out_node.dim() != 2:
        raise SpecTreeError("out_node must be [B][depth + 1]")
    stride = out_node.shape[1]
    accept_at = _int_rows("accept_len", accept_len, B, device)
    node_at = _int_rows("out_node", out_node, (cache.B, stride), device)
    new_at = _int_rows("new_len", new_len, B, device)
    stream = _ready(device, status, stream)
    _check(_lib.spec_tree_kv_commit(cache.B, cache.at, accept_at, node_at, stride, new_at, status.data_ptr(), stream))
