"""ctypes binding of libgdn.so (include/gdn.h), with the same names as the C entry points.

Argument marshalling only: tensors are passed as device pointers, the current torch stream as
the HIP stream, and every non-zero status becomes a ``GdnError``.  There is no fallback: if the
library is missing, loading fails loudly.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libgdn.so")

GDN_OK, GDN_ERR_ARG, GDN_ERR_SHAPE, GDN_ERR_DTYPE, GDN_ERR_RANGE, GDN_ERR_HIP = range(6)
GDN_F32, GDN_BF16, GDN_E4M3, GDN_I8 = range(4)
GDN_CHAIN, GDN_TREE = 0, 1
GDN_F_QK_NORM_SILU = 0x1
GDN_F_CHECK_INDICES = 0x2
GDN_F_DEFER_COMMIT = 0x4
GDN_ROPE_HALF, GDN_ROPE_INTERLEAVED = 0, 1
GDN_ROPE_PLAIN, GDN_ROPE_LINEAR, GDN_ROPE_NTK, GDN_ROPE_YARN = range(4)
GDN_KV_BF16, GDN_KV_E4M3, GDN_KV_I8 = range(3)
GDN_NORM_RMS, GDN_NORM_NONE = 0, 1
GDN_ACT_NONE, GDN_ACT_SILU, GDN_ACT_GELU, GDN_ACT_GELU_TANH, GDN_ACT_RELU, GDN_ACT_SIGMOID = range(6)

EXPORTS = ("gdn_verify", "gdn_verify_resume", "gdn_verify_tree", "gdn_rollback", "gdn_rollback_batch", "gdn_rollback_trim",
           "gdn_prefill", "gdn_prefill_noalloc", "gdn_prefill_workspace_bytes", "gdn_capture_bytes", "gdn_reset",
           "gdn_snapshot", "gdn_restore", "gdn_rollback_layers", "gdn_graph_create", "gdn_graph_launch",
           "gdn_graph_destroy", "gdn_linear", "gdn_rope_init", "gdn_rope", "gdn_kv_bytes", "gdn_kv_write",
           "gdn_kv_read", "gdn_kv_commit", "gdn_attn_verify", "gdn_attn_workspace_bytes", "gdn_norm", "gdn_linear_act",
           "gdn_linear_act_workspace_bytes", "gdn_logprob", "gdn_logprob_workspace_bytes", "gdn_last_error", "gdn_version")


class GdnError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[gdn status {code}] {msg}")
        self.code = code


class gdn_dims(ctypes.Structure):
    _fields_ = [("n_kh", ctypes.c_int32), ("n_vh", ctypes.c_int32), ("d_k", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("d_conv", ctypes.c_int32), ("n_pool", ctypes.c_int32),
                ("act_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("eps", ctypes.c_float)]


class gdn_capture(ctypes.Structure):
    _fields_ = [("dims", gdn_dims), ("ssm", ctypes.c_void_p), ("conv", ctypes.c_void_p),
                ("state", ctypes.c_void_p), ("conv_state", ctypes.c_void_p),
                ("t_cap", ctypes.c_int32), ("mode", ctypes.c_int32)]


class gdn_layer(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("state", "conv_state", "qkv", "z", "alpha", "beta", "A_log",
                                                "dt_bias", "conv_w", "norm_w", "cap_ssm", "cap_conv", "out")]


class gdn_out_seg(ctypes.Structure):
    _fields_ = [("n0", ctypes.c_int32), ("n1", ctypes.c_int32), ("ld", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("sigmoid", ctypes.c_int32), ("ptr", ctypes.c_void_p)]


class gdn_rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("ld", ctypes.c_int64), ("hd", ctypes.c_int64),
                ("n_heads", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class gdn_mat(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("ld", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class gdn_rope_params(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("orig_ctx", ctypes.c_int32), ("sections", ctypes.c_int32 * 4), ("theta", ctypes.c_double),
                ("factor", ctypes.c_double), ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("mscale", ctypes.c_double)]


class gdn_rope_table(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("n_axes", ctypes.c_int32),
                ("axis_end", ctypes.c_int32 * 4), ("mscale", ctypes.c_float), ("turns", ctypes.c_double * 128)]


class gdn_kv(ctypes.Structure):
    _fields_ = [("n_kv", ctypes.c_int32), ("d", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("format", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


class gdn_kv_batch(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("start", ctypes.c_void_p), ("n_new", ctypes.c_void_p),
                ("max_pages", ctypes.c_int32), ("n_batch", ctypes.c_int32), ("n_tok", ctypes.c_int32)]


GDN_GRAPH_VERIFY = 0x1
GDN_GRAPH_ROLLBACK = 0x2

_lib = None


def lib() -> ctypes.CDLL:
    """Load libgdn.so (built in-tree by ``gated_deltanet_linear_verify_amd.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m gated_deltanet_linear_verify_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, S = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        D = ctypes.POINTER(gdn_dims)
        Cp = ctypes.POINTER(gdn_capture)
        L.gdn_verify.argtypes = [D, P, P, P, P, P, P, P, P, P, P, Cp, P, I, P, I, P]
        L.gdn_verify_tree.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P, Cp, P, I, P, I, P]
        L.gdn_verify_resume.argtypes = [D, P, P, P, P, P, P, P, P, P, P, Cp, P, I, P, P, I, P]
        L.gdn_rollback.argtypes = [Cp, I, I, P]
        L.gdn_rollback_batch.argtypes = [Cp, P, P, I, P]
        L.gdn_rollback_trim.argtypes = [Cp, I, I, I, P]
        L.gdn_prefill.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P, I, I, P, S, P]
        L.gdn_prefill_noalloc.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P, I, I, P]
        L.gdn_prefill_workspace_bytes.argtypes = [D, I]
        L.gdn_prefill_workspace_bytes.restype = S
        L.gdn_capture_bytes.argtypes = [D, I, I, ctypes.POINTER(S)]
        L.gdn_capture_bytes.restype = S
        L.gdn_reset.argtypes = [D, P, P, I, P]
        L.gdn_snapshot.argtypes = [D, P, P, P, P, P, I, P]
        L.gdn_restore.argtypes = [D, P, P, P, P, P, I, P]
        L.gdn_rollback_layers.argtypes = [Cp, I, P, P, I, P]
        L.gdn_graph_create.argtypes = [D, ctypes.POINTER(gdn_layer), I, I, I, P, I, P, ctypes.c_uint32,
                                       ctypes.POINTER(ctypes.c_void_p)]
        L.gdn_graph_launch.argtypes = [P, P]
        L.gdn_linear.argtypes = [P, P, I, I, I, ctypes.POINTER(gdn_out_seg), I, P]
        L.gdn_graph_destroy.argtypes = [P]
        R, T = ctypes.POINTER(gdn_rows), ctypes.POINTER(gdn_rope_table)
        K, B = ctypes.POINTER(gdn_kv), ctypes.POINTER(gdn_kv_batch)
        L.gdn_rope_init.argtypes = [ctypes.POINTER(gdn_rope_params), T]
        L.gdn_rope.argtypes = [T, R, R, I, I, P, I, I, P]
        L.gdn_kv_bytes.argtypes = [K, ctypes.POINTER(S)]
        L.gdn_kv_bytes.restype = S
        L.gdn_kv_write.argtypes = [K, B, R, R, T, P, P]
        L.gdn_kv_read.argtypes = [K, B, R, R, P]
        L.gdn_kv_commit.argtypes = [K, B, P, P, I, P]
        L.gdn_attn_verify.argtypes = [K, B, P, P, I, P, R, R, ctypes.c_float, P, S, P]
        L.gdn_attn_workspace_bytes.argtypes = [K, I, I, I, I]
        L.gdn_attn_workspace_bytes.restype = S
        A, F = ctypes.POINTER(gdn_mat), ctypes.c_float
        L.gdn_norm.argtypes = [R, R, R, P, R, P, I, I, F, I, P]
        L.gdn_linear_act.argtypes = [A, A, I, I, I, P, I, I, A, A, P, S, P]
        L.gdn_linear_act_workspace_bytes.argtypes = [I, I, I, I, I]
        L.gdn_linear_act_workspace_bytes.restype = S
        L.gdn_logprob.argtypes = [A, I, I, F, P, I, P, P, P, P, P, P, I, P, S, P]
        L.gdn_logprob_workspace_bytes.argtypes = [I, I, I, I, I]
        L.gdn_logprob_workspace_bytes.restype = S
        for f in ("gdn_verify", "gdn_verify_resume", "gdn_verify_tree", "gdn_rollback", "gdn_rollback_batch",
                  "gdn_rollback_trim", "gdn_prefill", "gdn_prefill_noalloc", "gdn_reset", "gdn_snapshot", "gdn_restore",
                  "gdn_rollback_layers", "gdn_graph_create", "gdn_graph_launch", "gdn_graph_destroy",
                  "gdn_linear", "gdn_rope_init", "gdn_rope", "gdn_kv_write", "gdn_kv_read", "gdn_kv_commit",
                  "gdn_attn_verify", "gdn_norm", "gdn_linear_act", "gdn_logprob"):
            getattr(L, f).restype = ctypes.c_int
        L.gdn_last_error.restype = ctypes.c_char_p
        L.gdn_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def last_error() -> str:
    return lib().gdn_last_error().decode()


def version() -> str:
    return lib().gdn_version().decode()


def _check(rc: int) -> None:
    if rc != GDN_OK:
        raise GdnError(rc, last_error())


def make_dims(shape, *, flags: int = 0, eps: float = 1e-6, n_pool: Optional[int] = None) -> gdn_dims:
    """gdn_dims from a workloads.Shape."""
    return gdn_dims(shape.n_kh, shape.n_vh, shape.d_k, shape.d_v, shape.d_conv,
                    shape.n_pool if n_pool is None else n_pool, shape.act_dtype, shape.out_dtype,
                    flags, eps)


def _p(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


class _Torch:
    """What the bindings below need of torch for every call, looked up once: a call of a small kernel is
    bound by the host, and torch.cuda.current_stream() alone builds a Stream object in 2.9 us where the
    handle is a query of 0.1 us."""

    def __init__(self):
        import torch
        torch.cuda.current_device()  # initialises the runtime, or says why it cannot
        self.dtypes = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}
        self.codes = {torch.float8_e4m3fn: GDN_E4M3, torch.int8: GDN_I8}
        self.all = {**self.dtypes, **self.codes}
        self.int32, self.float32 = torch.int32, torch.float32
        self.device = torch.cuda.current_device
        self.stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None)

    def stream(self, stream, here: int):
        if stream is None and self.stream_of is not None:
            return self.stream_of(here)
        return _stream(stream)


_torch_state = None


def _torch() -> _Torch:
    global _torch_state
    if _torch_state is None:
        _torch_state = _Torch()
    return _torch_state


class Capture:
    """Per-position capture buffers (torch tensors) plus the restore targets."""

    def __init__(self, dims: gdn_dims, ssm, conv, state, conv_state, t_cap: int, mode: int):
        self.dims, self.ssm, self.conv = dims, ssm, conv
        self.state, self.conv_state = state, conv_state
        self.t_cap, self.mode = t_cap, mode
        self.c = gdn_capture(dims, _p(ssm), _p(conv), _p(state), _p(conv_state), t_cap, mode)

    @property
    def ref(self):
        return ctypes.byref(self.c)


def capture_bytes(dims: gdn_dims, t_cap: int, mode: int) -> tuple:
    cb = ctypes.c_size_t(0)
    sb = lib().gdn_capture_bytes(ctypes.byref(dims), t_cap, mode, ctypes.byref(cb))
    return sb, cb.value


def gdn_verify(dims, state, conv_state, qkv, z, alpha, beta, A_log, dt_bias, conv_w, norm_w,
               capture: Optional[Capture], out, n_tok: int, slot_ids, n_batch: int,
               stream=None) -> None:
    _check(lib().gdn_verify(ctypes.byref(dims), _p(state), _p(conv_state), _p(qkv), _p(z),
                            _p(alpha), _p(beta), _p(A_log), _p(dt_bias), _p(conv_w), _p(norm_w),
                            capture.ref if capture is not None else None, _p(out), n_tok,
                            _p(slot_ids), n_batch, _stream(stream)))


def gdn_verify_resume(dims, state, conv_state, qkv, z, alpha, beta, A_log, dt_bias, conv_w, norm_w,
                      capture: Capture, out, n_tok: int, slot_ids, resume_idx, n_batch: int,
                      stream=None) -> None:
    _check(lib().gdn_verify_resume(ctypes.byref(dims), _p(state), _p(conv_state), _p(qkv), _p(z),
                                   _p(alpha), _p(beta), _p(A_log), _p(dt_bias), _p(conv_w),
                                   _p(norm_w), capture.ref if capture is not None else None,
                                   _p(out), n_tok, _p(slot_ids), _p(resume_idx), n_batch,
                                   _stream(stream)))


def gdn_verify_tree(dims, state, conv_state, qkv, z, alpha, beta, A_log, dt_bias, conv_w, norm_w,
                    parent, capture: Capture, out, n_tok: int, slot_ids, n_batch: int,
                    stream=None) -> None:
    _check(lib().gdn_verify_tree(ctypes.byref(dims), _p(state), _p(conv_state), _p(qkv), _p(z),
                                 _p(alpha), _p(beta), _p(A_log), _p(dt_bias), _p(conv_w),
                                 _p(norm_w), _p(parent), capture.ref, _p(out), n_tok,
                                 _p(slot_ids), n_batch, _stream(stream)))


def gdn_rollback(capture: Capture, slot: int, accepted_idx: int, stream=None) -> None:
    _check(lib().gdn_rollback(capture.ref, slot, accepted_idx, _stream(stream)))


def gdn_rollback_batch(capture: Capture, slots, accepted_idx, n: int, stream=None) -> None:
    _check(lib().gdn_rollback_batch(capture.ref, _p(slots), _p(accepted_idx), n, _stream(stream)))


def gdn_rollback_layers(layers, slots, accepted_idx, n: int, stream=None) -> None:
    """One launch (per 64 layers) restoring every layer's capture for the listed slots."""
    arr = (gdn_capture * len(layers))(*[c.c for c in layers])
    _check(lib().gdn_rollback_layers(arr, len(layers), _p(slots), _p(accepted_idx), n, _stream(stream)))


def gdn_linear(x, w, M: int, N: int, K: int, segs, stream=None) -> None:
    """y = x W^T into column segments: segs is a list of (n0, n1, tensor, ld, sigmoid) with the
    tensor's dtype (bf16 or fp32) as the storage type."""
    import torch
    arr = (gdn_out_seg * len(segs))(*[
        gdn_out_seg(n0, n1, ld, GDN_BF16 if t.dtype == torch.bfloat16 else GDN_F32, int(bool(sg)), _p(t))
        for (n0, n1, t, ld, sg) in segs])
    _check(lib().gdn_linear(_p(x), _p(w), M, N, K, arr, len(segs), _stream(stream)))


class Graph:
    """A recorded spec-decode step (gdn_graph_create) over layers given as dicts of torch tensors
    with the gdn_layer field names; replay with launch(), freed by close() or on collection."""

    def __init__(self, dims, layers, t_cap: int, n_tok: int, slot_ids, n_batch: int, accepted_idx,
                 phases: int = GDN_GRAPH_VERIFY | GDN_GRAPH_ROLLBACK):
        arr = (gdn_layer * len(layers))(*[gdn_layer(*[_p(L[n]) for n, _ in gdn_layer._fields_])
                                          for L in layers])
        self._h = ctypes.c_void_p(None)
        self._keep = (layers, slot_ids, accepted_idx)  # the graph holds raw pointers into these
        _check(lib().gdn_graph_create(ctypes.byref(dims), arr, len(layers), t_cap, n_tok, _p(slot_ids),
                                      n_batch, _p(accepted_idx), phases, ctypes.byref(self._h)))

    def launch(self, stream=None) -> None:
        _check(lib().gdn_graph_launch(self._h, _stream(stream)))

    def close(self) -> None:
        if self._h:
            _check(lib().gdn_graph_destroy(self._h))
            self._h = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gdn_rollback_trim(capture: Capture, slot: int, trim: int, n_tok: int, stream=None) -> None:
    _check(lib().gdn_rollback_trim(capture.ref, slot, trim, n_tok, _stream(stream)))


def gdn_prefill_workspace_bytes(dims, n_tok: int) -> int:
    return lib().gdn_prefill_workspace_bytes(ctypes.byref(dims), n_tok)


def gdn_prefill(dims, state, conv_state, qkv, z, alpha, beta, A_log, dt_bias, conv_w, norm_w, out,
                n_tok: int, slot: int, workspace, ws_bytes: int, stream=None) -> None:
    _check(lib().gdn_prefill(ctypes.byref(dims), _p(state), _p(conv_state), _p(qkv), _p(z),
                             _p(alpha), _p(beta), _p(A_log), _p(dt_bias), _p(conv_w), _p(norm_w),
                             _p(out), n_tok, slot, _p(workspace), ws_bytes, _stream(stream)))


def gdn_prefill_noalloc(dims, state, conv_state, qkv, z, alpha, beta, A_log, dt_bias, conv_w, norm_w,
                        out, n_tok: int, slot: int, stream=None) -> None:
    _check(lib().gdn_prefill_noalloc(ctypes.byref(dims), _p(state), _p(conv_state), _p(qkv), _p(z),
                                     _p(alpha), _p(beta), _p(A_log), _p(dt_bias), _p(conv_w),
                                     _p(norm_w), _p(out), n_tok, slot, _stream(stream)))


def gdn_reset(dims, state, conv_state, slot: int, stream=None) -> None:
    _check(lib().gdn_reset(ctypes.byref(dims), _p(state), _p(conv_state), slot, _stream(stream)))


def gdn_snapshot(dims, state, conv_state, snap_state, snap_conv, slots, n: int, stream=None) -> None:
    _check(lib().gdn_snapshot(ctypes.byref(dims), _p(state), _p(conv_state), _p(snap_state), _p(snap_conv),
                              _p(slots), n, _stream(stream)))


def gdn_restore(dims, state, conv_state, snap_state, snap_conv, slots, n: int, stream=None) -> None:
    _check(lib().gdn_restore(ctypes.byref(dims), _p(state), _p(conv_state), _p(snap_state), _p(snap_conv),
                             _p(slots), n, _stream(stream)))


# ---- the full-attention layers: rotary positions, the paged KV cache, attention ----

def _bad(msg: str) -> GdnError:
    return GdnError(GDN_ERR_ARG, msg)


def _elsewhere(fn: str, t, here: int) -> GdnError:
    return _bad(f"{fn}: a tensor is on {t.device}, not on the current device cuda:{here}, where the launch goes")


def _ints(fn: str, name: str, t, here: int, T: _Torch, n0: int, n1: int = -1) -> int:
    """Address of a contiguous int32 tensor [n0] or [n0][n1] (the first size may be larger)."""
    if t.get_device() != here:
        raise _elsewhere(fn, t, here)
    if t.dtype is not T.int32 or not t.is_contiguous():
        raise _bad(f"{fn}: {name} must be a contiguous int32 tensor")
    shape = t.shape
    if len(shape) != (1 if n1 < 0 else 2) or shape[0] < n0 or (n1 >= 0 and shape[1] != n1):
        raise _bad(f"{fn}: {name} has shape {tuple(shape)}, expected {(n0,) if n1 < 0 else (n0, n1)}")
    return t.data_ptr()


def _rows(fn: str, name: str, t, here: int, T: _Torch, n_rows: int, d: int, codes: bool = False) -> gdn_rows:
    """gdn_rows of a [n_rows][n_heads][d] tensor whose channels are contiguous (other strides are free)."""
    if t.get_device() != here:
        raise _elsewhere(fn, t, here)
    dtype = (T.all if codes else T.dtypes).get(t.dtype)
    if dtype is None:
        raise GdnError(GDN_ERR_DTYPE, f"{fn}: {name} must be bfloat16 or float32, not {t.dtype}")
    shape, strides = t.shape, t.stride()
    if len(shape) != 3 or shape[0] < n_rows or shape[2] != d or (strides[2] != 1 and d > 1):
        raise _bad(f"{fn}: {name} must be [{n_rows}][heads][{d}] with contiguous channels, got {tuple(shape)} "
                   f"with strides {strides}")
    # a single row or head may carry any stride in torch; it is never stepped over
    return gdn_rows(t.data_ptr(), strides[0] if shape[0] > 1 else 0, strides[1] if shape[1] > 1 else 0, shape[1], dtype)


def gdn_rope_init(rot_dim: int, *, theta: float = 1e4, layout: int = GDN_ROPE_HALF, scaling: int = GDN_ROPE_PLAIN,
                  factor: float = 1.0, orig_ctx: int = 0, sections=None, beta_fast: float = 0.0,
                  beta_slow: float = 0.0, mscale: float = 0.0) -> gdn_rope_table:
    """The rotary table of the parameters (host memory, kept by the caller)."""
    sections = list(sections or ())
    if len(sections) > 4:
        raise GdnError(GDN_ERR_SHAPE, f"gdn_rope_init: {len(sections)} sections, at most 4 position axes")
    sec = (ctypes.c_int32 * 4)(*sections)
    p = gdn_rope_params(rot_dim, layout, scaling, orig_ctx, sec, theta, factor, beta_fast, beta_slow, mscale)
    t = gdn_rope_table()
    _check(lib().gdn_rope_init(ctypes.byref(p), ctypes.byref(t)))
    return t


def gdn_rope(table: gdn_rope_table, segs, positions, n_tok: int, *, inverse: bool = False, stream=None) -> None:
    """Rotate segs, a list of (x, out) tensors [n_tok][heads][d] (out may be x); positions int32
    [n_axes][n_tok]."""
    fn, T, n = "gdn_rope", _torch(), len(segs)
    here = T.device()
    if not n:
        raise GdnError(GDN_ERR_SHAPE, "gdn_rope: no rows given")
    d = segs[0][0].shape[-1]
    xs, outs = (gdn_rows * n)(), (gdn_rows * n)()
    for i, (x, out) in enumerate(segs):
        xs[i], outs[i] = _rows(fn, "x", x, here, T, n_tok, d), _rows(fn, "out", out, here, T, n_tok, d)
    _check(lib().gdn_rope(table, xs, outs, n, d, _ints(fn, "positions", positions, here, T, table.n_axes, n_tok), n_tok,
                          1 if inverse else 0, T.stream(stream, here)))


class KvCache:
    """A layer's paged KV cache over caller-owned tensors: k and v [n_pages][n_kv][page_size][d] in
    bfloat16, float8_e4m3fn or int8, the 8-bit ones with fp32 k_scale and v_scale [n_pages][n_kv][page_size]."""

    def __init__(self, k, v, k_scale=None, v_scale=None, *, flags: int = 0):
        import torch
        formats = {torch.bfloat16: GDN_KV_BF16, torch.float8_e4m3fn: GDN_KV_E4M3, torch.int8: GDN_KV_I8}
        if k.dtype not in formats or v.dtype != k.dtype:
            raise GdnError(GDN_ERR_DTYPE, f"KvCache: k and v must both be one of {list(formats)}")
        tensors = [t for t in (k, v, k_scale, v_scale) if t is not None]
        if k.dim() != 4 or v.shape != k.shape or any(s.shape != k.shape[:3] or s.dtype != torch.float32 for s in tensors[2:]):
            raise _bad("KvCache: k and v are [n_pages][n_kv][page_size][d], scales their first three sizes in float32")
        if not all(t.is_contiguous() for t in tensors) or any(t.device != k.device for t in tensors):
            raise _bad("KvCache: the cache's tensors must be contiguous and on one device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device = k.get_device()
        n_pages, n_kv, page_size, d = k.shape
        self.c = gdn_kv(n_kv, d, page_size, n_pages, formats[k.dtype], flags, _p(k), _p(v), _p(k_scale), _p(v_scale))

    @property
    def ref(self):
        return ctypes.byref(self.c)

    def _here(self, fn: str, T: _Torch) -> int:
        """The current device, which has to hold the cache."""
        here = T.device()
        if self.device != here:
            raise _elsewhere(fn, self.k, here)
        return here


def gdn_kv_bytes(n_kv: int, d: int, page_size: int, n_pages: int, fmt: int) -> tuple:
    """(bytes of k, bytes of k_scale) of a cache of these sizes; v takes as much again."""
    kv = gdn_kv(n_kv, d, page_size, n_pages, fmt, 0, None, None, None, None)
    sb = ctypes.c_size_t(0)
    return lib().gdn_kv_bytes(ctypes.byref(kv), ctypes.byref(sb)), sb.value


def _batch(fn: str, here: int, T: _Torch, block_table, start, n_new, n_batch: int, n_tok: int) -> gdn_kv_batch:
    wide = block_table.shape[1] if block_table.dim() == 2 else 0
    return gdn_kv_batch(_ints(fn, "block_table", block_table, here, T, n_batch, wide),
                        _ints(fn, "start", start, here, T, n_batch),
                        None if n_new is None else _ints(fn, "n_new", n_new, here, T, n_batch), wide, n_batch, n_tok)


def gdn_kv_write(kv: KvCache, k, v, block_table, start, n_new, n_batch: int, n_tok: int, *,
                 rope: Optional[gdn_rope_table] = None, positions=None, stream=None) -> None:
    """k and v [n_batch * n_tok][n_kv][d] into the cache at positions start[b] + t, k rotated by ``rope`` on the
    way; positions int32 [n_axes][n_batch * n_tok]."""
    fn, T, n, d = "gdn_kv_write", _torch(), n_batch * n_tok, kv.c.d
    here = kv._here(fn, T)
    b = _batch(fn, here, T, block_table, start, n_new, n_batch, n_tok)
    if rope is not None and positions is None:
        raise _bad("gdn_kv_write: rope needs positions")
    pos = _ints(fn, "positions", positions, here, T, rope.n_axes, n) if rope is not None else None
    _check(lib().gdn_kv_write(kv.c, b, _rows(fn, "k", k, here, T, n, d), _rows(fn, "v", v, here, T, n, d), rope, pos,
                              T.stream(stream, here)))


def gdn_kv_read(kv: KvCache, block_table, start, n_new, k, v, n_batch: int, n_tok: int, *, stream=None) -> None:
    """Positions start[b] + t of the cache into k and v [n_batch * n_tok][n_kv][d]."""
    fn, T, n, d = "gdn_kv_read", _torch(), n_batch * n_tok, kv.c.d
    here = kv._here(fn, T)
    b = _batch(fn, here, T, block_table, start, n_new, n_batch, n_tok)
    _check(lib().gdn_kv_read(kv.c, b, _rows(fn, "k", k, here, T, n, d), _rows(fn, "v", v, here, T, n, d),
                             T.stream(stream, here)))


def gdn_kv_commit(kv: KvCache, block_table, start, path, n_path, n_batch: int, n_tok: int, *, n_new=None,
                  stream=None) -> None:
    """Move the cache rows of the accepted nodes path[b][:n_path[b]] (of n_tok per entry) to start[b], start[b] + 1, ..."""
    fn, T = "gdn_kv_commit", _torch()
    here = kv._here(fn, T)
    b = _batch(fn, here, T, block_table, start, n_new, n_batch, n_tok)
    wide = path.shape[1] if path.dim() == 2 else 0
    _check(lib().gdn_kv_commit(kv.c, b, _ints(fn, "path", path, here, T, n_batch, wide),
                               _ints(fn, "n_path", n_path, here, T, n_batch), wide, T.stream(stream, here)))


def gdn_attn_workspace_bytes(kv: KvCache, n_q: int, n_batch: int, n_tok: int, prefix: bool = False) -> int:
    return lib().gdn_attn_workspace_bytes(kv.c, n_q, n_batch, n_tok, int(bool(prefix)))


def gdn_attn_verify(kv: KvCache, q, block_table, start, n_new, parent, prefix_pages, prefix_len, out, n_batch: int,
                    n_tok: int, scale: float, workspace, *, stream=None) -> None:
    """Attention of q [n_batch * n_tok][n_q][d] over the cache into out, a chain (parent None) or a tree, with an
    optional prefix shared by the batch: prefix_pages int32 [pages], prefix_len int32 [1]."""
    fn, T, n, d = "gdn_attn_verify", _torch(), n_batch * n_tok, kv.c.d
    here = kv._here(fn, T)
    b = _batch(fn, here, T, block_table, start, n_new, n_batch, n_tok)
    par = None if parent is None else _ints(fn, "parent", parent, here, T, n_batch, n_tok)
    pre = None if prefix_pages is None else _ints(fn, "prefix_pages", prefix_pages, here, T, 1)
    plen = None if prefix_len is None else _ints(fn, "prefix_len", prefix_len, here, T, 1)
    if workspace.get_device() != here:
        raise _elsewhere(fn, workspace, here)
    if not workspace.is_contiguous():  # an expanded tensor has less memory than elements
        raise _bad("gdn_attn_verify: workspace must be contiguous")
    _check(lib().gdn_attn_verify(kv.c, b, par, pre, 0 if pre is None else prefix_pages.shape[0], plen,
                                 _rows(fn, "q", q, here, T, n, d), _rows(fn, "out", out, here, T, n, d), scale,
                                 workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                 T.stream(stream, here)))


# ---- between the mixers and behind the last one: norms, products with an epilogue, log probabilities ----

def _floats(fn: str, name: str, t, here: int, T: _Torch, n0: int, n1: int = -1) -> int:
    """Address of a contiguous float32 tensor [n0] or [n0][n1] (the first size may be larger)."""
    if t.get_device() != here:
        raise _elsewhere(fn, t, here)
    if t.dtype is not T.float32 or not t.is_contiguous():
        raise _bad(f"{fn}: {name} must be a contiguous float32 tensor")
    shape = t.shape
    if len(shape) != (1 if n1 < 0 else 2) or shape[0] < n0 or (n1 >= 0 and shape[1] != n1):
        raise _bad(f"{fn}: {name} has shape {tuple(shape)}, expected {(n0,) if n1 < 0 else (n0, n1)}")
    return t.data_ptr()


def _mat(fn: str, name: str, t, here: int, T: _Torch, rows: int, cols: int, types: dict, scale=None) -> gdn_mat:
    """gdn_mat of a [rows][cols] tensor whose columns are contiguous (more rows are left alone)."""
    if t.get_device() != here:
        raise _elsewhere(fn, t, here)
    dtype = types.get(t.dtype)
    if dtype is None:
        raise GdnError(GDN_ERR_DTYPE, f"{fn}: {name} must be one of {list(types)}, not {t.dtype}")
    shape, strides = t.shape, t.stride()
    if len(shape) != 2 or shape[0] < rows or shape[1] != cols or (strides[1] != 1 and cols > 1):
        raise _bad(f"{fn}: {name} must be [{rows}][{cols}] with contiguous columns, got {tuple(shape)} with strides {strides}")
    return gdn_mat(t.data_ptr(), None if scale is None else _floats(fn, name + "_scale", scale, here, T, rows),
                   strides[0] if shape[0] > 1 else cols, dtype)


def _scratch(fn: str, t, here: int) -> tuple:
    """(address, bytes) of a workspace tensor, or nothing."""
    if t is None:
        return None, 0
    if t.get_device() != here:
        raise _elsewhere(fn, t, here)
    if not t.is_contiguous():  # an expanded tensor has less memory than elements
        raise _bad(f"{fn}: workspace must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


def gdn_norm(x, weight, out, n_tok: int, *, residual=None, total=None, scale=None, eps: float = 1e-6,
             mode: int = GDN_NORM_RMS, stream=None) -> None:
    """RMS norm of x (+ residual) [n_tok][heads][d] by weight (float32 [d], or None) into out: bfloat16, float32, or
    float8_e4m3fn / int8 with scale float32 [n_tok][heads]; total receives x + residual."""
    fn, T = "gdn_norm", _torch()
    here = T.device()
    d, heads = x.shape[-1], x.shape[1] if x.dim() == 3 else 0
    r = [None if t is None else _rows(fn, n, t, here, T, n_tok, d, n == "out")
         for n, t in (("x", x), ("residual", residual), ("total", total), ("out", out))]
    if weight is not None and tuple(weight.shape) != (d,):  # one of all heads would be cut to its first d values
        raise _bad(f"{fn}: weight has shape {tuple(weight.shape)}, expected {(d,)}")
    _check(lib().gdn_norm(r[0], r[1], r[2], None if weight is None else _floats(fn, "weight", weight, here, T, d), r[3],
                          None if scale is None else _floats(fn, "scale", scale, here, T, n_tok, heads), d, n_tok, eps, mode,
                          T.stream(stream, here)))


def gdn_linear_act_workspace_bytes(M: int, N: int, K: int, dtype, gated: bool = False) -> int:
    """Of a gdn_linear_act call with x and w of the torch type ``dtype``."""
    import torch
    codes = {torch.bfloat16: GDN_BF16, torch.float8_e4m3fn: GDN_E4M3, torch.int8: GDN_I8}
    return lib().gdn_linear_act_workspace_bytes(M, N, K, codes.get(dtype, -1), int(bool(gated)))


def gdn_linear_act(x, w, out, M: int, N: int, K: int, *, x_scale=None, w_scale=None, bias=None, act: int = GDN_ACT_NONE,
                   gated: bool = False, residual=None, workspace=None, stream=None) -> None:
    """out [M][N] = act(x w^T + bias) + residual, or act(gate) * up of w's first and last N rows where gated; x [M][K] and
    w [N or 2 N][K] in bfloat16, or float8_e4m3fn or int8 with float32 scales per row.  w and bias may have more rows where not
    gated; those are left alone."""
    fn, T, rows = "gdn_linear_act", _torch(), 2 * N if gated else N
    here = T.device()
    if gated:  # of more rows the up rows would be taken from among the gate's
        for name, t in (("w", w), ("w_scale", w_scale), ("bias", bias)):
            if t is not None and t.shape[0] != rows:
                raise _bad(f"{fn}: {name} has {t.shape[0]} rows, a gated product of {N} columns takes {rows}")
    ws, ws_bytes = _scratch(fn, workspace, here)
    _check(lib().gdn_linear_act(
        _mat(fn, "x", x, here, T, M, K, T.all, x_scale), _mat(fn, "w", w, here, T, rows, K, T.all, w_scale), M, N, K,
        None if bias is None else _floats(fn, "bias", bias, here, T, rows), act, 1 if gated else 0,
        None if residual is None else _mat(fn, "residual", residual, here, T, M, N, T.dtypes),
        _mat(fn, "out", out, here, T, M, N, T.dtypes), ws, ws_bytes, T.stream(stream, here)))


def gdn_logprob_workspace_bytes(n_rows: int, n_vocab: int, dtype, n_ids: int = 0, top_k: int = 0) -> int:
    """Of a gdn_logprob call with logits of the torch type ``dtype``."""
    import torch
    codes = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}
    return lib().gdn_logprob_workspace_bytes(n_rows, n_vocab, codes.get(dtype, -1), n_ids, top_k)


def gdn_logprob(logits, n_rows: int, n_vocab: int, *, ids=None, temperature: float = 1.0, logprob=None, rank=None,
                lse=None, entropy=None, top_ids=None, top_logprob=None, workspace=None, stream=None) -> None:
    """Of logits [n_rows][n_vocab]: log probabilities and ranks of ids (int32 [n_rows][n_ids], -1: none), log sum exp,
    entropy, and the first top_k alternatives (top_ids int32 and top_logprob [n_rows][top_k])."""
    fn, T = "gdn_logprob", _torch()
    here = T.device()
    n_ids = 0 if ids is None else ids.shape[-1]
    k = 0 if top_ids is None else top_ids.shape[-1]
    at = lambda get, n, t, *sizes: None if t is None else get(fn, n, t, here, T, n_rows, *sizes)  # noqa: E731
    ws, ws_bytes = _scratch(fn, workspace, here)
    _check(lib().gdn_logprob(
        _mat(fn, "logits", logits, here, T, n_rows, n_vocab, T.dtypes), n_rows, n_vocab, temperature,
        at(_ints, "ids", ids, n_ids), n_ids, at(_floats, "logprob", logprob, n_ids), at(_ints, "rank", rank, n_ids),
        at(_floats, "lse", lse), at(_floats, "entropy", entropy), at(_ints, "top_ids", top_ids, k),
        at(_floats, "top_logprob", top_logprob, k), k, ws, ws_bytes, T.stream(stream, here)))
