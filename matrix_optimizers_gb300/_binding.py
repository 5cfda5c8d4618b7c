"""ctypes binding of libmatrixopt (include/matrixopt.h): argument marshalling only.

Every function here has the name of the C entry point it calls, converts
torch tensors / Python values into the C structures and pointers, and raises
``MoError`` on a non-zero status.  No arithmetic of the method happens here:
every step runs in the library's CUDA kernels (or, for ``plan_owners``, in
its host C++).  If the library has not been built the first call raises.
"""
import bisect
import ctypes
import os
import struct
import threading

import torch  # loads the CUDA runtime the library links against

from . import build as _build

c_int32, c_uint32, c_int64, c_float, c_double, c_void_p, c_size_t = (
    ctypes.c_int32, ctypes.c_uint32, ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.c_void_p, ctypes.c_size_t)

MO_OK, MO_ERR_INVALID_ARG, MO_ERR_ALIGNMENT, MO_ERR_WORKSPACE, MO_ERR_CUDA, MO_ERR_TIMEOUT, \
    MO_ERR_UNSUPPORTED = 0, -1, -2, -3, -4, -5, -6
MO_F32, MO_BF16, MO_I32, MO_I64, MO_E4M3 = 0, 1, 2, 3, 4
MO_NS_BF16, MO_NS_FP32 = 0, 1


class MoError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{msg} (status {status})")
        self.status = status


class mo_matrix(ctypes.Structure):
    _fields_ = [("rows", c_int64), ("cols", c_int64), ("ld", c_int64),
                ("w_dtype", c_int32), ("m_dtype", c_int32), ("g_dtype", c_int32),
                ("reserved", c_int32),
                ("W", c_void_p), ("M", c_void_p), ("G", c_void_p)]


class mo_muon_cfg(ctypes.Structure):
    _fields_ = [("mu", c_float), ("lr", c_float), ("update_scale", c_float),
                ("weight_decay", c_float), ("ns_steps", c_int32),
                ("a", c_float), ("b", c_float), ("c", c_float),
                ("ns_precision", c_int32), ("apply_update", c_int32),
                ("out_dtype", c_int32), ("spectral_iters", c_int32)]


class mo_adamw_tail(ctypes.Structure):
    _fields_ = [("numel", c_int64), ("W", c_void_p), ("g", c_void_p), ("m", c_void_p),
                ("v", c_void_p), ("lr", c_float), ("beta1", c_float), ("beta2", c_float),
                ("eps", c_float), ("weight_decay", c_float), ("reserved", c_int32),
                ("step", c_int64)]


class mo_ns_view(ctypes.Structure):
    _fields_ = [("m", c_int64), ("n", c_int64), ("ldx", c_int64), ("lda", c_int64),
                ("transposed", c_int32), ("precision", c_int32),
                ("x_op", c_int64 * 2), ("diag_res", c_int64), ("gram", c_int64),
                ("poly", c_int64), ("deps", c_int64), ("tiles_sym", c_int32), ("tiles_apply", c_int32),
                ("releases_per_tile", c_int32), ("reserved", c_int32)]


class mo_distill(ctypes.Structure):
    _fields_ = [("n", c_int64), ("vocab", c_int64), ("ldl", c_int64),
                ("top", c_int32), ("logits_dtype", c_int32), ("idx_dtype", c_int32), ("teacher_dtype", c_int32),
                ("temperature", c_float), ("grad_scale", c_float),
                ("logits", c_void_p), ("idx", c_void_p), ("teacher", c_void_p), ("row_weight", c_void_p)]


class mo_route(ctypes.Structure):
    _fields_ = [("n", c_int64), ("ldl", c_int64),
                ("experts", c_int32), ("top", c_int32), ("logits_dtype", c_int32), ("renormalise", c_int32),
                ("logits", c_void_p), ("mask", c_void_p)]


class mo_block_norm(ctypes.Structure):
    _fields_ = [("n", c_int64), ("dim", c_int64), ("ldx", c_int64), ("ldr", c_int64), ("rows_per_gate", c_int64),
                ("ldgate", c_int64),
                ("x_dtype", c_int32), ("stream_dtype", c_int32), ("param_dtype", c_int32),
                ("eps", c_float), ("residual_scale", c_float), ("block_scale", c_float),
                ("x", c_void_p), ("residual", c_void_p), ("post", c_void_p), ("gate", c_void_p), ("pre", c_void_p)]


class mo_adamw_tensor(ctypes.Structure):
    _fields_ = [("numel", c_int64), ("W", c_void_p), ("g", c_void_p), ("m", c_void_p), ("v", c_void_p),
                ("m_scale", c_void_p), ("v_scale", c_void_p),
                ("w_dtype", c_int32), ("g_dtype", c_int32), ("state_dtype", c_int32),
                ("lr", c_float), ("weight_decay", c_float), ("reserved", c_int32)]


class mo_adamw_cfg(ctypes.Structure):
    _fields_ = [("beta1", c_float), ("beta2", c_float), ("eps", c_float), ("grad_scale", c_float),
                ("step", c_int64), ("step_ptr", c_void_p), ("grad_mul", c_void_p),
                ("seed", c_uint32), ("dither", c_int32)]


_CODES = {c_int32: "i", c_uint32: "I", c_int64: "q", c_float: "f", c_void_p: "P"}


def _packer(structure):
    """A function from a structure's values (addresses as integers, 0 for null) to its bytes, which
    an argument of type c_void_p takes: half the time of filling the structure itself."""
    return struct.Struct("@" + "".join(_CODES[kind] for _, kind in structure._fields_)).pack


_pack_route, _pack_norm, _pack_adamw_cfg = _packer(mo_route), _packer(mo_block_norm), _packer(mo_adamw_cfg)


# (name, restype, argtypes) of every exported symbol declared in include/*.h
_SIGNATURES = [
    ("mo_workspace_bytes", c_int32, [ctypes.POINTER(mo_matrix), c_int32, ctypes.POINTER(mo_muon_cfg),
                                     ctypes.POINTER(c_size_t)]),
    ("muon_step_batched", c_int32, [ctypes.POINTER(mo_matrix), c_int32, ctypes.POINTER(mo_muon_cfg),
                                    ctypes.POINTER(mo_adamw_tail), ctypes.POINTER(c_void_p),
                                    c_void_p, c_size_t, c_void_p]),
    ("muon_step_sign_packed", c_int32, [ctypes.POINTER(mo_matrix), c_int32, ctypes.POINTER(mo_muon_cfg),
                                        ctypes.POINTER(c_void_p), c_void_p, c_size_t, c_void_p]),
    ("muon_step_sign_vote", c_int32, [ctypes.POINTER(mo_matrix), c_int32, ctypes.POINTER(mo_muon_cfg),
                                      ctypes.POINTER(c_void_p), c_void_p, c_int32, c_int64, c_float, c_void_p,
                                      c_size_t, c_void_p]),
    ("ns_workspace_bytes", c_int32, [ctypes.POINTER(c_int64), ctypes.POINTER(c_int64), c_int32, c_int32,
                                     ctypes.POINTER(c_size_t)]),
    ("ns_orthogonalize", c_int32, [ctypes.POINTER(c_void_p), ctypes.POINTER(c_void_p),
                                   ctypes.POINTER(c_int64), ctypes.POINTER(c_int64),
                                   ctypes.POINTER(c_int64), c_int32, c_int32, c_int32, c_int32,
                                   c_float, c_float, c_float, c_int32, c_void_p, c_size_t, c_void_p]),
    ("ns_orthogonalize_noalloc", c_int32, [c_void_p, c_void_p, c_int64, c_int64, c_int64, c_int32, c_int32,
                                           c_int32, c_float, c_float, c_float, c_void_p]),
    ("ns_orthogonalize_noalloc_status", c_int32, [c_void_p]),
    ("sign_pack", c_int32, [c_void_p, c_int32, c_int64, c_int64, c_int64, c_void_p, c_void_p]),
    ("sign_vote_update", c_int32, [ctypes.POINTER(c_void_p), c_int32, c_int64, c_int64, c_void_p,
                                   c_int32, c_int64, c_float, c_void_p]),
    ("sign_vote_polar_workspace_bytes", c_int32, [c_int64, c_int64, c_int64, ctypes.POINTER(c_size_t)]),
    ("sign_vote_polar_update", c_int32, [ctypes.POINTER(c_void_p), c_int32, c_int64, c_int64, c_void_p, c_int32,
                                         c_int64, c_float, c_int32, c_float, c_float, c_float, c_void_p,
                                         c_size_t, c_void_p]),
    ("sign_pack_batched", c_int32, [ctypes.POINTER(c_void_p), c_int32, c_int32, c_int64, c_int64, c_int64,
                                    ctypes.POINTER(c_void_p), c_void_p]),
    ("sign_int8", c_int32, [c_void_p, c_int32, c_int64, c_int64, c_int64, c_void_p, c_void_p]),
    ("sign_vote_update_int8", c_int32, [ctypes.POINTER(c_void_p), c_int32, c_int64, c_int64, c_void_p,
                                        c_int32, c_int64, c_float, c_void_p]),
    ("plan_owners", c_int32, [ctypes.POINTER(c_int64), ctypes.POINTER(c_int64), c_int32, c_int32,
                              c_int32, c_double, c_double, ctypes.POINTER(c_int32),
                              ctypes.POINTER(c_double)]),
    ("embedding_lookup", c_int32, [c_void_p, c_int32, c_int64, c_int64, c_int64, c_void_p, c_int32, c_int64, c_float,
                                   c_void_p, c_int32, c_int64, c_void_p]),
    ("embedding_grad_workspace_bytes", c_int32, [c_int64, c_int64, c_int64, ctypes.POINTER(c_size_t)]),
    ("embedding_grad", c_int32, [c_void_p, c_int32, c_int64, c_int64, c_int64, c_void_p, c_int32, c_int64, c_float,
                                 c_void_p, c_int32, c_int64, c_int32, c_void_p, c_size_t, c_void_p]),
    ("expert_linear_workspace_bytes", c_int32, [c_int64, c_int64, c_int64, c_int32, ctypes.POINTER(c_size_t)]),
    ("expert_linear", c_int32, [c_void_p, c_int64, c_void_p, c_int64, c_int64, c_void_p, c_int64, c_int64, c_int64,
                                c_int32, c_void_p, c_int32, c_int64, c_void_p, c_size_t, c_void_p]),
    ("expert_linear_dgrad", c_int32, [c_void_p, c_int64, c_void_p, c_int64, c_int64, c_void_p, c_int64, c_int64,
                                      c_int64, c_int32, c_void_p, c_int32, c_int64, c_void_p, c_size_t, c_void_p]),
    ("expert_linear_wgrad", c_int32, [c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_int64, c_int64,
                                      c_int32, c_void_p, c_int32, c_int64, c_int64, c_int32, c_void_p, c_size_t,
                                      c_void_p]),
    ("distill_topk_loss", c_int32, [ctypes.POINTER(mo_distill), c_void_p, c_void_p, c_void_p]),
    ("distill_topk_grad", c_int32, [ctypes.POINTER(mo_distill), c_void_p, c_void_p, c_int32, c_int64, c_void_p]),
    ("distill_topk_loss_grad", c_int32, [ctypes.POINTER(mo_distill), c_void_p, c_void_p, c_int32, c_int64, c_void_p]),
    ("expert_route_workspace_bytes", c_int32, [c_int64, c_int32, c_int32, ctypes.POINTER(c_size_t)]),
    ("expert_route", c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                               c_void_p, c_void_p, c_size_t, c_void_p]),
    ("expert_route_grad", c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_float, c_float, c_void_p,
                                    c_int32, c_int64, c_void_p]),
    ("expert_scatter", c_int32, [c_void_p, c_int32, c_int64, c_int64, c_int64, c_void_p, c_int32, c_void_p, c_int32,
                                 c_int64, c_int64, c_void_p]),
    ("expert_combine", c_int32, [c_void_p, c_int32, c_int64, c_int64, c_void_p, c_void_p, c_int64, c_int32, c_int64,
                                 c_void_p, c_int32, c_int64, c_int32, c_void_p]),
    ("expert_combine_grad", c_int32, [c_void_p, c_int32, c_int64, c_void_p, c_int32, c_int64, c_int64, c_void_p,
                                      c_void_p, c_int64, c_int32, c_int64, c_void_p, c_int64, c_void_p, c_void_p]),
    ("block_norm", c_int32, [c_void_p, c_void_p, c_int64, c_void_p, c_int64, c_void_p]),
    ("block_norm_grad_workspace_bytes", c_int32, [c_int64, c_int64, c_int64, ctypes.POINTER(c_size_t)]),
    ("block_norm_grad", c_int32, [c_void_p, c_void_p, c_int64, c_void_p, c_int64, c_void_p,
                                  c_int64, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_void_p, c_void_p, c_int32,
                                  c_void_p, c_size_t, c_void_p]),
    ("adamw_step_batched", c_int32, [ctypes.POINTER(mo_adamw_tensor), c_int32, c_void_p, c_void_p]),
    ("mo_check_device_status", c_int32, [c_void_p, c_void_p]),
    ("mo_status_string", ctypes.c_char_p, [c_int32]),
    ("mo_version", c_int32, []),
    ("mo_debug_ns_view", c_int32, [ctypes.POINTER(c_int64), ctypes.POINTER(c_int64), c_int32, c_int32,
                                   c_int32, ctypes.POINTER(mo_ns_view)]),
    ("mo_debug_sm_count", c_int32, []),
    ("mo_debug_set_ns_fused", c_int32, [c_int32]),
    ("mo_debug_inject_dep_stall", c_int32, [c_int32, c_int64]),
    ("mo_debug_set_ns_pair", c_int32, [c_int32]),
    ("mo_debug_set_expert_shape", c_int32, [c_int32]),
    ("mo_debug_cta_stamps", c_int32, [c_void_p, c_int32, c_int32, ctypes.POINTER(c_int32)]),
    ("mo_trace_enable", c_int32, [c_int32]),
    ("mo_trace_read", c_int32, [ctypes.POINTER(c_int32), ctypes.POINTER(c_float), c_int32,
                                ctypes.POINTER(c_int32)]),
]

TRACE_KINDS = {1: "momentum_norm", 2: "norm_finalize", 3: "ns_gram", 4: "ns_poly", 5: "ns_apply",
               6: "ns_k0", 7: "adamw", 8: "sign_pack", 9: "vote_update", 10: "spectral_estimate",
               11: "ns_fused", 12: "embedding_lookup", 13: "embedding_sort", 14: "embedding_grad",
               15: "expert_linear", 16: "expert_linear_dgrad", 17: "expert_linear_wgrad", 18: "distill_topk",
               19: "expert_route", 20: "expert_route_grad", 21: "expert_scatter", 22: "expert_combine",
               23: "expert_combine_grad", 24: "block_norm", 25: "block_norm_grad", 26: "adamw_step_batched"}

_lib = None
_lock = threading.Lock()


def library_path():
    return _build.lib_path()


def load():
    """Load libmatrixopt.so (built in-tree by ``matrix_optimizers_gb300.build``)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise ImportError(
                f"{path} is missing: build the CUDA library first "
                "(python -m matrix_optimizers_gb300.build or __graft_entry__.build())")
        lib = ctypes.CDLL(path)
        for name, res, args in _SIGNATURES:
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _check(status):
    if status != MO_OK:
        msg = load().mo_status_string(status).decode()
        raise MoError(status, msg)


def dtype_code(dt):
    if dt == torch.float32:
        return MO_F32
    if dt == torch.bfloat16:
        return MO_BF16
    raise MoError(MO_ERR_INVALID_ARG, f"unsupported dtype {dt}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _ld(t):
    if t.dim() != 2 or (t.size(1) > 1 and t.stride(1) != 1):
        raise MoError(MO_ERR_INVALID_ARG, "matrices must be 2D with unit column stride")
    return t.stride(0) if t.size(0) > 1 else max(t.size(1), t.stride(0))


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_matrix(W, M, G):
    """mo_matrix for one parameter: W, M, G same shape and leading dimension."""
    if not (W.shape == M.shape == G.shape):
        raise MoError(MO_ERR_INVALID_ARG, "W, M and G must have one shape")
    ld = _ld(W)
    if _ld(M) != ld or _ld(G) != ld:
        raise MoError(MO_ERR_INVALID_ARG, "W, M and G must share the leading dimension")
    return mo_matrix(W.size(0), W.size(1), ld, dtype_code(W.dtype), dtype_code(M.dtype),
                     dtype_code(G.dtype), 0, W.data_ptr(), M.data_ptr(), G.data_ptr())


def make_cfg(mu=0.95, lr=0.02, ns_steps=5, a=3.4445, b=-4.7750, c=2.0315,
             precision=MO_NS_BF16, update_scale=1.0, weight_decay=0.0, apply_update=True,
             out_dtype=MO_BF16, spectral_iters=0):
    return mo_muon_cfg(mu, lr, update_scale, weight_decay, ns_steps, a, b, c, precision,
                       1 if apply_update else 0, out_dtype, spectral_iters)


def make_tail(W, g, m, v, step, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0):
    for t in (W, g, m, v):
        if t.dtype != torch.float32 or not t.is_contiguous():
            raise MoError(MO_ERR_INVALID_ARG, "the AdamW tail is contiguous float32")
    return mo_adamw_tail(W.numel(), W.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr(),
                         lr, beta1, beta2, eps, weight_decay, 0, step)


def _mat_array(mats):
    arr = (mo_matrix * max(1, len(mats)))()
    for i, m in enumerate(mats):
        arr[i] = m
    return arr


def mo_workspace_bytes(mats, cfg):
    out = c_size_t(0)
    _check(load().mo_workspace_bytes(_mat_array(mats), len(mats), ctypes.byref(cfg), ctypes.byref(out)))
    return out.value


def muon_step_batched(mats, cfg, ws, tail=None, out=None, stream=None):
    """One Muon step over ``mats`` (list of mo_matrix); ``ws`` a CUDA uint8
    tensor of at least mo_workspace_bytes(); ``out`` a list of tensors when
    cfg.apply_update is 0."""
    outs = None
    if out is not None:
        outs = (c_void_p * max(1, len(out)))(*[o.data_ptr() for o in out])
    _check(load().muon_step_batched(
        _mat_array(mats), len(mats), ctypes.byref(cfg),
        ctypes.byref(tail) if tail is not None else None, outs,
        _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream)))


def muon_step_sign_packed(mats, cfg, words, ws, stream=None):
    """Sign-Muon worker step: momentum + NS with the packed signs of the
    direction written to ``words`` (list of int32 tensors) in the last epilogue."""
    arr = (c_void_p * max(1, len(words)))(*[w.data_ptr() for w in words])
    _check(load().muon_step_sign_packed(_mat_array(mats), len(mats), ctypes.byref(cfg), arr, _ptr(ws),
                                        ws.numel() if ws is not None else 0, _stream(stream)))


def muon_step_sign_vote(mats, cfg, words, W, lr, ws, stream=None):
    """The Sign-Muon step of the M workers ``mats``: momentum + NS with fused
    sign packing into ``words``, then the majority vote W <- W - lr * vote."""
    arr = (c_void_p * max(1, len(words)))(*[w.data_ptr() for w in words])
    _check(load().muon_step_sign_vote(_mat_array(mats), len(mats), ctypes.byref(cfg), arr, _ptr(W),
                                      dtype_code(W.dtype), _ld(W), lr, _ptr(ws),
                                      ws.numel() if ws is not None else 0, _stream(stream)))


def ns_workspace_bytes(shapes, precision=MO_NS_BF16):
    n = len(shapes)
    rows = (c_int64 * max(1, n))(*[s[0] for s in shapes])
    cols = (c_int64 * max(1, n))(*[s[1] for s in shapes])
    out = c_size_t(0)
    _check(load().ns_workspace_bytes(rows, cols, n, precision, ctypes.byref(out)))
    return out.value


def ns_orthogonalize(X, out, steps, ws, a=3.4445, b=-4.7750, c=2.0315, precision=MO_NS_BF16,
                     stream=None):
    """out[i] = NS_steps(X[i]/||X[i]||_F) for lists of tensors (one dtype each)."""
    n = len(X)
    xs = (c_void_p * max(1, n))(*[x.data_ptr() for x in X])
    os_ = (c_void_p * max(1, n))(*[o.data_ptr() for o in out])
    rows = (c_int64 * max(1, n))(*[x.size(0) for x in X])
    cols = (c_int64 * max(1, n))(*[x.size(1) for x in X])
    lds = []
    for x, o in zip(X, out):
        if _ld(x) != _ld(o):
            raise MoError(MO_ERR_INVALID_ARG, "X[i] and out[i] must share the leading dimension")
        lds.append(_ld(x))
    ld = (c_int64 * max(1, n))(*lds)
    in_dt = dtype_code(X[0].dtype) if n else MO_F32
    out_dt = dtype_code(out[0].dtype) if n else MO_F32
    _check(load().ns_orthogonalize(xs, os_, rows, cols, ld, n, in_dt, out_dt, steps, a, b, c,
                                   precision, _ptr(ws), ws.numel() if ws is not None else 0,
                                   _stream(stream)))


def ns_orthogonalize_noalloc(X, out, steps, a=3.4445, b=-4.7750, c=2.0315, stream=None):
    """out = NS_steps(X/||X||_F) for one matrix, using the library's fixed
    device scratch instead of a workspace (for callers that cannot allocate
    device memory; see include/matrixopt.h for the size limit)."""
    if _ld(X) != _ld(out):
        raise MoError(MO_ERR_INVALID_ARG, "X and out must share the leading dimension")
    _check(load().ns_orthogonalize_noalloc(_ptr(X), _ptr(out), X.size(0), X.size(1), _ld(X),
                                           dtype_code(X.dtype), dtype_code(out.dtype), steps, a, b, c,
                                           _stream(stream)))


def ns_orthogonalize_noalloc_status(stream=None):
    """MO_OK, or MO_ERR_TIMEOUT if an allocation-free run's bounded device
    wait gave up since the last check (the record is then cleared)."""
    return load().ns_orthogonalize_noalloc_status(_stream(stream))


def sign_pack(U, words, stream=None):
    """Pack the signs of U (2D float32/bf16) into the uint32 words tensor
    (int32 storage, ceil(numel/32) entries)."""
    _check(load().sign_pack(_ptr(U), dtype_code(U.dtype), U.size(0), U.size(1), _ld(U),
                            _ptr(words), _stream(stream)))


def sign_vote_update(words, W, lr, stream=None):
    """W -= lr * majority_vote(words) for a list of packed word tensors."""
    M = len(words)
    arr = (c_void_p * max(1, M))(*[w.data_ptr() for w in words])
    _check(load().sign_vote_update(arr, M, W.size(0), W.size(1), _ptr(W), dtype_code(W.dtype),
                                   _ld(W), lr, _stream(stream)))


def sign_vote_polar_workspace_bytes(W):
    out = c_size_t(0)
    _check(load().sign_vote_polar_workspace_bytes(W.size(0), W.size(1), _ld(W), ctypes.byref(out)))
    return out.value


def sign_vote_polar_update(words, W, lr, ws, steps=5, a=3.4445, b=-4.7750, c=2.0315, stream=None):
    """W -= lr * NS(majority_vote(words)): the vote followed by the local polar step."""
    M = len(words)
    arr = (c_void_p * max(1, M))(*[w.data_ptr() for w in words])
    _check(load().sign_vote_polar_update(arr, M, W.size(0), W.size(1), _ptr(W), dtype_code(W.dtype), _ld(W),
                                         lr, steps, a, b, c, _ptr(ws), ws.numel() if ws is not None else 0,
                                         _stream(stream)))


def sign_pack_batched(U, words, stream=None):
    """sign_pack of M same-shaped matrices (lists U, words) in one launch."""
    M = len(U)
    us = (c_void_p * max(1, M))(*[u.data_ptr() for u in U])
    ws = (c_void_p * max(1, M))(*[w.data_ptr() for w in words])
    lds = {_ld(u) for u in U}
    if len(lds) != 1 or len({tuple(u.shape) for u in U}) != 1 or len({u.dtype for u in U}) != 1:
        raise MoError(MO_ERR_INVALID_ARG, "sign_pack_batched wants one shape, dtype and ld")
    _check(load().sign_pack_batched(us, M, dtype_code(U[0].dtype), U[0].size(0), U[0].size(1), lds.pop(),
                                    ws, _stream(stream)))


def sign_int8(U, out, stream=None):
    """int8 signs (-1/+1) of U into ``out`` (int8, rows*cols entries)."""
    _check(load().sign_int8(_ptr(U), dtype_code(U.dtype), U.size(0), U.size(1), _ld(U), _ptr(out),
                            _stream(stream)))


def sign_vote_update_int8(signs, W, lr, stream=None):
    """W -= lr * sign(sum of the workers' int8 signs), ties -> +1."""
    M = len(signs)
    arr = (c_void_p * max(1, M))(*[s.data_ptr() for s in signs])
    _check(load().sign_vote_update_int8(arr, M, W.size(0), W.size(1), _ptr(W), dtype_code(W.dtype),
                                        _ld(W), lr, _stream(stream)))


def plan_owners(shapes, world, ns_steps=5, w_bytes=1.0, w_flops=1.0):
    """Host-only owner plan: returns (owner list, per-rank load list)."""
    n = len(shapes)
    rows = (c_int64 * max(1, n))(*[s[0] for s in shapes])
    cols = (c_int64 * max(1, n))(*[s[1] for s in shapes])
    owner = (c_int32 * max(1, n))()
    load_ = (c_double * max(1, world))() if world > 0 else None
    _check(load().plan_owners(rows, cols, n, world, ns_steps, w_bytes, w_flops, owner, load_))
    return list(owner)[:n], list(load_)[:world]


# The training-step operators' calls are short, so their wrappers keep to few
# Python operations: plain integers for addresses (ctypes converts them) and
# one entry of _calls for each function, filled on first use.
_calls = {}


def _call(name):
    f = _calls.get(name)
    if f is None:
        f = _calls[name] = getattr(load(), name)
    return f


_current_raw_stream = torch._C._cuda_getCurrentRawStream   # current_stream() without building a Stream object
_current_device = torch._C._cuda_getDevice                 # (a CUDA tensor is at hand: initialised)
_DTYPES = {torch.float32: MO_F32, torch.bfloat16: MO_BF16}
_ID_DTYPES = {torch.int32: MO_I32, torch.int64: MO_I64}


def _invalid(msg):
    raise MoError(MO_ERR_INVALID_ARG, msg)


def _op_stream(stream, tensors):
    """Raw stream of a call whose tensors (the first is one, others may be None) share
    the current CUDA device (the library takes addresses only and launches there):
    `stream`, which must be of that device too, or its current one."""
    devices = [t.get_device() for t in tensors if t is not None]
    dev = devices[0]
    if dev < 0:
        _invalid("tensors must be on a CUDA device")
    if devices.count(dev) != len(devices):
        _invalid("tensors must share one CUDA device")
    if dev != _current_device():
        _invalid(f"tensors on cuda:{dev}, which is not the current device")
    if stream is None:
        return _current_raw_stream(dev)
    if stream.device.index != dev:
        _invalid(f"tensors on cuda:{dev}, stream on {stream.device}")
    return stream.cuda_stream


def _row_pitch(cols):
    """The leading dimension given for a single row, on which nothing depends: any aligned
    value, the same for every tensor of that row."""
    return (cols + 7) // 8 * 8


def _matrix(t, what):
    """(address, type code, rows, cols, ld) of a float32 or bf16 matrix."""
    try:
        (rows, cols), (ld, unit) = t.shape, t.stride()
    except ValueError:
        _invalid(f"{what} must be 2D")
    if unit != 1 and cols > 1:
        _invalid(f"{what} must have unit column stride")
    if rows <= 1:
        ld = _row_pitch(cols)
    code = _DTYPES.get(t.dtype)
    if code is None:
        _invalid(f"{what}: unsupported dtype {t.dtype}")
    return t.data_ptr(), code, rows, cols, ld


def _ids(t):
    """(address, type code, count) of a vector of token ids."""
    code = _ID_DTYPES.get(t.dtype)
    if code is None:
        _invalid(f"ids: unsupported dtype {t.dtype}")
    if t.dim() != 1 or not t.is_contiguous():
        _invalid("ids must be 1D and contiguous")
    return t.data_ptr(), code, t.shape[0]


def _size(name, *args):
    out = c_size_t(0)
    _check(_call(name)(*args, ctypes.byref(out)))
    return out.value


def _nbytes(ws):
    if not ws.is_contiguous():
        _invalid("a workspace must be contiguous")
    return ws.nbytes


def embedding_lookup(W, ids, out, scale=1.0, stream=None):
    """out[i] = scale * W[ids[i]] for W (vocab x dim), ids (n, int32 or int64)
    and out (n x dim); ids outside the table give zeros."""
    s = _op_stream(stream, (W, ids, out))
    w, w_code, vocab, dim, ldw = _matrix(W, "W")
    o, o_code, n, cols, ldo = _matrix(out, "out")
    i, i_code, count = _ids(ids)
    if n != count or cols != dim:
        _invalid("out must be len(ids) x dim")
    _check(_call("embedding_lookup")(w, w_code, vocab, dim, ldw, i, i_code, n, scale, o, o_code, ldo, s))


def embedding_grad_workspace_bytes(n, vocab, dim):
    return _size("embedding_grad_workspace_bytes", n, vocab, dim)


def embedding_grad(dY, ids, dW, ws, scale=1.0, accumulate=False, stream=None):
    """dW[v] (+)= scale * sum of dY[i] over ids[i] == v, dense (vocab x dim);
    a contiguous float32 dW is what make_tail takes as g."""
    s = _op_stream(stream, (dY, ids, dW, ws))
    y, y_code, n, dim, ldy = _matrix(dY, "dY")
    w, w_code, vocab, cols, ldw = _matrix(dW, "dW")
    i, i_code, count = _ids(ids)
    if n != count or cols != dim:
        _invalid("dY must be len(ids) x dim")
    _check(_call("embedding_grad")(y, y_code, n, dim, ldy, i, i_code, vocab, scale, w, w_code, ldw,
                                   1 if accumulate else 0, ws.data_ptr(), _nbytes(ws), s))


def expert_linear_workspace_bytes(rows, n, k, experts):
    return _size("expert_linear_workspace_bytes", rows, n, k, experts)


def _stack(t, what):
    """(address, type code, experts, rows, cols, ld, stride) of a stack of matrices."""
    if t.dim() != 3:
        _invalid(f"{what} must be 3D")
    (experts, rows, cols), (stride, ld, unit) = t.shape, t.stride()
    if cols > 1 and unit != 1:
        _invalid(f"{what} must have unit column stride")
    if rows <= 1:
        ld = stride if rows == 1 and experts > 1 else _row_pitch(cols)   # (the stride's own checks hold for it)
    if experts <= 1 or rows == 0:
        stride = rows * ld
    code = _DTYPES.get(t.dtype)
    if code is None:
        _invalid(f"{what}: unsupported dtype {t.dtype}")
    return t.data_ptr(), code, experts, rows, cols, ld, stride


def _offsets(offsets, experts):
    if offsets.dtype != torch.int32 or offsets.shape != (experts + 1,) or not offsets.is_contiguous():
        _invalid("offsets must be experts + 1 contiguous int32")
    return offsets.data_ptr()


def expert_linear(X, W, offsets, Y, ws, stream=None):
    """Y[r] = X[r] W_e^T for the rows r of expert e (offsets[e] .. offsets[e+1] - 1):
    X rows x k and W experts x n x k in bf16, Y rows x n float32 or bf16."""
    s = _op_stream(stream, (X, W, offsets, Y, ws))
    x, x_code, rows, k, ldx = _matrix(X, "X")
    y, y_code, y_rows, y_cols, ldy = _matrix(Y, "Y")
    w, w_code, experts, n, w_cols, ldw, stride = _stack(W, "W")
    if x_code != MO_BF16 or w_code != MO_BF16:
        _invalid("operands must be bfloat16")
    if y_rows != rows or w_cols != k or y_cols != n:
        _invalid("X must be rows x k and Y rows x n of W's experts x n x k")
    _check(_call("expert_linear")(x, ldx, w, ldw, stride, _offsets(offsets, experts), rows, n, k, experts, y, y_code,
                                  ldy, ws.data_ptr(), _nbytes(ws), s))


def expert_linear_dgrad(dY, W, offsets, dX, ws, stream=None):
    """dX[r] = dY[r] W_e: the input's gradient of expert_linear."""
    s = _op_stream(stream, (dY, W, offsets, dX, ws))
    y, y_code, rows, n, ldy = _matrix(dY, "dY")
    x, x_code, x_rows, k, ldx = _matrix(dX, "dX")
    w, w_code, experts, w_rows, w_cols, ldw, stride = _stack(W, "W")
    if y_code != MO_BF16 or w_code != MO_BF16:
        _invalid("operands must be bfloat16")
    if x_rows != rows or w_rows != n or w_cols != k:
        _invalid("dY must be rows x n and dX rows x k of W's experts x n x k")
    _check(_call("expert_linear_dgrad")(y, ldy, w, ldw, stride, _offsets(offsets, experts), rows, n, k, experts, x,
                                        x_code, ldx, ws.data_ptr(), _nbytes(ws), s))


def expert_linear_wgrad(dY, X, offsets, dW, ws, accumulate=False, stream=None):
    """dW[e] (+)= dY_e^T X_e: the weights' gradients of expert_linear; each dW[e]
    is the G of one make_matrix."""
    s = _op_stream(stream, (dY, X, offsets, dW, ws))
    y, y_code, rows, n, ldy = _matrix(dY, "dY")
    x, x_code, x_rows, k, ldx = _matrix(X, "X")
    w, w_code, experts, w_rows, w_cols, ldw, stride = _stack(dW, "dW")
    if y_code != MO_BF16 or x_code != MO_BF16:
        _invalid("operands must be bfloat16")
    if x_rows != rows or w_rows != n or w_cols != k:
        _invalid("dY must be rows x n and X rows x k of dW's experts x n x k")
    _check(_call("expert_linear_wgrad")(y, ldy, x, ldx, _offsets(offsets, experts), rows, n, k, experts, w, w_code,
                                        ldw, stride, 1 if accumulate else 0, ws.data_ptr(), _nbytes(ws), s))


def _distill(logits, idx, teacher, temperature, row_weight, grad_scale):
    p, code, n, vocab, ld = _matrix(logits, "logits")
    t_code, i_code = _DTYPES.get(teacher.dtype), _ID_DTYPES.get(idx.dtype)
    if t_code is None or i_code is None:
        _invalid("teacher must be float32 or bfloat16, idx int32 or int64")
    if (idx.dim() != 2 or idx.shape != teacher.shape or idx.shape[0] != n or not idx.is_contiguous() or
            not teacher.is_contiguous()):
        _invalid("idx and teacher must be contiguous, rows x top")
    w = None
    if row_weight is not None:
        if row_weight.dtype != torch.float32 or row_weight.shape != (n,) or not row_weight.is_contiguous():
            _invalid("row_weight must be contiguous float32, one per row")
        w = row_weight.data_ptr()
    return mo_distill(n, vocab, ld, idx.shape[1], code, i_code, t_code, temperature, grad_scale, p, idx.data_ptr(),
                      teacher.data_ptr(), w)


def _f32_out(t, shape, name):
    if t.dtype != torch.float32 or t.shape != shape or not t.is_contiguous():
        _invalid(f"{name} must be contiguous float32 of shape {shape}")
    return t.data_ptr()


def _dlogits(dlogits, logits):
    if dlogits.shape != logits.shape:
        _invalid("dlogits must have the logits' shape")
    p, code, _, _, ld = _matrix(dlogits, "dlogits")
    return p, code, ld


def distill_topk_loss(logits, idx, teacher, loss, stats, temperature=1.0, row_weight=None, stream=None):
    """Per-row distillation loss from the teacher's top logits (include/matrixopt.h)
    and the row statistics distill_topk_grad takes (rows x 2)."""
    s = _op_stream(stream, (logits, idx, teacher, loss, stats) + (() if row_weight is None else (row_weight,)))
    d = _distill(logits, idx, teacher, temperature, row_weight, 1.0)
    _check(_call("distill_topk_loss")(d, _f32_out(loss, (d.n,), "loss"), _f32_out(stats, (d.n, 2), "stats"), s))


def distill_topk_grad(logits, idx, teacher, stats, dlogits, temperature=1.0, row_weight=None, grad_scale=1.0,
                      stream=None):
    """The loss's gradient by the logits, from distill_topk_loss's statistics;
    dlogits may be the logits themselves."""
    s = _op_stream(stream, (logits, idx, teacher, stats, dlogits) + (() if row_weight is None else (row_weight,)))
    d = _distill(logits, idx, teacher, temperature, row_weight, grad_scale)
    g, code, ld = _dlogits(dlogits, logits)
    _check(_call("distill_topk_grad")(d, _f32_out(stats, (d.n, 2), "stats"), g, code, ld, s))


def distill_topk_loss_grad(logits, idx, teacher, loss, dlogits, temperature=1.0, row_weight=None, grad_scale=1.0,
                           stream=None):
    """Loss and gradient in one call, which reads the logits a second time mostly from L2;
    dlogits may be the logits."""
    s = _op_stream(stream, (logits, idx, teacher, loss, dlogits) + (() if row_weight is None else (row_weight,)))
    d = _distill(logits, idx, teacher, temperature, row_weight, grad_scale)
    g, code, ld = _dlogits(dlogits, logits)
    _check(_call("distill_topk_loss_grad")(d, _f32_out(loss, (d.n,), "loss"), g, code, ld, s))


def expert_route_workspace_bytes(n, experts, top):
    return _size("expert_route_workspace_bytes", n, experts, top)


_I32, _F32, _MASKS = torch.int32, torch.float32, (torch.bool, torch.uint8)


def _dense(t, dtype, shape, name):
    """Address of a contiguous tensor of that type and shape."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _invalid(f"{name} must be contiguous {dtype} of shape {shape}")
    return t.data_ptr()


def _route(logits, top, mask, renormalise):
    p, code, n, experts, ld = _matrix(logits, "logits")
    m = 0
    if mask is not None:
        if mask.dtype not in _MASKS or mask.shape != (n,) or not mask.is_contiguous():
            _invalid("mask must be contiguous bool or uint8, one per row")
        m = mask.data_ptr()
    return _pack_route(n, ld, experts, top, code, 1 if renormalise else 0, p, m), n, experts


def expert_route(logits, idx, gates, pos, offsets, counts, loss, ws, order=None, mask=None, renormalise=False,
                 stream=None):
    """Routes each row of logits (n x experts) to its `top` experts of largest logit
    (idx.shape[1]): idx, gates (float32) and pos are n x top, offsets and counts
    experts + 1 int32, loss two float32 (balance, z) or None, order n * top int32 or
    None; see include/matrixopt.h."""
    s = _op_stream(stream, (logits, idx, gates, pos, offsets, counts, ws, loss, order, mask))
    if idx.dim() != 2:
        _invalid("idx must be rows x top")
    rows, top = each = idx.shape
    r, n, experts = _route(logits, top, mask, renormalise)
    if n != rows:
        _invalid("idx must have a row for each of the logits'")
    ends = (experts + 1,)
    _check(_call("expert_route")(
        r, _dense(idx, _I32, each, "idx"), _dense(gates, _F32, each, "gates"), _dense(pos, _I32, each, "pos"),
        None if order is None else _dense(order, _I32, (n * top,), "order"), _dense(offsets, _I32, ends, "offsets"),
        _dense(counts, _I32, ends, "counts"), None if loss is None else _dense(loss, _F32, (2,), "loss"),
        ws.data_ptr(), _nbytes(ws), s))


def expert_route_grad(logits, idx, counts, dgates, dlogits, mask=None, renormalise=False, balance_coef=0.0, z_coef=0.0,
                      stream=None):
    """dlogits = gradient of sum(dgates * gates) + balance_coef * balance + z_coef * z by
    the logits; dgates (n x top float32) may be None, dlogits may be the logits."""
    s = _op_stream(stream, (logits, idx, counts, dlogits, dgates, mask))
    if idx.dim() != 2:
        _invalid("idx must be rows x top")
    top = idx.shape[1]
    r, n, experts = _route(logits, top, mask, renormalise)
    each = (n, top)
    g, code, ld = _dlogits(dlogits, logits)
    _check(_call("expert_route_grad")(r, _dense(idx, _I32, each, "idx"), _dense(counts, _I32, (experts + 1,), "counts"),
                                      None if dgates is None else _dense(dgates, _F32, each, "dgates"), balance_coef,
                                      z_coef, g, code, ld, s))


def _places(pos, n):
    shape = pos.shape
    if pos.dtype is not _I32 or len(shape) != 2 or shape[0] != n or not pos.is_contiguous():
        _invalid("pos must be contiguous int32, rows x top")
    return pos.data_ptr(), shape[1]


def expert_scatter(X, pos, Xs, stream=None):
    """Xs[pos[r, j]] = X[r]: each row of X (n x dim) to its places among the rows sorted
    by expert; places outside Xs are absent."""
    s = _op_stream(stream, (X, pos, Xs))
    x, x_code, n, dim, ldx = _matrix(X, "X")
    y, y_code, slots, cols, ldy = _matrix(Xs, "Xs")
    if cols != dim:
        _invalid("X and Xs must have rows of one length")
    p, top = _places(pos, n)
    _check(_call("expert_scatter")(x, x_code, n, dim, ldx, p, top, y, y_code, slots, ldy, s))


def expert_combine(Ys, pos, Y, gates=None, accumulate=False, stream=None):
    """Y[r] (+)= sum over j of gates[r, j] * Ys[pos[r, j]]; without gates the gradient of
    expert_scatter."""
    s = _op_stream(stream, (Ys, pos, Y, gates))
    x, x_code, slots, cols, ldx = _matrix(Ys, "Ys")
    y, y_code, n, dim, ldy = _matrix(Y, "Y")
    if cols != dim:
        _invalid("Y and Ys must have rows of one length")
    p, top = _places(pos, n)
    _check(_call("expert_combine")(x, x_code, slots, ldx, p,
                                   None if gates is None else _dense(gates, _F32, (n, top), "gates"), n, top, dim, y,
                                   y_code, ldy, 1 if accumulate else 0, s))


def expert_combine_grad(dY, Ys, pos, gates, dYs, dgates, stream=None):
    """dYs[pos[r, j]] = gates[r, j] * dY[r] and dgates[r, j] = dY[r] . Ys[pos[r, j]]; gates may
    be None (1), dgates None (not wanted), dYs may be Ys itself."""
    s = _op_stream(stream, (dY, Ys, pos, dYs, gates, dgates))
    d, d_code, n, dim, ldd = _matrix(dY, "dY")
    x, x_code, slots, cols, ldx = _matrix(Ys, "Ys")
    y, y_code, y_slots, y_cols, ldy = _matrix(dYs, "dYs")
    if (cols, y_cols) != (dim, dim) or y_slots != slots or y_code != x_code:
        _invalid("dYs must have Ys's shape and type, and their rows the length of dY's")
    p, top = _places(pos, n)
    _check(_call("expert_combine_grad")(d, d_code, ldd, x, x_code, slots, ldx, p,
                                        None if gates is None else _dense(gates, _F32, (n, top), "gates"), n, top, dim, y,
                                        ldy, None if dgates is None else _dense(dgates, _F32, (n, top), "dgates"), s))


def _gain(t, shape, name, dtype):
    """(address, type) of a gain vector, whose type is that of the other parameters."""
    own = t.dtype
    if own not in _DTYPES or t.shape != shape or not t.is_contiguous():
        _invalid(f"{name} must be {shape[0]} contiguous float32 or bfloat16 values")
    if own is not dtype and dtype is not None:
        _invalid("post, gate and pre must have one type")
    return t.data_ptr(), own


def _norm_args(x, post, gate, pre, eps, residual_scale, block_scale, rows_per_gate):
    """The values of mo_block_norm, those of the stream to be filled in, and x's shape, its type and
    the rows of gate."""
    x_p, code, n, dim, ldx = _matrix(x, "x")
    vector = (dim,)
    post_p = gate_p = pre_p = 0
    dtype = None
    ldgate, gates = dim, 0
    if post is not None:
        post_p, dtype = _gain(post, vector, "post", dtype)
    if pre is not None:
        pre_p, dtype = _gain(pre, vector, "pre", dtype)
    if gate is not None:
        if gate.dim() == 1:
            gate_p, dtype = _gain(gate, vector, "gate", dtype)
            gates = 1
        else:
            gate_p, _, gates, cols, ldgate = _matrix(gate, "gate")
            if dtype is not None and gate.dtype is not dtype:
                _invalid("post, gate and pre must have one type")
            dtype = gate.dtype
            if cols != dim:
                _invalid("gate must have rows of x's length")
        if rows_per_gate is None:
            if n > 0 and (gates == 0 or n % gates):
                _invalid("rows_per_gate is needed where the gate's rows do not divide x's")
            rows_per_gate = n // gates if n > 0 else 1
        if rows_per_gate < 1 or (n > 0 and gates != -(-n // rows_per_gate)):
            _invalid("gate must be ceil(rows / rows_per_gate) x dim")
    values = [n, dim, ldx, 0, rows_per_gate or 1, ldgate, code, MO_F32, _DTYPES.get(dtype, MO_F32), eps, residual_scale,
              block_scale, x_p, 0, post_p, gate_p, pre_p]
    return values, x.shape, code, gates


def _like(t, shape, what, code):
    """(address, ld, type code) of an optional matrix of that shape, whose type is `code` unless
    that is None: then the type that is returned is wanted of the next."""
    if t is None:
        return None, shape[1], code
    if t.shape != shape:
        _invalid(f"{what} must have x's shape")
    rows, cols = shape
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        _invalid(f"{what} must have unit column stride")
    own = _DTYPES.get(t.dtype)
    if own is None or (own != code and code is not None):
        _invalid(f"{what}: unsupported dtype {t.dtype}, or another than the matrices it goes with")
    return t.data_ptr(), ld if rows > 1 else _row_pitch(cols), own


def block_norm(x, y, h, residual=None, post=None, gate=None, pre=None, eps=1e-6, residual_scale=1.0, block_scale=1.0,
               rows_per_gate=None, stream=None):
    """y = residual_scale * residual + block_scale * gate * post * norm(x) and h = pre * norm(y)
    over rows (norm by the root mean square).  post, gate, pre and residual may be None, and y
    or (with pre) h; gate is dim values or a row for every rows_per_gate rows of x.  y may be
    the residual, h may be x."""
    s = _op_stream(stream, (x, y, h, residual, post, gate, pre))
    p, shape, code, _ = _norm_args(x, post, gate, pre, eps, residual_scale, block_scale, rows_per_gate)
    y_p, ldy, stream_code = _like(y, shape, "y", None)
    r_p, p[3], stream_code = _like(residual, shape, "residual", stream_code)
    h_p, ldh, _ = _like(h, shape, "h", code)
    p[7], p[13] = stream_code or MO_F32, r_p or 0
    _check(_call("block_norm")(_pack_norm(*p), y_p, ldy, h_p, ldh, s))


def block_norm_grad_workspace_bytes(n, dim, gates):
    return _size("block_norm_grad_workspace_bytes", n, dim, gates)


def block_norm_grad(x, y, dy, dh, dx, ws, dresidual=None, post=None, gate=None, pre=None, dpost=None, dgate=None,
                    dpre=None, eps=1e-6, residual_scale=1.0, block_scale=1.0, rows_per_gate=None, accumulate=False,
                    stream=None):
    """block_norm's gradients from x, the y it wrote (None without pre), dy (or None) and dh
    (None without pre): dx, dresidual (or None; may be dy), and the float32 gradients of the
    parameters (each may be None; accumulate=True adds to them).  Without rows these are 0, dgate
    with all rows that it has."""
    s = _op_stream(stream, (x, dx, ws, y, dy, dh, dresidual, post, gate, pre, dpost, dgate, dpre))
    p, shape, code, gates = _norm_args(x, post, gate, pre, eps, residual_scale, block_scale, rows_per_gate)
    y_p, ldy, stream_code = _like(y, shape, "y", None)
    dy_p, lddy, stream_code = _like(dy, shape, "dy", stream_code)
    dr_p, lddr, stream_code = _like(dresidual, shape, "dresidual", stream_code)
    dh_p, lddh, _ = _like(dh, shape, "dh", code)
    dx_p, lddx, _ = _like(dx, shape, "dx", code)
    p[7] = stream_code or MO_F32
    vector = (shape[1],)
    if dgate is not None:
        each = vector if gates == 1 and dgate.dim() == 1 else (gates, shape[1])
    _check(_call("block_norm_grad")(
        _pack_norm(*p), y_p, ldy, dy_p, lddy, dh_p, lddh, dx_p, lddx, dr_p, lddr,
        None if dpost is None else _dense(dpost, _F32, vector, "dpost"),
        None if dgate is None else _dense(dgate, _F32, each, "dgate"),
        None if dpre is None else _dense(dpre, _F32, vector, "dpre"), 1 if accumulate else 0, ws.data_ptr(), _nbytes(ws),
        s))
    if shape[0] == 0 and dgate is not None and not accumulate:
        # the library takes a gate's rows from x's (none here), a tensor has its own
        if stream is None:
            dgate.zero_()
        else:
            with torch.cuda.stream(stream):
                dgate.zero_()


ADAMW_BLOCK = 256      # values of one scale of the 8-bit states


def make_adamw_tensor(W, g, m, v, m_scale=None, v_scale=None, lr=1e-3, weight_decay=0.0):
    """mo_adamw_tensor for one parameter: W and g contiguous float32 or bfloat16, and the
    states m and v float32, or float8_e4m3fn with a float32 scale in m_scale and v_scale for
    each ADAMW_BLOCK values (zeros to begin with)."""
    n = W.numel()
    for t, name in ((W, "W"), (g, "g"), (m, "m"), (v, "v")):
        if t.numel() != n or not t.is_contiguous():
            _invalid(f"{name} must be contiguous, of W's size")
    w_code, g_code = _DTYPES.get(W.dtype), _DTYPES.get(g.dtype)
    if w_code is None or g_code is None:
        _invalid("W and g must be float32 or bfloat16")
    if m.dtype != v.dtype or m.dtype not in (torch.float32, torch.float8_e4m3fn):
        _invalid("m and v must both be float32 or both float8_e4m3fn")
    scales = ()
    if m.dtype == torch.float32:
        if m_scale is not None or v_scale is not None:
            _invalid("float32 states have no scales")
    else:
        if m_scale is None or v_scale is None:
            _invalid("float8_e4m3fn states need m_scale and v_scale")
        scales = (m_scale, v_scale)
        for t in scales:
            _dense(t, _F32, (-(-n // ADAMW_BLOCK),), "a scale")
    t = mo_adamw_tensor(n, W.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr(),
                        *([c.data_ptr() for c in scales] or [None, None]), w_code, g_code,
                        MO_E4M3 if scales else MO_F32, lr, weight_decay, 0)
    t.tensors = (W, g, m, v) + scales
    return t


def _check_apart(written, read):
    """Refuses contiguous tensors that are written and overlap, with each other or with one that is read."""
    spans = sorted([(t.data_ptr(), t.nbytes) for t in written])
    begins, ends = [at for at, size in spans if size], [at + size for at, size in spans if size]
    apart = all(map(int.__le__, ends, begins[1:]))
    for t in read if apart else ():
        at, size = t.data_ptr(), t.nbytes
        k = bisect.bisect_right(begins, at)                    # the spans before k begin at or before t
        if size and ((k > 0 and ends[k - 1] > at) or (k < len(begins) and begins[k] < at + size)):
            apart = False
    if not apart:
        _invalid("the tensors that are written must overlap neither each other nor a gradient (is one of them in the "
                 "list twice?)")


class adamw_tensors:
    """A list of make_adamw_tensor results laid out once, for adamw_step_batched; it keeps
    their tensors alive.  `array` holds the descriptors, which every call reads anew: a rate that changes
    is written to array[i].lr (or .weight_decay) between steps.  A captured step keeps those of its capture."""

    def __init__(self, tensors):
        self.count = len(tensors)
        self.array = (mo_adamw_tensor * max(1, self.count))(*tensors)
        self.tensors = [t for d in tensors for t in d.tensors]
        devices = {t.get_device() for t in self.tensors}
        if len(devices) > 1 or min(devices, default=0) < 0:
            _invalid("tensors must share one CUDA device")
        _check_apart([t for d in tensors for t in d.tensors[:1] + d.tensors[2:]], [d.tensors[1] for d in tensors])


def adamw_step_batched(tensors, step, beta1=0.9, beta2=0.95, eps=1e-8, grad_scale=1.0, grad_mul=None, seed=None,
                       stream=None):
    """One AdamW step at step number `step` (>= 1; or a CUDA int64 tensor of one value, read on
    the device) for a list of make_adamw_tensor results or an adamw_tensors.  The gradients are
    scaled by grad_scale and by *grad_mul (a CUDA float32 tensor of one value).  With a seed the
    8-bit states are rounded at random, else to nearest."""
    if not isinstance(tensors, adamw_tensors):
        tensors = adamw_tensors(tensors)
    if tensors.count == 0:
        return
    scalars = ()
    step_ptr = mul = 0
    if isinstance(step, torch.Tensor):
        if step.dtype != torch.int64 or step.numel() != 1:
            _invalid("step must be a number or one int64 value")
        scalars, step_ptr, step = (step,), step.data_ptr(), 0
    if grad_mul is not None:
        if grad_mul.dtype != torch.float32 or grad_mul.numel() != 1:
            _invalid("grad_mul must be one float32 value")
        scalars += (grad_mul,)
        mul = grad_mul.data_ptr()
    s = _op_stream(stream, (tensors.tensors[0],) + scalars)
    cfg = _pack_adamw_cfg(beta1, beta2, eps, grad_scale, step, step_ptr, mul, 0 if seed is None else seed & 0xFFFFFFFF,
                          0 if seed is None else 1)
    _check(_call("adamw_step_batched")(tensors.array, tensors.count, cfg, s))


def mo_check_device_status(ws, stream=None):
    """Returns the status word the kernels left in ``ws`` (and clears it)."""
    return load().mo_check_device_status(_ptr(ws), _stream(stream))


def mo_debug_ns_view(shapes, index, precision=MO_NS_BF16):
    n = len(shapes)
    rows = (c_int64 * max(1, n))(*[s[0] for s in shapes])
    cols = (c_int64 * max(1, n))(*[s[1] for s in shapes])
    v = mo_ns_view()
    _check(load().mo_debug_ns_view(rows, cols, n, precision, index, ctypes.byref(v)))
    return v


def mo_debug_inject_dep_stall(matrix, wait_cycles=2_000_000):
    """Makes the fused NS launch's dependency waits of matrix `matrix` run out
    after `wait_cycles` SM cycles (matrix -1 turns it off)."""
    _check(load().mo_debug_inject_dep_stall(matrix, wait_cycles))


def mo_debug_set_ns_pair(on):
    """Selects 256 x 256 CTA-pair tiles (True) or 128 x 256 single-CTA tiles
    (False) for the NS kernel; returns the previous setting."""
    prev = load().mo_debug_set_ns_pair(1 if on else 0)
    _check(prev if prev < 0 else 0)
    return bool(prev)


def mo_debug_set_ns_fused(on):
    """Selects the NS launch schedule: 1 / True fused with per-matrix
    counters, 2 fused with grid-wide counters, 3 (default) either by size,
    0 / False one launch per phase; returns the previous setting."""
    prev = load().mo_debug_set_ns_fused(int(on))
    _check(prev if prev < 0 else 0)
    return prev


def mo_debug_set_expert_shape(shape):
    """Tile geometry of the expert products: 0 single CTAs, 1 CTA pairs, 2 few
    tokens, -1 (default) by the sizes; returns the previous setting."""
    prev = load().mo_debug_set_expert_shape(int(shape))
    _check(prev if prev < 0 else 0)
    return prev - 1


def mo_debug_cta_stamps(buf, capacity, max_ctas):
    """Start recording per-CTA stamps (start, end, dependency-wait ns,
    spinning waits) into ``buf`` (int64 CUDA tensor of 4*capacity*max_ctas
    entries); ``buf=None`` stops.  Returns the number of launches recorded
    since the previous call."""
    rec = c_int32(0)
    _check(load().mo_debug_cta_stamps(_ptr(buf), capacity, max_ctas, ctypes.byref(rec)))
    return rec.value


def mo_trace_enable(capacity):
    """Record a CUDA event pair around each of the next ``capacity`` launches
    issued from this thread (0 disables)."""
    _check(load().mo_trace_enable(capacity))


def mo_trace_read(cap=1 << 16):
    """[(kind name, milliseconds), ...] of the launches traced since the last read."""
    kinds = (c_int32 * cap)()
    ms = (c_float * cap)()
    count = c_int32(0)
    _check(load().mo_trace_read(kinds, ms, cap, ctypes.byref(count)))
    return [(TRACE_KINDS.get(kinds[i], str(kinds[i])), ms[i]) for i in range(min(cap, count.value))]
