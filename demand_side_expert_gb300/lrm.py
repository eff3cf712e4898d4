"""ctypes binding of liblrm.so: argument marshalling only.

Every function has the name and argument order of its C entry point in
include/lrm.h; tensors are passed as device pointers (torch tensors are
accepted and their data_ptr() is used), ``stream`` defaults to torch's
current CUDA stream. A status other than LRM_OK raises LrmError. The library
is required: importing this module without a built liblrm.so raises.
"""

from __future__ import annotations

import ctypes
import os

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblrm.so")

LRM_OK, LRM_ERR_INVALID_ARG, LRM_ERR_UNSUPPORTED, LRM_ERR_WORKSPACE, LRM_ERR_CUDA = range(5)
LRM_F32, LRM_BF16 = 0, 1
LRM_DEVERR_EXPERT_ID, LRM_DEVERR_QUOTA, LRM_DEVERR_INDEX, LRM_DEVERR_TIMEOUT = 1, 2, 4, 8
LRM_DEVERR_QUEUE = 16

# Every symbol include/lrm.h declares.
EXPORTS = (
    "lrm_workspace_bytes", "lrm_clear_device_error", "lrm_get_device_error",
    "lrm_status_string", "lrm_dispatch_permute", "lrm_permute_rows",
    "lrm_quota_from_rate", "lrm_score", "lrm_select_quota", "lrm_compact",
    "lrm_expert_bwd_grouped", "lrm_expert_fc2_dgrad", "lrm_expert_fc2_wgrad",
    "lrm_expert_fc1_wgrad", "lrm_expert_fc1_dgrad", "lrm_scatter_dx",
    "lrm_dispatch_permute_noalloc", "lrm_selftest_wait_timeout", "lrm_score_variant",
    "lrm_gather_tokens", "lrm_expert_fc1_fwd", "lrm_expert_fc2_fwd", "lrm_combine",
    "lrm_expert_fwd_grouped", "lrm_expert_fc1_recompute", "lrm_expert_bwd_gathered",
    "lrm_select_rate", "lrm_router_workspace_bytes", "lrm_route", "lrm_route_bwd",
    "lrm_gate_grad", "lrm_norm_workspace_bytes", "lrm_add_rmsnorm", "lrm_add_rmsnorm_bwd",
    "lrm_adamw_step",
)
LRM_BWD_FC2_DGRAD, LRM_BWD_FC2_WGRAD, LRM_BWD_FC1_WGRAD = 1, 2, 4
LRM_BWD_FC1_DGRAD, LRM_BWD_SCATTER_DX, LRM_BWD_ALL = 8, 16, 31
LRM_METRIC_LRM, LRM_METRIC_GRAD_SQ, LRM_METRIC_GRAD_ABS, LRM_METRIC_RANDOM = range(4)
LRM_NOALLOC_MAX_CHUNK_ENTRIES = 65536
LRM_STATE_F32, LRM_STATE_F8 = 0, 1


class LrmError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {status_string(status)}")


class lrm_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("D", ctypes.c_int32), ("H", ctypes.c_int32),
                ("E", ctypes.c_int32), ("K", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class lrm_router(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("K", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("stride", ctypes.c_int64),
                ("renorm", ctypes.c_int32), ("balance_coef", ctypes.c_float),
                ("z_coef", ctypes.c_float)]


class lrm_norm(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("D", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("q_cols", ctypes.c_int32),
                ("eps", ctypes.c_float), ("x_stride", ctypes.c_int64),
                ("res_stride", ctypes.c_int64)]


class lrm_adamw_tensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("master", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("state", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("weight_decay", ctypes.c_double)]


class lrm_adamw(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64),
                ("grad_scale", ctypes.c_void_p)]


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"liblrm.so not built at {_LIB_PATH}; run "
            "`python -m demand_side_expert_gb300.build` (needs nvcc)")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
    sp = ctypes.POINTER(lrm_shape)
    rp, np_ = ctypes.POINTER(lrm_router), ctypes.POINTER(lrm_norm)
    ap, tp = ctypes.POINTER(lrm_adamw), ctypes.POINTER(lrm_adamw_tensor)
    sig = {
        "lrm_workspace_bytes": (sz, [sp]),
        "lrm_clear_device_error": (i32, [vp, sz, vp]),
        "lrm_get_device_error": (i32, [vp, sz, ctypes.POINTER(i32), vp]),
        "lrm_status_string": (ctypes.c_char_p, [i32]),
        "lrm_dispatch_permute": (i32, [sp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "lrm_permute_rows": (i32, [vp, i32, vp, vp, i64, vp]),
        "lrm_quota_from_rate": (i32, [vp, i32, i32, i32, i32, vp, vp]),
        "lrm_score": (i32, [sp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "lrm_select_quota": (i32, [sp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "lrm_compact": (i32, [sp] + [vp] * 15 + [vp, sz, vp]),
        "lrm_expert_bwd_grouped": (i32, [sp] + [vp] * 16 + [vp, sz, vp]),
        "lrm_expert_fc2_dgrad": (i32, [sp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "lrm_expert_fc2_wgrad": (i32, [sp, vp, vp, vp, vp, vp, sz, vp]),
        "lrm_expert_fc1_wgrad": (i32, [sp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "lrm_expert_fc1_dgrad": (i32, [sp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "lrm_scatter_dx": (i32, [sp, vp, vp, vp, vp, vp, sz, vp]),
        "lrm_dispatch_permute_noalloc": (i32, [sp, vp, vp, vp, vp, vp, vp, vp]),
        "lrm_selftest_wait_timeout": (i32, [vp, sz, vp]),
        "lrm_score_variant": (i32, [sp, i32, ctypes.c_uint64, vp, vp, vp, vp, vp, vp, sz, vp]),
        "lrm_gather_tokens": (i32, [sp, vp, vp, vp, vp, sz, vp]),
        "lrm_expert_fc1_fwd": (i32, [sp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "lrm_expert_fc2_fwd": (i32, [sp, vp, vp, vp, vp, vp, sz, vp]),
        "lrm_combine": (i32, [sp, vp, vp, vp, vp, vp, sz, vp]),
        "lrm_expert_fwd_grouped": (i32, [sp] + [vp] * 13 + [vp, sz, vp]),
        "lrm_expert_fc1_recompute": (i32, [sp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "lrm_expert_bwd_gathered": (i32, [sp, i32] + [vp] * 18 + [vp, sz, vp]),
        "lrm_select_rate": (i32, [sp, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]),
        "lrm_router_workspace_bytes": (sz, [rp]),
        "lrm_route": (i32, [rp] + [vp] * 8 + [sz, vp]),
        "lrm_route_bwd": (i32, [rp] + [vp] * 8 + [sz, vp]),
        "lrm_gate_grad": (i32, [sp] + [vp] * 5 + [sz, vp]),
        "lrm_norm_workspace_bytes": (sz, [np_]),
        "lrm_add_rmsnorm": (i32, [np_] + [vp] * 9),
        "lrm_add_rmsnorm_bwd": (i32, [np_] + [vp] * 8 + [sz, vp]),
        "lrm_adamw_step": (i32, [ap, tp, i32, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib = _load()


def library_path() -> str:
    return _LIB_PATH


def _p(x):
    """Device pointer of a tensor (or an int address, or None)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _current_stream_fn():
    """A function that returns torch's current stream as an address. The one that
    torch's own compiled kernels are launched with takes 0.2 us, making a Stream
    object for it (the public way, kept where the other is missing) 3 us: more than
    a launch."""
    import torch

    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    if raw is None or device is None:
        return lambda: torch.cuda.current_stream().cuda_stream
    torch.cuda.init()
    return lambda: raw(device())


_current_stream = None


def current_device() -> int:
    """Index of the device that kernels launch on: torch's current one."""
    global _current_device
    if _current_device is None:
        import torch

        torch.cuda.init()
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return _current_device()


_current_device = None


def _s(stream):
    if stream is None:
        global _current_stream
        if _current_stream is None:
            _current_stream = _current_stream_fn()
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, status: int):
    if status != LRM_OK:
        raise LrmError(fn, status)


def entry(name: str):
    """An entry point for callers that keep its arguments as ctypes ones (descriptors
    by reference, addresses, the stream): no marshalling, the same errors."""
    fn = getattr(_lib, name)

    def call(*args):
        status = fn(*args)
        if status != LRM_OK:
            raise LrmError(name, status)

    return call


def stream_address(stream=None) -> int:
    """Address of a stream (a torch stream, an address, None: torch's current one)."""
    return _s(stream)


def make_shape(T: int, D: int, H: int, E: int, K: int, dtype: int) -> lrm_shape:
    return lrm_shape(T, D, H, E, K, dtype)


def status_string(status: int) -> str:
    return _lib.lrm_status_string(status).decode()


def lrm_status_string(status: int) -> str:
    return status_string(status)


def lrm_workspace_bytes(shape: lrm_shape) -> int:
    return int(_lib.lrm_workspace_bytes(ctypes.byref(shape)))


def lrm_clear_device_error(ws, ws_bytes: int, stream=None):
    _check("lrm_clear_device_error", _lib.lrm_clear_device_error(_p(ws), ws_bytes, _s(stream)))


def lrm_get_device_error(ws, ws_bytes: int, stream=None) -> int:
    out = ctypes.c_int32(0)
    _check("lrm_get_device_error",
           _lib.lrm_get_device_error(_p(ws), ws_bytes, ctypes.byref(out), _s(stream)))
    return int(out.value)


def lrm_dispatch_permute(shape, topk_idx, perm, inv, counts, off, ws, ws_bytes, stream=None):
    _check("lrm_dispatch_permute", _lib.lrm_dispatch_permute(
        ctypes.byref(shape), _p(topk_idx), _p(perm), _p(inv), _p(counts), _p(off),
        _p(ws), ws_bytes, _s(stream)))


def lrm_permute_rows(perm, n_rows: int, src, dst, row_bytes: int, stream=None):
    _check("lrm_permute_rows", _lib.lrm_permute_rows(
        _p(perm), n_rows, _p(src), _p(dst), row_bytes, _s(stream)))


def lrm_quota_from_rate(counts, E: int, num: int, den: int, cap: int, quota, stream=None):
    _check("lrm_quota_from_rate", _lib.lrm_quota_from_rate(
        _p(counts), E, num, den, cap, _p(quota), _s(stream)))


def lrm_score(shape, g, phi, alpha, inv, score, ws, ws_bytes, stream=None):
    _check("lrm_score", _lib.lrm_score(
        ctypes.byref(shape), _p(g), _p(phi), _p(alpha), _p(inv), _p(score),
        _p(ws), ws_bytes, _s(stream)))


def lrm_select_quota(shape, score, off, quota, keep, sel_off, sel_pos, ws, ws_bytes,
                     stream=None):
    _check("lrm_select_quota", _lib.lrm_select_quota(
        ctypes.byref(shape), _p(score), _p(off), _p(quota), _p(keep), _p(sel_off),
        _p(sel_pos), _p(ws), ws_bytes, _s(stream)))


def lrm_compact(shape, perm, keep, sel_off, sel_pos, alpha, x, g, ab, phi, dy_c, x_c, ab_c,
                phi_c, tok_c, row_of_pos, ws, ws_bytes, stream=None):
    _check("lrm_compact", _lib.lrm_compact(
        ctypes.byref(shape), _p(perm), _p(keep), _p(sel_off), _p(sel_pos), _p(alpha), _p(x),
        _p(g), _p(ab), _p(phi), _p(dy_c), _p(x_c), _p(ab_c), _p(phi_c), _p(tok_c),
        _p(row_of_pos), _p(ws), ws_bytes, _s(stream)))


def lrm_expert_bwd_grouped(shape, sel_off, w_gate, w_up, w_down, dy_c, x_c, ab_c, phi_c, inv,
                           row_of_pos, dab_c, dx_c, dw_gate, dw_up, dw_down, dx, ws, ws_bytes,
                           stream=None):
    _check("lrm_expert_bwd_grouped", _lib.lrm_expert_bwd_grouped(
        ctypes.byref(shape), _p(sel_off), _p(w_gate), _p(w_up), _p(w_down), _p(dy_c), _p(x_c),
        _p(ab_c), _p(phi_c), _p(inv), _p(row_of_pos), _p(dab_c), _p(dx_c), _p(dw_gate),
        _p(dw_up), _p(dw_down), _p(dx), _p(ws), ws_bytes, _s(stream)))


def lrm_expert_fc2_dgrad(shape, sel_off, w_down, dy_c, ab_c, dab_c, ws, ws_bytes, stream=None):
    _check("lrm_expert_fc2_dgrad", _lib.lrm_expert_fc2_dgrad(
        ctypes.byref(shape), _p(sel_off), _p(w_down), _p(dy_c), _p(ab_c), _p(dab_c), _p(ws),
        ws_bytes, _s(stream)))


def lrm_expert_fc2_wgrad(shape, sel_off, phi_c, dy_c, dw_down, ws, ws_bytes, stream=None):
    _check("lrm_expert_fc2_wgrad", _lib.lrm_expert_fc2_wgrad(
        ctypes.byref(shape), _p(sel_off), _p(phi_c), _p(dy_c), _p(dw_down), _p(ws), ws_bytes,
        _s(stream)))


def lrm_expert_fc1_wgrad(shape, sel_off, x_c, dab_c, dw_gate, dw_up, ws, ws_bytes, stream=None):
    _check("lrm_expert_fc1_wgrad", _lib.lrm_expert_fc1_wgrad(
        ctypes.byref(shape), _p(sel_off), _p(x_c), _p(dab_c), _p(dw_gate), _p(dw_up), _p(ws),
        ws_bytes, _s(stream)))


def lrm_expert_fc1_dgrad(shape, sel_off, w_gate, w_up, dab_c, dx_c, ws, ws_bytes, stream=None):
    _check("lrm_expert_fc1_dgrad", _lib.lrm_expert_fc1_dgrad(
        ctypes.byref(shape), _p(sel_off), _p(w_gate), _p(w_up), _p(dab_c), _p(dx_c), _p(ws),
        ws_bytes, _s(stream)))


def lrm_scatter_dx(shape, dx_c, inv, row_of_pos, dx, ws, ws_bytes, stream=None):
    _check("lrm_scatter_dx", _lib.lrm_scatter_dx(
        ctypes.byref(shape), _p(dx_c), _p(inv), _p(row_of_pos), _p(dx), _p(ws), ws_bytes,
        _s(stream)))


def lrm_dispatch_permute_noalloc(shape, topk_idx, perm, inv, counts, off, dev_err=None,
                                 stream=None):
    """Dispatch permutation that allocates nothing (scratch built into the library).

    For callers that may not allocate device memory; see include/lrm.h for
    the size limit and the rule that overlapping calls race.
    """
    _check("lrm_dispatch_permute_noalloc", _lib.lrm_dispatch_permute_noalloc(
        ctypes.byref(shape), _p(topk_idx), _p(perm), _p(inv), _p(counts), _p(off),
        _p(dev_err), _s(stream)))


def lrm_selftest_wait_timeout(ws, ws_bytes, stream=None):
    _check("lrm_selftest_wait_timeout",
           _lib.lrm_selftest_wait_timeout(_p(ws), ws_bytes, _s(stream)))


def lrm_score_variant(shape, metric, seed, g, phi, alpha, inv, score, ws, ws_bytes, stream=None):
    _check("lrm_score_variant", _lib.lrm_score_variant(
        ctypes.byref(shape), metric, seed, _p(g), _p(phi), _p(alpha), _p(inv), _p(score),
        _p(ws), ws_bytes, _s(stream)))


def lrm_gather_tokens(shape, perm, x, x_disp, ws, ws_bytes, stream=None):
    _check("lrm_gather_tokens", _lib.lrm_gather_tokens(
        ctypes.byref(shape), _p(perm), _p(x), _p(x_disp), _p(ws), ws_bytes, _s(stream)))


def lrm_expert_fc1_fwd(shape, off, x_disp, w_gate, w_up, ab, phi, ws, ws_bytes, stream=None):
    _check("lrm_expert_fc1_fwd", _lib.lrm_expert_fc1_fwd(
        ctypes.byref(shape), _p(off), _p(x_disp), _p(w_gate), _p(w_up), _p(ab), _p(phi),
        _p(ws), ws_bytes, _s(stream)))


def lrm_expert_fc2_fwd(shape, off, phi, w_down, y, ws, ws_bytes, stream=None):
    _check("lrm_expert_fc2_fwd", _lib.lrm_expert_fc2_fwd(
        ctypes.byref(shape), _p(off), _p(phi), _p(w_down), _p(y), _p(ws), ws_bytes,
        _s(stream)))


def lrm_combine(shape, y, alpha, inv, out, ws, ws_bytes, stream=None):
    _check("lrm_combine", _lib.lrm_combine(
        ctypes.byref(shape), _p(y), _p(alpha), _p(inv), _p(out), _p(ws), ws_bytes,
        _s(stream)))


def lrm_expert_fwd_grouped(shape, perm, inv, off, alpha, x, w_gate, w_up, w_down, x_disp, ab,
                           phi, y, out, ws, ws_bytes, stream=None):
    _check("lrm_expert_fwd_grouped", _lib.lrm_expert_fwd_grouped(
        ctypes.byref(shape), _p(perm), _p(inv), _p(off), _p(alpha), _p(x), _p(w_gate),
        _p(w_up), _p(w_down), _p(x_disp), _p(ab), _p(phi), _p(y), _p(out), _p(ws), ws_bytes,
        _s(stream)))


def lrm_expert_fc1_recompute(shape, sel_off, x_c, w_gate, w_up, ab_c, ws, ws_bytes,
                             stream=None):
    _check("lrm_expert_fc1_recompute", _lib.lrm_expert_fc1_recompute(
        ctypes.byref(shape), _p(sel_off), _p(x_c), _p(w_gate), _p(w_up), _p(ab_c), _p(ws),
        ws_bytes, _s(stream)))


def lrm_expert_bwd_gathered(shape, parts, sel_off, sel_pos, tok_c, w_gate, w_up, w_down, dy_c,
                            x, ab, phi, inv, row_of_pos, dab_c, dx_c, dw_gate, dw_up, dw_down,
                            dx, ws, ws_bytes, stream=None):
    _check("lrm_expert_bwd_gathered", _lib.lrm_expert_bwd_gathered(
        ctypes.byref(shape), parts, _p(sel_off), _p(sel_pos), _p(tok_c), _p(w_gate), _p(w_up),
        _p(w_down), _p(dy_c), _p(x), _p(ab), _p(phi), _p(inv), _p(row_of_pos), _p(dab_c),
        _p(dx_c), _p(dw_gate), _p(dw_up), _p(dw_down), _p(dx), _p(ws), ws_bytes, _s(stream)))


def lrm_select_rate(shape, score, off, num, den, cap, quota, keep, sel_off, sel_pos, ws, ws_bytes,
                    stream=None):
    _check("lrm_select_rate", _lib.lrm_select_rate(
        ctypes.byref(shape), _p(score), _p(off), num, den, cap, _p(quota), _p(keep), _p(sel_off),
        _p(sel_pos), _p(ws), ws_bytes, _s(stream)))


def lrm_router_workspace_bytes(router: lrm_router) -> int:
    return int(_lib.lrm_router_workspace_bytes(ctypes.byref(router)))


def lrm_route(router, logits, mask, topk_idx, alpha, counts, prob_sum, loss, ws, ws_bytes,
              stream=None):
    _check("lrm_route", _lib.lrm_route(
        ctypes.byref(router), _p(logits), _p(mask), _p(topk_idx), _p(alpha), _p(counts),
        _p(prob_sum), _p(loss), _p(ws), ws_bytes, _s(stream)))


def lrm_route_bwd(router, logits, mask, topk_idx, counts, dalpha, dloss, dlogits, ws, ws_bytes,
                  stream=None):
    _check("lrm_route_bwd", _lib.lrm_route_bwd(
        ctypes.byref(router), _p(logits), _p(mask), _p(topk_idx), _p(counts), _p(dalpha),
        _p(dloss), _p(dlogits), _p(ws), ws_bytes, _s(stream)))


def lrm_gate_grad(shape, g, y, inv, dalpha, ws, ws_bytes, stream=None):
    _check("lrm_gate_grad", _lib.lrm_gate_grad(
        ctypes.byref(shape), _p(g), _p(y), _p(inv), _p(dalpha), _p(ws), ws_bytes, _s(stream)))


def lrm_norm_workspace_bytes(norm: lrm_norm) -> int:
    return int(_lib.lrm_norm_workspace_bytes(ctypes.byref(norm)))


def lrm_add_rmsnorm(norm, x, res, w, h, y, q, q_scale, rstd, stream=None):
    _check("lrm_add_rmsnorm", _lib.lrm_add_rmsnorm(
        ctypes.byref(norm), _p(x), _p(res), _p(w), _p(h), _p(y), _p(q), _p(q_scale), _p(rstd),
        _s(stream)))


def lrm_add_rmsnorm_bwd(norm, dy, dh, h, w, rstd, dx, dw, ws, ws_bytes, stream=None):
    _check("lrm_add_rmsnorm_bwd", _lib.lrm_add_rmsnorm_bwd(
        ctypes.byref(norm), _p(dy), _p(dh), _p(h), _p(w), _p(rstd), _p(dx), _p(dw), _p(ws),
        ws_bytes, _s(stream)))


def lrm_adamw_step(adamw, tensors, count: int, stream=None):
    """``tensors``: a ctypes array of lrm_adamw_tensor."""
    _check("lrm_adamw_step", _lib.lrm_adamw_step(
        ctypes.byref(adamw), tensors, count, _s(stream)))
