"""Python binding of libdmuon.so, the GB300 (sm_103a) owner-side Muon step.

Argument marshalling only: every step of the Muon update runs in the
library's CUDA kernels.  The functions keep the C names of
``include/dmuon.h``; PyTorch tensors are accepted for convenience (their
device pointers and shapes are passed through), raw device pointers with
explicit shapes are accepted by the ``*_ptrs`` variants.

There is no CPU fallback: if ``lib/libdmuon.so`` has not been built,
``load()`` raises.
"""
import ctypes
import struct
import os

__all__ = [
    "DmuonError", "load", "lib_path", "dmuon_create", "dmuon_destroy",
    "dmuon_step", "dmuon_step_ptrs", "dmuon_newton_schulz",
    "dmuon_newton_schulz_ptrs", "dmuon_newton_schulz_noalloc", "dmuon_get_status",
    "dmuon_gram_newton_schulz", "dmuon_gram_newton_schulz_ptrs", "BACKENDS",
    "dmuon_adamw_step", "dmuon_adamw_step_ptrs", "dmuon_clip_grad_norm", "dmuon_clip_grad_norm_ptrs",
    "dmuon_workspace_bytes", "dmuon_polar_express_coefficients", "dmuon_gram_check_coefficients",
    "dmuon_plan_preview",
    "dmuon_mxfp4_bytes", "dmuon_mxfp4_empty", "dmuon_mxfp4_quantize", "dmuon_mxfp4_dequantize", "dmuon_mxfp4_gemm",
    "dmuon_block_norm_forward", "dmuon_block_norm_backward",
    "dmuon_mxfp8_bytes", "dmuon_mxfp8_empty", "dmuon_mxfp8_quantize", "dmuon_mxfp8_dequantize", "dmuon_mx_linear",
    "dmuon_act_backward", "dmuon_add_norm_forward", "dmuon_add_norm_backward", "dmuon_dropout", "ACTIVATIONS",
    "dmuon_launch_count", "dmuon_last_error", "dmuon_profile_enable", "dmuon_profile_read",
    "dmuon_plan_summary", "dmuon_error_string", "dmuon_version", "Handle",
    "KIND_NAMES", "STATUS",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "lib", "libdmuon.so")
_lib = None

STATUS = {
    0: "DMUON_OK", -1: "DMUON_ERR_ARG", -2: "DMUON_ERR_ALIGN", -3: "DMUON_ERR_OOM",
    -4: "DMUON_ERR_CUDA", -5: "DMUON_ERR_NONFINITE", -6: "DMUON_ERR_TIMEOUT",
    -7: "DMUON_ERR_UNSUPPORTED",
}
KIND_NAMES = ("momentum", "finalize", "gram", "gram2", "apply", "update0", "adamw", "clip", "small",
              "gs_gram", "gs_prod", "ns_fused", "mx_quantize", "mx_dequantize", "mx_gemm", "norm_fwd", "norm_bwd",
              "act_bwd", "add_norm_fwd", "add_norm_bwd", "dropout")


class DmuonError(RuntimeError):
    def __init__(self, code, what=""):
        self.code = code
        msg = "%s (%d)" % (STATUS.get(code, "unknown"), code)
        if _lib is not None:
            msg += ": " + _lib.dmuon_error_string(code).decode()
        super().__init__(what + ": " + msg if what else msg)


class Shape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class Opts(ctypes.Structure):
    _fields_ = [("weight_decay", ctypes.c_float), ("eps", ctypes.c_float),
                ("nesterov", ctypes.c_int), ("scale_mode", ctypes.c_int),
                ("coeffs", ctypes.POINTER(ctypes.c_float)), ("backend", ctypes.c_int),
                ("restarts", ctypes.POINTER(ctypes.c_int)), ("n_restarts", ctypes.c_int)]


class BlockNorm(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("dtype", ctypes.c_int), ("eps", ctypes.c_float),
                ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("f", ctypes.c_void_p), ("ldf", ctypes.c_int64),
                ("post_w", ctypes.c_void_p), ("pre_w", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("rows_per_gate", ctypes.c_int64), ("res_scale", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("h", ctypes.c_void_p), ("ldh", ctypes.c_int64),
                ("rstd", ctypes.c_void_p)]


class BlockNormGrad(ctypes.Structure):
    _fields_ = [("dy", ctypes.c_void_p), ("lddy", ctypes.c_int64), ("dh", ctypes.c_void_p), ("lddh", ctypes.c_int64),
                ("dx", ctypes.c_void_p), ("lddx", ctypes.c_int64), ("df", ctypes.c_void_p), ("lddf", ctypes.c_int64),
                ("d_post_w", ctypes.c_void_p), ("d_pre_w", ctypes.c_void_p), ("d_gate", ctypes.c_void_p),
                ("d_res_scale", ctypes.c_void_p)]


class MxLinear(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64), ("bits", ctypes.c_int), ("dtype", ctypes.c_int),
                ("a_data", ctypes.c_void_p), ("a_scales", ctypes.c_void_p), ("b_data", ctypes.c_void_p), ("b_scales", ctypes.c_void_p),
                ("alpha", ctypes.c_float), ("beta", ctypes.c_float), ("bias", ctypes.c_void_p), ("act", ctypes.c_int),
                ("c", ctypes.c_void_p), ("ldc", ctypes.c_int64), ("pre", ctypes.c_void_p), ("ldpre", ctypes.c_int64),
                ("d", ctypes.c_void_p), ("ldd", ctypes.c_int64)]


class ActBackward(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("dtype", ctypes.c_int), ("act", ctypes.c_int),
                ("dout", ctypes.c_void_p), ("lddout", ctypes.c_int64), ("pre", ctypes.c_void_p), ("ldpre", ctypes.c_int64),
                ("dz", ctypes.c_void_p), ("lddz", ctypes.c_int64), ("d_bias", ctypes.c_void_p), ("scale_mode", ctypes.c_int),
                ("row_data", ctypes.c_void_p), ("row_scales", ctypes.c_void_p), ("col_data", ctypes.c_void_p),
                ("col_scales", ctypes.c_void_p)]


class AddNorm(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("dtype", ctypes.c_int), ("eps", ctypes.c_float),
                ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("f", ctypes.c_void_p), ("ldf", ctypes.c_int64), ("w", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("h", ctypes.c_void_p), ("ldh", ctypes.c_int64),
                ("q_data", ctypes.c_void_p), ("q_scales", ctypes.c_void_p), ("scale_mode", ctypes.c_int), ("p", ctypes.c_float),
                ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64), ("rstd", ctypes.c_void_p)]


class AddNormGrad(ctypes.Structure):
    _fields_ = [("dy", ctypes.c_void_p), ("lddy", ctypes.c_int64), ("dh", ctypes.c_void_p), ("lddh", ctypes.c_int64),
                ("dx", ctypes.c_void_p), ("lddx", ctypes.c_int64), ("df", ctypes.c_void_p), ("lddf", ctypes.c_int64),
                ("d_w", ctypes.c_void_p)]


# The same fields for struct.pack, which fills them in half the time.
_NORM = struct.Struct("qqifPqPqPPPqPPqPqP")
_NORM_GRAD = struct.Struct("PqPqPqPqPPPP")
_LINEAR = struct.Struct("qqqiiPPPPffPiPqPqPq")
_ACT_BACKWARD = struct.Struct("qqiiPqPqPqPiPPPP")
_ADD_NORM = struct.Struct("qqifPqPqPPqPqPPifQQP")
_ADD_NORM_GRAD = struct.Struct("PqPqPqPqP")
assert _NORM.size == ctypes.sizeof(BlockNorm) and _NORM_GRAD.size == ctypes.sizeof(BlockNormGrad)
assert _LINEAR.size == ctypes.sizeof(MxLinear) and _ACT_BACKWARD.size == ctypes.sizeof(ActBackward)
assert _ADD_NORM.size == ctypes.sizeof(AddNorm) and _ADD_NORM_GRAD.size == ctypes.sizeof(AddNormGrad)


BACKENDS = {"direct": 0, "gram": 1}
SCALE_MODES = {"floor": 0, "ceil": 1}
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
_TYPES = {}  # torch dtype -> type code of include/dmuon.h, filled with the first tensor


def _types():
    if not _TYPES:
        import torch
        _TYPES.update({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2, torch.uint8: 3})
    return _TYPES


def lib_path():
    return _LIB_PATH


def load(path=None):
    """Load libdmuon.so (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or _LIB_PATH
    if not os.path.exists(p):
        raise ImportError("libdmuon.so not built (%s); run __graft_entry__.build()" % p)
    L = ctypes.CDLL(p)
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    pp = ctypes.POINTER(ctypes.c_void_p)
    L.dmuon_default_opts.argtypes = [ctypes.POINTER(Opts)]
    L.dmuon_default_opts.restype = None
    L.dmuon_create.argtypes = [ctypes.POINTER(vp), i32]
    L.dmuon_create.restype = i32
    L.dmuon_destroy.argtypes = [vp]
    L.dmuon_destroy.restype = None
    L.dmuon_workspace_bytes.argtypes = [ctypes.POINTER(Shape), i32, ctypes.POINTER(ctypes.c_size_t)]
    L.dmuon_workspace_bytes.restype = i32
    L.dmuon_workspace_bytes_ex.argtypes = [ctypes.POINTER(Shape), i32, i32, ctypes.POINTER(ctypes.c_size_t)]
    L.dmuon_workspace_bytes_ex.restype = i32
    L.dmuon_gram_newton_schulz.argtypes = [vp, pp, pp, ctypes.POINTER(Shape), i32, i32,
                                           ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int),
                                           i32, f32, vp]
    L.dmuon_gram_newton_schulz.restype = i32
    L.dmuon_step.argtypes = [vp, pp, pp, pp, ctypes.POINTER(Shape), i32, f32, f32, i32,
                             ctypes.POINTER(Opts), vp]
    L.dmuon_step.restype = i32
    L.dmuon_newton_schulz.argtypes = [vp, pp, pp, ctypes.POINTER(Shape), i32, i32,
                                      ctypes.POINTER(ctypes.c_float), f32, vp]
    L.dmuon_newton_schulz.restype = i32
    L.dmuon_newton_schulz_noalloc.argtypes = [vp, vp, i64, i64, i32, ctypes.POINTER(ctypes.c_float),
                                              f32, i32, vp]
    L.dmuon_newton_schulz_noalloc.restype = i32
    L.dmuon_adamw_step.argtypes = [vp, pp, pp, pp, pp, ctypes.POINTER(i64), i32, f32, f32, f32, f32,
                                   f32, i32, vp]
    L.dmuon_adamw_step.restype = i32
    L.dmuon_clip_grad_norm.argtypes = [vp, pp, ctypes.POINTER(i64), i32, ctypes.POINTER(ctypes.c_int), i32,
                                       f32, ctypes.POINTER(f32), ctypes.POINTER(f32), vp]
    L.dmuon_clip_grad_norm.restype = i32
    L.dmuon_get_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int), i32]
    L.dmuon_get_status.restype = i32
    L.dmuon_last_error.argtypes = [vp]
    L.dmuon_last_error.restype = ctypes.c_char_p
    L.dmuon_set_overlap.argtypes = [vp, i32]
    L.dmuon_set_overlap.restype = i32
    L.dmuon_set_balanced_dealing.argtypes = [vp, i32]
    L.dmuon_set_balanced_dealing.restype = i32
    L.dmuon_set_fused_phases.argtypes = [vp, i32]
    L.dmuon_set_fused_phases.restype = i32
    L.dmuon_set_fp16_iterations.argtypes = [vp, i32]
    L.dmuon_set_fp16_iterations.restype = i32
    L.dmuon_set_small_path.argtypes = [vp, i32]
    L.dmuon_set_small_path.restype = i32
    L.dmuon_set_chunk_elements.argtypes = [vp, i64]
    L.dmuon_set_chunk_elements.restype = i32
    L.dmuon_set_tile_mode.argtypes = [vp, i32]
    L.dmuon_set_tile_mode.restype = i32
    L.dmuon_set_wait_timeout.argtypes = [vp, ctypes.c_uint64]
    L.dmuon_set_wait_timeout.restype = i32
    L.dmuon_launch_count.argtypes = [vp]
    L.dmuon_launch_count.restype = i64
    L.dmuon_profile_enable.argtypes = [vp, i32]
    L.dmuon_profile_enable.restype = i32
    L.dmuon_profile_read.argtypes = [vp, ctypes.POINTER(ctypes.c_double),
                                     ctypes.POINTER(ctypes.c_int64), i32]
    L.dmuon_profile_read.restype = i32
    L.dmuon_plan_summary.argtypes = [vp, ctypes.c_char_p, ctypes.c_size_t]
    L.dmuon_plan_summary.restype = i32
    L.dmuon_error_string.argtypes = [i32]
    L.dmuon_error_string.restype = ctypes.c_char_p
    L.dmuon_version.argtypes = []
    L.dmuon_version.restype = ctypes.c_char_p
    L.dmuon_plan_preview.argtypes = [ctypes.POINTER(Shape), i32, i32, i32, i32, i32, i32, ctypes.c_char_p,
                                     ctypes.c_size_t]
    L.dmuon_plan_preview.restype = i32
    L.dmuon_polar_express_coefficients.argtypes = [i32, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                                                   ctypes.POINTER(ctypes.c_float)]
    L.dmuon_polar_express_coefficients.restype = i32
    L.dmuon_gram_check_coefficients.argtypes = [i32, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int),
                                                i32, ctypes.c_char_p, ctypes.c_size_t]
    L.dmuon_gram_check_coefficients.restype = i32
    sz = ctypes.POINTER(ctypes.c_size_t)
    L.dmuon_mxfp4_bytes.argtypes = [i64, i64, sz, sz]
    L.dmuon_mxfp4_bytes.restype = i32
    L.dmuon_mxfp4_quantize.argtypes = [vp, vp, i32, i64, i64, i64, i32, vp, i64, vp, vp, vp, vp, vp]
    L.dmuon_mxfp4_quantize.restype = i32
    L.dmuon_mxfp4_dequantize.argtypes = [vp, vp, vp, i64, i64, vp, i32, i64, vp]
    L.dmuon_mxfp4_dequantize.restype = i32
    L.dmuon_mxfp4_gemm.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp, i32, i64, f32, f32, vp]
    L.dmuon_mxfp4_gemm.restype = i32
    L.dmuon_block_norm_forward.argtypes = [vp, ctypes.POINTER(BlockNorm), vp]
    L.dmuon_block_norm_forward.restype = i32
    L.dmuon_block_norm_backward.argtypes = [vp, ctypes.POINTER(BlockNorm), ctypes.POINTER(BlockNormGrad), vp]
    L.dmuon_block_norm_backward.restype = i32
    L.dmuon_mxfp8_bytes.argtypes = [i64, i64, sz, sz]
    L.dmuon_mxfp8_bytes.restype = i32
    L.dmuon_mxfp8_quantize.argtypes = [vp, vp, i32, i64, i64, i64, i32, vp, vp, vp, vp, vp]
    L.dmuon_mxfp8_quantize.restype = i32
    L.dmuon_mxfp8_dequantize.argtypes = [vp, vp, vp, i64, i64, vp, i32, i64, vp]
    L.dmuon_mxfp8_dequantize.restype = i32
    L.dmuon_mx_linear.argtypes = [vp, ctypes.POINTER(MxLinear), vp]
    L.dmuon_mx_linear.restype = i32
    L.dmuon_act_backward.argtypes = [vp, ctypes.POINTER(ActBackward), vp]
    L.dmuon_act_backward.restype = i32
    L.dmuon_add_norm_forward.argtypes = [vp, ctypes.POINTER(AddNorm), vp]
    L.dmuon_add_norm_forward.restype = i32
    L.dmuon_add_norm_backward.argtypes = [vp, ctypes.POINTER(AddNorm), ctypes.POINTER(AddNormGrad), vp]
    L.dmuon_add_norm_backward.restype = i32
    L.dmuon_dropout.argtypes = [vp, vp, i32, i64, i64, i64, vp, i64, vp, i64, f32, ctypes.c_uint64, ctypes.c_uint64, vp]
    L.dmuon_dropout.restype = i32
    _lib = L
    return L


def _check(code, what, h=None):
    if code != 0:
        if h is not None and _lib is not None:
            what = what + " [" + _lib.dmuon_last_error(h).decode() + "]"
        raise DmuonError(code, what)


def _ptr_array(ptrs):
    arr = (ctypes.c_void_p * max(1, len(ptrs)))()
    for i, p in enumerate(ptrs):
        arr[i] = int(p)
    return arr


def _shape_array(shapes):
    arr = (Shape * max(1, len(shapes)))()
    for i, (r, c) in enumerate(shapes):
        arr[i].rows, arr[i].cols = int(r), int(c)
    return arr


def _coeff_array(coeffs):
    if coeffs is None:
        return None
    flat = [float(v) for row in coeffs for v in row]
    return (ctypes.c_float * max(1, len(flat)))(*flat)


def _stream_handle(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream
    return int(stream)


def _tensor_args(tensors, name):
    ptrs, shapes = [], []
    for t in tensors:
        if t.dim() != 2 or not t.is_cuda or not t.is_contiguous() or str(t.dtype) != "torch.float32":
            raise ValueError("%s: each matrix must be a contiguous 2-D float32 CUDA tensor" % name)
        ptrs.append(t.data_ptr())
        shapes.append(tuple(t.shape))
    return ptrs, shapes


# ---------------------------------------------------------------- C calls

def dmuon_version():
    return load().dmuon_version().decode()


def dmuon_error_string(code):
    return load().dmuon_error_string(int(code)).decode()


class _RawHandle(ctypes.c_void_p):
    """A dmuon handle that knows its device."""


def dmuon_create(device=0):
    h = _RawHandle()
    _check(load().dmuon_create(ctypes.byref(h), int(device)), "dmuon_create")
    h.device = int(device)
    return h


def dmuon_destroy(h):
    if h is not None:
        load().dmuon_destroy(h)


def dmuon_workspace_bytes(shapes, backend="direct"):
    out = ctypes.c_size_t(0)
    _check(load().dmuon_workspace_bytes_ex(_shape_array(shapes), len(shapes), BACKENDS[backend],
                                           ctypes.byref(out)), "dmuon_workspace_bytes")
    return out.value


def dmuon_polar_express_coefficients(steps=5, lower=1e-3, upper=1.0, safety=1.05):
    """Polar Express table (host only): ``steps`` rows (a, b, c) as floats."""
    out = (ctypes.c_float * (3 * max(1, int(steps))))()
    _check(load().dmuon_polar_express_coefficients(int(steps), float(lower), float(upper), float(safety), out),
           "dmuon_polar_express_coefficients")
    return [(out[3 * k], out[3 * k + 1], out[3 * k + 2]) for k in range(int(steps))]


def dmuon_plan_preview(shapes, backend="direct", tile_mode=0, clusters=76, sms=152, balanced=True):
    """Host-only summary of the plan a handle would build for ``shapes`` on a
    device with ``clusters`` 2-CTA clusters and ``sms`` SMs (GB300: 76, 152)."""
    buf = ctypes.create_string_buffer(512)
    rc = load().dmuon_plan_preview(_shape_array(shapes), len(shapes), BACKENDS[backend], int(tile_mode),
                                   int(clusters), int(sms), 1 if balanced else 0, buf, 512)
    if rc < 0:
        raise DmuonError(rc, "dmuon_plan_preview")
    return buf.value.decode()


def dmuon_gram_check_coefficients(ns_steps=5, coeffs=None, restarts=None):
    """The Gram-space backend's fp16 range check (host only): (True, "") or
    (False, reason)."""
    carr = _coeff_array(coeffs)
    rarr, nr = _restart_array(restarts)
    why = ctypes.create_string_buffer(256)
    rc = load().dmuon_gram_check_coefficients(int(ns_steps), carr, rarr, nr, why, 256)
    if rc not in (0, -1):
        raise DmuonError(rc, "dmuon_gram_check_coefficients")
    return rc == 0, why.value.decode()


def _restart_array(restarts):
    """None -> NULL (the default {2}); a sequence -> (int array, count)."""
    if restarts is None:
        return None, 0
    rs = [int(k) for k in restarts]
    return (ctypes.c_int * max(1, len(rs)))(*rs), len(rs)


def dmuon_step_ptrs(h, w_ptrs, g_ptrs, m_ptrs, shapes, lr, mu, ns_steps=5,
                    weight_decay=0.0, eps=1e-7, nesterov=True, scale_mode=0,
                    coeffs=None, stream=None, check=True, backend="direct", restarts=None):
    """dmuon_step on raw device pointers; returns the status code.
    backend "gram" selects the Gram-space iteration with restart positions
    `restarts` (None = the default [2])."""
    L = load()
    opts = Opts()
    L.dmuon_default_opts(ctypes.byref(opts))
    opts.weight_decay = float(weight_decay)
    opts.eps = float(eps)
    opts.nesterov = 1 if nesterov else 0
    opts.scale_mode = int(scale_mode)
    opts.backend = BACKENDS[backend]
    rarr, nr = _restart_array(restarts)
    if rarr is not None:
        opts.restarts = ctypes.cast(rarr, ctypes.POINTER(ctypes.c_int))
        opts.n_restarts = nr
    carr = _coeff_array(coeffs)
    if carr is not None:
        opts.coeffs = ctypes.cast(carr, ctypes.POINTER(ctypes.c_float))
    rc = L.dmuon_step(h, _ptr_array(w_ptrs), _ptr_array(g_ptrs), _ptr_array(m_ptrs),
                      _shape_array(shapes), len(shapes), float(lr), float(mu), int(ns_steps),
                      ctypes.byref(opts), ctypes.c_void_p(_stream_handle(stream)))
    if check:
        _check(rc, "dmuon_step", h)
    return rc


def dmuon_step(h, params, grads, momentum, lr=0.02, mu=0.95, ns_steps=5, **kw):
    """One Muon step over lists of CUDA fp32 tensors (updated in place)."""
    wp, ws = _tensor_args(params, "params")
    gp, gs = _tensor_args(grads, "grads")
    mp, ms = _tensor_args(momentum, "momentum")
    if ws != gs or ws != ms:
        raise ValueError("params, grads and momentum must have matching shapes")
    return dmuon_step_ptrs(h, wp, gp, mp, ws, lr, mu, ns_steps, **kw)


def dmuon_newton_schulz_ptrs(h, in_ptrs, out_ptrs, shapes, ns_steps=5, coeffs=None,
                             eps=1e-7, stream=None, check=True):
    L = load()
    carr = _coeff_array(coeffs)
    rc = L.dmuon_newton_schulz(h, _ptr_array(in_ptrs), _ptr_array(out_ptrs), _shape_array(shapes),
                               len(shapes), int(ns_steps),
                               None if carr is None else ctypes.cast(carr, ctypes.POINTER(ctypes.c_float)),
                               float(eps), ctypes.c_void_p(_stream_handle(stream)))
    if check:
        _check(rc, "dmuon_newton_schulz", h)
    return rc


def dmuon_newton_schulz(h, inputs, outputs, ns_steps=5, coeffs=None, eps=1e-7, stream=None):
    ip, is_ = _tensor_args(inputs, "inputs")
    op, os_ = _tensor_args(outputs, "outputs")
    if is_ != os_:
        raise ValueError("inputs and outputs must have matching shapes")
    return dmuon_newton_schulz_ptrs(h, ip, op, is_, ns_steps, coeffs, eps, stream)


def dmuon_gram_newton_schulz_ptrs(h, in_ptrs, out_ptrs, shapes, ns_steps=5, coeffs=None, restarts=None,
                                  eps=1e-7, stream=None, check=True):
    L = load()
    carr = _coeff_array(coeffs)
    rarr, nr = _restart_array(restarts)
    rc = L.dmuon_gram_newton_schulz(
        h, _ptr_array(in_ptrs), _ptr_array(out_ptrs), _shape_array(shapes), len(shapes), int(ns_steps),
        None if carr is None else ctypes.cast(carr, ctypes.POINTER(ctypes.c_float)),
        None if rarr is None else ctypes.cast(rarr, ctypes.POINTER(ctypes.c_int)), nr, float(eps),
        ctypes.c_void_p(_stream_handle(stream)))
    if check:
        _check(rc, "dmuon_gram_newton_schulz", h)
    return rc


def dmuon_gram_newton_schulz(h, inputs, outputs, ns_steps=5, coeffs=None, restarts=None, eps=1e-7,
                             stream=None):
    """Standalone Newton-Schulz with the Gram-space backend."""
    ip, is_ = _tensor_args(inputs, "inputs")
    op, os_ = _tensor_args(outputs, "outputs")
    if is_ != os_:
        raise ValueError("inputs and outputs must have matching shapes")
    return dmuon_gram_newton_schulz_ptrs(h, ip, op, is_, ns_steps, coeffs, restarts, eps, stream)


def dmuon_newton_schulz_noalloc(input_ptr, output_ptr, rows, cols, ns_steps=5, coeffs=None,
                                eps=1e-7, sync_status=True, stream=None):
    """Allocation-free standalone NS of one matrix (raw device pointers);
    returns the status code."""
    carr = _coeff_array(coeffs)
    return load().dmuon_newton_schulz_noalloc(
        ctypes.c_void_p(int(input_ptr)), ctypes.c_void_p(int(output_ptr)), int(rows), int(cols),
        int(ns_steps), None if carr is None else ctypes.cast(carr, ctypes.POINTER(ctypes.c_float)),
        float(eps), 1 if sync_status else 0, ctypes.c_void_p(_stream_handle(stream)))


def _flat_args(tensors, name):
    ptrs, numels = [], []
    for t in tensors:
        if not t.is_cuda or not t.is_contiguous() or str(t.dtype) != "torch.float32":
            raise ValueError("%s: each tensor must be a contiguous float32 CUDA tensor" % name)
        ptrs.append(t.data_ptr())
        numels.append(t.numel())
    return ptrs, numels


def dmuon_adamw_step_ptrs(h, p_ptrs, g_ptrs, m_ptrs, v_ptrs, numels, lr=1e-3, beta1=0.9,
                          beta2=0.999, eps=1e-8, weight_decay=0.01, step=1, stream=None, check=True):
    n = len(numels)
    nums = (ctypes.c_int64 * max(1, n))(*[int(x) for x in numels])
    rc = load().dmuon_adamw_step(h, _ptr_array(p_ptrs), _ptr_array(g_ptrs), _ptr_array(m_ptrs),
                                 _ptr_array(v_ptrs), nums, n, float(lr), float(beta1), float(beta2),
                                 float(eps), float(weight_decay), int(step),
                                 ctypes.c_void_p(_stream_handle(stream)))
    if check:
        _check(rc, "dmuon_adamw_step", h)
    return rc


def dmuon_adamw_step(h, params, grads, exp_avg, exp_avg_sq, **kw):
    """AdamW over lists of contiguous fp32 CUDA tensors (updated in place)."""
    pp_, nums = _flat_args(params, "params")
    gp, gn = _flat_args(grads, "grads")
    mp, mn = _flat_args(exp_avg, "exp_avg")
    vp_, vn = _flat_args(exp_avg_sq, "exp_avg_sq")
    if not (nums == gn == mn == vn):
        raise ValueError("params, grads, exp_avg, exp_avg_sq must have matching sizes")
    return dmuon_adamw_step_ptrs(h, pp_, gp, mp, vp_, nums, **kw)


def dmuon_clip_grad_norm_ptrs(h, g_ptrs, numels, max_norm, buckets=None, n_buckets=None,
                              stats=True, stream=None, check=True):
    """Returns (status, norms, coefs); norms/coefs are None when stats=False."""
    n = len(numels)
    nb = 1 if buckets is None else int(n_buckets if n_buckets is not None else max(buckets) + 1)
    nums = (ctypes.c_int64 * max(1, n))(*[int(x) for x in numels])
    bk = None if buckets is None else (ctypes.c_int * max(1, n))(*[int(b) for b in buckets])
    norms = (ctypes.c_float * nb)() if stats else None
    coefs = (ctypes.c_float * nb)() if stats else None
    rc = load().dmuon_clip_grad_norm(h, _ptr_array(g_ptrs), nums, n, bk, nb, float(max_norm),
                                     norms, coefs, ctypes.c_void_p(_stream_handle(stream)))
    if check:
        _check(rc, "dmuon_clip_grad_norm", h)
    if not stats:
        return rc, None, None
    return rc, [norms[i] for i in range(nb)], [coefs[i] for i in range(nb)]


def dmuon_clip_grad_norm(h, grads, max_norm, buckets=None, n_buckets=None, stats=True, stream=None):
    """Segmented clipping of CUDA fp32 gradients in place; returns (norms, coefs)."""
    gp, nums = _flat_args(grads, "grads")
    _, norms, coefs = dmuon_clip_grad_norm_ptrs(h, gp, nums, max_norm, buckets, n_buckets, stats, stream)
    return norms, coefs


# ------------------------------------ 4- and 8-bit projections and their norms

def _device(h, t, name):
    """Index of the handle's device, on which every tensor of a call has to be;
    that of ``t``, the first one, for a handle that does not tell."""
    try:
        return h.device
    except AttributeError:
        index = t.get_device()
    if index < 0:
        raise ValueError("%s: a CUDA tensor is wanted" % name)
    return index


def _matrix(t, name, index, dtype=None, shape=None):
    """(pointer, leading dimension, type code, shape) of a 2-D tensor on the
    device ``index`` whose rows are contiguous; ``dtype`` and ``shape``, where
    given, have to match."""
    code = (_TYPES or _types()).get(t.dtype, 3)
    size = t.shape
    if code > 2 or t.get_device() != index or len(size) != 2 or (dtype is not None and code != dtype):
        raise ValueError("%s: a 2-D tensor of float32, bfloat16 or float16%s on the handle's device is wanted"
                         % (name, "" if dtype is None else " (the type of the others)"))
    if shape is not None and size != shape:
        raise ValueError("%s: shape %s, %s wanted" % (name, tuple(size), tuple(shape)))
    return t.data_ptr(), _pitch(t, size, name), code, size


def _pitch(t, size, name):
    rows, cols = size
    ld, inner = t.stride()
    if cols > 1 and inner != 1 or rows > 1 and ld < cols:
        raise ValueError("%s: rows must be contiguous and not overlap" % name)
    return ld if rows > 1 else max(ld, cols)


def _like(t, name, first):
    """(pointer, leading dimension) of a matrix of the device, type, type code
    and shape ``first``; None gives (0, 0)."""
    if t is None:
        return 0, 0
    index, dtype, code, size = first
    if t.dtype is dtype and t.shape == size and t.get_device() == index and t.is_contiguous():
        return t.data_ptr(), size[1]
    return _matrix(t, name, index, code, size)[:2]


def _floats(t, name, index, shape):
    """Pointer of a contiguous fp32 tensor of ``shape`` on the device; None gives 0."""
    if t is None:
        return 0
    if (_TYPES or _types()).get(t.dtype) != 0 or t.get_device() != index or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s: a contiguous float32 tensor of shape %s on the handle's device is wanted" % (name, tuple(shape)))
    return t.data_ptr()


def _mx(q, name, index, rows, k, bits):
    """(data pointer, scales pointer) of an MXFP4 or MXFP8 matrix (data, scales)."""
    data, scales = q
    nb = -(-k // 32)
    types = _TYPES or _types()
    if (types.get(data.dtype) != 3 or types.get(scales.dtype) != 3 or data.numel() != rows * nb * 4 * bits or
            scales.numel() != -(-rows // 128) * -(-nb // 4) * 512 or data.get_device() != index or scales.get_device() != index or
            not data.is_contiguous() or not scales.is_contiguous()):
        raise ValueError("%s: contiguous uint8 tensors of the sizes dmuon_mxfp%d_empty(%d, %d) gives on the handle's device are wanted"
                         % (name, bits, rows, k))
    return data.data_ptr(), scales.data_ptr()


def _mxfp4(q, name, index, rows, k):
    return _mx(q, name, index, rows, k, 4)


def _mxfp8(q, name, index, rows, k):
    """The same of an MXFP8 matrix; None gives (None, None)."""
    return (None, None) if q is None else _mx(q, name, index, rows, k, 8)


_raw_stream = None  # torch's current stream of a device as an integer


def _stream_of(stream, index):
    """Handle of ``stream``, or of the device's current stream."""
    global _raw_stream
    if stream is not None:
        return _stream_handle(stream)
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
    return _raw_stream(index)


def dmuon_mxfp4_bytes(rows, k):
    """(data bytes, scale bytes) of a rows x k MXFP4 matrix (host only)."""
    d, s = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(load().dmuon_mxfp4_bytes(int(rows), int(k), ctypes.byref(d), ctypes.byref(s)), "dmuon_mxfp4_bytes")
    return d.value, s.value


def dmuon_mxfp4_empty(rows, k, device="cuda"):
    """Uninitialised buffers (data, scales) of a rows x k MXFP4 matrix."""
    import torch
    d, s = dmuon_mxfp4_bytes(rows, k)
    return (torch.empty((rows, d // max(1, rows)), dtype=torch.uint8, device=device),
            torch.empty(s, dtype=torch.uint8, device=device))


def dmuon_mxfp4_quantize(h, src, by_rows=None, by_cols=None, noise=None, scale="floor", stream=None):
    """Quantise the matrix ``src`` [r, c] along its rows into ``by_rows`` (an
    r x c MXFP4 matrix) and / or along its columns into ``by_cols`` (c x r).
    ``noise``: uint8 [r, c] of random bytes for stochastic rounding."""
    index = _device(h, src, "src")
    ptr, ld, code, size = _matrix(src, "src", index)
    r, c = size
    nptr, nld = None, 0
    if noise is not None:
        if noise.get_device() != index or (_TYPES or _types()).get(noise.dtype) != 3 or noise.shape != size:
            raise ValueError("noise: a uint8 tensor of src's shape on the handle's device is wanted")
        nptr, nld = noise.data_ptr(), _pitch(noise, size, "noise")
    rd, rs = (None, None) if by_rows is None else _mxfp4(by_rows, "by_rows", index, r, c)
    cd, cs = (None, None) if by_cols is None else _mxfp4(by_cols, "by_cols", index, c, r)
    mode = SCALE_MODES[scale]
    if r == 0 or c == 0:
        return
    rc = load().dmuon_mxfp4_quantize(h, ptr, code, r, c, ld, mode, nptr, nld, rd, rs, cd, cs, _stream_of(stream, index))
    if rc:
        _check(rc, "dmuon_mxfp4_quantize", h)


def dmuon_mxfp4_dequantize(h, q, out, stream=None):
    """The values of the MXFP4 matrix ``q`` into ``out`` [rows, k]."""
    index = _device(h, out, "out")
    ptr, ld, code, (r, k) = _matrix(out, "out", index)
    d, s = _mxfp4(q, "q", index, r, k)
    if r == 0 or k == 0:
        return
    rc = load().dmuon_mxfp4_dequantize(h, d, s, r, k, ptr, code, ld, _stream_of(stream, index))
    if rc:
        _check(rc, "dmuon_mxfp4_dequantize", h)


def _zero_block(rows, stream, index, bits=4):
    """A zero matrix of one block of columns: buffers of the stream (raw handle),
    which an empty sum is taken over since the library wants k >= 1."""
    import contextlib
    import torch
    d, s = dmuon_mxfp4_bytes(rows, 32) if bits == 4 else dmuon_mxfp8_bytes(rows, 32)
    here = torch.cuda.current_stream(index)
    on = contextlib.nullcontext() if here.cuda_stream == stream else torch.cuda.stream(torch.cuda.ExternalStream(stream, index))
    with on:
        buf = torch.zeros(d + s, dtype=torch.uint8, device="cuda:%d" % index)
    return buf, buf.data_ptr(), buf.data_ptr() + d


def dmuon_mxfp4_gemm(h, a, b, out, k, alpha=1.0, beta=0.0, stream=None):
    """out = alpha * a b^T + beta * out of MXFP4 matrices a [m, k] and
    b [n, k]; out is [m, n] in float32, bfloat16 or float16.  k = 0, a sum over
    no rows, gives beta * out."""
    index = _device(h, out, "out")
    ptr, ld, code, (m, n) = _matrix(out, "out", index)
    ad, as_ = _mxfp4(a, "a", index, m, k)
    bd, bs = _mxfp4(b, "b", index, n, k)
    if m == 0 or n == 0:
        return
    stream = _stream_of(stream, index)
    if k == 0:
        zeros, ad, as_ = _zero_block(max(m, n), stream, index)
        bd, bs, k = ad, as_, 32
    rc = load().dmuon_mxfp4_gemm(h, ad, as_, bd, bs, m, n, k, ptr, code, ld, alpha, beta, stream)
    if rc:
        _check(rc, "dmuon_mxfp4_gemm", h)


def _block_norm(h, x, f, y, post_w, pre_w, rstd, gate, rows_per_gate, res_scale, eps, out):
    """The fields that forward and backward share; x and out may be None."""
    index = _device(h, f, "f")
    fp, ldf, code, shape = _matrix(f, "f", index)
    rows, cols = shape
    first = index, f.dtype, code, shape
    xp, ldx = _like(x, "x", first)
    yp, ldy = _like(y, "y", first)
    hp, ldh = _like(out, "out", first)
    per = max(1, rows) if rows_per_gate is None else int(rows_per_gate)
    if per < 1:
        raise ValueError("rows_per_gate must be at least 1")
    line = (cols,)
    packed = _NORM.pack(rows, cols, code, eps, xp, ldx, fp, ldf, _floats(post_w, "post_w", index, line),
                        _floats(pre_w, "pre_w", index, line), _floats(gate, "gate", index, (-(-rows // per), cols)), per,
                        _floats(res_scale, "res_scale", index, line), yp, ldy, hp, ldh, _floats(rstd, "rstd", index, (2, rows)))
    return BlockNorm.from_buffer_copy(packed), first


def dmuon_block_norm_forward(h, x, f, post_w, pre_w, y, out, rstd, gate=None, rows_per_gate=None, res_scale=None,
                             eps=1e-6, stream=None):
    """y = res_scale * x + gate * rms(f) * post_w and out = rms(y) * pre_w over
    the rows of x and f [rows, cols]; rstd [2, rows] is what the backward needs.
    ``gate`` [ceil(rows / rows_per_gate), cols] (rows_per_gate None: one row for all)."""
    p, first = _block_norm(h, x, f, y, post_w, pre_w, rstd, gate, rows_per_gate, res_scale, eps, out)
    rc = load().dmuon_block_norm_forward(h, p, _stream_of(stream, first[0]))
    if rc:
        _check(rc, "dmuon_block_norm_forward", h)


def dmuon_block_norm_backward(h, dy, dh, x, f, y, post_w, pre_w, rstd, dx, df, d_post_w, d_pre_w, gate=None,
                              d_gate=None, rows_per_gate=None, res_scale=None, d_res_scale=None, stream=None):
    """Gradients of dmuon_block_norm_forward from dh (of its out) and dy (of y,
    None = 0).  x may be None unless d_res_scale is wanted."""
    p, first = _block_norm(h, x, f, y, post_w, pre_w, rstd, gate, rows_per_gate, res_scale, 0.0, None)
    if d_gate is not None and gate is None:
        raise ValueError("d_gate without a gate")
    index, line = first[0], (first[3][1],)
    q = BlockNormGrad.from_buffer_copy(_NORM_GRAD.pack(
        *_like(dy, "dy", first), *_like(dh, "dh", first), *_like(dx, "dx", first), *_like(df, "df", first),
        _floats(d_post_w, "d_post_w", index, line), _floats(d_pre_w, "d_pre_w", index, line),
        0 if d_gate is None else _floats(d_gate, "d_gate", index, gate.shape), _floats(d_res_scale, "d_res_scale", index, line)))
    rc = load().dmuon_block_norm_backward(h, p, q, _stream_of(stream, first[0]))
    if rc:
        _check(rc, "dmuon_block_norm_backward", h)


def dmuon_mxfp8_bytes(rows, k):
    """(data bytes, scale bytes) of a rows x k MXFP8 matrix (host only)."""
    d, s = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(load().dmuon_mxfp8_bytes(int(rows), int(k), ctypes.byref(d), ctypes.byref(s)), "dmuon_mxfp8_bytes")
    return d.value, s.value


def dmuon_mxfp8_empty(rows, k, device="cuda"):
    """Uninitialised buffers (data, scales) of a rows x k MXFP8 matrix."""
    import torch
    d, s = dmuon_mxfp8_bytes(rows, k)
    return (torch.empty((rows, d // max(1, rows)), dtype=torch.uint8, device=device),
            torch.empty(s, dtype=torch.uint8, device=device))


def dmuon_mxfp8_quantize(h, src, by_rows=None, by_cols=None, scale="floor", stream=None):
    """Quantise the matrix ``src`` [r, c] along its rows into ``by_rows`` (an
    r x c MXFP8 matrix) and / or along its columns into ``by_cols`` (c x r)."""
    index = _device(h, src, "src")
    ptr, ld, code, (r, c) = _matrix(src, "src", index)
    rd, rs = _mxfp8(by_rows, "by_rows", index, r, c)
    cd, cs = _mxfp8(by_cols, "by_cols", index, c, r)
    mode = SCALE_MODES[scale]
    if r == 0 or c == 0:
        return
    rc = load().dmuon_mxfp8_quantize(h, ptr, code, r, c, ld, mode, rd, rs, cd, cs, _stream_of(stream, index))
    if rc:
        _check(rc, "dmuon_mxfp8_quantize", h)


def dmuon_mxfp8_dequantize(h, q, out, stream=None):
    """The values of the MXFP8 matrix ``q`` into ``out`` [rows, k]."""
    index = _device(h, out, "out")
    ptr, ld, code, (r, k) = _matrix(out, "out", index)
    d, s = _mx(q, "q", index, r, k, 8)
    if r == 0 or k == 0:
        return
    rc = load().dmuon_mxfp8_dequantize(h, d, s, r, k, ptr, code, ld, _stream_of(stream, index))
    if rc:
        _check(rc, "dmuon_mxfp8_dequantize", h)


def dmuon_mx_linear(h, a, b, out, k, bias=None, act="none", pre=None, residual=None, alpha=1.0, beta=1.0, bits=8, stream=None):
    """z = alpha * a b^T + bias, out = act(z) + beta * residual, pre = z of
    MXFP8 (bits=4: MXFP4) matrices a [m, k] and b [n, k]; out, pre and residual
    (which may be out) are [m, n] of one type, bias [n] float32.  k = 0, a sum over
    no rows, gives z = bias."""
    index = _device(h, out, "out")
    ptr, ld, code, size = _matrix(out, "out", index)
    m, n = size
    if bits not in (4, 8):
        raise ValueError("bits must be 4 or 8")
    ad, as_ = _mx(a, "a", index, m, k, bits)
    bd, bs = _mx(b, "b", index, n, k, bits)
    first = index, out.dtype, code, size
    pp, ldp = _like(pre, "pre", first)
    cp, ldc = _like(residual, "residual", first)
    bp = _floats(bias, "bias", index, (n,))
    kind = ACTIVATIONS[act]
    if m == 0 or n == 0:
        return
    stream = _stream_of(stream, index)
    if k == 0:
        zeros, ad, as_ = _zero_block(max(m, n), stream, index, bits)
        bd, bs, k = ad, as_, 32
    p = MxLinear.from_buffer_copy(_LINEAR.pack(m, n, k, bits, code, ad, as_, bd, bs, alpha, beta, bp, kind, cp, ldc, pp, ldp, ptr, ld))
    rc = load().dmuon_mx_linear(h, p, stream)
    if rc:
        _check(rc, "dmuon_mx_linear", h)


def dmuon_act_backward(h, dout, pre, act, dz=None, d_bias=None, by_rows=None, by_cols=None, scale="floor", stream=None):
    """dz = dout * act'(pre) of dout and pre [r, c] into ``dz``, by rows and / or
    columns into the MXFP8 matrices ``by_rows`` (r x c) and ``by_cols`` (c x r),
    and its column sums into ``d_bias`` [c] float32; None for what is not wanted.
    ``pre`` may be None for act "none"."""
    index = _device(h, dout, "dout")
    ptr, ld, code, size = _matrix(dout, "dout", index)
    r, c = size
    kind = ACTIVATIONS[act]
    if pre is None and kind != 0:
        raise ValueError("pre is wanted for this activation")
    first = index, dout.dtype, code, size
    pp, ldp = _like(pre, "pre", first)
    zp, ldz = _like(dz, "dz", first)
    rd, rs = _mxfp8(by_rows, "by_rows", index, r, c)
    cd, cs = _mxfp8(by_cols, "by_cols", index, c, r)
    p = ActBackward.from_buffer_copy(_ACT_BACKWARD.pack(r, c, code, kind, ptr, ld, pp, ldp, zp, ldz, _floats(d_bias, "d_bias", index, (c,)),
                                                        SCALE_MODES[scale], rd or 0, rs or 0, cd or 0, cs or 0))
    if dz is None and d_bias is None and by_rows is None and by_cols is None:
        raise ValueError("no output is given")
    rc = load().dmuon_act_backward(h, p, _stream_of(stream, index))
    if rc:
        _check(rc, "dmuon_act_backward", h)


def _check_uint64(seed, offset):
    if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
        raise ValueError("seed and offset must be from 0 to 2^64 - 1")


def _add_norm(h, x, f, y, w, rstd, out, q, mode, p, seed, offset, eps, like):
    """The fields that forward and backward share; ``like`` is f, or df."""
    _check_uint64(seed, offset)
    index = _device(h, like, "f")
    fp, ldf, code, size = _matrix(like, "f", index)
    rows, cols = size
    first = index, like.dtype, code, size
    xp, ldx = _like(x, "x", first)
    yp, ldy = _like(y, "y", first)
    hp, ldh = _like(out, "out", first)
    qd, qs = _mxfp8(q, "q", index, rows, cols)
    packed = _ADD_NORM.pack(rows, cols, code, eps, xp, ldx, fp, ldf, _floats(w, "w", index, (cols,)), yp, ldy, hp, ldh, qd or 0, qs or 0,
                            SCALE_MODES[mode], p, seed, offset, _floats(rstd, "rstd", index, (rows,)))
    return AddNorm.from_buffer_copy(packed), first


def dmuon_add_norm_forward(h, x, f, w, y, rstd, out=None, q=None, p=0.0, seed=0, offset=0, eps=1e-6, scale="floor", stream=None):
    """y = x + dropout(f) (x None: 0) and rms(y) * w over the rows of x and f
    [rows, cols], into ``out`` (their type) and / or ``q`` (an MXFP8 matrix);
    rstd [rows] is what the backward needs."""
    if y is None or w is None or rstd is None or out is None and q is None:
        raise ValueError("y, w, rstd and out or q are wanted")
    s, first = _add_norm(h, x, f, y, w, rstd, out, q, scale, p, seed, offset, eps, f)
    rc = load().dmuon_add_norm_forward(h, s, _stream_of(stream, first[0]))
    if rc:
        _check(rc, "dmuon_add_norm_forward", h)


def dmuon_add_norm_backward(h, dy, dh, y, w, rstd, dx, df, d_w, p=0.0, seed=0, offset=0, stream=None):
    """Gradients of dmuon_add_norm_forward from dh (of its normalised values) and
    dy (of y, None = 0): dx (None: not wanted; without dropout it is df), df and
    d_w [cols] float32.  y, rstd, p, seed and offset as in the forward."""
    if dh is None or df is None or y is None or w is None or rstd is None or d_w is None:
        raise ValueError("dh, y, w, rstd, df and d_w are wanted")
    s, first = _add_norm(h, None, None, y, w, rstd, None, None, "floor", p, seed, offset, 0.0, df)
    index, line = first[0], (first[3][1],)
    g = AddNormGrad.from_buffer_copy(_ADD_NORM_GRAD.pack(*_like(dy, "dy", first), *_like(dh, "dh", first), *_like(dx, "dx", first),
                                                         *_like(df, "df", first), _floats(d_w, "d_w", index, line)))
    rc = load().dmuon_add_norm_backward(h, s, g, _stream_of(stream, index))
    if rc:
        _check(rc, "dmuon_add_norm_backward", h)


def dmuon_dropout(h, x, out, p, seed, offset=0, residual=None, stream=None):
    """out = dropout(x) (+ residual) over [rows, cols]: an element stays with
    probability 1 - p, as (p, seed, offset, row, column) tell, and is then scaled
    by 1 / (1 - p).  The same call on a gradient is the backward pass; out may be
    x or residual."""
    _check_uint64(seed, offset)
    index = _device(h, x, "x")
    ptr, ld, code, size = _matrix(x, "x", index)
    first = index, x.dtype, code, size
    if out is None:
        raise ValueError("out is wanted")
    op, ldo = _like(out, "out", first)
    rp, ldr = _like(residual, "residual", first)
    rc = load().dmuon_dropout(h, ptr, code, size[0], size[1], ld, rp or None, ldr, op, ldo, p, seed, offset, _stream_of(stream, index))
    if rc:
        _check(rc, "dmuon_dropout", h)


def dmuon_get_status(h, n_flags=0):
    """Synchronise and return (status_code, per-matrix flags list)."""
    flags = (ctypes.c_int * max(1, n_flags))()
    rc = load().dmuon_get_status(h, flags, int(n_flags))
    return rc, [flags[i] for i in range(n_flags)]


def dmuon_set_overlap(h, on=True):  # default off in the library
    """Overlap the next chunk's momentum pass with the current chunk's products."""
    _check(load().dmuon_set_overlap(h, 1 if on else 0), "dmuon_set_overlap")


def dmuon_set_chunk_elements(h, elems):
    """Chunk size of later plans in matrix elements (0 = default 2^29)."""
    _check(load().dmuon_set_chunk_elements(h, int(elems)), "dmuon_set_chunk_elements")


def dmuon_set_balanced_dealing(h, on=True):  # default on in the library
    """Longest-first dealing of work items to the least-loaded CTA (pair) for later plans."""
    _check(load().dmuon_set_balanced_dealing(h, 1 if on else 0), "dmuon_set_balanced_dealing")


def dmuon_set_fp16_iterations(h, iters=3):  # default 3 in the library
    """Direct backend: leading Newton-Schulz iterations with fp16 operands
    (later ones bf16); 64 or more: every iteration."""
    _check(load().dmuon_set_fp16_iterations(h, int(iters)), "dmuon_set_fp16_iterations")


def dmuon_set_fused_phases(h, mode=2):  # default 2 (automatic) in the library
    """Direct backend: every product of every iteration of a chunk in one
    persistent launch -- 0 never, 1 always (True), 2 for chunks of few work
    items (the default); False selects 0."""
    m = 1 if mode is True else (0 if mode is False else int(mode))
    _check(load().dmuon_set_fused_phases(h, m), "dmuon_set_fused_phases")


def dmuon_set_small_path(h, on=True):  # default on in the library
    """Route small matrices (oriented m <= 128, n <= 512) through the fused
    one-CTA-per-matrix kernel (on) or through the chunked GEMM path (off)."""
    _check(load().dmuon_set_small_path(h, 1 if on else 0), "dmuon_set_small_path")


def dmuon_set_tile_mode(h, mode):
    """0 automatic, 1 single-CTA 128x256 tiles, 2 CTA-pair 256x256 tiles,
    3 single-CTA 128x128 tiles."""
    _check(load().dmuon_set_tile_mode(h, int(mode)), "dmuon_set_tile_mode")


def dmuon_set_wait_timeout(h, ns):
    _check(load().dmuon_set_wait_timeout(h, int(ns)), "dmuon_set_wait_timeout")


def dmuon_last_error(h):
    return load().dmuon_last_error(h).decode()


def dmuon_launch_count(h):
    return int(load().dmuon_launch_count(h))


def dmuon_profile_enable(h, on=True):
    _check(load().dmuon_profile_enable(h, 1 if on else 0), "dmuon_profile_enable")


def dmuon_profile_read(h):
    """{kind: (ms_total, launches)} accumulated since the last read."""
    n = len(KIND_NAMES)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int64 * n)()
    _check(load().dmuon_profile_read(h, ms, cnt, n), "dmuon_profile_read")
    return {KIND_NAMES[k]: (ms[k], cnt[k]) for k in range(n)}


def dmuon_plan_summary(h):
    L = load()
    need = L.dmuon_plan_summary(h, None, 0)
    buf = ctypes.create_string_buffer(need + 1)
    L.dmuon_plan_summary(h, buf, need + 1)
    return buf.value.decode()


class Handle:
    """Owning wrapper of a dmuon handle (destroyed on close / exit)."""

    def __init__(self, device=0):
        self.h = dmuon_create(device)

    def close(self):
        if self.h is not None:
            dmuon_destroy(self.h)
            self.h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def step(self, params, grads, momentum, lr=0.02, mu=0.95, ns_steps=5, **kw):
        return dmuon_step(self.h, params, grads, momentum, lr, mu, ns_steps, **kw)

    def newton_schulz(self, inputs, outputs, ns_steps=5, coeffs=None, eps=1e-7, stream=None):
        return dmuon_newton_schulz(self.h, inputs, outputs, ns_steps, coeffs, eps, stream)

    def gram_newton_schulz(self, inputs, outputs, ns_steps=5, coeffs=None, restarts=None, eps=1e-7,
                           stream=None):
        return dmuon_gram_newton_schulz(self.h, inputs, outputs, ns_steps, coeffs, restarts, eps, stream)

    def status(self, n_flags=0):
        return dmuon_get_status(self.h, n_flags)

    def mxfp4_quantize(self, src, by_rows=None, by_cols=None, noise=None, scale="floor", stream=None):
        return dmuon_mxfp4_quantize(self.h, src, by_rows, by_cols, noise, scale, stream)

    def mxfp4_dequantize(self, q, out, stream=None):
        return dmuon_mxfp4_dequantize(self.h, q, out, stream)

    def mxfp4_gemm(self, a, b, out, k, alpha=1.0, beta=0.0, stream=None):
        return dmuon_mxfp4_gemm(self.h, a, b, out, k, alpha, beta, stream)

    def block_norm_forward(self, x, f, post_w, pre_w, y, out, rstd, **kw):
        return dmuon_block_norm_forward(self.h, x, f, post_w, pre_w, y, out, rstd, **kw)

    def block_norm_backward(self, dy, dh, x, f, y, post_w, pre_w, rstd, dx, df, d_post_w, d_pre_w, **kw):
        return dmuon_block_norm_backward(self.h, dy, dh, x, f, y, post_w, pre_w, rstd, dx, df, d_post_w, d_pre_w, **kw)

    def mxfp8_quantize(self, src, by_rows=None, by_cols=None, scale="floor", stream=None):
        return dmuon_mxfp8_quantize(self.h, src, by_rows, by_cols, scale, stream)

    def mxfp8_dequantize(self, q, out, stream=None):
        return dmuon_mxfp8_dequantize(self.h, q, out, stream)

    def mx_linear(self, a, b, out, k, **kw):
        return dmuon_mx_linear(self.h, a, b, out, k, **kw)

    def act_backward(self, dout, pre, act, **kw):
        return dmuon_act_backward(self.h, dout, pre, act, **kw)

    def add_norm_forward(self, x, f, w, y, rstd, **kw):
        return dmuon_add_norm_forward(self.h, x, f, w, y, rstd, **kw)

    def add_norm_backward(self, dy, dh, y, w, rstd, dx, df, d_w, **kw):
        return dmuon_add_norm_backward(self.h, dy, dh, y, w, rstd, dx, df, d_w, **kw)

    def dropout(self, x, out, p, seed, offset=0, residual=None, stream=None):
        return dmuon_dropout(self.h, x, out, p, seed, offset, residual, stream)
