"""Thin Python binding of libfp8q's C ABI (include/fp8q.h).

Argument marshalling only: every step of the path runs in the CUDA kernels of
libfp8q.so.  Tensors are torch CUDA tensors (torch supplies device memory and
streams); the functions keep the C names and raise Fp8qError on a non-OK
status.  The first nine calls go through ctypes, the 4-bit calls and those behind
them through a compiled module (csrc/binding.cpp), which takes 2 to 3 us a call where
a single token's kernel takes 2 to 5; either lets other Python threads run
meanwhile.  If the library has not been built, loading fails loudly -- there is
no fallback.
"""
from __future__ import annotations

import ctypes
import os

E4M3FN = 0
E5M2 = 1
MXFP4 = 2
NVFP4 = 3
ACT_NONE = 0
ACT_GELU = 1
ALGO_MAX = 0
ALGO_MOST_RECENT = 1
MAX_TENSORS = 512

STATUS = {0: "FP8Q_OK", 1: "FP8Q_ERR_INVALID_ARG", 2: "FP8Q_ERR_UNSUPPORTED", 3: "FP8Q_ERR_CUDA",
          4: "FP8Q_ERR_TOO_MANY_TENSORS"}

# Every symbol the header declares, but the five that only count bytes.
EXPORTS = ("fp8q_quantize_amax", "fp8q_multi_quantize_amax", "fp8q_dequantize",
           "fp8q_amax_scale_update", "fp8q_qdq_amax", "fp8q_amax_scale_update_ring",
           "fp8q_gelu_quantize_amax", "fp8q_layernorm_quantize_amax",
           "fp8q_amax_scale_update_ring_quantize", "fp8q_fp4_quantize_amax", "fp8q_fp4_dequantize",
           "fp8q_fp4_matmul", "fp8q_residual_norm_quantize_amax", "fp8q_residual_norm_backward",
           "fp8q_matmul", "fp8q_grouped_matmul", "fp8q_grouped_weight_gradient", "fp8q_checkpoint_quantize",
           "fp8q_checkpoint_dequantize", "fp8q_gelu_backward_quantize_amax",
           "fp8q_status_string", "fp8q_last_cuda_error")

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfp8q.so")


class Fp8qError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        msg = f"{where}: {STATUS.get(status, status)}"
        if detail:
            msg += f" ({detail})"
        super().__init__(msg)


class Tensor(ctypes.Structure):
    """fp8q_tensor: one entry of a ragged list."""
    _fields_ = [("x_bf16", ctypes.c_void_p), ("q", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("scale", ctypes.c_void_p), ("amax", ctypes.c_void_p)]


class ResidualNorm(ctypes.Structure):
    """fp8q_residual_norm: the arguments of fp8q_residual_norm_quantize_amax."""
    _fields_ = [("rows", ctypes.c_int64), ("hidden", ctypes.c_int32), ("fmt", ctypes.c_int), ("residual", ctypes.c_void_p),
                ("block", ctypes.c_void_p), ("post_weight", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("rows_per_gate", ctypes.c_int64), ("gate_is_bf16", ctypes.c_int32), ("alpha", ctypes.c_float),
                ("eps", ctypes.c_float), ("pre_weight", ctypes.c_void_p), ("residual_out", ctypes.c_void_p),
                ("h", ctypes.c_void_p), ("q", ctypes.c_void_p), ("sf", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("amax", ctypes.c_void_p), ("rstd_post", ctypes.c_void_p), ("rstd_pre", ctypes.c_void_p)]


class ResidualNormGrad(ctypes.Structure):
    """fp8q_residual_norm_grad: the arguments of fp8q_residual_norm_backward."""
    _fields_ = [("rows", ctypes.c_int64), ("hidden", ctypes.c_int32), ("gate_is_bf16", ctypes.c_int32),
                ("d_residual_out", ctypes.c_void_p), ("d_h", ctypes.c_void_p), ("residual_out", ctypes.c_void_p),
                ("rstd_pre", ctypes.c_void_p), ("pre_weight", ctypes.c_void_p), ("block", ctypes.c_void_p),
                ("rstd_post", ctypes.c_void_p), ("post_weight", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("rows_per_gate", ctypes.c_int64), ("alpha", ctypes.c_float), ("d_residual", ctypes.c_void_p),
                ("d_block", ctypes.c_void_p), ("d_pre_weight", ctypes.c_void_p), ("d_post_weight", ctypes.c_void_p),
                ("d_gate", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


class Product(ctypes.Structure):
    """fp8q_product: the arguments of fp8q_matmul, fp8q_grouped_matmul and fp8q_grouped_weight_gradient."""
    _fields_ = [("m", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64), ("a", ctypes.c_void_p), ("b", ctypes.c_void_p),
                ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64), ("a_fmt", ctypes.c_int), ("b_fmt", ctypes.c_int),
                ("a_trans", ctypes.c_int32), ("b_trans", ctypes.c_int32), ("a_scale", ctypes.c_void_p), ("b_scale", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("bias_is_bf16", ctypes.c_int32), ("act", ctypes.c_int), ("residual", ctypes.c_void_p),
                ("d", ctypes.c_void_p), ("out", ctypes.c_int), ("q_fmt", ctypes.c_int), ("q", ctypes.c_void_p),
                ("q_scale", ctypes.c_void_p), ("amax", ctypes.c_void_p), ("h", ctypes.c_void_p), ("h_sf", ctypes.c_void_p)]


class GeluGrad(ctypes.Structure):
    """fp8q_gelu_grad: the arguments of fp8q_gelu_backward_quantize_amax."""
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("fmt", ctypes.c_int), ("d_y", ctypes.c_void_p), ("h", ctypes.c_void_p),
                ("h_sf", ctypes.c_void_p), ("d_x", ctypes.c_void_p), ("q", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("amax", ctypes.c_void_p), ("d_bias", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libfp8q.so (built by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build the CUDA library first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, c_int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
        L.fp8q_quantize_amax.argtypes = [vp, vp, i64, c_int, vp, vp, vp]
        L.fp8q_multi_quantize_amax.argtypes = [vp, i32, c_int, vp]
        L.fp8q_dequantize.argtypes = [vp, vp, i64, c_int, vp, vp]
        L.fp8q_amax_scale_update.argtypes = [vp, i32, i32, vp, vp, vp, vp, c_int, c_int, i32, vp]
        L.fp8q_qdq_amax.argtypes = [vp, vp, i64, c_int, vp, vp, vp]
        L.fp8q_amax_scale_update_ring.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp, c_int, c_int, i32,
                                                  vp]
        L.fp8q_gelu_quantize_amax.argtypes = [vp, vp, vp, i64, c_int, vp, vp, vp]
        L.fp8q_layernorm_quantize_amax.argtypes = [vp, vp, vp, i64, i32, vp, vp, ctypes.c_float, c_int,
                                                   vp, vp, vp]
        L.fp8q_amax_scale_update_ring_quantize.argtypes = [vp, vp, vp, i32, i32, vp, vp, vp, vp, c_int, c_int,
                                                           i32, vp, vp, i64, i32, vp, vp]
        L.fp8q_fp4_quantize_amax.argtypes = [vp, i64, i64, vp, vp, vp, vp, c_int, vp, vp, vp]
        L.fp8q_fp4_dequantize.argtypes = [vp, vp, vp, i64, i64, c_int, vp, vp]
        L.fp8q_fp4_matmul.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, c_int, c_int, vp, vp, vp]
        L.fp8q_residual_norm_quantize_amax.argtypes = [vp, vp]
        L.fp8q_residual_norm_backward.argtypes = [vp, vp]
        L.fp8q_residual_norm_backward_workspace.argtypes = [i64, i32, i64]
        L.fp8q_residual_norm_backward_workspace.restype = i64
        L.fp8q_matmul.argtypes = [vp, vp]
        L.fp8q_grouped_matmul.argtypes = [vp, vp, i32, vp]
        L.fp8q_grouped_weight_gradient.argtypes = [vp, vp, i32, vp]
        L.fp8q_checkpoint_scale_bytes.argtypes = [i64, i64]
        L.fp8q_checkpoint_scale_bytes.restype = i64
        L.fp8q_checkpoint_quantize.argtypes = [vp, vp, vp, i64, i64, vp]
        L.fp8q_checkpoint_dequantize.argtypes = [vp, vp, vp, i64, i64, vp]
        L.fp8q_gelu_backward_workspace.argtypes = [i64, i64]
        L.fp8q_gelu_backward_workspace.restype = i64
        L.fp8q_gelu_backward_quantize_amax.argtypes = [vp, vp]
        for f in ("fp8q_quantize_amax", "fp8q_multi_quantize_amax", "fp8q_dequantize",
                  "fp8q_amax_scale_update", "fp8q_qdq_amax", "fp8q_amax_scale_update_ring",
                  "fp8q_gelu_quantize_amax", "fp8q_layernorm_quantize_amax",
                  "fp8q_amax_scale_update_ring_quantize", "fp8q_fp4_quantize_amax", "fp8q_fp4_dequantize",
                  "fp8q_fp4_matmul", "fp8q_residual_norm_quantize_amax", "fp8q_residual_norm_backward", "fp8q_matmul",
                  "fp8q_grouped_matmul", "fp8q_grouped_weight_gradient", "fp8q_checkpoint_quantize",
                  "fp8q_checkpoint_dequantize", "fp8q_gelu_backward_quantize_amax"):
            getattr(L, f).restype = c_int
        L.fp8q_status_string.argtypes = [c_int]
        L.fp8q_status_string.restype = ctypes.c_char_p
        L.fp8q_last_cuda_error.argtypes = []
        L.fp8q_last_cuda_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


_binding = None


def _native():
    """The compiled marshalling (csrc/binding.cpp) of the calls from the 4-bit ones on, on libfp8q's entry points."""
    global _binding
    if _binding is not None:
        return _binding
    L = lib()
    from . import build
    made_for, runs = build.binding_made_for(), build.binding_for()  # the import of torch also loads the libraries the module needs
    if made_for != runs:
        raise RuntimeError(f"_binding.so was made for {made_for or 'nothing yet'}, this is {runs or 'a Python without torch'}: "
                           "run python -m quantize_amax_scaling_gb300.build")
    from . import _binding as b
    at = lambda *fs: (ctypes.cast(f, ctypes.c_void_p).value for f in fs)  # noqa: E731
    b.bind(*at(L.fp8q_fp4_quantize_amax, L.fp8q_fp4_dequantize, L.fp8q_fp4_matmul, L.fp8q_residual_norm_quantize_amax,
               L.fp8q_residual_norm_backward, L.fp8q_residual_norm_backward_workspace))
    b.bind_products(*at(L.fp8q_matmul, L.fp8q_grouped_matmul, L.fp8q_grouped_weight_gradient, L.fp8q_checkpoint_quantize,
                        L.fp8q_checkpoint_dequantize, L.fp8q_gelu_backward_quantize_amax, L.fp8q_gelu_backward_workspace))
    _binding = b
    return b


def _check(status: int, where: str):
    if status != 0:
        detail = lib().fp8q_last_cuda_error().decode() if status == 3 else ""
        raise Fp8qError(status, where, detail)


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


_FP8_DTYPES = None


def _dev(t, kind, name):
    """Reject anything but a contiguous CUDA tensor of the right element type
    on the current CUDA device.

    Pointers reach the kernels unchanged, so a host tensor must never get
    through, and the library launches on the current device, so a tensor on
    another GPU must not either.  ``kind`` is "bf16", "u8" (uint8 or a float8
    dtype), "f32" or "i32".
    """
    global _FP8_DTYPES
    if _FP8_DTYPES is None:
        import torch
        _FP8_DTYPES = (torch.uint8, torch.float8_e4m3fn, torch.float8_e5m2)
    if t is None:
        return
    import torch
    ok = {"bf16": (torch.bfloat16,), "u8": _FP8_DTYPES, "f32": (torch.float32,),
          "i32": (torch.int32,)}[kind]
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in ok:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {ok}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    cur = torch.cuda.current_device()
    if t.device.index != cur:
        raise ValueError(f"{name} is on {t.device} but the current CUDA device is cuda:{cur}; "
                         "the kernels launch on the current device (wrap the call in torch.cuda.device)")


def _numel(t):
    return 0 if t is None else t.numel()


def fp8q_quantize_amax(x, q, fmt, scale, amax, stream=None):
    """q = FP8(x / scale) (saturating RNE) and amax = max(amax, max|x|) in one launch."""
    n = _numel(x)
    if q is not None and _numel(q) != n:
        raise ValueError("q must have as many elements as x")
    for t, k, nm in ((x, "bf16", "x"), (q, "u8", "q"), (scale, "f32", "scale"), (amax, "f32", "amax")):
        _dev(t, k, nm)
    _check(lib().fp8q_quantize_amax(_ptr(x), _ptr(q), n, fmt, _ptr(scale), _ptr(amax),
                                    _stream(stream)), "fp8q_quantize_amax")


def fp8q_qdq_amax(x, y, fmt, scale, amax, stream=None):
    """y = DQ(Q(x)) in bf16 and amax = max(amax, max|x|) in one launch (y may be x)."""
    n = _numel(x)
    if y is not None and _numel(y) != n:
        raise ValueError("y must have as many elements as x")
    for t, k, nm in ((x, "bf16", "x"), (y, "bf16", "y"), (scale, "f32", "scale"), (amax, "f32", "amax")):
        _dev(t, k, nm)
    _check(lib().fp8q_qdq_amax(_ptr(x), _ptr(y), n, fmt, _ptr(scale), _ptr(amax), _stream(stream)),
           "fp8q_qdq_amax")


def fp8q_gelu_quantize_amax(h, y, q, fmt, scale, amax, stream=None):
    """y = bf16(GELU(h)) (y may be None), q = FP8(y / scale), amax = max(amax, max|y|), one launch."""
    n = _numel(h)
    for t, nm in ((y, "y"), (q, "q")):
        if t is not None and _numel(t) != n:
            raise ValueError(f"{nm} must have as many elements as h")
    for t, k, nm in ((h, "bf16", "h"), (y, "bf16", "y"), (q, "u8", "q"), (scale, "f32", "scale"),
                     (amax, "f32", "amax")):
        _dev(t, k, nm)
    _check(lib().fp8q_gelu_quantize_amax(_ptr(h), _ptr(y), _ptr(q), n, fmt, _ptr(scale), _ptr(amax),
                                         _stream(stream)), "fp8q_gelu_quantize_amax")


def fp8q_layernorm_quantize_amax(x, y, q, gamma, beta, fmt, scale, amax, eps=1e-6, stream=None):
    """y = bf16(LayerNorm(x) * gamma + beta) (y may be None), q = FP8(y / scale),
    amax = max(amax, max|y|), one launch.

    ``x`` is bf16 [rows, hidden]; ``gamma`` and ``beta`` are float32 [hidden].
    """
    if x.dim() != 2:
        raise ValueError("x must be [rows, hidden]")
    rows, hidden = x.shape
    for t, nm in ((y, "y"), (q, "q")):
        if t is not None and _numel(t) != rows * hidden:
            raise ValueError(f"{nm} must have as many elements as x")
    for t, nm in ((gamma, "gamma"), (beta, "beta")):
        if _numel(t) != hidden:
            raise ValueError(f"{nm} must have hidden={hidden} elements")
    for t, k, nm in ((x, "bf16", "x"), (y, "bf16", "y"), (q, "u8", "q"), (gamma, "f32", "gamma"),
                     (beta, "f32", "beta"), (scale, "f32", "scale"), (amax, "f32", "amax")):
        _dev(t, k, nm)
    _check(lib().fp8q_layernorm_quantize_amax(_ptr(x), _ptr(y), _ptr(q), rows, hidden, _ptr(gamma),
                                              _ptr(beta), float(eps), fmt, _ptr(scale), _ptr(amax),
                                              _stream(stream)), "fp8q_layernorm_quantize_amax")


class TensorList:
    """A ragged list checked and marshalled once into the ``fp8q_tensor`` array that
    ``fp8q_multi_quantize_amax`` takes.

    ``scales`` and ``amaxes`` are sequences of one-element float32 tensors (or views
    into one vector) aligned with ``xs``.  Passing a TensorList instead of the four
    sequences skips the per-tensor checks on every call, which for hundreds of small
    tensors take longer than the launch itself.  The list keeps the tensors alive; it
    reads their storage when called, so tensors resized or replaced since it was built
    need a new list.
    """

    def __init__(self, xs, qs, scales, amaxes):
        count = len(xs)
        if not (len(qs) == len(scales) == len(amaxes) == count):
            raise ValueError("xs, qs, scales and amaxes must have the same length")
        import torch
        _dev(None, "bf16", "")
        cur = None
        kinds = ((torch.bfloat16,), _FP8_DTYPES, (torch.float32,), (torch.float32,))
        arr = (Tensor * max(1, count))()
        for i in range(count):
            ts = (xs[i], qs[i], scales[i], amaxes[i])
            for t, ok, k, nm in zip(ts, kinds, ("bf16", "u8", "f32", "f32"), ("x", "q", "scale", "amax")):
                if t is None:
                    raise ValueError(f"{nm}[{i}] is None")
                # the common case in one expression; anything else gets _dev's message
                if t.dtype not in ok or not t.is_cuda or not t.is_contiguous():
                    _dev(t, k, f"{nm}[{i}]")
                if cur is None:
                    cur = torch.cuda.current_device()
                if t.get_device() != cur:
                    _dev(t, k, f"{nm}[{i}]")
            n = ts[0].numel()
            if ts[1].numel() != n:
                raise ValueError(f"tensor {i}: q must have as many elements as x")
            arr[i].x_bf16 = ts[0].data_ptr()
            arr[i].q = ts[1].data_ptr()
            arr[i].n = n
            arr[i].scale = ts[2].data_ptr()
            arr[i].amax = ts[3].data_ptr()
        self.count = count
        self.array = arr
        self.address = ctypes.cast(arr, ctypes.c_void_p)
        self._keep = (list(xs), list(qs), list(scales), list(amaxes))


def fp8q_multi_quantize_amax(xs, qs=None, fmt=E4M3FN, scales=None, amaxes=None, stream=None):
    """fp8q_quantize_amax over a ragged list of tensors, one launch.

    Either the four aligned sequences (xs, qs, scales, amaxes: see TensorList),
    checked on every call, or a TensorList built once as ``xs`` (leave qs, scales
    and amaxes out).
    """
    if isinstance(xs, TensorList):
        if qs is not None or scales is not None or amaxes is not None:
            raise ValueError("pass either a TensorList or xs, qs, scales and amaxes")
        tl = xs
    else:
        tl = TensorList(xs, qs, scales, amaxes)
    _check(lib().fp8q_multi_quantize_amax(tl.address, tl.count, fmt, _stream(stream)),
           "fp8q_multi_quantize_amax")


def fp8q_dequantize(q, y, fmt, scale, stream=None):
    """y = bf16_rne(float(q) * scale)."""
    n = _numel(q)
    if y is not None and _numel(y) != n:
        raise ValueError("y must have as many elements as q")
    for t, k, nm in ((q, "u8", "q"), (y, "bf16", "y"), (scale, "f32", "scale")):
        _dev(t, k, nm)
    _check(lib().fp8q_dequantize(_ptr(q), _ptr(y), n, fmt, _ptr(scale), _stream(stream)),
           "fp8q_dequantize")


def fp8q_amax_scale_update(history, amax_new, scale, scale_inv, fmt=E4M3FN, algo=ALGO_MAX,
                           margin=0, slot_format=None, stream=None):
    """In-place amax-history roll, amax selection and scale/scale_inv update.

    ``history`` is a float32 [history_len, num_slots] tensor, row 0 newest.
    """
    if history.dim() != 2:
        raise ValueError("history must be [history_len, num_slots]")
    H, S = history.shape
    for t, k, nm in ((history, "f32", "history"), (amax_new, "f32", "amax_new"),
                     (scale, "f32", "scale"), (scale_inv, "f32", "scale_inv"),
                     (slot_format, "u8", "slot_format")):
        _dev(t, k, nm)
    for t, nm in ((amax_new, "amax_new"), (scale, "scale"), (scale_inv, "scale_inv"),
                  (slot_format, "slot_format")):
        if t is not None and t.numel() != S:
            raise ValueError(f"{nm} must have num_slots={S} elements")
    _check(lib().fp8q_amax_scale_update(_ptr(history), H, S, _ptr(amax_new), _ptr(scale),
                                        _ptr(scale_inv), _ptr(slot_format), fmt, algo, margin,
                                        _stream(stream)), "fp8q_amax_scale_update")


def fp8q_amax_scale_update_ring(history, head, amax_new, scale, scale_inv, fmt=E4M3FN,
                                algo=ALGO_MAX, margin=0, slot_format=None, stream=None):
    """Ring-buffer amax history update: overwrite each slot's oldest row, advance head.

    ``history`` is float32 [history_len, num_slots]; ``head`` is int32 [num_slots],
    the row of each slot's newest entry.
    """
    if history.dim() != 2:
        raise ValueError("history must be [history_len, num_slots]")
    H, S = history.shape
    for t, k, nm in ((history, "f32", "history"), (head, "i32", "head"), (amax_new, "f32", "amax_new"),
                     (scale, "f32", "scale"), (scale_inv, "f32", "scale_inv"),
                     (slot_format, "u8", "slot_format")):
        if t is None and nm == "head":
            raise ValueError("head must be a contiguous int32 CUDA tensor")
        _dev(t, k, nm)
    for t, nm in ((head, "head"), (amax_new, "amax_new"), (scale, "scale"), (scale_inv, "scale_inv"),
                  (slot_format, "slot_format")):
        if t is not None and t.numel() != S:
            raise ValueError(f"{nm} must have num_slots={S} elements")
    _check(lib().fp8q_amax_scale_update_ring(_ptr(history), _ptr(head), H, S, _ptr(amax_new),
                                             _ptr(scale), _ptr(scale_inv), _ptr(slot_format), fmt,
                                             algo, margin, _stream(stream)),
           "fp8q_amax_scale_update_ring")


def fp8q_amax_scale_update_ring_quantize(history, head_in, head_out, amax_new, scale, scale_inv, x, q, slot,
                                         amax, fmt=E4M3FN, algo=ALGO_MAX, margin=0, slot_format=None,
                                         stream=None):
    """The ring-buffer update of every slot, then q = FP8(x / scale[slot]) with the
    new scale and amax = max(amax, max|x|), in one launch.  head_in is read,
    head_out written (two int32 [num_slots] arrays, swapped between steps)."""
    if history.dim() != 2:
        raise ValueError("history must be [history_len, num_slots]")
    H, S = history.shape
    n = _numel(x)
    if q is not None and _numel(q) != n:
        raise ValueError("q must have as many elements as x")
    for t, k, nm in ((history, "f32", "history"), (amax_new, "f32", "amax_new"), (scale, "f32", "scale"),
                     (scale_inv, "f32", "scale_inv"), (slot_format, "u8", "slot_format"), (x, "bf16", "x"),
                     (q, "u8", "q"), (amax, "f32", "amax")):
        _dev(t, k, nm)
    for t, nm in ((head_in, "head_in"), (head_out, "head_out")):
        if t is None:
            raise ValueError(f"{nm} must be a contiguous int32 CUDA tensor")
        _dev(t, "i32", nm)
    for t, nm in ((head_in, "head_in"), (head_out, "head_out"), (amax_new, "amax_new"), (scale, "scale"),
                  (scale_inv, "scale_inv"), (slot_format, "slot_format")):
        if t is not None and t.numel() != S:
            raise ValueError(f"{nm} must have num_slots={S} elements")
    _check(lib().fp8q_amax_scale_update_ring_quantize(
        _ptr(history), _ptr(head_in), _ptr(head_out), H, S, _ptr(amax_new), _ptr(scale), _ptr(scale_inv),
        _ptr(slot_format), fmt, algo, margin, _ptr(x), _ptr(q), n, slot, _ptr(amax), _stream(stream)),
        "fp8q_amax_scale_update_ring_quantize")


_FP4_MAX_DIM = 2 ** 31 - 1024  # rows and columns of a packed operand


def fp4_row_bytes(cols):
    """Bytes of a row's codes in a packed 4-bit operand: two codes a byte, rows of whole 32-column groups."""
    return (cols + 31) // 32 * 16


def fp4_scale_bytes(rows, cols, fmt):
    """Bytes of a packed 4-bit operand's block scales: tiles of 128 rows x 4 blocks."""
    return (rows + 127) // 128 * ((cols + 127) // 128 if fmt == MXFP4 else (cols + 63) // 64) * 512


def fp4_empty(rows, cols, fmt, device="cuda"):
    """Room for a packed 4-bit operand of an [rows, cols] matrix: (codes [rows, row bytes], scales); on the
    current CUDA device one allocation holds both."""
    if device == "cuda":
        return _native().fp4_empty(rows, cols, fmt)
    import torch
    if not (0 <= rows <= _FP4_MAX_DIM and 0 <= cols <= _FP4_MAX_DIM) or fmt not in (MXFP4, NVFP4):
        raise ValueError("fp4_empty takes rows and cols from 0 to 2^31 - 1024 and MXFP4 or NVFP4")
    return (torch.empty((rows, fp4_row_bytes(cols)), dtype=torch.uint8, device=device),
            torch.empty(fp4_scale_bytes(rows, cols, fmt), dtype=torch.uint8, device=device))


def fp8q_fp4_quantize_amax(x, q, sf, fmt, scale=None, amax=None, qt=None, sft=None, stream=None):
    """The packed 4-bit operand (q, sf) of x [rows, cols], and (qt, sft) of its transpose, either
    pair None, with amax = max(amax, max|x|), in one launch.  scale (NVFP4): the tensor scale, None for 1."""
    st = _native().fp4_quantize_amax(x, q, sf, fmt, scale, amax, qt, sft, stream)
    if st:
        _check(st, "fp8q_fp4_quantize_amax")


def fp8q_fp4_dequantize(q, sf, y, fmt, scale=None, stream=None):
    """y [rows, cols] = bf16 of what the packed 4-bit operand (q, sf) stands for."""
    st = _native().fp4_dequantize(q, sf, y, fmt, scale, stream)
    if st:
        _check(st, "fp8q_fp4_dequantize")


def fp8q_fp4_matmul(a, a_sf, b, b_sf, d, k, fmt, a_scale=None, b_scale=None, stream=None):
    """d [m, n] (bf16 or float32) = A [m, k] times the transpose of B [n, k], both packed 4-bit operands."""
    st = _native().fp4_matmul(a, a_sf, b, b_sf, d, k, fmt, a_scale, b_scale, stream)
    if st:
        _check(st, "fp8q_fp4_matmul")


def fp8q_residual_norm_quantize_amax(residual, residual_out, block=None, post_weight=None, gate=None, rows_per_gate=0,
                                     alpha=1.0, pre_weight=None, h=None, q=None, sf=None, fmt=E4M3FN, scale=None,
                                     amax=None, rstd_post=None, rstd_pre=None, eps=1e-6, stream=None):
    """residual_out = residual + alpha * gate * RMSnorm(block) * post_weight, and of it
    h = RMSnorm(residual_out) * pre_weight, its codes q (FP8, or 4 bits with sf) and amax, one launch.

    ``residual`` is bf16 [rows, hidden]; ``gate`` is float32 or bf16 [ceil(rows / rows_per_gate), hidden].
    Parts left None are left out (no ``post_weight``: block is added as it is); ``residual_out`` may be
    ``residual``.  ``rstd_post`` and ``rstd_pre`` (float32 [rows]) keep what the backward pass needs.
    """
    st = _native().residual_norm_quantize_amax(residual, residual_out, block, post_weight, gate, rows_per_gate, alpha,
                                               pre_weight, h, q, sf, fmt, scale, amax, rstd_post, rstd_pre, eps, stream)
    if st:
        _check(st, "fp8q_residual_norm_quantize_amax")


def residual_norm_backward_workspace(rows, hidden, rows_per_gate=0):
    """Bytes of workspace of fp8q_residual_norm_backward (rows_per_gate 0: no gate)."""
    return _native().residual_norm_backward_workspace(rows, hidden, rows_per_gate)


def fp8q_residual_norm_backward(d_residual_out, d_h, residual_out, rstd_pre, pre_weight, d_residual, d_pre_weight,
                                block=None, rstd_post=None, post_weight=None, gate=None, rows_per_gate=0, alpha=1.0,
                                d_block=None, d_post_weight=None, d_gate=None, workspace=None, stream=None):
    """Gradients of fp8q_residual_norm_quantize_amax.  ``d_residual_out`` and ``d_h`` (with residual_out,
    rstd_pre and pre_weight) come from what follows, either may be None; gradients left None are not
    computed.  ``workspace``: residual_norm_backward_workspace bytes (uint8), for one call at a time.
    """
    st = _native().residual_norm_backward(d_residual_out, d_h, residual_out, rstd_pre, pre_weight, d_residual,
                                          d_pre_weight, block, rstd_post, post_weight, gate, rows_per_gate, alpha,
                                          d_block, d_post_weight, d_gate, workspace, stream)
    if st:
        _check(st, "fp8q_residual_norm_backward")


def fp8q_matmul(a, b, d=None, a_fmt=E4M3FN, b_fmt=E4M3FN, a_scale=None, b_scale=None, a_trans=False, b_trans=False, bias=None,
                act=ACT_NONE, residual=None, q=None, q_fmt=E4M3FN, q_scale=None, amax=None, h=None, h_sf=None, stream=None):
    """d [m, n] = act(A B^T a_scale b_scale + bias) + residual, of A [m, k] (stored [k, m] with ``a_trans``) and
    B [n, k] ([k, n] with ``b_trans``), both FP8 codes whose rows may lie any multiple of 16 bytes apart.

    ``d`` is bf16 or float32; beside it or in its place q = FP8(bf16 result / q_scale), amax = max(amax, max|bf16
    result|), and (h, h_sf), the checkpoint of what ``act`` is applied to.  ``bias`` is float32 or bf16 [n];
    ``residual`` has d's type (bf16 without d) and may be d.
    Codes are uint8 of either format, or of the float8 type that the call's format names.
    """
    st = _native().matmul(a, b, d, a_fmt, b_fmt, a_scale, b_scale, a_trans, b_trans, bias, act, residual, q, q_fmt, q_scale,
                          amax, h, h_sf, stream)
    if st:
        _check(st, "fp8q_matmul")


def fp8q_grouped_matmul(a, b, offsets, d=None, a_fmt=E4M3FN, b_fmt=E4M3FN, a_scale=None, b_scale=None, b_trans=False, bias=None,
                        act=ACT_NONE, residual=None, q=None, q_fmt=E4M3FN, q_scale=None, amax=None, h=None, h_sf=None,
                        stream=None):
    """fp8q_matmul of each group's rows of ``a`` [m, k] by its own matrix of ``b`` [groups, n, k] ([groups, k, n] with
    ``b_trans``) and its own ``bias`` [groups, n].  Group g is rows offsets[g] to offsets[g + 1] - 1 (int32 on the
    device, read by the kernel); rows of no group are left as they were."""
    st = _native().grouped_matmul(a, b, d, a_fmt, b_fmt, a_scale, b_scale, False, b_trans, bias, act, residual, q, q_fmt, q_scale,
                                  amax, h, h_sf, offsets, stream)
    if st:
        _check(st, "fp8q_grouped_matmul")


def fp8q_grouped_weight_gradient(a, b, offsets, d, a_fmt=E5M2, b_fmt=E4M3FN, a_scale=None, b_scale=None, residual=None, stream=None):
    """d [groups, m, n] (bf16 or float32): for each group the sum over its rows t of a[t]^T b[t] a_scale b_scale, plus
    ``residual`` (d's type, may be d).  ``a`` is [rows, m], ``b`` [rows, n]; an empty group's sum is zeros."""
    st = _native().grouped_weight_gradient(a, b, offsets, d, a_fmt, b_fmt, a_scale, b_scale, residual, stream)
    if st:
        _check(st, "fp8q_grouped_weight_gradient")


def checkpoint_empty(rows, cols, device="cuda"):
    """Room for the 8-bit checkpoint of an [rows, cols] activation: (codes [rows, cols], scales [rows, blocks of 32]); on
    the current CUDA device one allocation holds both."""
    if device == "cuda":
        return _native().checkpoint_empty(rows, cols)
    import torch
    if not (0 <= rows <= _FP4_MAX_DIM and 0 <= cols <= _FP4_MAX_DIM):
        raise ValueError("checkpoint_empty takes rows and cols from 0 to 2^31 - 1024")
    return (torch.empty((rows, cols), dtype=torch.uint8, device=device),
            torch.empty((rows, (cols + 31) // 32), dtype=torch.uint8, device=device))


def fp8q_checkpoint_quantize(x, q, sf, stream=None):
    """(q, sf) = the 8-bit checkpoint of x [rows, cols]: e4m3 codes under a power of two for each 32 columns of a row."""
    st = _native().checkpoint_quantize(x, q, sf, stream)
    if st:
        _check(st, "fp8q_checkpoint_quantize")


def fp8q_checkpoint_dequantize(q, sf, y, stream=None):
    """y [rows, cols] = bf16 of what the checkpoint (q, sf) stands for."""
    st = _native().checkpoint_dequantize(q, sf, y, stream)
    if st:
        _check(st, "fp8q_checkpoint_dequantize")


def gelu_backward_workspace(rows, cols):
    """Bytes of workspace of fp8q_gelu_backward_quantize_amax with d_bias."""
    return _native().gelu_backward_workspace(rows, cols)


def fp8q_gelu_backward_quantize_amax(d_y, h, h_sf, q=None, fmt=E5M2, scale=None, amax=None, d_x=None, d_bias=None, workspace=None,
                                     stream=None):
    """D = d_y GELU'(h) from the checkpoint (h, h_sf) of the GELU's input (both None: D = d_y); d_x = bf16(D), q = FP8(d_x /
    scale), amax = max(amax, max|d_x|) and d_bias (float32 [cols]) = the sum of D over rows, each where it is given.
    ``workspace``: gelu_backward_workspace bytes (uint8) with d_bias, for one call at a time."""
    st = _native().gelu_backward_quantize_amax(d_y, h, h_sf, q, fmt, scale, amax, d_x, d_bias, workspace, stream)
    if st:
        _check(st, "fp8q_gelu_backward_quantize_amax")


def status_string(status: int) -> str:
    return lib().fp8q_status_string(status).decode()
